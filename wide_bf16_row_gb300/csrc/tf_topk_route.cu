// Expert routing for GB300 (sm_103a): the best k experts of each token with
// renormalised weights, and the gradient of those weights.
//
// What is computed, for a token's row x of E expert logits:
//   score   s_e = 1 / (1 + exp(-x_e))                  (sigmoid), or
//           s_e = exp(x_e) / sum_f exp(x_f)            (softmax),
//           over the experts within reach: an expert whose logit is NaN or
//           -inf is out of reach (no score, no part in the sum, never
//           chosen); +inf stands for the largest finite float;
//   choice  c_e = s_e + bias_e; the bias moves the choice only;
//   groups  E / G consecutive experts each; a group's value is the sum of its
//           best one or two choices, and only the experts of the best groups
//           remain (ties: the lower group);
//   the k largest choices, in descending order (ties: the lower expert);
//   weight  w_i = scale * s_i, or scale * s_i / (sum over the chosen s).
// Empty places (fewer than k experts remain) hold -1 and weight 0.
//
// The choice is the one the formula gives in 64 bits.  Scores are computed
// in 32 bits with a known error; where two neighbours in the order that
// decides (the first k + 1 choices; the groups on either side of the cut)
// come closer than twice that error, the row is decided again in 64 bits.
// Neighbours with the same logit and the same bias are an exact tie and need
// no second look, and without a bias the logits themselves are the order.
//
// One warp per token, expert e in lane e / P, register e % P (P = experts a
// lane holds), so that a lower lane holds lower experts and ties fall right.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "tf_topk.h"

int tf_topk_internal_fail_cuda(int cuda_error);
int tf_topk_internal_device(int *sm_count);

namespace {

constexpr int kRouteWarps = 8; // warps (tokens in flight) per CTA
constexpr int kRouteThreads = 32 * kRouteWarps;
constexpr int kMaxExperts = TF_TOPK_ROUTE_MAX_EXPERTS;
constexpr int kMaxRouteK = TF_TOPK_ROUTE_MAX_K;
constexpr uint32_t kAll = 0xFFFFFFFFu;
template <int P> constexpr int kRouteCtas = P <= 8 ? 4 : P <= 16 ? 2 : 1; // CTAs an SM holds at a time
// Errors of the 32-bit scores, rounded up (u = 2^-24).  Sigmoid: exp2 of a
// rounded product, |x| s(1 - s) <= 0.23 bounding the share of the rounded
// exponent and s(1 - s) <= 1/4 that of exp2's 2 ulp; a sum and a reciprocal
// of at most 1: under 6 u.  Softmax: |x| exp(-|x|) <= 0.37, a sum of 32 lanes'
// at most 32 terms (36 u), a reciprocal, a product: under 45 u.  Adding the
// bias rounds by u of the sum.
constexpr float kSigmoidError = 5e-7f;
constexpr float kSoftmaxError = 4e-6f;
constexpr float kSumError = 1.2e-7f;

static_assert(kMaxRouteK <= 32, "a lane per chosen expert");
static_assert(kMaxExperts == 32 * 32, "at most 32 experts a lane");

struct RouteArgs {
    int64_t tokens, row_stride;
    int32_t experts, k, softmax, groups, kept, best, renorm;
    float scale;
    bool vec; // rows are whole vectors (load_row)
    const float *bias;
    int32_t *idx;
    float *weight;
    int32_t *load;
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// Whether an expert with this logit can be chosen (not NaN, not -inf).
__device__ __forceinline__ bool in_reach(float x) { return x > -INFINITY; }

// Order-preserving key of a number (NaN excluded); both zeros give one key,
// and 0 stays free for "none".
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t order_key64(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum64(double v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(kAll, v, d);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
    return key_value(__reduce_max_sync(kAll, order_key(v)));
}

// Takes the largest remaining key of the warp out of `key`: its value and
// its expert (the lowest on ties); 0 and -1 when none is left.
template <int P>
__device__ __forceinline__ uint32_t take_best(uint32_t (&key)[P], int lane, int &expert)
{
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) mine = max(mine, key[j]);
    const uint32_t best = __reduce_max_sync(kAll, mine);
    if (best == 0) {
        expert = -1;
        return 0;
    }
    const int owner = __ffs(__ballot_sync(kAll, mine == best)) - 1;
    int at = 0;
#pragma unroll
    for (int j = P - 1; j >= 0; --j) at = key[j] == best ? j : at;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (lane == owner && j == at) key[j] = 0;
    expert = __shfl_sync(kAll, lane * P + at, owner);
    return best;
}

template <int P>
__device__ __forceinline__ uint64_t take_best64(uint64_t (&key)[P], int lane, int &expert)
{
    uint64_t mine = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) mine = key[j] > mine ? key[j] : mine;
    const uint64_t best = warp_max64(mine);
    if (best == 0) {
        expert = -1;
        return 0;
    }
    const int owner = __ffs(__ballot_sync(kAll, mine == best)) - 1;
    int at = 0;
#pragma unroll
    for (int j = P - 1; j >= 0; --j) at = key[j] == best ? j : at;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (lane == owner && j == at) key[j] = 0;
    expert = __shfl_sync(kAll, lane * P + at, owner);
    return best;
}

// The groups kept, as a mask, from the groups' values: lane g < groups holds
// group g's key.  `cut`: the first key left out (0 when none is left out).
template <typename K>
__device__ __forceinline__ uint32_t best_groups(K mine, int groups, int kept, int lane, K &last, K &cut)
{
    uint32_t rank = 0;
    for (int g = 0; g < groups; ++g) {
        const K other = __shfl_sync(kAll, mine, g);
        rank += other > mine || (other == mine && g < lane);
    }
    const bool keep = lane < groups && rank < (uint32_t)kept;
    const uint32_t on_edge = __ballot_sync(kAll, lane < groups && rank == (uint32_t)kept - 1);
    const uint32_t past = __ballot_sync(kAll, lane < groups && rank == (uint32_t)kept);
    last = on_edge ? __shfl_sync(kAll, mine, __ffs(on_edge) - 1) : (K)0;
    cut = past ? __shfl_sync(kAll, mine, __ffs(past) - 1) : (K)0;
    return __ballot_sync(kAll, keep);
}

// The choice of one row in 64 bits: lane i gets the i-th chosen expert or -1.
template <typename T, int P>
__device__ __noinline__ int choose_in_64_bits(const T *row, const RouteArgs &a)
{
    const int lane = threadIdx.x & 31;
    double v[P];
    double top = -INFINITY;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int e = lane * P + j;
        const float x = e < a.experts ? load_logit(row + e) : -INFINITY;
        v[j] = in_reach(x) ? (double)fminf(x, FLT_MAX) : (double)-INFINITY;
        top = fmax(top, v[j]);
    }
    if (a.softmax) {
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, d));
        double sum = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) sum += v[j] > -INFINITY ? exp(v[j] - top) : 0.0;
        sum = warp_sum64(sum);
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (v[j] > -INFINITY) v[j] = exp(v[j] - top) / sum;
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (v[j] > -INFINITY) v[j] = 1.0 / (1.0 + exp(-v[j]));
    }
    uint64_t key[P], by_group[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int e = lane * P + j;
        double c = v[j];
        if (c > -INFINITY && a.bias) c += (double)a.bias[e];
        const bool ok = c > -INFINITY; // neither NaN nor -inf
        by_group[j] = ok ? order_key64(c) : 0ull;
        key[j] = by_group[j];
        if (ok && !a.bias) key[j] = order_key64((double)fminf(load_logit(row + e), FLT_MAX));
    }
    if (a.groups > 1) {
        const int per = a.experts / a.groups;
        uint64_t mine = 0;
        for (int g = 0; g < a.groups; ++g) {
            uint64_t members[P];
#pragma unroll
            for (int j = 0; j < P; ++j) members[j] = (lane * P + j) / per == g ? by_group[j] : 0ull;
            int e;
            const uint64_t first = take_best64<P>(members, lane, e);
            const uint64_t second = a.best > 1 && first ? take_best64<P>(members, lane, e) : 0ull;
            const auto value = [](uint64_t k) {
                return __longlong_as_double((long long)(k & 0x8000000000000000ull ? k ^ 0x8000000000000000ull : ~k));
            };
            const double sum = first ? value(first) + (second ? value(second) : 0.0) : 0.0;
            if (lane == g) mine = first ? order_key64(sum) : 0ull;
        }
        uint64_t last, cut;
        const uint32_t keep = best_groups<uint64_t>(mine, a.groups, a.kept, lane, last, cut);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = lane * P + j;
            if (e < a.experts && !((keep >> (e / per)) & 1u)) key[j] = 0;
        }
    }
    int chosen = -1;
    for (int i = 0; i < a.k; ++i) {
        int e;
        if (take_best64<P>(key, lane, e) == 0) break;
        if (lane == i) chosen = e;
    }
    return chosen;
}

// Sum and maximum over the W lanes (a power of two) that hold one token.
template <int W> __device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
template <int W> __device__ __forceinline__ float lanes_max(float v)
{
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

// The chosen scores of a token (a lane each, or `on` false) divided by their
// sum; where the scores themselves underflow, through their logarithms.
template <int W> __device__ __forceinline__ float share_of(float s, float x, bool on, bool softmax)
{
    float log_s = x;
    if (!softmax) {
        const float total = lanes_sum<W>(on ? s : 0.0f);
        if (__all_sync(kAll, total >= 1e-30f)) return on ? __fdividef(s, total) : 0.0f;
        log_s = fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
    }
    // softmax: the row's other experts cancel
    const float top = lanes_max<W>(on ? log_s : -INFINITY);
    const float q = on ? __expf(log_s - top) : 0.0f;
    const float total = lanes_sum<W>(q);
    return on ? __fdividef(q, total) : 0.0f;
}

// A lane's P logits of a row, its experts lane * P ..: -inf past the last
// expert and for NaN, +inf as the largest finite float.  `vec`: rows and the
// expert count are whole 16-byte (or, where a lane holds less, P-element)
// vectors.
template <typename T, int P>
__device__ __forceinline__ void load_row(const T *row, int experts, int lane, bool vec, float (&x)[P])
{
    constexpr int kBytes = P * (int)sizeof(T) < 16 ? P * (int)sizeof(T) : 16;
    constexpr int kEach = kBytes / (int)sizeof(T); // elements per vector
    if (vec) {
#pragma unroll
        for (int v = 0; v < P / kEach; ++v) {
            const int e = lane * P + v * kEach;
            alignas(16) T part[kEach];
            if (e < experts) {
                if (kBytes == 16) *reinterpret_cast<uint4 *>(part) = *reinterpret_cast<const uint4 *>(row + e);
                else if (kBytes == 8) *reinterpret_cast<uint2 *>(part) = *reinterpret_cast<const uint2 *>(row + e);
                else if (kBytes == 4) *reinterpret_cast<uint32_t *>(part) = *reinterpret_cast<const uint32_t *>(row + e);
                else *reinterpret_cast<uint16_t *>(part) = *reinterpret_cast<const uint16_t *>(row + e);
            }
#pragma unroll
            for (int j = 0; j < kEach; ++j) x[v * kEach + j] = e < experts ? load_logit(&part[j]) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = lane * P + j < experts ? load_logit(row + lane * P + j) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) x[j] = in_reach(x[j]) ? fminf(x[j], FLT_MAX) : -INFINITY;
}

// Largest and second largest (in that order) of two such pairs.
__device__ __forceinline__ void join_best_two(float &m1, float &m2, float o1, float o2)
{
    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
    m1 = fmaxf(m1, o1);
}

__device__ __forceinline__ float group_value(float m1, float m2, int best)
{
    return best > 1 && m2 > -INFINITY ? m1 + m2 : m1;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_fast(float x) { return reciprocal_fast(1.0f + exp2_fast(-kLog2e * x)); }

// Short keys: an order key whose low bits give way to the expert (lower
// experts larger), so that a warp maximum names the choice and its expert at
// once, and no two are equal.  What the cut bits held decides later, where
// two neighbours come close.
template <int P> struct ShortKey {
    static constexpr uint32_t kMask = 32 * P - 1;
    // the part of a value that the cut bits may hold
    static constexpr float kCut = (float)(32 * P) / (float)(1 << 23);
    __device__ static uint32_t make(float v, int expert) { return (order_key(v) & ~kMask) | (kMask - expert); }
    __device__ static float value(uint32_t key) { return key_value(key & ~kMask); }
    __device__ static int expert(uint32_t key) { return (int)(kMask - (key & kMask)); }
};

__device__ __forceinline__ void order_pair(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// A lane's D largest keys in descending order (D = P up to 4).
template <int P> struct LaneList {
    static constexpr int D = P < 4 ? P : 4;
    uint32_t at[D];

    __device__ static void sort4(uint32_t (&k)[4])
    {
        order_pair(k[0], k[1]);
        order_pair(k[2], k[3]);
        order_pair(k[0], k[2]);
        order_pair(k[1], k[3]);
        order_pair(k[1], k[2]);
    }
    __device__ explicit LaneList(const uint32_t (&key)[P])
    {
#pragma unroll
        for (int i = 0; i < D; ++i) at[i] = key[i];
        if constexpr (P == 2) order_pair(at[0], at[1]);
        if constexpr (P >= 4) sort4(at);
#pragma unroll
        for (int b = 4; b + 3 < P; b += 4) {
            uint32_t o[4] = {key[b], key[b + 1], key[b + 2], key[b + 3]};
            sort4(o);
            // the four largest of two descending fours: bitonic, then sorted
#pragma unroll
            for (int i = 0; i < 4; ++i) at[i] = max(at[i], o[3 - i]);
            order_pair(at[0], at[2]);
            order_pair(at[1], at[3]);
            order_pair(at[0], at[1]);
            order_pair(at[2], at[3]);
        }
    }
    // The warp's largest key, taken out of its lane's list.
    __device__ uint32_t take(const uint32_t (&key)[P])
    {
        const uint32_t best = __reduce_max_sync(kAll, at[0]);
        if (at[0] == best) {
#pragma unroll
            for (int i = 0; i + 1 < D; ++i) at[i] = at[i + 1];
            at[D - 1] = 0;
            if (D < P && at[0] == 0) // the list ran out: the next one of the lane
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (key[j] < best) at[0] = max(at[0], key[j]);
        }
        return best;
    }
};

// The k best experts of a row by the logits alone, from whole keys.
template <typename T, int P>
__device__ __noinline__ int choose_by_logits(const T *row, const RouteArgs &a)
{
    const int lane = threadIdx.x & 31;
    float x[P];
    load_row<T, P>(row, a.experts, lane, a.vec, x);
    uint32_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) key[j] = x[j] > -INFINITY ? order_key(x[j]) : 0u;
    int chosen = -1;
    for (int i = 0; i < a.k; ++i) {
        int e;
        if (take_best<P>(key, lane, e) == 0) break;
        if (lane == i) chosen = e;
    }
    return chosen;
}

// The order of up to 32 experts, one per lane (lanes < n), that short keys
// could not settle: by the logits, or with a bias by the choices, in 64 bits
// where 32 leave neighbours closer than their error.  `c` is the lane's choice
// in 32 bits.  Lane i gets the i-th.
template <typename T, int P>
__device__ __noinline__ int settle(const T *row, const RouteArgs &a, int expert, float c, int n, int *place)
{
    const int lane = threadIdx.x & 31;
    const bool mine = lane < n;
    int rank = 0;
    bool close = false;
    const float error = 2.0f * (a.softmax ? kSoftmaxError : kSigmoidError);
    for (int i = 0; i < n; ++i) {
        const float o = __shfl_sync(kAll, c, i);
        const int oe = __shfl_sync(kAll, expert, i);
        rank += o > c || (o == c && oe < expert);
        close |= mine && oe != expert && !(fabsf(o - c) > error + kSumError * (fabsf(o) + fabsf(c)));
    }
    if (a.bias && __any_sync(kAll, close)) {
        const float x = mine ? fminf(load_logit(row + expert), FLT_MAX) : 0.0f;
        double d;
        if (a.softmax) {
            float y[P];
            load_row<T, P>(row, a.experts, lane, a.vec, y);
            float top = y[0];
#pragma unroll
            for (int j = 1; j < P; ++j) top = fmaxf(top, y[j]);
            top = warp_max(top);
            double sum = 0;
#pragma unroll 1
            for (int j = 0; j < P; ++j) {
                const int e = lane * P + j;
                const float z = e < a.experts ? load_logit(row + e) : -INFINITY;
                if (in_reach(z)) sum += exp((double)fminf(z, FLT_MAX) - top);
            }
            sum = warp_sum64(sum);
            d = exp((double)x - top) / sum;
        } else {
            d = 1.0 / (1.0 + exp(-(double)x));
        }
        if (mine) d += (double)a.bias[expert];
        rank = 0;
        for (int i = 0; i < n; ++i) {
            const double o = __shfl_sync(kAll, d, i);
            const int oe = __shfl_sync(kAll, expert, i);
            rank += o > d || (o == d && oe < expert);
        }
    }
    if (mine) place[rank] = expert;
    __syncwarp();
    const int chosen = mine ? place[lane] : -1;
    __syncwarp();
    return chosen;
}

// One warp per token.  A lane sorts its best few experts' short keys; k warp
// maxima over the lanes' best then name the choices in order.  It is bound by
// the instructions of the scan over E logits (two special-function ones per
// sigmoid) and of the k rounds, not by the row's bytes.
template <typename T, int P>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<P>) route_kernel(const T *__restrict__ logits, RouteArgs a)
{
    __shared__ int32_t count[kMaxExperts];
    __shared__ int32_t place[kRouteWarps][32];
    using Key = ShortKey<P>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.load) {
        for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) count[e] = 0;
        __syncthreads();
    }
    grid_dependency_wait();
    float bias[P]; // -inf where no choice can come of it
#pragma unroll
    for (int j = 0; j < P; ++j) {
        bias[j] = a.bias && lane * P + j < a.experts ? a.bias[lane * P + j] : 0.0f;
        bias[j] = bias[j] > -INFINITY ? bias[j] : -INFINITY;
    }
    const int per = a.experts / a.groups;
    // lanes that hold one group, when whole lanes do and their count is a power of two
    const int group_lanes = per % P == 0 && ((per / P) & (per / P - 1)) == 0 ? per / P : 0;
    const bool scored = a.bias || a.groups > 1; // else the logits alone decide
    // errors of a choice: of the score, and relative to the sum with the bias
    const float error = !scored ? 0.0f : a.softmax ? kSoftmaxError : kSigmoidError;
    const float part = scored ? kSumError + 2.0f * Key::kCut : 0.0f;
    const int64_t step = (int64_t)gridDim.x * kRouteWarps;
    int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    float next[P];
    if (t < a.tokens) load_row<T, P>(logits + t * a.row_stride, a.experts, lane, a.vec, next);
    for (; t < a.tokens; t += step) {
        const T *row = logits + t * a.row_stride;
        float c[P];
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = next[j];
        if (t + step < a.tokens) load_row<T, P>(logits + (t + step) * a.row_stride, a.experts, lane, a.vec, next);
        float top = 0.0f, inverse = 1.0f;
        if (a.softmax && (scored || !a.renorm)) {
            float m = c[0], sum = 0.0f, q[P];
#pragma unroll
            for (int j = 1; j < P; ++j) m = fmaxf(m, c[j]);
            top = fmaxf(warp_max(m), -FLT_MAX); // finite: exp(-inf - top) is 0
#pragma unroll
            for (int j = 0; j < P; ++j) {
                q[j] = exp2_fast(kLog2e * (c[j] - top));
                sum += q[j];
            }
            inverse = reciprocal_fast(warp_sum(sum));
            if (scored)
#pragma unroll
                for (int j = 0; j < P; ++j) c[j] = c[j] > -INFINITY ? fmaf(q[j], inverse, bias[j]) : -INFINITY;
        } else if (scored) {
#pragma unroll
            for (int j = 0; j < P; ++j) c[j] = c[j] > -INFINITY ? sigmoid_fast(c[j]) + bias[j] : -INFINITY;
        }
        uint32_t key[P];
#pragma unroll
        for (int j = 0; j < P; ++j) key[j] = c[j] > -INFINITY ? Key::make(c[j], lane * P + j) : 0u;
        bool again = false; // too close to call in 32 bits
        if (a.groups > 1 && !group_lanes) {
            uint32_t mine = 0;
            float most = 0.0f;
            for (int g = 0; g < a.groups; ++g) {
                uint32_t members[P];
#pragma unroll
                for (int j = 0; j < P; ++j) members[j] = (lane * P + j) / per == g ? key[j] : 0u;
                int e;
                const uint32_t first = take_best<P>(members, lane, e);
                const uint32_t second = a.best > 1 && first ? take_best<P>(members, lane, e) : 0u;
                const float u = first ? Key::value(first) : 0.0f, w = second ? Key::value(second) : 0.0f;
                if (lane == g) mine = first ? order_key(u + w) : 0u;
                most = fmaxf(most, fabsf(u) + fabsf(w));
            }
            uint32_t last, cut;
            const uint32_t keep = best_groups<uint32_t>(mine, a.groups, a.kept, lane, last, cut);
            if (cut) again = !(key_value(last) - key_value(cut) > 4.0f * error + 4.0f * part * most);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int e = lane * P + j;
                if (e < a.experts && !((keep >> (e / per)) & 1u)) key[j] = 0;
            }
        }
        LaneList<P> list(key);
        if (a.groups > 1 && group_lanes) {
            float m1 = c[0], m2 = -INFINITY; // whole values: a cut between groups must not hang on short keys
#pragma unroll
            for (int j = 1; j < P; ++j) {
                m2 = fmaxf(m2, fminf(m1, c[j]));
                m1 = fmaxf(m1, c[j]);
            }
            for (int d = 1; d < group_lanes; d <<= 1)
                join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, d), __shfl_xor_sync(kAll, m2, d));
            const bool any = m1 > -INFINITY && lane < a.groups * group_lanes;
            const uint32_t mine = any ? order_key(group_value(m1, m2, a.best)) : 0u;
            uint32_t left = mine, last = 0;
            for (int g = 0; g < a.kept; ++g) { // equal values go at once; the cut is then not clear
                last = __reduce_max_sync(kAll, left);
                if (left == last) left = 0;
            }
            const uint32_t cut = __reduce_max_sync(kAll, left);
            const bool keep = mine >= last;
            if (cut) {
                const float size = any ? fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f) : 0.0f;
                const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
                again = !(key_value(last) - key_value(cut) > 4.0f * error + 4.0f * kSumError * most);
            }
            // equal values among the kept ones: more groups than asked for
            again = again || __popc(__ballot_sync(kAll, keep && any)) > a.kept * group_lanes;
            if (!keep)
#pragma unroll
                for (int i = 0; i < LaneList<P>::D; ++i) list.at[i] = 0;
        }
        uint32_t mine = 0, prev = 0;
        for (int i = 0; i < a.k; ++i) {
            prev = list.take(key);
            if (lane == i) mine = prev;
        }
        int chosen = lane < a.k && mine ? Key::expert(mine) : -1;
        // neighbours that the short keys do not settle, the one behind the k-th among them
        const auto close = [&](uint32_t p, uint32_t q) {
            const float u = Key::value(p), w = Key::value(q);
            return p && q && !(u - w > 2.0f * error + part * (fabsf(u) + fabsf(w)));
        };
        const uint32_t below = __shfl_down_sync(kAll, mine, 1);
        uint32_t past = list.take(key);
        const bool over = close(prev, past);
        if (!again && __any_sync(kAll, over || (lane < a.k - 1 && close(mine, below)))) {
            int n = a.k;
            if (over) { // everything that could still belong before the cut
                while (n < 32) {
                    if (lane == n) chosen = Key::expert(past);
                    ++n;
                    prev = past;
                    past = list.take(key);
                    if (!close(prev, past)) break;
                }
                again = n == 32 && close(prev, past);
            }
            if (!again) {
                const int found = __popc(__ballot_sync(kAll, chosen >= 0));
                float mine_c = chosen >= 0 ? fminf(load_logit(row + chosen), FLT_MAX) : 0.0f; // the logits decide
                if (a.bias && chosen >= 0)
                    mine_c = (a.softmax ? exp2_fast(kLog2e * (mine_c - top)) * inverse : sigmoid_fast(mine_c)) + a.bias[chosen];
                chosen = settle<T, P>(row, a, chosen, mine_c, min(n, found), place[warp]);
            }
        }
        if (again) chosen = scored ? choose_in_64_bits<T, P>(row, a) : choose_by_logits<T, P>(row, a);
        // weights of the chosen
        const bool on = lane < a.k && chosen >= 0;
        const float x = on ? fminf(load_logit(row + chosen), FLT_MAX) : 0.0f;
        float w = !on ? 0.0f : a.softmax ? exp2_fast(kLog2e * (x - top)) * inverse : sigmoid_fast(x);
        if (a.renorm) w = share_of<32>(w, x, on, a.softmax != 0);
        if (lane < a.k) {
            a.idx[t * a.k + lane] = on ? chosen : -1;
            a.weight[t * a.k + lane] = w * a.scale;
        }
        if (a.load && on) atomicAdd(&count[chosen], 1);
    }
    grid_dependents_go();
    if (a.load) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.experts; e += kRouteThreads)
            if (count[e]) atomicAdd(a.load + e, count[e]);
    }
}

struct RouteGradArgs {
    int64_t tokens, row_stride;
    int32_t experts, k, softmax, renorm;
    float scale;
    bool vec, vec_row; // the gradient's and the logits' rows are whole vectors
    const int32_t *idx;
    const float *grad;
};

__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// A lane's P values of a row (as load_row holds them).
template <typename T, int P>
__device__ __forceinline__ void store_row(T *row, int experts, int lane, bool vec, const float (&x)[P])
{
    constexpr int kBytes = P * (int)sizeof(T) < 16 ? P * (int)sizeof(T) : 16;
    constexpr int kEach = kBytes / (int)sizeof(T);
    if (vec) {
#pragma unroll
        for (int v = 0; v < P / kEach; ++v) {
            const int e = lane * P + v * kEach;
            alignas(16) T part[kEach];
#pragma unroll
            for (int j = 0; j < kEach; ++j) store_grad(&part[j], x[v * kEach + j]);
            if (e < experts) {
                if (kBytes == 16) *reinterpret_cast<uint4 *>(row + e) = *reinterpret_cast<const uint4 *>(part);
                else if (kBytes == 8) *reinterpret_cast<uint2 *>(row + e) = *reinterpret_cast<const uint2 *>(part);
                else if (kBytes == 4) *reinterpret_cast<uint32_t *>(row + e) = *reinterpret_cast<const uint32_t *>(part);
                else *reinterpret_cast<uint16_t *>(row + e) = *reinterpret_cast<const uint16_t *>(part);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (lane * P + j < experts) store_grad(row + lane * P + j, x[j]);
    }
}

// An expert named twice for a token (a list this library never writes) adds
// up, in the lanes' order, in its first lane; false in the others.
template <int W> __device__ __forceinline__ bool add_twins(float &d, bool on, int expert, int k)
{
    const int lane = threadIdx.x & 31, first = lane & ~(W - 1);
    const uint32_t twins = __match_any_sync(kAll, on ? first * kMaxExperts + expert : -1 - lane);
    if (__any_sync(kAll, (twins & (twins - 1)) != 0)) {
        float sum = 0.0f;
        for (int i = 0; i < k; ++i) {
            const float o = __shfl_sync(kAll, d, first + i);
            if ((twins >> (first + i)) & 1u) sum += o;
        }
        d = sum;
    }
    return on && lane == __ffs(twins) - 1;
}

// Gradient of the weights for the logits:
//   per chosen score  g_i = scale * dw_i, renormalised: (g_i - sum_j g_j r_j) / S
//                     with r_j = s_j / S, S the chosen scores' sum;
//   sigmoid  dx_i = g_i s_i (1 - s_i), others 0;
//   softmax  dx_e = s_e (g_e - sum_j g_j s_j), g_e = 0 for the others -- and
//            with renormalised weights that sum is 0, so only the chosen
//            experts' logits count.
// This kernel: all but the plain softmax.  W lanes per token, 32 / W tokens
// per warp; their rows are cleared, then the chosen experts' values stored.
template <typename T, int W>
__global__ void __launch_bounds__(kRouteThreads)
route_grad_kernel(const T *__restrict__ logits, T *__restrict__ out, RouteGradArgs a)
{
    constexpr int kTokens = 32 / W;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, place = lane & (W - 1);
    grid_dependency_wait();
    const int64_t step = (int64_t)gridDim.x * kRouteWarps * kTokens;
    for (int64_t t0 = ((int64_t)blockIdx.x * kRouteWarps + warp) * kTokens; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + lane / W;
        const int64_t cells = (a.tokens - t0 < kTokens ? a.tokens - t0 : kTokens) * a.experts;
        T *rows = out + t0 * a.experts;
        if (a.vec) {
            uint4 *v = reinterpret_cast<uint4 *>(rows);
            for (int i = lane; i < (int)(cells * (int)sizeof(T) / 16); i += 32) v[i] = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = lane; i < (int)cells; i += 32) store_grad(rows + i, 0.0f);
        }
        const bool mine = place < a.k && t < a.tokens;
        const int e = mine ? a.idx[t * a.k + place] : -1;
        const float g_in = mine ? a.grad[t * a.k + place] : 0.0f;
        float x = e >= 0 && e < a.experts ? load_logit(logits + t * a.row_stride + e) : -INFINITY;
        const bool on = in_reach(x);
        x = fminf(x, FLT_MAX);
        const float g = on ? a.scale * g_in : 0.0f;
        const float below = on && !a.softmax ? 1.0f / (1.0f + expf(x)) : 1.0f; // 1 - s
        const float s = on && !a.softmax ? 1.0f / (1.0f + expf(-x)) : 0.0f;
        float d;
        if (a.renorm) {
            const float r = share_of<W>(s, x, on, a.softmax != 0);
            const float dot = lanes_sum<W>(on ? g * r : 0.0f);
            d = on ? r * (g - dot) * below : 0.0f;
        } else {
            d = g * below * s;
        }
        __syncwarp(); // the rows are cleared
        if (add_twins<W>(d, on, e, a.k)) store_grad(out + t * a.experts + e, d);
    }
    grid_dependents_go();
}

// The plain softmax (no renormalising): every expert within reach has a
// gradient.  One warp per token, the row's exponentials in registers.
template <typename T, int P>
__global__ void __launch_bounds__(kRouteThreads)
route_softmax_grad_kernel(const T *__restrict__ logits, T *__restrict__ out, RouteGradArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T *row = logits + t * a.row_stride;
        T *dst = out + t * a.experts;
        const int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
        const float g_in = lane < a.k ? a.grad[t * a.k + lane] : 0.0f;
        float s[P];
        load_row<T, P>(row, a.experts, lane, a.vec_row, s);
        float top = s[0], sum = 0.0f;
#pragma unroll
        for (int j = 1; j < P; ++j) top = fmaxf(top, s[j]);
        top = fmaxf(warp_max(top), -FLT_MAX);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            s[j] = expf(s[j] - top);
            sum += s[j];
        }
        const float total = fmaxf(warp_sum(sum), FLT_MIN); // no expert within reach: all 0
        const float x = e >= 0 && e < a.experts ? load_logit(row + e) : -INFINITY;
        const bool on = in_reach(x);
        const float own = on ? expf(fminf(x, FLT_MAX) - top) / total : 0.0f;
        const float g = on ? a.scale * g_in : 0.0f;
        const float dot = warp_sum(g * own);
#pragma unroll
        for (int j = 0; j < P; ++j) s[j] = -dot * (s[j] / total);
        store_row<T, P>(dst, a.experts, lane, a.vec, s);
        __syncwarp(); // the chosen experts' values replace the row's
        float d = g;
        const bool first = add_twins<32>(d, on, e, a.k);
        if (first) store_grad(dst + e, own * (d - dot));
    }
    grid_dependents_go();
}

// ---------------------------------------------------------------- host side

template <typename T> using RouteKernel = void (*)(const T *, RouteArgs);

template <typename T> RouteKernel<T> route_kernel_for(int experts)
{
    const int per = (experts + 31) / 32;
    return per <= 1 ? route_kernel<T, 1>
           : per <= 2 ? route_kernel<T, 2>
           : per <= 4 ? route_kernel<T, 4>
           : per <= 8 ? route_kernel<T, 8>
           : per <= 16 ? route_kernel<T, 16>
                       : route_kernel<T, 32>;
}

// CTAs for a warp per token (or group of tokens), `each` per SM at most.
int64_t route_grid(int64_t warps, int sm_count, int each)
{
    const int64_t need = (warps + kRouteWarps - 1) / kRouteWarps;
    const int64_t most = (int64_t)sm_count * each;
    return need < most ? need : most;
}

cudaLaunchConfig_t route_config(int64_t grid, cudaStream_t stream, cudaLaunchAttribute *attr)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Whether a lane's experts can be read as whole vectors.
bool whole_vectors(const void *logits, size_t size, int experts, int64_t row_stride)
{
    int per = 1;
    while (32 * per < experts) per *= 2;
    const size_t bytes = per * size < 16 ? per * size : 16;
    return (reinterpret_cast<uintptr_t>(logits) & (bytes - 1)) == 0 && experts * size % bytes == 0 &&
           (size_t)row_stride * size % bytes == 0;
}

template <typename T> cudaError_t launch_route(const void *logits, RouteArgs a, int sm_count, void *stream)
{
    a.vec = whole_vectors(logits, sizeof(T), a.experts, a.row_stride);
    cudaLaunchAttribute attr[1];
    const int each = a.experts <= 256 ? kRouteCtas<8> : a.experts <= 512 ? kRouteCtas<16> : kRouteCtas<32>;
    const cudaLaunchConfig_t cfg =
        route_config(route_grid(a.tokens, sm_count, each), static_cast<cudaStream_t>(stream), attr);
    return cudaLaunchKernelEx(&cfg, route_kernel_for<T>(a.experts), static_cast<const T *>(logits), a);
}

template <typename T> using RouteGradKernel = void (*)(const T *, T *, RouteGradArgs);

template <typename T> RouteGradKernel<T> softmax_grad_kernel_for(int experts)
{
    const int per = (experts + 31) / 32;
    return per <= 1 ? route_softmax_grad_kernel<T, 1>
           : per <= 2 ? route_softmax_grad_kernel<T, 2>
           : per <= 4 ? route_softmax_grad_kernel<T, 4>
           : per <= 8 ? route_softmax_grad_kernel<T, 8>
           : per <= 16 ? route_softmax_grad_kernel<T, 16>
                       : route_softmax_grad_kernel<T, 32>;
}

template <typename T>
cudaError_t launch_route_grad(const void *logits, void *out, RouteGradArgs a, int sm_count, void *stream)
{
    RouteGradKernel<T> kernel;
    int tokens_per_warp = 1;
    if (a.softmax && !a.renorm) {
        a.vec = whole_vectors(out, sizeof(T), a.experts, a.experts);
        a.vec_row = whole_vectors(logits, sizeof(T), a.experts, a.row_stride);
        kernel = softmax_grad_kernel_for<T>(a.experts);
    } else {
        a.vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && a.experts * sizeof(T) % 16 == 0;
        kernel = a.k <= 8 ? route_grad_kernel<T, 8> : a.k <= 16 ? route_grad_kernel<T, 16> : route_grad_kernel<T, 32>;
        tokens_per_warp = a.k <= 8 ? 4 : a.k <= 16 ? 2 : 1;
    }
    cudaLaunchAttribute attr[1];
    const int64_t warps = (a.tokens + tokens_per_warp - 1) / tokens_per_warp;
    const cudaLaunchConfig_t cfg = route_config(route_grid(warps, sm_count, 8), static_cast<cudaStream_t>(stream), attr);
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(logits), static_cast<T *>(out), a);
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The shape guards both entry points share.
int check_shape(int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride, int32_t k)
{
    if (dtype != TF_TOPK_DTYPE_BF16 && dtype != TF_TOPK_DTYPE_F16 && dtype != TF_TOPK_DTYPE_F32)
        return TF_TOPK_ERR_DTYPE;
    if (k < 1 || k > kMaxRouteK) return TF_TOPK_ERR_K;
    if (tokens < 0 || experts < 1 || experts > kMaxExperts || row_stride < experts ||
        (tokens > 0 && row_stride > INT64_MAX / 8 / tokens))
        return TF_TOPK_ERR_SHAPE;
    return TF_TOPK_OK;
}

} // namespace

extern "C" {

int tf_topk_route(const void *logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride, int32_t k,
                  const float *bias, int32_t score, int32_t groups, int32_t groups_kept, int32_t group_best,
                  int32_t renormalize, float scale, int32_t *out_idx, float *out_weight, int32_t *load, void *stream)
{
    int st = check_shape(dtype, tokens, experts, row_stride, k);
    if (st != TF_TOPK_OK) return st;
    if ((score != TF_TOPK_ROUTE_SOFTMAX && score != TF_TOPK_ROUTE_SIGMOID) || groups < 1 ||
        groups > TF_TOPK_ROUTE_MAX_GROUPS || experts % groups != 0 || groups_kept < 1 || groups_kept > groups ||
        (group_best != 1 && group_best != 2) || !isfinite(scale))
        return TF_TOPK_ERR_ARG;
    if (tokens == 0) return TF_TOPK_OK;
    if (!logits || !out_idx || !out_weight) return TF_TOPK_ERR_NULL;
    if (!aligned(logits, dtype == TF_TOPK_DTYPE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(out_idx, 4) ||
        !aligned(out_weight, 4) || !aligned(load, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    RouteArgs a;
    a.tokens = tokens;
    a.row_stride = row_stride;
    a.experts = experts;
    a.k = k;
    a.softmax = score == TF_TOPK_ROUTE_SOFTMAX;
    a.groups = groups_kept < groups ? groups : 1; // every group kept: none decides
    a.kept = groups_kept;
    a.best = group_best;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.bias = bias;
    a.idx = out_idx;
    a.weight = out_weight;
    a.load = load;
    cudaError_t e = dtype == TF_TOPK_DTYPE_F32   ? launch_route<float>(logits, a, sm_count, stream)
                    : dtype == TF_TOPK_DTYPE_F16 ? launch_route<__half>(logits, a, sm_count, stream)
                                                 : launch_route<__nv_bfloat16>(logits, a, sm_count, stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}

int tf_topk_route_grad(const void *logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride,
                       int32_t k, const int32_t *idx, const float *grad_weight, int32_t score, int32_t renormalize,
                       float scale, void *out_grad_logits, void *stream)
{
    int st = check_shape(dtype, tokens, experts, row_stride, k);
    if (st != TF_TOPK_OK) return st;
    if ((score != TF_TOPK_ROUTE_SOFTMAX && score != TF_TOPK_ROUTE_SIGMOID) || !isfinite(scale)) return TF_TOPK_ERR_ARG;
    if (tokens == 0) return TF_TOPK_OK;
    if (!logits || !idx || !grad_weight || !out_grad_logits) return TF_TOPK_ERR_NULL;
    const size_t size = dtype == TF_TOPK_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(out_grad_logits, size) || !aligned(idx, 4) || !aligned(grad_weight, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    RouteGradArgs a;
    a.tokens = tokens;
    a.row_stride = row_stride;
    a.experts = experts;
    a.k = k;
    a.softmax = score == TF_TOPK_ROUTE_SOFTMAX;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.idx = idx;
    a.grad = grad_weight;
    cudaError_t e = dtype == TF_TOPK_DTYPE_F32 ? launch_route_grad<float>(logits, out_grad_logits, a, sm_count, stream)
                    : dtype == TF_TOPK_DTYPE_F16
                        ? launch_route_grad<__half>(logits, out_grad_logits, a, sm_count, stream)
                        : launch_route_grad<__nv_bfloat16>(logits, out_grad_logits, a, sm_count, stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}

} // extern "C"
