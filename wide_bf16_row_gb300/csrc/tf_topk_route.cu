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
// of at most 1: under 6 u.  Softmax: the exponent's roundings and that of
// log2 e (2.3 u |x| relative, with |x| exp(-|x|) <= 0.37), a sum (32 lanes of at
// most 32 terms: 36 u; four lanes of 64 terms in four chains: 19 u), exp2 in the
// sum and in the score (4 u each), a reciprocal, a product: under 50 u; relative
// to the score, with |x| <= 88 where it is not flushed to 0: under 253 u.  Adding
// the bias rounds by u of the sum.
constexpr float kSigmoidError = 5e-7f;
constexpr float kSoftmaxError = 4e-6f;
constexpr float kSoftmaxPart = 1.6e-5f;
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

// The kernel before this one, which may write its inputs, has ended.  (Inputs are
// not __restrict__: their loads could be taken for loads of constants and move
// across the wait.)
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
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
    return key_value(__reduce_max_sync(kAll, order_key(v)));
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
// sum; where a token's scores themselves underflow, through their logarithms
// (whatever the warp's other tokens need).  An only one's share is 1, not its
// product with a reciprocal: the gradient is then 0.
template <int W> __device__ __forceinline__ float share_of(float s, float x, bool on, bool softmax)
{
    float log_s = x, plain = 0.0f;
    bool enough = false;
    if (!softmax) {
        const float total = lanes_sum<W>(on ? s : 0.0f);
        enough = total >= 1e-30f;
        plain = !on ? 0.0f : s == total ? 1.0f : __fdividef(s, total);
        if (__all_sync(kAll, enough)) return plain;
        log_s = fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
    }
    // softmax: the row's other experts cancel
    const float top = lanes_max<W>(on ? log_s : -INFINITY);
    const float q = on ? __expf(log_s - top) : 0.0f;
    const float total = lanes_sum<W>(q);
    return enough ? plain : !on ? 0.0f : q == total ? 1.0f : __fdividef(q, total);
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

// A lane's biases; -inf where no choice can come of one.
template <int P> __device__ __forceinline__ void load_bias(const RouteArgs &a, int lane, float (&bias)[P])
{
#pragma unroll
    for (int j = 0; j < P; ++j) {
        bias[j] = a.bias && lane * P + j < a.experts ? a.bias[lane * P + j] : 0.0f;
        bias[j] = bias[j] > -INFINITY ? bias[j] : -INFINITY;
    }
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

// What two groups' values have to differ by to be told apart in 32 bits:
// four scores' errors and four roundings of sums; `most` bounds the sum of a
// group's best two (which without a bias are scores, whose errors are relative
// too).
__device__ __forceinline__ float groups_margin(const RouteArgs &a, float most)
{
    float errors = 4.0f * (a.softmax ? kSoftmaxError : kSigmoidError);
    if (a.softmax && !a.bias) errors = fminf(errors, 3.0f * kSoftmaxPart * most + 1e-37f);
    return errors + 4.0f * kSumError * most;
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
    // of a choice that is no -0, -inf included
    __device__ static uint32_t make_plain(float v, int expert)
    {
        const uint32_t b = __float_as_uint(v);
        return ((b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) & ~kMask) | (kMask - expert);
    }
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

// What of a row's softmax the weights need.
struct RowSoftmax {
    float top, inverse; // exp(x - top) * inverse
};

// The slow parts below run for a token in some thousands, whose warp the
// kernel then waits for: their loops stay rolled, because fetching code that
// no other warp has run takes longer than running it (unrolled, they were 31
// us of a 74 us kernel).

// Sum of exp(x - top) over a row in 64 bits, in every lane.
template <typename T> __device__ __noinline__ double sum_in_64_bits(const T *row, int experts, float top)
{
    double sum = 0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < experts; e += 32) {
        const float x = load_logit(row + e);
        if (in_reach(x)) sum += exp((double)fminf(x, FLT_MAX) - (double)top);
    }
#pragma unroll 1
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    return sum;
}

// A logit's score in 64 bits (`top` and `sum` of its row's softmax); -inf for
// an expert out of reach.
__device__ __noinline__ double score_in_64_bits(const RouteArgs &a, float x, float top, double sum)
{
    if (!in_reach(x)) return -INFINITY;
    const double e = exp(a.softmax ? (double)fminf(x, FLT_MAX) - (double)top : -(double)fminf(x, FLT_MAX));
    return a.softmax ? e / sum : 1.0 / (1.0 + e);
}

// An expert's choice in 64 bits; -inf where it has none.
template <typename T>
__device__ __noinline__ double choice_in_64_bits(const T *row, const RouteArgs &a, int expert, float top, double sum)
{
    double c = score_in_64_bits(a, load_logit(row + expert), top, sum);
    if (a.bias) c += (double)a.bias[expert];
    return c > -INFINITY ? c : -INFINITY;
}

// The groups kept, where the values around the cut are too close to call
// (`last` the last kept, `cut` the first left out, `margin` their error): the
// groups in between are valued again in 64 bits.  `value`: the groups' values,
// or null to value them all.  Without a bias a group's best are those of the
// largest logits, so only they are scored in 64 bits.
template <typename T>
__device__ __noinline__ uint32_t decide_groups(const T *row, const RouteArgs &a, const float *value, float last, float cut,
                                               float margin, float top)
{
    const int lane = threadIdx.x & 31, per = a.experts / a.groups;
    const float v = value && lane < a.groups ? value[lane] : -INFINITY;
    const bool open = lane < a.groups && (!value || (!(v < cut - margin) && !(v > last + margin) && v > -INFINITY));
    const uint32_t unsure = __ballot_sync(kAll, open);
    const uint32_t in = __ballot_sync(kAll, lane < a.groups && !open && v > last);
    const double sum = a.softmax ? sum_in_64_bits(row, a.experts, top) : 1.0;
    double mine = 0;
    float x1 = -INFINITY, x2 = -INFINITY; // the lane's group's best logits
#pragma unroll 1
    for (uint32_t left = unsure; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        if (!a.bias) {
            float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 1
            for (int i = lane; i < per; i += 32) {
                const float x = load_logit(row + g * per + i);
                const float c = in_reach(x) ? fminf(x, FLT_MAX) : -INFINITY;
                m2 = fmaxf(m2, fminf(m1, c));
                m1 = fmaxf(m1, c);
            }
#pragma unroll 1
            for (int d = 16; d; d >>= 1) join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, d), __shfl_xor_sync(kAll, m2, d));
            if (lane == g) x1 = m1, x2 = a.best > 1 ? m2 : -INFINITY;
        } else {
            double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 1
            for (int i = lane; i < per; i += 32) {
                const double c = choice_in_64_bits(row, a, g * per + i, top, sum);
                m2 = fmax(m2, fmin(m1, c));
                m1 = fmax(m1, c);
            }
#pragma unroll 1
            for (int d = 16; d; d >>= 1) {
                const double o1 = __shfl_xor_sync(kAll, m1, d), o2 = __shfl_xor_sync(kAll, m2, d);
                m2 = fmax(fmin(m1, o1), fmax(m2, o2));
                m1 = fmax(m1, o1);
            }
            if (lane == g) mine = a.best > 1 && m2 > -INFINITY ? m1 + m2 : m1;
        }
    }
    if (!a.bias) {
        mine = score_in_64_bits(a, x1, top, sum);
        if (x2 > -INFINITY) mine += score_in_64_bits(a, x2, top, sum);
    }
    int rank = __popc(in);
#pragma unroll 1
    for (uint32_t left = unsure; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const double o = __shfl_sync(kAll, mine, g);
        rank += o > mine || (o == mine && g < lane);
    }
    return in | __ballot_sync(kAll, open && rank < a.kept);
}

// As decide_groups, from the values of the groups as the lanes have them:
// group g's `value`, if there is `any`, in several lanes or none.
template <typename T>
__device__ __noinline__ uint32_t settle_groups(const T *row, const RouteArgs &a, bool any, int g, float value, float margin,
                                               float top, float *place)
{
    const int lane = threadIdx.x & 31;
    place[lane] = -INFINITY;
    __syncwarp();
    if (any) place[g] = value;
    __syncwarp();
    const float mine = place[lane];
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < a.groups; ++o) {
        const float v = place[o];
        rank += v > mine || (v == mine && o < lane);
    }
    const bool in = lane < a.groups;
    const int last = __ffs(__ballot_sync(kAll, in && rank == a.kept - 1)) - 1;
    const int cut = __ffs(__ballot_sync(kAll, in && rank == a.kept)) - 1;
    const uint32_t kept =
        decide_groups(row, a, place, __shfl_sync(kAll, mine, last), __shfl_sync(kAll, mine, cut), margin, top);
    __syncwarp();
    return kept;
}

// The choice of a row whose order short keys and 32 bits left open, given the
// groups kept and a bound that no chosen expert's choice lies below: the few
// experts from there on, in order by the logits, or with a bias in 64 bits.
// Lane i < k gets the i-th or -1; `lost` where there are too many of them.
template <typename T>
__device__ __noinline__ int choose_from(const T *row, const RouteArgs &a, uint32_t keep, float least, RowSoftmax soft,
                                        int32_t *place, bool &lost)
{
    const int lane = threadIdx.x & 31, per = a.experts / a.groups;
    int n = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        float c = -INFINITY;
        if (e < a.experts && in_reach(load_logit(row + e)) && (a.groups == 1 || ((keep >> (e / per)) & 1u))) {
            c = fminf(load_logit(row + e), FLT_MAX);
            if (a.bias)
                c = (a.softmax ? exp2_fast(kLog2e * (c - soft.top)) * soft.inverse : sigmoid_fast(c)) + a.bias[e];
        }
        const bool in = c > -INFINITY && c >= least;
        const uint32_t mask = __ballot_sync(kAll, in);
        const int at = n + __popc(mask & ((1u << lane) - 1u));
        if (in && at < 32) place[at] = e;
        n += __popc(mask);
    }
    __syncwarp();
    lost = n > 32;
    if (lost) return -1;
    const int expert = lane < n ? place[lane] : -1;
    double c = expert < 0 ? -INFINITY : (double)fminf(load_logit(row + expert), FLT_MAX);
    if (a.bias) { // without one the logits decide
        const double sum = a.softmax ? sum_in_64_bits(row, a.experts, soft.top) : 1.0;
        c = expert < 0 ? -INFINITY : choice_in_64_bits(row, a, expert, soft.top, sum);
    }
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double o = __shfl_sync(kAll, c, i);
        const int oe = __shfl_sync(kAll, expert, i);
        rank += o > c || (o == c && oe < expert);
    }
    __syncwarp();
    if (expert >= 0) place[rank] = expert;
    __syncwarp();
    const int chosen = lane < n && lane < a.k ? place[lane] : -1;
    __syncwarp();
    return chosen;
}

// The whole choice of a row in 64 bits, or without a bias by the logits (heavy
// ties): one expert at a time.  Lane i < k gets the i-th or -1.
template <typename T> __device__ __noinline__ int choose_slowly(const T *row, const RouteArgs &a)
{
    const int lane = threadIdx.x & 31, per = a.experts / a.groups;
    float top = -INFINITY;
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 32) {
        const float x = load_logit(row + e);
        if (in_reach(x)) top = fmaxf(top, fminf(x, FLT_MAX));
    }
    top = warp_max(top);
    const double sum = a.softmax && a.bias ? sum_in_64_bits(row, a.experts, top) : 1.0;
    const uint32_t keep = a.groups > 1 ? decide_groups(row, a, nullptr, 0.0f, 0.0f, 0.0f, top) : 0xFFFFFFFFu;
    double c[kMaxExperts / 32];
#pragma unroll 1
    for (int i = 0, e = lane; e < a.experts; ++i, e += 32) {
        const float x = load_logit(row + e);
        c[i] = -INFINITY;
        if (in_reach(x) && ((keep >> (a.groups > 1 ? e / per : 0)) & 1u))
            c[i] = a.bias ? choice_in_64_bits(row, a, e, top, sum) : (double)fminf(x, FLT_MAX);
    }
    int chosen = -1;
#pragma unroll 1
    for (int round = 0; round < a.k; ++round) {
        double best = -INFINITY;
        int at = kMaxExperts;
#pragma unroll 1
        for (int i = 0, e = lane; e < a.experts; ++i, e += 32)
            if (c[i] > best) {
                best = c[i];
                at = e;
            }
        const int own = at;
#pragma unroll 1
        for (int d = 16; d; d >>= 1) {
            const double o = __shfl_xor_sync(kAll, best, d);
            const int oe = __shfl_xor_sync(kAll, at, d);
            if (o > best || (o == best && oe < at)) {
                best = o;
                at = oe;
            }
        }
        if (!(best > -INFINITY)) break;
        if (own == at) c[at >> 5] = -INFINITY;
        if (lane == round) chosen = at;
    }
    return chosen;
}

// The order of up to 32 experts, one per lane (lanes < n), that short keys
// could not settle: by the logits, or with a bias by the choices, in 64 bits
// where 32 leave neighbours closer than their error.  `c` is the lane's choice
// in 32 bits.  Lane i gets the i-th.
template <typename T>
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
        float top = -INFINITY;
#pragma unroll 1
        for (int e = lane; a.softmax && e < a.experts; e += 32) {
            const float x = load_logit(row + e);
            if (in_reach(x)) top = fmaxf(top, fminf(x, FLT_MAX));
        }
        top = warp_max(top);
        const double sum = a.softmax ? sum_in_64_bits(row, a.experts, top) : 1.0;
        const double d = mine ? choice_in_64_bits(row, a, expert, top, sum) : -INFINITY;
        rank = 0;
#pragma unroll 1
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

// The lanes that value one group, a power of two of them: those that hold it,
// when whole lanes do (`own`); else its members change hands through shared
// memory.
struct GroupLanes {
    bool own;
    int per, lanes;             // experts of a group, lanes that value it
    int group, begin, end;      // the lane's group; the members it looks at, `lanes` apart
    int first_lane, first_left; // of the lane's first expert's group: its first lane, its experts from there on
};

template <int P> __device__ __forceinline__ GroupLanes group_lanes(const RouteArgs &a, int lane)
{
    GroupLanes of;
    of.per = a.experts / a.groups;
    const int whole = of.per / P;
    of.own = of.per % P == 0 && (whole & (whole - 1)) == 0;
    of.lanes = of.own ? whole : 1 << (31 - __clz(32 / a.groups));
    of.group = lane / of.lanes;
    of.begin = of.group * of.per + lane % of.lanes;
    of.end = of.group < a.groups ? (of.group + 1) * of.per : 0;
    const int first = lane * P / of.per;
    of.first_lane = first * of.lanes; // past the last group too, where no key is
    of.first_left = (first + 1) * of.per - lane * P;
    return of;
}

// The choice of one row by a whole warp, from its logits (load_row) in `c`
// (overwritten): lane i < k gets the i-th expert or -1.  A lane sorts its best
// few experts' short keys; k warp maxima over the lanes' best then name the
// choices in order.
template <typename T, int P>
__device__ __forceinline__ int choose_row(const T *row, const RouteArgs &a, float (&c)[P], const float (&bias)[P],
                                          const GroupLanes &of, int32_t *place, float *swap, RowSoftmax &soft)
{
    using Key = ShortKey<P>;
    const int lane = threadIdx.x & 31;
    const bool scored = a.bias || a.groups > 1; // else the logits alone decide
    // errors of a choice: of the score, and relative to the sum with the bias
    const float error = !scored ? 0.0f : a.softmax ? kSoftmaxError : kSigmoidError;
    const float part = scored ? kSumError + 2.0f * Key::kCut : 0.0f;
    soft = {0.0f, 1.0f};
    float &top = soft.top, &inverse = soft.inverse;
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
    if (a.groups > 1) {
        float m1 = -INFINITY, m2 = -INFINITY; // whole values: a cut between groups must not hang on short keys
        if (of.own) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                m2 = fmaxf(m2, fminf(m1, c[j]));
                m1 = fmaxf(m1, c[j]);
            }
        } else { // the groups' members change hands
#pragma unroll
            for (int j = 0; j < P; ++j) swap[lane * P + j + (lane * P >> 5)] = c[j];
            __syncwarp();
            for (int e = of.begin; e < of.end; e += of.lanes) {
                const float v = swap[e + (e >> 5)];
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
            __syncwarp();
        }
        for (int d = 1; d < of.lanes; d <<= 1)
            join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, d), __shfl_xor_sync(kAll, m2, d));
        const bool any = m1 > -INFINITY && of.group < a.groups;
        const uint32_t mine = any ? order_key(group_value(m1, m2, a.best)) : 0u;
        uint32_t left = mine, last = 0;
        for (int g = 0; g < a.kept; ++g) { // equal values go at once; the cut is then not clear
            last = __reduce_max_sync(kAll, left);
            if (left == last) left = 0;
        }
        const uint32_t cut = __reduce_max_sync(kAll, left);
        const float size = any ? fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f) : 0.0f;
        const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
        const float margin = groups_margin(a, most);
        bool keep = any && mine >= last;
        uint32_t kept = __ballot_sync(kAll, keep);
        // too close to call, or of equal values more kept than asked for
        if ((cut && !(key_value(last) - key_value(cut) > margin)) || __popc(kept) > a.kept * of.lanes) {
            kept = settle_groups(row, a, any, of.group, group_value(m1, m2, a.best), margin, top, swap);
            keep = any && ((kept >> of.group) & 1u);
            kept = __ballot_sync(kAll, keep);
        }
        if (of.own) {
#pragma unroll
            for (int j = 0; j < P; ++j) key[j] = keep ? key[j] : 0u;
        } else {
            int at = of.first_lane, left = of.first_left;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (left == 0) {
                    at += of.lanes;
                    left = of.per;
                }
                --left;
                if (!((kept >> (at & 31)) & 1u)) key[j] = 0;
            }
        }
    }
    LaneList<P> list(key);
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
            chosen = settle(row, a, chosen, mine_c, min(n, found), place);
        }
    }
    if (again) chosen = choose_slowly(row, a);
    return chosen;
}

// One warp per token: bound by the instructions of the scan over E logits (two
// special-function ones per sigmoid) and of the k rounds, not by the row's
// bytes.  For what route_quad_kernel does not take.
template <typename T, int P>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<P>) route_kernel(const T *logits, RouteArgs a)
{
    __shared__ int32_t count[kMaxExperts];
    __shared__ int32_t place[kRouteWarps][32];
    __shared__ float swap[kRouteWarps][33 * P];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.load) {
        for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) count[e] = 0;
        __syncthreads();
    }
    grid_dependency_wait();
    float bias[P];
    load_bias<P>(a, lane, bias);
    const GroupLanes of = group_lanes<P>(a, lane);
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
        RowSoftmax soft;
        const int chosen = choose_row<T, P>(row, a, c, bias, of, place[warp], swap[warp], soft);
        // weights of the chosen
        const bool on = lane < a.k && chosen >= 0;
        const float x = on ? fminf(load_logit(row + chosen), FLT_MAX) : 0.0f;
        float w = !on ? 0.0f : a.softmax ? exp2_fast(kLog2e * (x - soft.top)) * soft.inverse : sigmoid_fast(x);
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


// ------------------------------------------------ four lanes per token

constexpr int kQuadExperts = 256; // the most a quad holds: 64 a lane
constexpr int kQuadK = 8;
constexpr int kQuadTokens = 8; // tokens a warp has at a time
constexpr int kQuadGroups = 16;
enum QuadMode { kQuadVec, kQuadElement, kQuadGroup };
static_assert(kQuadExperts == 16 * 16, "sixteen steps of sixteen experts");

// Eight keys into descending order (odd-even merges).
__device__ __forceinline__ void sort8(uint32_t (&k)[8])
{
    constexpr int a[19] = {0, 2, 4, 6, 0, 1, 4, 5, 1, 5, 0, 1, 2, 3, 2, 3, 1, 3, 5};
    constexpr int b[19] = {1, 3, 5, 7, 2, 3, 6, 7, 2, 6, 4, 5, 6, 7, 4, 5, 2, 4, 6};
#pragma unroll
    for (int i = 0; i < 19; ++i) order_pair(k[a[i]], k[b[i]]);
}

// The eight largest of two descending eights, in order, into k; `dropped`
// keeps the largest of those left out.
__device__ __forceinline__ void keep8(uint32_t (&k)[8], const uint32_t (&o)[8], uint32_t &dropped)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t mine = k[i], other = o[7 - i];
        k[i] = max(mine, other);
        dropped = max(dropped, min(mine, other));
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) // bitonic: half-cleaners
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order_pair(k[i], k[i + d]);
}

// A choice's error in 32 bits, but for the sum with its bias.
__device__ __forceinline__ float score_error(bool softmax, float s) { return softmax ? kSoftmaxPart * s : kSigmoidError; }

// Whether an expert that was left out -- short key below `below` -- could
// belong in front of the k-th choice `kth` (expert `ke`, logit `kx`).  Without
// a bias the logits tell; with one, what equals the k-th in logit and bias is
// a tie, and in order.  By the whole warp.
template <typename T>
__device__ __noinline__ bool left_out_matters(const T *row, const RouteArgs &a, uint32_t keep, uint32_t below, float kth,
                                              float kx, int ke, RowSoftmax soft)
{
    using Key = ShortKey<kQuadExperts / 32>;
    const int per = a.experts / a.groups;
    const bool scored = a.bias || a.groups > 1, softmax = a.softmax != 0;
    const float kb = a.bias ? a.bias[ke] : 0.0f;
    const float ks = score_error(softmax, a.bias ? kth - kb : 0.0f);
    bool matters = false;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.experts; e += 32) {
        const float x = load_logit(row + e);
        if (!in_reach(x) || !((keep >> (a.groups > 1 ? e / per : 0)) & 1u)) continue;
        const float z = fminf(x, FLT_MAX);
        const float b = a.bias ? a.bias[e] : 0.0f;
        // c to the last bit as the tokens' lanes have it: its key tells whether it was left out
        const float q = softmax ? exp2_fast(kLog2e * (z - soft.top)) : sigmoid_fast(z);
        const float s = softmax ? q * soft.inverse : q;
        const float c = !scored ? z + 0.0f : softmax ? fmaf(q, soft.inverse, b) : q + b;
        if (!(c > -INFINITY) || Key::make_plain(c, e) >= below) continue;
        if (!a.bias) matters = matters || z > kx;
        else if (z != kx || b != kb)
            matters = matters || !(kth - c > ks + score_error(softmax, s) + kSumError * (fabsf(kth) + fabsf(c)));
    }
    return __any_sync(kAll, matters);
}

// Four lanes per token, eight tokens per warp, for up to 256 experts and k up
// to 8: expert 16 s + 4 l + j is lane l's j-th of step s, so that a token's
// lanes read 16 experts side by side.  Every lane sorts its short keys in
// eights and keeps the best eight, and two exchanges join the four lanes'.
// Against one warp per token the fixed work is shared by eight: 65536 x 256
// fp32 with groups and bias takes 53 us here and took 94 there.  Rows are read
// by aligned vectors of four (kQuadVec) or by elements.  Groups are whole
// steps, valued on the way; or of any size (kQuadGroup, up to 128 experts),
// valued from a copy of the choices in shared memory.
template <typename T, int S, QuadMode kMode>
__global__ void __launch_bounds__(kRouteThreads, 2) route_quad_kernel(const T *logits, RouteArgs a)
{
    constexpr int P = 4 * S;
    constexpr bool kVec = kMode == kQuadVec, kAny = kMode == kQuadGroup;
    static_assert(!kAny || P <= 32, "a lane's experts have a bit each");
    using Key = ShortKey<kQuadExperts / 32>;
    constexpr uint32_t kLeast = 0x00800000u; // keys below: out of reach
    __shared__ int32_t count[kQuadExperts];
    alignas(16) __shared__ float bias[kQuadExperts];
    __shared__ float group[kRouteWarps][kQuadTokens][kQuadGroups];
    __shared__ int32_t place[kRouteWarps][32];
    __shared__ int32_t redone[kRouteWarps][kQuadTokens][kQuadK];
    // kAny: choices (tokens four banks apart), and a lane's experts by group
    alignas(16) __shared__ float value[kAny ? kRouteWarps : 1][kQuadTokens][kAny ? 16 * S + 4 : 4];
    __shared__ uint32_t members[kQuadGroups][4];
    const int per = a.experts / a.groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 3, mine = lane >> 2;
    const bool scored = a.bias || a.groups > 1;
    for (int e = threadIdx.x; e < kQuadExperts; e += kRouteThreads) count[e] = 0;
    grid_dependency_wait();
    for (int e = threadIdx.x; e < kQuadExperts; e += kRouteThreads) {
        const float b = a.bias && e < a.experts ? a.bias[e] : 0.0f;
        bias[e] = b > -INFINITY ? b : -INFINITY; // no choice can come of NaN
    }
    if (kAny)
        for (int m = threadIdx.x; m < 4 * a.groups; m += kRouteThreads) {
            uint32_t bits = 0;
            for (int i = 0; i < P; ++i) {
                const int e = 16 * (i / 4) + 4 * (m & 3) + i % 4;
                bits |= (uint32_t)(e / per == m / 4) << i;
            }
            members[m / 4][m & 3] = bits;
        }
    __syncthreads();
    const int steps_each = a.groups > 1 && !kAny ? per / 16 : S + 1; // steps of a group
    const float error = !scored ? 0.0f : a.softmax ? kSoftmaxError : kSigmoidError;
    // 16-bit logits fit a short key whole: what ties there is a tie
    const bool exact = !scored && sizeof(T) == 2;
    const int64_t step = (int64_t)gridDim.x * kRouteWarps * kQuadTokens;
    for (int64_t t0 = ((int64_t)blockIdx.x * kRouteWarps + warp) * kQuadTokens; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + mine;
        const bool live = t < a.tokens;
        const T *row = logits + (live ? t : t0) * a.row_stride;
        float c[P];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = 16 * s + 4 * sub;
            alignas(16) T x[4];
            const bool in = live && e < a.experts;
            if (kVec && in) {
                if (sizeof(T) == 4) *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(row + e);
                else *reinterpret_cast<uint2 *>(x) = *reinterpret_cast<const uint2 *>(row + e);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (kVec) c[4 * s + j] = in ? load_logit(&x[j]) : -INFINITY;
                else c[4 * s + j] = live && e + j < a.experts ? load_logit(row + e + j) : -INFINITY;
                c[4 * s + j] = in_reach(c[4 * s + j]) ? fminf(c[4 * s + j], FLT_MAX) : -INFINITY;
            }
        }
        float top = 0.0f, inverse = 1.0f;
        if (a.softmax && (scored || !a.renorm)) {
            float m = c[0], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}; // in chains: their error is what the margins count on
#pragma unroll
            for (int i = 1; i < P; ++i) m = fmaxf(m, c[i]);
            top = fmaxf(lanes_max<4>(m), -FLT_MAX);
            if (scored) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float q = exp2_fast(kLog2e * (c[i] - top));
                    sum[i & 3] += q;
                    c[i] = c[i] > -INFINITY ? q : -1.0f; // a score may underflow to 0 and still be chosen
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) sum[i & 3] += exp2_fast(kLog2e * (c[i] - top));
            }
            inverse = reciprocal_fast(lanes_sum<4>((sum[0] + sum[1]) + (sum[2] + sum[3])));
        }
        float most = 0.0f;
        if (scored) {
            float m1 = -INFINITY, m2 = -INFINITY;
            int left = steps_each, g = 0;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float4 b4 = *reinterpret_cast<const float4 *>(bias + 16 * s + 4 * sub);
                const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float &v = c[4 * s + j];
                    if (a.softmax) v = v >= 0.0f ? fmaf(v, inverse, b[j]) : -INFINITY;
                    else v = v > -INFINITY ? sigmoid_fast(v) + b[j] : -INFINITY;
                    if (!kAny) {
                        m2 = fmaxf(m2, fminf(m1, v));
                        m1 = fmaxf(m1, v);
                    }
                }
                if (kAny)
                    *reinterpret_cast<float4 *>(&value[warp][mine][16 * s + 4 * sub]) =
                        make_float4(c[4 * s], c[4 * s + 1], c[4 * s + 2], c[4 * s + 3]);
                else if (--left == 0) { // a group's last step
                    join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, 1), __shfl_xor_sync(kAll, m2, 1));
                    join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, 2), __shfl_xor_sync(kAll, m2, 2));
                    if (sub == 0) group[warp][mine][g] = group_value(m1, m2, a.best);
                    if (m1 > -INFINITY) most = fmaxf(most, fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f));
                    m1 = m2 = -INFINITY;
                    left = steps_each;
                    ++g;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) c[i] += 0.0f; // one zero
        }
        uint32_t keep = 0xFFFFFFFFu;
        if (kAny) {
            __syncwarp();
            for (int g = 0; g < a.groups; ++g) {
                float m1 = -INFINITY, m2 = -INFINITY;
                for (int i = sub; i < per; i += 4) {
                    const float v = value[warp][mine][g * per + i];
                    m2 = fmaxf(m2, fminf(m1, v));
                    m1 = fmaxf(m1, v);
                }
                join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, 1), __shfl_xor_sync(kAll, m2, 1));
                join_best_two(m1, m2, __shfl_xor_sync(kAll, m1, 2), __shfl_xor_sync(kAll, m2, 2));
                if (sub == 0) group[warp][mine][g] = group_value(m1, m2, a.best);
                if (m1 > -INFINITY) most = fmaxf(most, fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f));
            }
        }
        if (a.groups > 1) {
            __syncwarp();
            keep = 0;
            float last = -INFINITY, cut = -INFINITY;
            for (int g = sub; g < a.groups; g += 4) {
                const float v = group[warp][mine][g];
                int rank = 0;
                for (int o = 0; o < a.groups; ++o) {
                    const float u = group[warp][mine][o];
                    rank += u > v || (u == v && o < g);
                }
                if (rank < a.kept) keep |= 1u << g;
                if (rank == a.kept - 1) last = v;
                if (rank == a.kept) cut = v;
            }
            keep |= __shfl_xor_sync(kAll, keep, 1);
            keep |= __shfl_xor_sync(kAll, keep, 2);
            last = lanes_max<4>(last);
            cut = lanes_max<4>(cut);
            const float margin = groups_margin(a, most);
            const bool unsure = live && cut > -INFINITY && !(last - cut > margin);
            for (uint32_t left = __ballot_sync(kAll, unsure) & 0x11111111u; left; left &= left - 1) {
                const int first = __ffs(left) - 1, q = first >> 2;
                const uint32_t kept = decide_groups(
                    logits + (t0 + q) * a.row_stride, a, group[warp][q], __shfl_sync(kAll, last, first),
                    __shfl_sync(kAll, cut, first), __shfl_sync(kAll, margin, first), __shfl_sync(kAll, top, first));
                if (mine == q) keep = kept;
            }
            __syncwarp(); // the groups are read before the next tokens' are written
        }
        uint32_t within = 0; // kAny: the lane's experts in the groups kept
        if (kAny)
            for (int g = 0; g < a.groups; ++g) within |= (keep >> g) & 1u ? members[g][sub] : 0u;
        uint32_t best[8], dropped = 0;
        {
            int left = steps_each, g = 0;
#pragma unroll
            for (int b = 0; b < S / 2; ++b) {
                uint32_t k[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int s = 2 * b + h;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        k[4 * h + j] = (kAny ? within >> (kAny ? 4 * s + j : 0) : keep >> g) & 1u ? Key::make_plain(c[4 * s + j], 16 * s + 4 * sub + j) : 0u;
                    if (--left == 0) {
                        left = steps_each;
                        ++g;
                    }
                }
                sort8(k);
                if (b == 0)
#pragma unroll
                    for (int i = 0; i < 8; ++i) best[i] = k[i];
                else keep8(best, k, dropped);
            }
        }
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_xor_sync(kAll, best[i], d);
            const uint32_t od = __shfl_xor_sync(kAll, dropped, d);
            dropped = max(dropped, od);
            keep8(best, o, dropped);
        }
        // places 2 sub and 2 sub + 1: experts, logits, scores and whole choices
        const uint32_t k0 = sub == 0 ? best[0] : sub == 1 ? best[2] : sub == 2 ? best[4] : best[6];
        const uint32_t k1 = sub == 0 ? best[1] : sub == 1 ? best[3] : sub == 2 ? best[5] : best[7];
        int e0 = k0 >= kLeast ? Key::expert(k0) : -1, e1 = k1 >= kLeast ? Key::expert(k1) : -1;
        float x0 = e0 >= 0 ? fminf(load_logit(row + e0), FLT_MAX) : 0.0f;
        float x1 = e1 >= 0 ? fminf(load_logit(row + e1), FLT_MAX) : 0.0f;
        bool again = false, edge = false; // open: the order of the chosen, and what they leave out
        float least = -FLT_MAX;           // nothing below it is chosen
        float kth = -INFINITY, kx = 0.0f; // the k-th choice, its logit and expert
        int ke = -1;
        const auto score = [&](float x) { return a.softmax ? exp2_fast(kLog2e * (x - top)) * inverse : sigmoid_fast(x); };
        if (!exact) {
            // (without a bias the logits are the order, whatever the keys hold)
            float c0 = e0 < 0 ? -INFINITY : a.bias ? score(x0) + bias[e0] : x0;
            float c1 = e1 < 0 ? -INFINITY : a.bias ? score(x1) + bias[e1] : x1;
            float next = __shfl_down_sync(kAll, c0, 1, 4);
            if (__any_sync(kAll, c1 > c0 || (sub < 3 && next > c1))) { // the short keys hid an order
                for (int pass = 0; pass < 4; ++pass) { // odd-even exchanges; equal choices keep theirs (the index's)
                    if (c1 > c0) {
                        const float tc = c0, tx = x0;
                        const int te = e0;
                        c0 = c1, x0 = x1, e0 = e1;
                        c1 = tc, x1 = tx, e1 = te;
                    }
                    const float nc = __shfl_down_sync(kAll, c0, 1, 4), nx = __shfl_down_sync(kAll, x0, 1, 4);
                    const float pc = __shfl_up_sync(kAll, c1, 1, 4), px = __shfl_up_sync(kAll, x1, 1, 4);
                    const int ne = __shfl_down_sync(kAll, e0, 1, 4), pe = __shfl_up_sync(kAll, e1, 1, 4);
                    const bool give = sub < 3 && nc > c1, take = sub > 0 && c0 > pc;
                    if (give) c1 = nc, x1 = nx, e1 = ne;
                    if (take) c0 = pc, x0 = px, e0 = pe;
                }
                next = __shfl_down_sync(kAll, c0, 1, 4);
            }
            const int last = (a.k - 1) / 2; // the k-th choice's lane
            kth = __shfl_sync(kAll, (a.k & 1) ? c0 : c1, last, 4);
            kx = __shfl_sync(kAll, (a.k & 1) ? x0 : x1, last, 4);
            ke = __shfl_sync(kAll, (a.k & 1) ? e0 : e1, last, 4);
            // Still too close: neighbours up to the k-th, the k-th and any
            // behind it (whose errors may be larger than its neighbour's),
            // unless they are one choice twice (same logit, same bias: a tie,
            // and in order), or a choice left out.
            const auto close = [&](float u, float w, float errors) {
                return w > -INFINITY && !(u - w > errors + (scored ? kSumError : 0.0f) * (fabsf(u) + fabsf(w)));
            };
            if (a.bias) {
                const float r0 = e0 < 0 ? 0.0f : score_error(a.softmax != 0, c0 - bias[e0]);
                const float r1 = e1 < 0 ? 0.0f : score_error(a.softmax != 0, c1 - bias[e1]);
                const float rn = __shfl_down_sync(kAll, r0, 1, 4);
                const float xn = __shfl_down_sync(kAll, x0, 1, 4);
                const int en = __shfl_down_sync(kAll, e0, 1, 4);
                const float kb = ke < 0 ? 0.0f : bias[ke], kr = score_error(a.softmax != 0, kth - kb);
                const int at = 2 * sub;
                if (at + 1 < a.k && close(c0, c1, r0 + r1)) again = x0 != x1 || bias[e0] != bias[e1];
                if (at + 2 < a.k && close(c1, next, r1 + rn)) again = again || x1 != xn || bias[e1] != bias[en];
                if (at >= a.k && close(kth, c0, kr + r0)) again = again || kx != x0 || kb != bias[e0];
                if (at + 1 >= a.k && close(kth, c1, kr + r1)) again = again || kx != x1 || kb != bias[e1];
            }
            if (kth > -INFINITY) least = a.bias && kth < INFINITY ? kth - 3.0f * error - 3.0f * kSumError * fabsf(kth) : kth;
            // anything left out has at most the largest value of its short key
            edge = ke >= 0 && dropped >= kLeast &&
                   close(a.bias || !scored ? kth : score(kx), key_value(dropped | Key::kMask), 2.0f * error);
        }
        // a token's bit in its first lane
        const auto by_token = [&](uint32_t lanes) {
            lanes |= lanes >> 1;
            return (lanes | lanes >> 2) & 0x11111111u;
        };
        uint32_t redo = by_token(__ballot_sync(kAll, (again || edge) && live));
        if (redo) {
            const uint32_t order = by_token(__ballot_sync(kAll, again && live));
            for (uint32_t left = redo; left; left &= left - 1) {
                const int first = __ffs(left) - 1, q = first >> 2;
                const T *other = logits + (t0 + q) * a.row_stride;
                const RowSoftmax soft = {__shfl_sync(kAll, top, first), __shfl_sync(kAll, inverse, first)};
                const uint32_t kept = __shfl_sync(kAll, keep, first);
                bool lost;
                int chosen = choose_from(other, a, kept, __shfl_sync(kAll, least, first), soft, place[warp], lost);
                if (lost) { // heavy ties: are they only that?
                    const float u = __shfl_sync(kAll, kth, first), x = __shfl_sync(kAll, kx, first);
                    const int e = __shfl_sync(kAll, ke, first);
                    if (!left_out_matters(other, a, kept, __shfl_sync(kAll, best[7], first), u, x, e, soft) &&
                        !((order >> first) & 1u)) {
                        redo &= ~(1u << first);
                        continue;
                    }
                    chosen = choose_slowly(other, a);
                }
                if (lane < kQuadK) redone[warp][q][lane] = chosen;
                __syncwarp();
            }
            if ((redo >> (4 * mine)) & 1u) {
                e0 = redone[warp][mine][2 * sub];
                e1 = redone[warp][mine][2 * sub + 1];
                x0 = e0 >= 0 ? fminf(load_logit(row + e0), FLT_MAX) : 0.0f;
                x1 = e1 >= 0 ? fminf(load_logit(row + e1), FLT_MAX) : 0.0f;
            }
            __syncwarp();
        }
        // weights of the two
        const bool on0 = live && 2 * sub < a.k && e0 >= 0, on1 = live && 2 * sub + 1 < a.k && e1 >= 0;
        float w0, w1;
        if (a.softmax && a.renorm) { // the row's other experts cancel
            const float lead = lanes_max<4>(fmaxf(on0 ? x0 : -FLT_MAX, on1 ? x1 : -FLT_MAX));
            w0 = on0 ? exp2_fast(kLog2e * (x0 - lead)) : 0.0f;
            w1 = on1 ? exp2_fast(kLog2e * (x1 - lead)) : 0.0f;
        } else {
            w0 = on0 ? score(x0) : 0.0f;
            w1 = on1 ? score(x1) : 0.0f;
        }
        if (a.renorm) {
            float sum = lanes_sum<4>(w0 + w1);
            if (__any_sync(kAll, sum < 1e-30f)) { // scores that underflow (or none chosen): by their logarithms
                const float l0 = on0 ? fminf(x0, 0.0f) - log1pf(expf(-fabsf(x0))) : -FLT_MAX;
                const float l1 = on1 ? fminf(x1, 0.0f) - log1pf(expf(-fabsf(x1))) : -FLT_MAX;
                const float lead = lanes_max<4>(fmaxf(l0, l1));
                const float v0 = on0 ? __expf(l0 - lead) : 0.0f, v1 = on1 ? __expf(l1 - lead) : 0.0f;
                const float all = lanes_sum<4>(v0 + v1);
                if (sum < 1e-30f) {
                    w0 = v0;
                    w1 = v1;
                    sum = all;
                }
            }
            w0 = on0 ? __fdividef(w0, sum) : 0.0f;
            w1 = on1 ? __fdividef(w1, sum) : 0.0f;
        }
        if (live) {
            const int64_t o = t * a.k + 2 * sub;
            if (2 * sub < a.k) {
                a.idx[o] = on0 ? e0 : -1;
                a.weight[o] = w0 * a.scale;
            }
            if (2 * sub + 1 < a.k) {
                a.idx[o + 1] = on1 ? e1 : -1;
                a.weight[o + 1] = w1 * a.scale;
            }
            if (a.load) {
                if (on0) atomicAdd(&count[e0], 1);
                if (on1) atomicAdd(&count[e1], 1);
            }
        }
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
route_grad_kernel(const T *logits, T *__restrict__ out, RouteGradArgs a)
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
route_softmax_grad_kernel(const T *logits, T *__restrict__ out, RouteGradArgs a)
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
        for (int j = 0; j < P; ++j) s[j] = s[j] > 0.0f ? -dot * (s[j] / total) : 0.0f; // 0 times an infinite dot too
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

template <typename T, QuadMode kMode> RouteKernel<T> quad_kernel_for(int experts)
{
    if (experts <= 32) return route_quad_kernel<T, 2, kMode>;
    if (experts <= 64) return route_quad_kernel<T, 4, kMode>;
    if (experts <= 128) return route_quad_kernel<T, 8, kMode>;
    if constexpr (kMode != kQuadGroup) return route_quad_kernel<T, 16, kMode>;
    return nullptr;
}

// Whether four lanes per token do: experts, groups and k that fit their layout,
// and so many tokens per SM that they beat a warp per token.  Eight warps of
// eight tokens are a CTA, so that up to 64 tokens per SM some SMs have none; a
// quad's time hardly grows until then, a warp's does from the first.  Both (us,
// four lanes / a warp per token, on 152 SMs, in a graph; with a bias a few of the
// rows are settled in 64 bits, which 3 to 6 us depend on):
//   tokens                       1216      2432      3648      6080      9728
//   60 fp16, k 4                 2.9/3.2   2.9/3.8   2.9/4.6   3.0/6.0   3.0/7.4
//   128 bf16, k 8                4.1/3.9   4.2/5.0   4.2/6.5   4.3/8.0   4.3/10
//   256 bf16, k 8                6.7/4.8   6.7/6.3   6.8/7.9   6.9/10    7.0/13
//   128 fp32, bias, k 8          8.7/4.4   8.5/5.4   8.7/6.5   9.1/9.8   9.3/12
//   256 fp32, bias, 8 groups     8.8/6.1    14/8.2    15/11     15/14     15/17
bool quads_fit(const RouteArgs &a, int sm_count)
{
    const int64_t each = a.bias || a.groups > 1 ? 40 : a.experts > 128 ? 16 : 8;
    return a.experts <= kQuadExperts && a.k <= kQuadK && a.groups <= kQuadGroups &&
           (a.groups == 1 || a.experts / a.groups % 16 == 0 || a.experts <= 128) && a.tokens >= sm_count * each;
}

template <typename T> cudaError_t launch_route(const void *logits, RouteArgs a, int sm_count, void *stream)
{
    if (quads_fit(a, sm_count)) {
        cudaLaunchAttribute attr[1];
        const int64_t warps = (a.tokens + kQuadTokens - 1) / kQuadTokens;
        const cudaLaunchConfig_t cfg =
            route_config(route_grid(warps, sm_count, 2), static_cast<cudaStream_t>(stream), attr);
        const bool vec = a.experts % 4 == 0 && a.row_stride % 4 == 0 &&
                         (reinterpret_cast<uintptr_t>(logits) & (4 * sizeof(T) - 1)) == 0;
        const auto kernel = a.groups > 1 && a.experts / a.groups % 16 ? quad_kernel_for<T, kQuadGroup>(a.experts)
                            : vec                                     ? quad_kernel_for<T, kQuadVec>(a.experts)
                                                                      : quad_kernel_for<T, kQuadElement>(a.experts);
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(logits), a);
    }
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
