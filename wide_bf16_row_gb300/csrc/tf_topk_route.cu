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
// Errors of the 32-bit scores, rounded up: a score is within 2e-6 of its
// value (exp2 of a rounded product, a sum of at most kMaxExperts of them, a
// reciprocal: under 8 * 2^-23 for a score of at most 1, with |x| s(1 - s) <=
// 0.23 and |x| exp(-|x|) <= 0.37 bounding the share of the rounded exponent),
// and adding the bias rounds by 2^-24 of the sum.
constexpr float kScoreError = 2e-6f;
constexpr float kSumError = 1.2e-7f;

static_assert(kMaxRouteK <= 32, "a lane per chosen expert");
static_assert(kMaxExperts == 32 * 32, "at most 32 experts a lane");

struct RouteArgs {
    int64_t tokens, row_stride;
    int32_t experts, k, softmax, groups, kept, best, renorm;
    float scale;
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

// The chosen scores of one row (lane i holds the i-th, or `on` false) divided
// by their sum; where the scores themselves underflow, through their
// logarithms.
__device__ __forceinline__ float share_of(float s, float x, bool on, bool softmax)
{
    if (softmax) { // exp(x_i) / sum over the chosen exp(x_j): the row's other experts cancel
        const float top = warp_max(on ? x : -INFINITY);
        const float q = on ? expf(x - top) : 0.0f;
        const float total = warp_sum(q);
        return on ? q / total : 0.0f;
    }
    const float total = warp_sum(on ? s : 0.0f);
    if (total >= 1e-30f) return on ? s / total : 0.0f;
    const float log_s = fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
    const float top = warp_max(on ? log_s : -INFINITY);
    const float q = on ? expf(log_s - top) : 0.0f;
    const float sum = warp_sum(q);
    return on ? q / sum : 0.0f;
}

template <typename T, int P>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const T *__restrict__ logits, RouteArgs a)
{
    __shared__ int32_t count[kMaxExperts];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.load) {
        for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) count[e] = 0;
        __syncthreads();
    }
    grid_dependency_wait();
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T *row = logits + t * a.row_stride;
        float x[P], s[P];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = lane * P + j;
            x[j] = e < a.experts ? fminf(load_logit(row + e), FLT_MAX) : -INFINITY;
            if (e < a.experts && isnan(load_logit(row + e))) x[j] = -INFINITY;
            top = fmaxf(top, x[j]);
        }
        float total = 1.0f;
        if (a.softmax) {
            top = warp_max(top);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                s[j] = in_reach(x[j]) ? __expf(x[j] - top) : 0.0f;
                sum += s[j];
            }
            total = warp_sum(sum);
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = s[j] / total;
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = __frcp_rn(1.0f + __expf(-x[j]));
        }
        // the order that decides: the biased scores, or the logits alone
        uint32_t key[P];
        float c[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            c[j] = s[j] + (a.bias && in_reach(x[j]) ? a.bias[lane * P + j] : 0.0f);
            const float v = a.bias ? c[j] : x[j];
            key[j] = in_reach(x[j]) && c[j] > -INFINITY ? order_key(v) : 0u;
        }
        bool again = false; // too close to call in 32 bits
        if (a.groups > 1) {
            const int per = a.experts / a.groups;
            uint32_t mine = 0;
            float size = 0.0f; // of the largest terms added up
            for (int g = 0; g < a.groups; ++g) {
                uint32_t members[P];
#pragma unroll
                for (int j = 0; j < P; ++j)
                    members[j] = key[j] && (lane * P + j) / per == g ? order_key(c[j]) : 0u;
                int e;
                const uint32_t first = take_best<P>(members, lane, e);
                const uint32_t second = a.best > 1 && first ? take_best<P>(members, lane, e) : 0u;
                const float u = first ? key_value(first) : 0.0f, w = second ? key_value(second) : 0.0f;
                if (lane == g) mine = first ? order_key(u + w) : 0u;
                size = fmaxf(size, fabsf(u) + fabsf(w));
            }
            uint32_t last, cut;
            const uint32_t keep = best_groups<uint32_t>(mine, a.groups, a.kept, lane, last, cut);
            // two scores, their biases and their sum on either side of the cut
            if (cut) again = !(key_value(last) - key_value(cut) > 4.0f * kScoreError + 4.0f * kSumError * size);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int e = lane * P + j;
                if (e < a.experts && !((keep >> (e / per)) & 1u)) key[j] = 0;
            }
        }
        int chosen = -1;
        float value = 0.0f;
        for (int i = 0; i < a.k; ++i) {
            int e;
            const uint32_t best = take_best<P>(key, lane, e);
            if (best == 0) break;
            if (lane == i) {
                chosen = e;
                value = key_value(best);
            }
        }
        if (a.bias) {
            int past; // the neighbour past the cut
            const float past_value = key_value(take_best<P>(key, lane, past));
            int en = __shfl_down_sync(kAll, chosen, 1);
            float vn = __shfl_down_sync(kAll, value, 1);
            if (lane == a.k - 1) {
                en = past;
                vn = past_value;
            }
            bool close = false;
            if (lane < a.k && chosen >= 0 && en >= 0 &&
                !(value - vn > 2.0f * kScoreError + kSumError * (fabsf(value) + fabsf(vn))))
                close = load_logit(row + chosen) != load_logit(row + en) || a.bias[chosen] != a.bias[en];
            again = again || __any_sync(kAll, close);
        }
        if (again) chosen = choose_in_64_bits<T, P>(row, a);
        // weights of the chosen
        const bool on = lane < a.k && chosen >= 0;
        const float xi = on ? fminf(load_logit(row + chosen), FLT_MAX) : 0.0f;
        const float si = !on ? 0.0f : a.softmax ? expf(xi - top) / total : 1.0f / (1.0f + expf(-xi));
        const float w = a.renorm ? share_of(si, xi, on, a.softmax != 0) : si;
        if (lane < a.k) {
            a.idx[t * a.k + lane] = on ? chosen : -1;
            a.weight[t * a.k + lane] = on ? w * a.scale : 0.0f;
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
    const int32_t *idx;
    const float *grad;
};

__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Gradient of the weights for the logits, one warp per token:
//   per chosen score  g_i = scale * dw_i, renormalised: (g_i - sum_j g_j r_j) / S
//                     with r_j = s_j / S, S the chosen scores' sum;
//   sigmoid  dx_i = g_i s_i (1 - s_i), others 0;
//   softmax  dx_e = s_e (g_e - sum_j g_j s_j), g_e = 0 for the others -- and
//            with renormalised weights that sum is 0, so only the chosen
//            experts' logits are read.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads)
route_grad_kernel(const T *__restrict__ logits, T *__restrict__ out, RouteGradArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T *row = logits + t * a.row_stride;
        T *dst = out + t * a.experts;
        int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
        float x = e >= 0 && e < a.experts ? load_logit(row + e) : -INFINITY;
        const bool on = in_reach(x);
        x = fminf(x, FLT_MAX);
        float g = on ? a.scale * a.grad[t * a.k + lane] : 0.0f;
        float d; // the chosen expert's gradient
        const float below = on && !a.softmax ? 1.0f / (1.0f + expf(x)) : 1.0f; // 1 - s
        float dot = 0.0f, top = 0.0f, total = 1.0f;
        if (a.renorm) {
            const float s = on && !a.softmax ? 1.0f / (1.0f + expf(-x)) : 0.0f;
            const float r = share_of(s, x, on, a.softmax != 0);
            dot = warp_sum(on ? g * r : 0.0f);
            d = r * (g - dot) * below;
        } else if (!a.softmax) {
            d = on ? g * below / (1.0f + expf(-x)) : 0.0f;
        } else {
            float m = -INFINITY;
            for (int i = lane; i < a.experts; i += 32) {
                const float y = load_logit(row + i);
                if (in_reach(y)) m = fmaxf(m, fminf(y, FLT_MAX));
            }
            top = warp_max(m);
            float sum = 0.0f;
            for (int i = lane; i < a.experts; i += 32) {
                const float y = load_logit(row + i);
                if (in_reach(y)) sum += expf(fminf(y, FLT_MAX) - top);
            }
            total = warp_sum(sum);
            const float s = on ? expf(x - top) / total : 0.0f;
            dot = warp_sum(on ? g * s : 0.0f);
            d = on ? s * (g - dot) : 0.0f;
        }
        if (a.softmax && !a.renorm) {
            for (int i = lane; i < a.experts; i += 32) {
                const float y = load_logit(row + i);
                store_grad(dst + i, in_reach(y) ? -dot * (expf(fminf(y, FLT_MAX) - top) / total) : 0.0f);
            }
        } else {
            for (int i = lane; i < a.experts; i += 32) store_grad(dst + i, 0.0f);
        }
        __syncwarp(); // the chosen experts' values replace those of the pass above
        // an expert named twice (a list this library never writes) adds up
        const uint32_t twins = __match_any_sync(kAll, on ? e : -1 - lane);
        if (__any_sync(kAll, on && (twins & (twins - 1)) != 0)) {
            const float extra = a.softmax && !a.renorm && on ? -dot * (expf(x - top) / total) : 0.0f;
            float sum = 0.0f; // each twin's own part, the shared part once
            for (int i = 0; i < a.k; ++i) {
                const float o = __shfl_sync(kAll, d - extra, i);
                if ((twins >> i) & 1u) sum += o;
            }
            d = sum + extra;
        }
        if (on && lane == __ffs(twins) - 1) store_grad(dst + e, d);
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

int64_t route_grid(int64_t tokens, int sm_count)
{
    const int64_t need = (tokens + kRouteWarps - 1) / kRouteWarps;
    const int64_t most = (int64_t)sm_count * 8;
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

template <typename T> cudaError_t launch_route(const void *logits, const RouteArgs &a, int sm_count, void *stream)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = route_config(route_grid(a.tokens, sm_count), static_cast<cudaStream_t>(stream), attr);
    return cudaLaunchKernelEx(&cfg, route_kernel_for<T>(a.experts), static_cast<const T *>(logits), a);
}

template <typename T>
cudaError_t launch_route_grad(const void *logits, void *out, const RouteGradArgs &a, int sm_count, void *stream)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = route_config(route_grid(a.tokens, sm_count), static_cast<cudaStream_t>(stream), attr);
    return cudaLaunchKernelEx(&cfg, route_grad_kernel<T>, static_cast<const T *>(logits), static_cast<T *>(out), a);
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
