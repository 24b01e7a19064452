// Tokens sorted by expert and back for GB300 (sm_103a): the way from
// tf_topk_route's choices to the experts' rows and from the experts' results
// to the tokens.
//
// What is computed, for tokens t with k choices idx[t][j] of E experts
// (choices outside [0, E) take no part), N = tokens * k, f = t * k + j:
//   order     the taking-part f's sorted by expert, and by f within an expert:
//             source[s] = f, slot[f] = s, offsets[e] = how many belong to
//             experts below e;
//   gather    rows[s] = x[source[s] / k], or in 8 bits with a scale per 128;
//   combine   out[t] = sum_j weight[t][j] * y[slot[t][j]];
//   gradients of both: d_y[s] = weight * d_out[t], d_weight[t][j] =
//             <d_out[t], y[s]>, d_x[t] = sum_j d_rows[slot[t][j]].
// Rows behind offsets[E] are written as zeros, so that nothing undefined is
// ever handed on.
//
// All of it is bound by bytes.  The kernels go by token, not by sorted row: a
// token's row is read once and written k times, or k rows are read and one is
// written, and no row is touched by two warps at once, so that there are no
// atomics and the same inputs give the same bits.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "tf_topk.h"

int tf_topk_internal_fail_cuda(int cuda_error);
int tf_topk_internal_device(int *sm_count);

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxExperts = TF_TOPK_ROUTE_MAX_EXPERTS;
constexpr int kMaxK = TF_TOPK_ROUTE_MAX_K;
constexpr int kMaxDim = 1 << 30; // so that the last step past a row's end still fits 32 bits
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 2048; // choices a CTA sorts at least, where there are several CTAs
constexpr int kSortKept = 4;     // choices a thread keeps in registers
// Choices that one CTA sorts by itself, in one launch and without a workspace.  One
// CTA / several (us, 256 experts): 2048 choices 7.4 (one chunk), 4096 11.3/8.1, 8192
// 19.5/8.5, 16384 35.5/9.7; with 16 experts 7.0/5.8, 10.9/6.0 and 18.8/7.2.
constexpr int kSortAlone = 8192;
constexpr int kRowWarps = 8;     // warps per CTA of the kernels over rows
constexpr int kRowThreads = 32 * kRowWarps;
// Gradient of combine: vectors that a thread has on their way, and CTAs of an SM, so
// many that their warps hide the latency as far as the registers go.  Whole vectors
// (16384 x 2048 bf16, k 8): 184 us with four CTAs, 169 with six.  Pairs (5001 x 1002
// bf16, k 3): 12.9 with four at a time and four CTAs, 16.2 with two and six.  Single
// elements (5001 x 1001 fp32; 40000 x 2049 bf16, k 6): 29.4 and 730 with four and
// four, 27.7 and 646 with two and six.
template <typename T, int kN> constexpr int kGradVecs = kN * sizeof(T) >= 16 ? 1 : kN > 1 ? 4 : 2;
template <typename T, int kN> constexpr int kGradCtas = kGradVecs<T, kN> == 4 ? 4 : 6;
constexpr int kScaleBlock = TF_TOPK_FP8_BLOCK;

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- the order

struct SortArgs {
    const int32_t *idx;
    int32_t *slot, *source, *offsets;
    int32_t *counts; // [chunks][experts], where there are several chunks
    int64_t n;
    int64_t chunk; // choices of a chunk, a multiple of 32 * kSortWarps
    int32_t experts;
};

// Counts of the experts in each chunk.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a)
{
    __shared__ int32_t count[kMaxExperts];
    grid_dependency_wait();
    grid_dependents_go();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * a.chunk, end = min(a.n, begin + a.chunk);
    for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
        const int e = a.idx[i];
        if ((uint32_t)e < (uint32_t)a.experts) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// A stable counting sort.  Each warp of a CTA owns consecutive choices, so
// that "before" means a lower chunk, a lower warp, an earlier step of 32 or a
// lower lane, in this order: the counts of the lower chunks, the prefix of the
// warps' counts, a running count, and the lanes with the same expert
// (match_any) give the place.  4 bytes are read per choice and 8 written; what it
// takes is the latency of its few steps, so a thread's first choices stay in
// registers, several counts are on their way at a time, and where the counts
// come from the kernel before, the CTA counts for itself while that runs.
template <bool kAlone> __global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a)
{
    extern __shared__ int32_t place[]; // [warps][experts]: counts, then the next place of each warp's choices
    __shared__ int32_t warp_sum[kSortWarps];
    __shared__ int32_t used;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // (the kernel that counts has waited for what comes before it, idx among it)
    if (kAlone) {
        grid_dependency_wait();
        grid_dependents_go();
    }
    const int64_t begin = blockIdx.x * a.chunk, end = min(a.n, begin + a.chunk);
    const int64_t share = ((end - begin + kSortWarps - 1) / kSortWarps + 31) / 32 * 32; // of a warp
    const int warps = (int)((end - begin + share - 1) / share);                         // that have any
    const int64_t w0 = begin + warp * share, w1 = min(end, w0 + share);
    int kept[kSortKept];
#pragma unroll
    for (int s = 0; s < kSortKept; ++s) kept[s] = w0 + 32 * s + lane < w1 ? a.idx[w0 + 32 * s + lane] : -1;
    for (int i = tid; i < warps * a.experts; i += kSortThreads) place[i] = 0;
    __syncthreads();
    int32_t *mine = place + warp * a.experts;
    // body(place in the order of the choices, expert or -1, lanes with the same) for the warp's choices
    const auto each_step = [&](auto body) {
        const auto step = [&](int64_t f, int e) {
            const int expert = (uint32_t)e < (uint32_t)a.experts ? e : -1;
            body(f, expert, __match_any_sync(kAll, expert));
        };
#pragma unroll
        for (int s = 0; s < kSortKept; ++s)
            if (w0 + 32 * s < w1) step(w0 + 32 * s + lane, kept[s]);
        for (int64_t i = w0 + 32 * kSortKept; i < w1; i += 32) step(i + lane, i + lane < w1 ? a.idx[i + lane] : -1);
    };
    const uint32_t lower_lanes = (1u << lane) - 1;
    each_step([&](int64_t, int e, uint32_t same) {
        if (e >= 0 && (same & lower_lanes) == 0) mine[e] += __popc(same);
        __syncwarp();
    });
    __syncthreads();
    if (!kAlone) {
        grid_dependency_wait();
        grid_dependents_go();
    }
    // thread e: the expert's choices in lower chunks and in all
    int32_t before = 0, total = 0;
    if (tid < a.experts) {
        if (kAlone) {
            for (int w = 0; w < warps; ++w) total += place[w * a.experts + tid];
        } else {
#pragma unroll 32
            for (int c = 0; c < (int)gridDim.x; ++c) {
                const int32_t v = a.counts[(int64_t)c * a.experts + tid];
                total += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
        }
    }
    int32_t upto = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int32_t s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(kAll, s, d);
            if (lane >= d) s += o;
        }
        warp_sum[lane] = s;
        if (lane == 31) used = s;
    }
    __syncthreads();
    const int32_t start = upto - total + (warp ? warp_sum[warp - 1] : 0); // of the expert's rows
    if (tid < a.experts) {
        int32_t at = start + before;
        for (int w0 = 0; w0 < warps; w0 += 8) { // eight counts on their way at a time
            int32_t v[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) v[w] = w0 + w < warps ? place[(w0 + w) * a.experts + tid] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) place[(w0 + w) * a.experts + tid] = at;
                at += v[w];
            }
        }
        if (blockIdx.x == 0) {
            a.offsets[tid] = start;
            if (tid == 0) a.offsets[a.experts] = used;
        }
    }
    __syncthreads();
    each_step([&](int64_t f, int e, uint32_t same) {
        const int lower = __popc(same & lower_lanes);
        const int32_t s = e >= 0 ? mine[e] + lower : -1;
        __syncwarp();
        if (e >= 0 && lower == 0) mine[e] += __popc(same);
        __syncwarp();
        if (f < w1) a.slot[f] = s;
        if (e >= 0) a.source[s] = (int32_t)f;
    });
    for (int64_t s = begin + tid; s < end; s += kSortThreads)
        if (s >= used) a.source[s] = -1;
}

// ---------------------------------------------------------------- vectors of a row

// kN elements of T, read and written at once (kN * sizeof(T) is 16, 4 or 2).
template <int kBytes> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int kN> struct Vec {
    union {
        typename Raw<kN * sizeof(T)>::type raw;
        T v[kN];
    };
    __device__ Vec() {}
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float &to, float x) { to = x; }
__device__ __forceinline__ void put(__half &to, float x) { to = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 &to, float x) { to = __float2bfloat16_rn(x); }

template <typename T, int kN> __device__ __forceinline__ Vec<T, kN> load(const T *p)
{
    Vec<T, kN> v;
    v.raw = *reinterpret_cast<const typename Raw<kN * sizeof(T)>::type *>(p);
    return v;
}
template <typename T, int kN> __device__ __forceinline__ void store(T *p, const Vec<T, kN> &v)
{
    *reinterpret_cast<typename Raw<kN * sizeof(T)>::type *>(p) = v.raw;
}
template <typename T, int kN> __device__ __forceinline__ Vec<T, kN> zeros()
{
    Vec<T, kN> v;
#pragma unroll
    for (int i = 0; i < kN; ++i) put(v.v[i], 0.0f);
    return v;
}

// body(row) for the rows that no choice has, a warp per row, shared out evenly:
// they lie together behind the last expert's.
template <typename F> __device__ __forceinline__ void unused_rows(const int32_t *source, int64_t n, F body)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * kRowWarps, me = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    for (int64_t first = me; first < n; first += 32 * warps) {
        const int64_t s = first + lane * warps;
        uint32_t none = __ballot_sync(kAll, s < n && source[s] < 0);
        for (; none; none &= none - 1) body(first + (__ffs(none) - 1) * warps);
    }
}

// ---------------------------------------------------------------- gather

struct GatherArgs {
    const int32_t *slot, *source;
    int64_t tokens, n;
    int64_t stride; // of x
    int32_t dim, k;
    int32_t segments; // of a row, kSegment vectors each
};

constexpr int kStep = 4; // vectors a lane has in flight

// A warp copies a segment of a token's row to its k places.
template <typename T, int kN> __global__ void __launch_bounds__(kRowThreads) gather_kernel(const T *x, T *out, GatherArgs a)
{
    grid_dependency_wait();
    grid_dependents_go();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t units = a.tokens * a.segments, warps = (int64_t)gridDim.x * kRowWarps;
    const int vecs = a.dim / kN;
    for (int64_t u = (int64_t)blockIdx.x * kRowWarps + warp; u < units; u += warps) {
        const int64_t t = u / a.segments;
        const int first = (int)(u - t * a.segments) * 32 * kStep + lane;
        const int32_t s = lane < a.k ? a.slot[t * a.k + lane] : -1;
        Vec<T, kN> v[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            if (first + 32 * i < vecs) v[i] = load<T, kN>(x + t * a.stride + (int64_t)(first + 32 * i) * kN);
        for (int j = 0; j < a.k; ++j) {
            const int64_t to = __shfl_sync(kAll, s, j);
            if (to < 0 || to >= a.n) continue;
#pragma unroll
            for (int i = 0; i < kStep; ++i)
                if (first + 32 * i < vecs) store(out + to * a.dim + (int64_t)(first + 32 * i) * kN, v[i]);
        }
    }
    unused_rows(a.source, a.n, [&](int64_t s) {
        for (int c = lane; c < vecs; c += 32) store(out + s * a.dim + (int64_t)c * kN, zeros<T, kN>());
    });
}

// ---------------------------------------------------------------- rows in 8 bits

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A warp turns kQuantVecs times 32 * kN values of a token's row into e4m3 with
// their scales, and writes them to the row's places, or to the row's own where
// there is no order.  The largest magnitude is taken on the bits, where NaN is
// above infinity above every number: a block that holds one gets a scale of
// NaN or infinity, and its products are NaN.  The quotient is rounded to 32
// bits, then to 8: two roundings, so that it is the same wherever it is
// computed with IEEE products and divisions.
template <typename T, int kN, bool kVec, int kQuantVecs>
__global__ void __launch_bounds__(kRowThreads) quantize_kernel(const T *x, uint8_t *q, float *scale, GatherArgs a)
{
    grid_dependency_wait();
    grid_dependents_go();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kLanes = kScaleBlock / kN; // that share a block
    const int blocks = (a.dim + kScaleBlock - 1) / kScaleBlock;
    const int64_t units = a.tokens * a.segments, warps = (int64_t)gridDim.x * kRowWarps;
    for (int64_t u = (int64_t)blockIdx.x * kRowWarps + warp; u < units; u += warps) {
        const int64_t t = u / a.segments;
        // dim is a multiple of 16: whole vectors
        const int first = ((int)(u - t * a.segments) * 32 * kQuantVecs + lane) * kN;
        const int32_t s = a.slot && lane < a.k ? a.slot[t * a.k + lane] : -1;
        Vec<T, kN> v[kQuantVecs];
#pragma unroll
        for (int n = 0; n < kQuantVecs; ++n) {
            const int at = first + 32 * kN * n;
            v[n] = zeros<T, kN>();
            if (at >= a.dim) continue;
            const T *p = x + t * a.stride + at;
            if (kVec) {
                v[n] = load<T, kN>(p);
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i) v[n].v[i] = p[i];
            }
        }
        uint32_t bits[kQuantVecs][kN / 4];
        float unit[kQuantVecs];
#pragma unroll
        for (int n = 0; n < kQuantVecs; ++n) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) most = max(most, __float_as_uint(as_float(v[n].v[i])) & 0x7FFFFFFFu);
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) most = max(most, __shfl_xor_sync(kAll, most, d));
            constexpr float kLeast = 7.888609052210118e-31f; // 2^-100
            const float top = __uint_as_float(most);
            unit[n] = __fmul_rn(top < kLeast ? kLeast : top, 1.0f / 448.0f);
#pragma unroll
            for (int i = 0; i < kN / 4; ++i) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] = __fdiv_rn(as_float(v[n].v[4 * i + c]), unit[n]);
                bits[n][i] = e4m3x2(w[0], w[1]) | (e4m3x2(w[2], w[3]) << 16);
            }
        }
        const auto put_row = [&](int64_t row) {
#pragma unroll
            for (int n = 0; n < kQuantVecs; ++n) {
                const int at = first + 32 * kN * n;
                if (at >= a.dim) continue;
                uint8_t *to = q + row * a.dim + at;
                if constexpr (kN == 8)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(bits[n][0], bits[n][1]);
                else
                    *reinterpret_cast<uint32_t *>(to) = bits[n][0];
                if (lane % kLanes == 0) scale[row * blocks + at / kScaleBlock] = unit[n];
            }
        };
        if (!a.slot) {
            put_row(t);
            continue;
        }
        for (int j = 0; j < a.k; ++j) {
            const int64_t to = __shfl_sync(kAll, s, j);
            if (to >= 0 && to < a.n) put_row(to);
        }
    }
    if (a.slot)
        unused_rows(a.source, a.n, [&](int64_t s) {
            for (int c = lane * 4; c < a.dim; c += 128) *reinterpret_cast<uint32_t *>(q + s * a.dim + c) = 0;
            for (int b = lane; b < blocks; b += 32) scale[s * blocks + b] = 0.0f;
        });
}

// ---------------------------------------------------------------- combine

struct CombineArgs {
    const int32_t *slot;
    const float *weight; // null: all 1
    int64_t tokens, n;
    int64_t stride; // of the rows
    int32_t dim, k;
    int32_t segments;
};

constexpr int kCombineVecs = 4; // vectors of a lane
constexpr int kCombineRows = 4; // rows in flight

// A warp adds up a segment of a token's k rows, in the order of its choices, in 32 bits.
template <typename T, int kN>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const T *rows, T *out, CombineArgs a)
{
    grid_dependency_wait();
    grid_dependents_go();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t units = a.tokens * a.segments, warps = (int64_t)gridDim.x * kRowWarps;
    const int vecs = a.dim / kN;
    for (int64_t u = (int64_t)blockIdx.x * kRowWarps + warp; u < units; u += warps) {
        const int64_t t = u / a.segments;
        const int first = (int)(u - t * a.segments) * 32 * kCombineVecs + lane;
        const int32_t s = lane < a.k ? a.slot[t * a.k + lane] : -1;
        const float w = lane < a.k && a.weight ? a.weight[t * a.k + lane] : 1.0f;
        float sum[kCombineVecs][kN];
#pragma unroll
        for (int i = 0; i < kCombineVecs; ++i)
#pragma unroll
            for (int c = 0; c < kN; ++c) sum[i][c] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kCombineRows) {
            Vec<T, kN> v[kCombineRows][kCombineVecs];
            float share[kCombineRows];
            bool has[kCombineRows];
#pragma unroll
            for (int j = 0; j < kCombineRows; ++j) {
                const int64_t from = __shfl_sync(kAll, s, (j0 + j) & 31);
                share[j] = __shfl_sync(kAll, w, (j0 + j) & 31);
                has[j] = j0 + j < a.k && from >= 0 && from < a.n;
                if (has[j]) {
#pragma unroll
                    for (int i = 0; i < kCombineVecs; ++i)
                        if (first + 32 * i < vecs)
                            v[j][i] = load<T, kN>(rows + from * a.stride + (int64_t)(first + 32 * i) * kN);
                }
            }
#pragma unroll
            for (int j = 0; j < kCombineRows; ++j) {
                if (!has[j]) continue;
#pragma unroll
                for (int i = 0; i < kCombineVecs; ++i)
#pragma unroll
                    for (int c = 0; c < kN; ++c) sum[i][c] = fmaf(share[j], as_float(v[j][i].v[c]), sum[i][c]);
            }
        }
#pragma unroll
        for (int i = 0; i < kCombineVecs; ++i) {
            if (first + 32 * i >= vecs) continue;
            Vec<T, kN> v;
#pragma unroll
            for (int c = 0; c < kN; ++c) put(v.v[c], sum[i][c]);
            store(out + t * a.dim + (int64_t)(first + 32 * i) * kN, v);
        }
    }
}

struct CombineGradArgs {
    const int32_t *slot, *source;
    const float *weight;
    float *grad_weight;
    int64_t tokens, n;
    int64_t grad_stride, row_stride;
    int32_t dim, k;
    int32_t token_warps; // warps of a token, a divisor of kRowWarps
};

constexpr int kGradRows = 4; // choices at a time

// A token's warps share its dims: each element of d_out is read once for four
// choices (more would take registers from the warps that hide the latency), whose
// rows of y are read and whose rows of d_y are written with it; the products' sums
// are joined through shared memory in the warps' order.  Where vectors are short a
// thread has several of them on their way.
template <typename T, int kN>
__global__ void __launch_bounds__(kRowThreads, kGradCtas<T, kN>)
    combine_grad_kernel(const T *grad_out, const T *rows, T *grad_rows, CombineGradArgs a)
{
    constexpr int kVecs = kGradVecs<T, kN>;
    __shared__ float part[2][kRowWarps][kGradRows];
    grid_dependency_wait();
    grid_dependents_go();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vecs = a.dim / kN;
    const int per_cta = kRowWarps / a.token_warps;
    const int of_token = warp % a.token_warps, stride = 32 * a.token_warps;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * per_cta; t0 < a.tokens; t0 += (int64_t)gridDim.x * per_cta) {
        const int64_t t = t0 + warp / a.token_warps;
        const bool in = t < a.tokens;
        const int32_t s = in && lane < a.k ? a.slot[t * a.k + lane] : -1;
        const float w = in && lane < a.k ? a.weight[t * a.k + lane] : 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kGradRows, turn ^= 1) {
            int32_t row[kGradRows];
            float share[kGradRows], dot[kGradRows];
#pragma unroll
            for (int j = 0; j < kGradRows; ++j) {
                row[j] = __shfl_sync(kAll, s, (j0 + j) & 31);
                share[j] = __shfl_sync(kAll, w, (j0 + j) & 31);
                if (j0 + j >= a.k || row[j] >= a.n) row[j] = -1;
                dot[j] = 0.0f;
            }
            if (in) {
                for (int c0 = of_token * 32 + lane; c0 < vecs; c0 += stride * kVecs) {
                    Vec<T, kN> d[kVecs], y[kGradRows][kVecs];
#pragma unroll
                    for (int n = 0; n < kVecs; ++n)
                        if (c0 + n * stride < vecs)
                            d[n] = load<T, kN>(grad_out + t * a.grad_stride + (int64_t)(c0 + n * stride) * kN);
#pragma unroll
                    for (int j = 0; j < kGradRows; ++j)
                        if (row[j] >= 0)
#pragma unroll
                            for (int n = 0; n < kVecs; ++n)
                                if (c0 + n * stride < vecs)
                                    y[j][n] = load<T, kN>(rows + row[j] * a.row_stride + (int64_t)(c0 + n * stride) * kN);
#pragma unroll
                    for (int j = 0; j < kGradRows; ++j) {
                        if (row[j] < 0) continue;
#pragma unroll
                        for (int n = 0; n < kVecs; ++n) {
                            if (c0 + n * stride >= vecs) continue;
                            Vec<T, kN> g;
#pragma unroll
                            for (int i = 0; i < kN; ++i) {
                                const float e = as_float(d[n].v[i]);
                                dot[j] = fmaf(e, as_float(y[j][n].v[i]), dot[j]);
                                put(g.v[i], e * share[j]);
                            }
                            store(grad_rows + (int64_t)row[j] * a.dim + (int64_t)(c0 + n * stride) * kN, g);
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kGradRows; ++j) {
#pragma unroll
                for (int m = 16; m; m >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], m);
                if (lane == 0) part[turn][warp][j] = dot[j];
            }
            // the other half is free: all have passed the barrier before
            if (a.token_warps > 1)
                __syncthreads();
            else
                __syncwarp();
            if (in && of_token == 0 && lane < kGradRows && j0 + lane < a.k) {
                float sum = 0.0f;
                for (int i = 0; i < a.token_warps; ++i) sum += part[turn][warp + i][lane];
                a.grad_weight[t * a.k + j0 + lane] = sum;
            }
        }
    }
    unused_rows(a.source, a.n, [&](int64_t s) {
        for (int c = lane; c < vecs; c += 32) store(grad_rows + s * a.dim + (int64_t)c * kN, zeros<T, kN>());
    });
}

// ---------------------------------------------------------------- host side

cudaLaunchConfig_t config(int64_t grid, int threads, size_t smem, void *stream, cudaLaunchAttribute *attr)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid < 1 ? 1 : grid), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs for so many warps' units, up to 16 rounds of what the SMs hold: short
// tails, and the last warps' zeros are shared out.
int64_t row_grid(int64_t units, int sm_count)
{
    const int64_t need = ceil_div(units, kRowWarps), most = (int64_t)sm_count * 8 * 16;
    return need < most ? need : most;
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The guards that the calls over rows share.
int check_rows(int32_t dtype, int64_t tokens, int32_t dim, int32_t k)
{
    if (dtype != TF_TOPK_DTYPE_BF16 && dtype != TF_TOPK_DTYPE_F16 && dtype != TF_TOPK_DTYPE_F32)
        return TF_TOPK_ERR_DTYPE;
    if (k < 1 || k > kMaxK) return TF_TOPK_ERR_K;
    if (tokens < 0 || dim < 1 || dim > kMaxDim || tokens > (int64_t)INT32_MAX / k) return TF_TOPK_ERR_SHAPE;
    return TF_TOPK_OK;
}

bool bad_stride(int64_t stride, int32_t dim, int64_t rows)
{
    return stride < dim || (rows > 0 && stride > INT64_MAX / 8 / rows);
}

size_t size_of(int32_t dtype) { return dtype == TF_TOPK_DTYPE_F32 ? 4 : 2; }

// Whether rows of `dim` elements at these strides are whole pieces of `bytes`.
bool whole(size_t bytes, size_t size, int32_t dim, int64_t stride, const void *a, const void *b, const void *c = nullptr)
{
    return aligned(a, bytes) && aligned(b, bytes) && aligned(c, bytes) && dim * size % bytes == 0 &&
           (size_t)stride * size % bytes == 0;
}

int done(cudaError_t e)
{
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}

template <typename T, int kN>
cudaError_t launch_gather(const void *x, void *out, GatherArgs a, int sm_count, void *stream)
{
    a.segments = (int32_t)ceil_div(a.dim / kN, 32 * kStep);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(row_grid(a.tokens * a.segments, sm_count), kRowThreads, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, gather_kernel<T, kN>, static_cast<const T *>(x), static_cast<T *>(out), a);
}

template <typename T, int kN>
cudaError_t launch_quantize(const void *x, void *q, float *scale, GatherArgs a, int sm_count, void *stream)
{
    const bool vec = whole(kN * sizeof(T), sizeof(T), a.dim, a.stride, x, nullptr);
    // Four vectors a lane where rows fill them and there are eight warps for each
    // SM, one otherwise (us, four / one, 2048 dims, k 8: 1 token 4.5/2.9, 64 5.0/3.1,
    // 512 5.1/5.6, 4096 15.5/20, 16384 56/77; 4001 x 1040, k 1, where a second four
    // hold 16 of 1024: 14/8.5).
    const int64_t segments = ceil_div(a.dim, 32 * kN * 4);
    const bool four = a.tokens * segments >= (int64_t)sm_count * 8 && 4 * (int64_t)a.dim >= 3 * segments * (32 * kN * 4);
    a.segments = (int32_t)ceil_div(a.dim, 32 * kN * (four ? 4 : 1));
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(row_grid(a.tokens * a.segments, sm_count), kRowThreads, 0, stream, attr);
    const auto kernel = four ? (vec ? quantize_kernel<T, kN, true, 4> : quantize_kernel<T, kN, false, 4>)
                             : (vec ? quantize_kernel<T, kN, true, 1> : quantize_kernel<T, kN, false, 1>);
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(x), static_cast<uint8_t *>(q), scale, a);
}

template <typename T, int kN>
cudaError_t launch_combine(const void *rows, void *out, CombineArgs a, int sm_count, void *stream)
{
    a.segments = (int32_t)ceil_div(a.dim / kN, 32 * kCombineVecs);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(row_grid(a.tokens * a.segments, sm_count), kRowThreads, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, combine_kernel<T, kN>, static_cast<const T *>(rows), static_cast<T *>(out), a);
}

template <typename T, int kN>
cudaError_t launch_combine_grad(const void *grad_out, const void *rows, void *grad_rows, CombineGradArgs a,
                                int sm_count, void *stream)
{
    // By the dims alone, so that a token's sums do not depend on the others.  Short
    // vectors: a warp takes up to 256 of a token, since more tokens under way hide
    // more than more warps for each (20000 x 65 fp32, k 6: 67 us with 32 a warp, 25
    // with 256; 5001 x 1002 bf16, k 3: 23 and 13; a call of 33 tokens 3.3 and 4.3).
    const int most = kGradVecs<T, kN> == 1 ? 32 : 256;
    a.token_warps = 1;
    while (a.token_warps < kRowWarps && a.token_warps * most < a.dim / kN) a.token_warps *= 2;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(row_grid(a.tokens * a.token_warps, sm_count), kRowThreads, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, combine_grad_kernel<T, kN>, static_cast<const T *>(grad_out),
                              static_cast<const T *>(rows), static_cast<T *>(grad_rows), a);
}

// CTAs of the sort: one up to kSortAlone choices, then one per kSortChunk, up to one per SM.
int64_t sort_chunks(int64_t n, int sm_count)
{
    if (n <= kSortAlone) return 1;
    const int64_t c = ceil_div(n, kSortChunk);
    return c < sm_count ? c : sm_count;
}

bool bad_sort(int64_t tokens, int32_t k, int32_t experts)
{
    return tokens < 0 || tokens > (int64_t)INT32_MAX / k || experts < 1 || experts > kMaxExperts;
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_sort_ready[kMaxDevices];
std::mutex g_sort_mutex;

// Per device, once: the sort's shared memory limit for the most experts.  A
// constant: the limit is the kernel's, not a call's, and one that a call set for
// itself another host thread could lower before the launch.
cudaError_t sort_setup()
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (e != cudaSuccess || g_sort_ready[dev].load(std::memory_order_acquire)) return e;
    std::lock_guard<std::mutex> lock(g_sort_mutex);
    constexpr int kMost = kSortWarps * kMaxExperts * (int)sizeof(int32_t);
    for (const auto kernel : {sort_place_kernel<false>, sort_place_kernel<true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess) g_sort_ready[dev].store(true, std::memory_order_release);
    return e;
}

} // namespace

extern "C" {

size_t tf_topk_sort_experts_workspace(int64_t tokens, int32_t k, int32_t experts)
{
    int sm_count = 0;
    if (k < 1 || k > kMaxK || bad_sort(tokens, k, experts) || tokens * k <= kSortAlone ||
        tf_topk_internal_device(&sm_count) != TF_TOPK_OK)
        return 0;
    return (size_t)sort_chunks(tokens * k, sm_count) * experts * sizeof(int32_t);
}

int tf_topk_sort_experts(const int32_t *idx, int64_t tokens, int32_t k, int32_t experts, void *workspace,
                         size_t workspace_bytes, int32_t *out_slot, int32_t *out_source, int32_t *out_offsets,
                         void *stream)
{
    if (k < 1 || k > kMaxK) return TF_TOPK_ERR_K;
    if (bad_sort(tokens, k, experts)) return TF_TOPK_ERR_SHAPE;
    if (!out_offsets || (tokens > 0 && (!idx || !out_slot || !out_source))) return TF_TOPK_ERR_NULL;
    if (!aligned(idx, 4) || !aligned(out_slot, 4) || !aligned(out_source, 4) || !aligned(out_offsets, 4) ||
        !aligned(workspace, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    const int st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    if (tokens == 0) {
        const cudaError_t e = cudaMemsetAsync(out_offsets, 0, (size_t)(experts + 1) * sizeof(int32_t),
                                              static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
    }
    SortArgs a;
    a.idx = idx;
    a.slot = out_slot;
    a.source = out_source;
    a.offsets = out_offsets;
    a.counts = static_cast<int32_t *>(workspace);
    a.n = tokens * k;
    a.experts = experts;
    const int64_t most = sort_chunks(a.n, sm_count);
    if (most > 1 && !workspace) return TF_TOPK_ERR_NULL;
    if (most > 1 && (size_t)most * experts * sizeof(int32_t) > workspace_bytes) return TF_TOPK_ERR_SCRATCH;
    a.chunk = ceil_div(ceil_div(a.n, most), kSortThreads) * kSortThreads;
    const int64_t chunks = ceil_div(a.n, a.chunk); // none of them empty
    const size_t smem = (size_t)kSortWarps * experts * sizeof(int32_t);
    const auto kernel = chunks == 1 ? sort_place_kernel<true> : sort_place_kernel<false>;
    cudaError_t e = sort_setup();
    cudaLaunchAttribute attr[1];
    if (e == cudaSuccess && chunks > 1) {
        const cudaLaunchConfig_t cfg = config(chunks, kSortThreads, 0, stream, attr);
        e = cudaLaunchKernelEx(&cfg, sort_count_kernel, a);
    }
    if (e == cudaSuccess) {
        const cudaLaunchConfig_t cfg = config(chunks, kSortThreads, smem, stream, attr);
        e = cudaLaunchKernelEx(&cfg, kernel, a);
    }
    return done(e);
}

int tf_topk_gather_tokens(const void *x, int32_t dtype, int64_t tokens, int32_t dim, int64_t row_stride, int32_t k,
                          const int32_t *slot, const int32_t *source, void *out_rows, void *stream)
{
    int st = check_rows(dtype, tokens, dim, k);
    if (st != TF_TOPK_OK) return st;
    if (bad_stride(row_stride, dim, tokens)) return TF_TOPK_ERR_SHAPE;
    if (tokens == 0) return TF_TOPK_OK;
    if (!x || !slot || !source || !out_rows) return TF_TOPK_ERR_NULL;
    const size_t size = size_of(dtype);
    if (!aligned(x, size) || !aligned(out_rows, size) || !aligned(slot, 4) || !aligned(source, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    GatherArgs a = {slot, source, tokens, tokens * k, row_stride, dim, k, 0};
    // a copy: the bits' width is all that matters
    if (whole(16, size, dim, row_stride, x, out_rows))
        return done(size == 4 ? launch_gather<float, 4>(x, out_rows, a, sm_count, stream)
                              : launch_gather<__half, 8>(x, out_rows, a, sm_count, stream));
    if (size == 4) return done(launch_gather<float, 1>(x, out_rows, a, sm_count, stream));
    return done(whole(4, size, dim, row_stride, x, out_rows) ? launch_gather<__half, 2>(x, out_rows, a, sm_count, stream)
                                                             : launch_gather<__half, 1>(x, out_rows, a, sm_count, stream));
}

int tf_topk_quantize_tokens(const void *x, int32_t dtype, int64_t tokens, int32_t dim, int64_t row_stride, int32_t k,
                            const int32_t *slot, const int32_t *source, void *out_q, float *out_scale, void *stream)
{
    int st = check_rows(dtype, tokens, dim, k);
    if (st != TF_TOPK_OK) return st;
    if (dim % 16 != 0 || bad_stride(row_stride, dim, tokens)) return TF_TOPK_ERR_SHAPE;
    if (tokens == 0) return TF_TOPK_OK;
    if (!slot && k != 1) return TF_TOPK_ERR_K;
    if (!x || !out_q || !out_scale || (slot && !source)) return TF_TOPK_ERR_NULL;
    if (!aligned(x, size_of(dtype)) || !aligned(out_q, 16) || !aligned(out_scale, 4) || !aligned(slot, 4) ||
        !aligned(source, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    GatherArgs a = {slot, source, tokens, tokens * k, row_stride, dim, k, 0};
    return done(dtype == TF_TOPK_DTYPE_F32   ? launch_quantize<float, 4>(x, out_q, out_scale, a, sm_count, stream)
                : dtype == TF_TOPK_DTYPE_F16 ? launch_quantize<__half, 8>(x, out_q, out_scale, a, sm_count, stream)
                                             : launch_quantize<__nv_bfloat16, 8>(x, out_q, out_scale, a, sm_count, stream));
}

int tf_topk_combine_tokens(const void *rows, int32_t dtype, int64_t tokens, int32_t dim, int64_t row_stride, int32_t k,
                           const int32_t *slot, const float *weight, void *out, void *stream)
{
    int st = check_rows(dtype, tokens, dim, k);
    if (st != TF_TOPK_OK) return st;
    if (bad_stride(row_stride, dim, tokens * k)) return TF_TOPK_ERR_SHAPE;
    if (tokens == 0) return TF_TOPK_OK;
    if (!rows || !slot || !out) return TF_TOPK_ERR_NULL;
    const size_t size = size_of(dtype);
    if (!aligned(rows, size) || !aligned(out, size) || !aligned(slot, 4) || !aligned(weight, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    CombineArgs a = {slot, weight, tokens, tokens * k, row_stride, dim, k, 0};
    const bool wide = whole(16, size, dim, row_stride, rows, out), pairs = whole(4, size, dim, row_stride, rows, out);
    if (dtype == TF_TOPK_DTYPE_F32)
        return done(wide ? launch_combine<float, 4>(rows, out, a, sm_count, stream)
                         : launch_combine<float, 1>(rows, out, a, sm_count, stream));
    if (dtype == TF_TOPK_DTYPE_F16)
        return done(wide    ? launch_combine<__half, 8>(rows, out, a, sm_count, stream)
                    : pairs ? launch_combine<__half, 2>(rows, out, a, sm_count, stream)
                            : launch_combine<__half, 1>(rows, out, a, sm_count, stream));
    return done(wide    ? launch_combine<__nv_bfloat16, 8>(rows, out, a, sm_count, stream)
                : pairs ? launch_combine<__nv_bfloat16, 2>(rows, out, a, sm_count, stream)
                        : launch_combine<__nv_bfloat16, 1>(rows, out, a, sm_count, stream));
}

int tf_topk_combine_tokens_grad(const void *grad_out, int32_t dtype, int64_t tokens, int32_t dim, int64_t grad_stride,
                                const void *rows, int64_t row_stride, int32_t k, const int32_t *slot,
                                const int32_t *source, const float *weight, void *out_grad_rows,
                                float *out_grad_weight, void *stream)
{
    int st = check_rows(dtype, tokens, dim, k);
    if (st != TF_TOPK_OK) return st;
    if (bad_stride(grad_stride, dim, tokens) || bad_stride(row_stride, dim, tokens * k)) return TF_TOPK_ERR_SHAPE;
    if (tokens == 0) return TF_TOPK_OK;
    if (!grad_out || !rows || !slot || !source || !weight || !out_grad_rows || !out_grad_weight)
        return TF_TOPK_ERR_NULL;
    const size_t size = size_of(dtype);
    if (!aligned(grad_out, size) || !aligned(rows, size) || !aligned(out_grad_rows, size) || !aligned(slot, 4) ||
        !aligned(source, 4) || !aligned(weight, 4) || !aligned(out_grad_weight, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0;
    st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    CombineGradArgs a = {slot, source, weight, out_grad_weight, tokens, tokens * k, grad_stride, row_stride, dim, k, 0};
    const auto fits = [&](size_t bytes) {
        return whole(bytes, size, dim, grad_stride, grad_out, rows, out_grad_rows) && (size_t)row_stride * size % bytes == 0;
    };
    const auto go = [&](auto launch) { return done(launch(grad_out, rows, out_grad_rows, a, sm_count, stream)); };
    if (dtype == TF_TOPK_DTYPE_F32) return go(fits(16) ? launch_combine_grad<float, 4> : launch_combine_grad<float, 1>);
    if (dtype == TF_TOPK_DTYPE_F16)
        return go(fits(16)  ? launch_combine_grad<__half, 8>
                  : fits(4) ? launch_combine_grad<__half, 2>
                            : launch_combine_grad<__half, 1>);
    return go(fits(16)  ? launch_combine_grad<__nv_bfloat16, 8>
              : fits(4) ? launch_combine_grad<__nv_bfloat16, 2>
                        : launch_combine_grad<__nv_bfloat16, 1>);
}

} // extern "C"
