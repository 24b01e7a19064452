// Logits made ready for sampling on GB300 (sm_103a): repetition, presence and
// frequency penalties for a request's tokens so far, biases and a grammar's
// mask, in one pass before tf_topk_select.
//
// What is computed, for a row x of logits whose request holds a prompt and an
// answer so far, n[c] being how often the answer has token c:
//   x[c] = x[c] > 0 ? x[c] / repetition : x[c] * repetition   if c is in either
//   x[c] = x[c] - frequency * n[c] - presence                 if n[c] > 0
//   x[c] = x[c] + bias                                        if c has one
//   x[c] = -inf                                               if c is not allowed
// in this order, each step rounded to 32 bits, the result once to its type.
//
// A CTA takes a chunk of a row's columns: it counts the request's tokens that
// fall into the chunk in shared memory (a word per column: the answer's count,
// the top bit for the prompt), then reads, changes and writes the chunk.  What
// bounds it is reading and writing the logits; every chunk reads the row's
// tokens again, from the L2, which is why a chunk is as wide as shared memory
// allows once there are CTAs enough.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "tf_topk.h"

int tf_topk_internal_fail_cuda(int cuda_error);
int tf_topk_internal_device(int *sm_count);

namespace {

constexpr int kThreads = 512;
constexpr int kMostChunk = 16384; // columns
constexpr int kLeastChunk = 2048;
constexpr int kPad = 16;          // words beside a chunk: its first vector may start off the 16-byte boundary
constexpr uint32_t kPrompt = 1u << 31;

struct PenaltyArgs {
    const void *logits;
    void *out;
    const int32_t *tokens, *lengths, *prompts;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_token;
    const float *bias_value;
    const uint32_t *allowed;
    int64_t cols, stride, out_stride, token_stride, bias_stride, allowed_stride;
    int32_t width, biases; // of a row
    int32_t chunk, chunks; // columns of a chunk, chunks of a row
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float &to, float x) { to = x; }
__device__ __forceinline__ void put(__half &to, float x) { to = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 &to, float x) { to = __float2bfloat16_rn(x); }

// What a request asks for.
struct Request {
    float repetition, presence, frequency;
    const float *bias;
};

template <typename T> __device__ __forceinline__ T changed(T logit, uint32_t word, uint32_t bias, const Request &r)
{
    float x = as_float(logit);
    if (word) x = x > 0.0f ? __fdiv_rn(x, r.repetition) : __fmul_rn(x, r.repetition);
    const uint32_t n = word & ~kPrompt;
    if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.frequency, (float)n)), r.presence);
    if (bias) x = __fadd_rn(x, r.bias[bias - 1]);
    T out;
    put(out, x);
    return out;
}

template <typename T> __global__ void __launch_bounds__(kThreads) penalize_kernel(const PenaltyArgs a)
{
    extern __shared__ uint4 smem[];
    grid_dependency_wait();
    grid_dependents_go();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.chunks;
    const int64_t c0 = (int64_t)(blockIdx.x - row * a.chunks) * a.chunk;
    const int cols = (int)min((int64_t)a.chunk, a.cols - c0); // of this chunk
    const T *in = static_cast<const T *>(a.logits) + row * a.stride + c0;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + c0;
    const uint32_t *allowed = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;

    // whole vectors from the first 16-byte boundary on, where input and output have it in the same place
    constexpr int kN = 16 / sizeof(T);
    const int off = (int)((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T));
    const bool vec = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int head = vec ? min(cols, (kN - off) % kN) : cols;
    const int vecs = (cols - head) / kN;

    // a column's words stand at base + column, so that a vector's words are whole 16 bytes
    const int base = kN - head % kN; // 1..kN
    uint32_t *words = reinterpret_cast<uint32_t *>(smem);
    uint16_t *places = reinterpret_cast<uint16_t *>(words + a.chunk + kPad);
    Request r;
    r.repetition = a.repetition ? a.repetition[row] : 1.0f;
    r.presence = a.presence ? a.presence[row] : 0.0f;
    r.frequency = a.frequency ? a.frequency[row] : 0.0f;
    r.bias = a.biases > 0 ? a.bias_value + row * a.bias_stride : nullptr;
    int length = a.lengths ? min(max(a.lengths[row], 0), a.width) : a.width;
    if (r.repetition == 1.0f && r.presence == 0.0f && r.frequency == 0.0f) length = 0; // asks for none
    const int prompt = a.prompts ? a.prompts[row] : 0;
    const bool counts = length > 0, biases = a.biases > 0;
    if (counts) {
        for (int i = tid; i < (a.chunk + kPad) / 4; i += kThreads) smem[i] = make_uint4(0, 0, 0, 0);
    }
    if (biases) {
        uint4 *p = reinterpret_cast<uint4 *>(places);
        for (int i = tid; i < (a.chunk + kPad) / 8; i += kThreads) p[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (counts) {
        const int32_t *tokens = a.tokens + row * a.token_stride;
        const auto note = [&](int i, int32_t token) {
            const int64_t c = token - c0;
            if (c < 0 || c >= cols) return;
            if (i < prompt)
                atomicOr(&words[base + c], kPrompt);
            else
                atomicAdd(&words[base + c], 1u);
        };
        const int lead = min(length, (int)((4 - (reinterpret_cast<uintptr_t>(tokens) / 4 & 3)) & 3));
        const int quads = (length - lead) / 4;
        if (tid < lead) note(tid, tokens[tid]);
#pragma unroll 4
        for (int i = tid; i < quads; i += kThreads) {
            const int4 t = *reinterpret_cast<const int4 *>(tokens + lead + 4 * i);
            const int at = lead + 4 * i;
            note(at, t.x), note(at + 1, t.y), note(at + 2, t.z), note(at + 3, t.w);
        }
        for (int i = lead + 4 * quads + tid; i < length; i += kThreads) note(i, tokens[i]);
    }
    if (biases) {
        // the last entry of a token counts
        for (int i = tid; i < a.biases; i += kThreads) {
            const int64_t c = a.bias_token[row * a.bias_stride + i] - c0;
            if (c < 0 || c >= cols) continue;
            uint16_t *p = &places[base + c], seen = *p;
            while (seen < (uint16_t)(i + 1)) {
                const uint16_t was = atomicCAS(p, seen, (uint16_t)(i + 1));
                if (was == seen) break;
                seen = was;
            }
        }
    }
    __syncthreads();

    T least;
    put(least, -INFINITY);
    const auto allow = [&](int c) { return !allowed || (allowed[(c0 + c) >> 5] >> ((c0 + c) & 31) & 1); };
    const auto one = [&](int c) {
        T x = in[c];
        const uint32_t w = counts ? words[base + c] : 0, b = biases ? places[base + c] : 0;
        if (w | b) x = changed(x, w, b, r);
        out[c] = allow(c) ? x : least;
    };
    for (int c = tid; c < head; c += kThreads) one(c);
    for (int c = head + vecs * kN + tid; c < cols; c += kThreads) one(c);
    constexpr int kStep = 4;
    for (int i0 = tid; i0 < vecs; i0 += kStep * kThreads) {
        union Piece {
            uint4 raw;
            T v[kN];
            __device__ Piece() {}
        } x[kStep];
        uint32_t bits[kStep];
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            const int i = i0 + s * kThreads, c = head + i * kN;
            bits[s] = 0xFFFFFFFFu;
            if (i >= vecs) continue;
            x[s].raw = *reinterpret_cast<const uint4 *>(in + c);
            if (allowed) {
                const int64_t at = c0 + c;
                const uint32_t lo = allowed[at >> 5], hi = allowed[(at + kN - 1) >> 5];
                bits[s] = __funnelshift_r(lo, hi, (uint32_t)(at & 31));
            }
        }
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            const int i = i0 + s * kThreads, c = head + i * kN;
            if (i >= vecs) continue;
            const int at = base + c; // a multiple of kN
            uint32_t any = 0;
            if (counts) {
#pragma unroll
                for (int j = 0; j < kN; j += 4) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(words + at + j);
                    any |= w.x | w.y | w.z | w.w;
                }
            }
            if (biases) {
                const uint2 p = *reinterpret_cast<const uint2 *>(places + at);
                any |= p.x | p.y;
                if (kN == 8) {
                    const uint2 o = *reinterpret_cast<const uint2 *>(places + at + 4);
                    any |= o.x | o.y;
                }
            }
            if (any) {
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const uint32_t w = counts ? words[at + j] : 0, b = biases ? places[at + j] : 0;
                    if (w | b) x[s].v[j] = changed(x[s].v[j], w, b, r);
                }
            }
#pragma unroll
            for (int j = 0; j < kN; ++j)
                if (!(bits[s] >> j & 1)) x[s].v[j] = least;
            *reinterpret_cast<uint4 *>(out + c) = x[s].raw;
        }
    }
}

// ---------------------------------------------------------------- host side

constexpr size_t smem_bytes(int chunk, bool biases) { return (size_t)(chunk + kPad) * (biases ? 6 : 4); }

constexpr int kMaxDevices = 64;
std::atomic<bool> g_ready[kMaxDevices];
std::mutex g_mutex;

using PenaltyKernel = void (*)(PenaltyArgs);

PenaltyKernel kernel_for(int32_t dtype)
{
    return dtype == TF_TOPK_DTYPE_F32   ? penalize_kernel<float>
           : dtype == TF_TOPK_DTYPE_F16 ? penalize_kernel<__half>
                                        : penalize_kernel<__nv_bfloat16>;
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool bad_stride(int64_t stride, int64_t width, int64_t rows)
{
    return stride < width || (rows > 0 && stride > INT64_MAX / 8 / rows);
}

} // namespace

extern "C" int tf_topk_penalize(const void *logits, int32_t dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t *tokens, int64_t token_stride, int32_t width, const int32_t *lengths,
                                const int32_t *prompts, const float *repetition, const float *presence,
                                const float *frequency, const int32_t *bias_token, const float *bias_value,
                                int64_t bias_stride, int32_t biases, const uint32_t *allowed, int64_t allowed_stride,
                                void *out, int64_t out_stride, void *stream)
{
    if (dtype != TF_TOPK_DTYPE_BF16 && dtype != TF_TOPK_DTYPE_F16 && dtype != TF_TOPK_DTYPE_F32)
        return TF_TOPK_ERR_DTYPE;
    if (rows < 0 || cols < 1 || cols > INT32_MAX || bad_stride(row_stride, cols, rows) ||
        bad_stride(out_stride, cols, rows) || width < 0 || (width > 0 && bad_stride(token_stride, width, rows)) ||
        biases < 0 || biases > TF_TOPK_PENALTY_MAX_BIASES || (biases > 0 && bad_stride(bias_stride, biases, rows)) ||
        (allowed && bad_stride(allowed_stride, (cols + 31) / 32, rows)) ||
        rows > INT32_MAX / ((cols + kLeastChunk - 1) / kLeastChunk))
        return TF_TOPK_ERR_SHAPE;
    if (rows == 0) return TF_TOPK_OK;
    if (!logits || !out || (width > 0 && !tokens) || (biases > 0 && (!bias_token || !bias_value))) return TF_TOPK_ERR_NULL;
    const size_t size = dtype == TF_TOPK_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(out, size) || !aligned(tokens, 4) || !aligned(lengths, 4) ||
        !aligned(prompts, 4) || !aligned(repetition, 4) || !aligned(presence, 4) || !aligned(frequency, 4) ||
        !aligned(bias_token, 4) || !aligned(bias_value, 4) || !aligned(allowed, 4))
        return TF_TOPK_ERR_ALIGN;
    int sm_count = 0, dev = 0;
    const int st = tf_topk_internal_device(&sm_count);
    if (st != TF_TOPK_OK) return st;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= kMaxDevices) return TF_TOPK_ERR_DEVICE;
    if (e == cudaSuccess && !g_ready[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_mutex);
        for (int32_t d : {TF_TOPK_DTYPE_BF16, TF_TOPK_DTYPE_F16, TF_TOPK_DTYPE_F32})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel_for(d), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_bytes(kMostChunk, true));
        if (e == cudaSuccess) g_ready[dev].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
    PenaltyArgs a;
    a.logits = logits;
    a.out = out;
    a.tokens = tokens;
    a.lengths = lengths;
    a.prompts = prompts;
    a.repetition = repetition;
    a.presence = presence;
    a.frequency = frequency;
    a.bias_token = bias_token;
    a.bias_value = bias_value;
    a.allowed = allowed;
    a.cols = cols;
    a.stride = row_stride;
    a.out_stride = out_stride;
    a.token_stride = token_stride;
    a.bias_stride = bias_stride;
    a.allowed_stride = allowed_stride;
    a.width = width;
    a.biases = biases;
    // the widest chunks that still give every SM two CTAs
    a.chunk = kMostChunk;
    while (a.chunk > kLeastChunk && rows * ((cols + a.chunk - 1) / a.chunk) < 2 * sm_count) a.chunk /= 2;
    a.chunks = (int32_t)((cols + a.chunk - 1) / a.chunk);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.chunks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = width > 0 || biases > 0 ? smem_bytes(a.chunk, biases > 0) : 0;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel_for(dtype), a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}
