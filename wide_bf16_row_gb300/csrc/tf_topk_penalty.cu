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
// Two kernels.  copy_kernel reads and writes the logits, with the mask: that is
// what bounds the whole.  name_kernel counts, in a table in shared memory, which
// columns a row's tokens and biases name, and how often, while the copy runs; when
// the copy is done it writes those columns again.  (In one kernel, with every
// CTA counting for its own columns, the counting took longer than the copy: 113
// us for 256 x 248320 with 4000 tokens against 56, of which the copy is 40, 0.95
// of the copy bandwidth.)
//
// The table: for up to kHashed tokens and biases a hash table of the columns, one
// CTA per row (16384 places of 10 bytes; twice as many do not fit an SM); for more,
// one word per column, the columns dealt out to several CTAs in turn (common tokens
// are neighbours), each of which reads all of the row's tokens.  Both (us, hash / words,
// 248320 columns, in place): 4000 tokens, 1 row 11.5/5.6, 33 rows 14/16, 256 rows 26/106;
// 8192 tokens 26/6.8, 31/20, 66/137: many rows want the hash, few rows, whose columns
// are shared out over the SMs, would not.

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

constexpr int kCopyThreads = 256;
constexpr int kStep = 4; // vectors of a thread
// One CTA per SM by its registers; two of fewer registers or threads were slower (55-67 us).
constexpr int kNameThreads = 1024;
constexpr int kBatch = 4;              // loads of a thread at once
constexpr int kHashed = 8192;          // tokens and biases that a hash table holds, in twice the places
constexpr int kMostPlaces = 32768;     // of a table without a hash: 192 KB with biases
constexpr int kLeastPlaces = 256;
// CTAs that share a row's columns for the sake of the SMs, at most.  With 4, 16 and
// 64 (us, 40000 tokens): 1 x 248320 15.4 (8 for the table's size), 10.7 and 6.8; 1 x 32771
// 9.1, 6.8 and 6.6; 33 x 32771 9.5, 15.2 and 15.2, where eight a row are more than one an SM.
constexpr int kMostShares = 16;
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30; // of a column's word; the answer's count below
constexpr int kMostWidth = 1 << 29;

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
    int32_t chunks;        // copy: CTAs of a row
    int32_t places;        // name: of the table, a power of two
    int32_t shares;        // name: CTAs of a row, a power of two
    int32_t hashed;        // name: the table is a hash table
    int32_t copied;        // name: a copy runs before
};

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float &to, float x) { to = x; }
__device__ __forceinline__ void put(__half &to, float x) { to = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 &to, float x) { to = __float2bfloat16_rn(x); }

// ---------------------------------------------------------------- the copy

template <typename T> union Piece {
    uint4 raw;
    T v[16 / sizeof(T)];
    __device__ Piece() {}
};

// A CTA copies up to kCopyThreads * kStep vectors of a row; out may be the input itself.
template <typename T> __global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PenaltyArgs a)
{
    grid_dependency_wait();
    grid_dependents_go();
    constexpr int kN = 16 / sizeof(T), kChunk = kCopyThreads * kStep * kN;
    const int tid = threadIdx.x;
    const uint32_t row = blockIdx.x / (uint32_t)a.chunks;
    const int64_t c0 = (int64_t)(blockIdx.x - row * (uint32_t)a.chunks) * kChunk;
    const int cols = (int)min((int64_t)kChunk, a.cols - c0);
    const T *in = static_cast<const T *>(a.logits) + row * a.stride + c0;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + c0;
    const uint32_t *allowed = a.allowed ? a.allowed + row * a.allowed_stride + (c0 >> 5) : nullptr; // chunks start on words
    // whole vectors from the first 16-byte boundary on, where input and output have it in the same place
    const int off = (int)((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T));
    const bool vec = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int head = vec ? min(cols, (kN - off) % kN) : cols;
    const int vecs = (cols - head) / kN;
    Piece<T> x[kStep];
    uint32_t low[kStep], high[kStep]; // the mask's words of a vector
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        const int i = tid + s * kCopyThreads, c = head + i * kN;
        low[s] = high[s] = kNone;
        if (i >= vecs) continue;
        x[s].raw = *reinterpret_cast<const uint4 *>(in + c);
        if (allowed) {
            low[s] = allowed[c >> 5];
            if (head % kN) high[s] = allowed[(c + kN - 1) >> 5];
        }
    }
    T least;
    put(least, -INFINITY);
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        const int i = tid + s * kCopyThreads, c = head + i * kN;
        if (i >= vecs) continue;
        if (allowed) {
            const uint32_t bits = __funnelshift_r(low[s], high[s], (uint32_t)c & 31);
            if ((bits & ((1u << kN) - 1)) != (1u << kN) - 1) {
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    if (!(bits >> j & 1)) x[s].v[j] = least;
            }
        }
        *reinterpret_cast<uint4 *>(out + c) = x[s].raw;
    }
    const auto one = [&](int c) { out[c] = !allowed || (allowed[c >> 5] >> (c & 31) & 1) ? in[c] : least; };
    for (int c = tid; c < head; c += kCopyThreads) one(c);
    for (int c = head + vecs * kN + tid; c < cols; c += kCopyThreads) one(c);
}

// ---------------------------------------------------------------- the named columns

// What a request asks for.
struct Request {
    float repetition, presence, frequency;
};

template <typename T> __device__ __forceinline__ T changed(T logit, uint32_t word, float bias, const Request &r)
{
    float x = as_float(logit);
    if (word & ~kBias) x = x > 0.0f ? __fdiv_rn(x, r.repetition) : __fmul_rn(x, r.repetition);
    const uint32_t n = word & ~(kPrompt | kBias);
    if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.frequency, (float)n)), r.presence);
    if (word & kBias) x = __fadd_rn(x, bias);
    T out;
    put(out, x);
    return out;
}

template <typename T, bool kHash> __global__ void __launch_bounds__(kNameThreads) name_kernel(const PenaltyArgs a)
{
    extern __shared__ uint4 smem[];
    // A copy before has waited for what comes before it, so that all but the
    // logits may be read while it runs.
    if (!a.copied) {
        grid_dependency_wait();
        grid_dependents_go();
    }
    const int tid = threadIdx.x;
    const uint32_t row = kHash ? blockIdx.x : blockIdx.x / (uint32_t)a.shares;
    const uint32_t share = kHash ? 0 : blockIdx.x & (uint32_t)(a.shares - 1);
    const int shift = kHash ? 0 : __ffs(a.shares) - 1, bits = __ffs(a.places) - 1;
    const uint32_t cols = (uint32_t)a.cols;
    uint32_t *words = reinterpret_cast<uint32_t *>(smem);                  // [places]
    uint32_t *keys = words + a.places;                                     // hash: [places], the columns
    uint16_t *last = reinterpret_cast<uint16_t *>(keys + (kHash ? a.places : 0)); // [places]: of a column's last bias, from 1
    // a thread's first tokens are on their way before their number is known
    const int32_t *tokens = a.tokens + (a.width > 0 ? row * a.token_stride : 0);
    // before the first 16 bytes
    const int lead = min(a.width, (int)((4 - (reinterpret_cast<uintptr_t>(tokens) / 4 & 3)) & 3));
    const int4 *vecs = reinterpret_cast<const int4 *>(tokens + lead);
    const int4 first = tid < (a.width - lead) / 4 ? vecs[tid] : make_int4(-1, -1, -1, -1);
    Request r;
    r.repetition = a.repetition ? a.repetition[row] : 1.0f;
    r.presence = a.presence ? a.presence[row] : 0.0f;
    r.frequency = a.frequency ? a.frequency[row] : 0.0f;
    int length = a.lengths ? min(max(a.lengths[row], 0), a.width) : a.width;
    const int prompt = a.prompts ? a.prompts[row] : 0;
    for (int i = tid; i < a.places / 4; i += kNameThreads) {
        smem[i] = make_uint4(0, 0, 0, 0);
        if (kHash) smem[i + a.places / 4] = make_uint4(kNone, kNone, kNone, kNone);
    }
    if (a.biases > 0)
        for (int i = tid; i < a.places / 8; i += kNameThreads) reinterpret_cast<uint4 *>(last)[i] = make_uint4(0, 0, 0, 0);
    if (r.repetition == 1.0f && r.presence == 0.0f && r.frequency == 0.0f) length = 0; // asks for none
    __syncthreads();

    // the place of a column in the table; the table is never full
    const auto place_of = [&](uint32_t c) {
        if (!kHash) return c >> shift;
        uint32_t h = (c * 2654435769u) >> (32 - bits);
        for (int i = 0; i < a.places; ++i) {
            const uint32_t k = keys[h];
            if (k == c) break;
            if (k == kNone) {
                const uint32_t was = atomicCAS(&keys[h], kNone, c);
                if (was == kNone || was == c) break;
            }
            h = (h + 1) & (uint32_t)(a.places - 1);
        }
        return h;
    };
    const auto mine = [&](int32_t token) { // a negative token is no column
        return (uint32_t)token < cols && (kHash || ((uint32_t)token & (uint32_t)(a.shares - 1)) == share);
    };
    if (length > 0) {
        const auto note = [&](int i, int32_t token) {
            if (!mine(token) || i >= length) return;
            const uint32_t p = place_of((uint32_t)token);
            if (i < prompt)
                atomicOr(&words[p], kPrompt);
            else
                atomicAdd(&words[p], 1u);
        };
        const auto note4 = [&](int i, const int4 &t) {
            const int at = lead + 4 * i;
            note(at, t.x), note(at + 1, t.y), note(at + 2, t.z), note(at + 3, t.w);
        };
        note4(tid, first);
        const int quads = (max(length - lead, 0)) / 4;
        for (int i0 = tid + kNameThreads; i0 < quads; i0 += kBatch * kNameThreads) {
            int4 t[kBatch];
#pragma unroll
            for (int s = 0; s < kBatch; ++s)
                t[s] = i0 + s * kNameThreads < quads ? vecs[i0 + s * kNameThreads] : make_int4(-1, -1, -1, -1);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) note4(i0 + s * kNameThreads, t[s]);
        }
        if (tid < min(lead, length)) note(tid, tokens[tid]);
        const int rest = lead + 4 * max(quads, min(kNameThreads, (a.width - lead) / 4)) + tid;
        if (rest < length) note(rest, tokens[rest]); // up to three
    }
    const int32_t *bias_token = a.bias_token + (a.biases > 0 ? row * a.bias_stride : 0);
    for (int i = tid; i < a.biases; i += kNameThreads) {
        const int32_t token = bias_token[i];
        if (!mine(token)) continue;
        const uint32_t p = place_of((uint32_t)token);
        atomicOr(&words[p], kBias);
        uint16_t seen = last[p]; // the last entry of a column counts
        while (seen < (uint16_t)(i + 1)) {
            const uint16_t was = atomicCAS(&last[p], seen, (uint16_t)(i + 1));
            if (was == seen) break;
            seen = was;
        }
    }
    __syncthreads();
    if (a.copied) {
        grid_dependency_wait();
        grid_dependents_go();
    }
    // Where out is the input itself, the copy has left a column as it was, or it is not allowed.
    const T *in = static_cast<const T *>(a.logits) + row * a.stride;
    T *out = static_cast<T *>(a.out) + row * a.out_stride;
    const uint32_t *allowed = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;
    const float *bias_value = a.bias_value + (a.biases > 0 ? row * a.bias_stride : 0);
    for (int p0 = tid; p0 < a.places; p0 += kBatch * kNameThreads) {
        uint32_t word[kBatch], c[kBatch], mask[kBatch];
        T x[kBatch];
        float bias[kBatch];
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            const int p = p0 + s * kNameThreads;
            word[s] = p < a.places ? words[p] : 0;
            if (word[s] == 0) continue;
            c[s] = kHash ? keys[p] : ((uint32_t)p << shift) | share;
            x[s] = in[c[s]];
            mask[s] = allowed ? allowed[c[s] >> 5] : kNone;
            bias[s] = word[s] & kBias ? bias_value[last[p] - 1] : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < kBatch; ++s)
            if (word[s] != 0 && (mask[s] >> (c[s] & 31) & 1)) out[c[s]] = changed(x[s], word[s], bias[s], r);
    }
}

// ---------------------------------------------------------------- host side

constexpr size_t table_bytes(int places, bool hashed, bool biases)
{
    return (size_t)places * (4 + (hashed ? 4 : 0) + (biases ? 2 : 0));
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_ready[kMaxDevices];
std::mutex g_mutex;

using PenaltyKernel = void (*)(PenaltyArgs);

PenaltyKernel copy_for(int32_t dtype)
{
    if (dtype == TF_TOPK_DTYPE_F32) return copy_kernel<float>;
    return dtype == TF_TOPK_DTYPE_F16 ? copy_kernel<__half> : copy_kernel<__nv_bfloat16>;
}

PenaltyKernel name_for(int32_t dtype, bool hashed)
{
    if (dtype == TF_TOPK_DTYPE_F32) return hashed ? name_kernel<float, true> : name_kernel<float, false>;
    if (dtype == TF_TOPK_DTYPE_F16) return hashed ? name_kernel<__half, true> : name_kernel<__half, false>;
    return hashed ? name_kernel<__nv_bfloat16, true> : name_kernel<__nv_bfloat16, false>;
}

cudaError_t launch(PenaltyKernel kernel, int64_t grid, int threads, size_t smem, const PenaltyArgs &a, void *stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool bad_stride(int64_t stride, int64_t width, int64_t rows)
{
    return stride < width || (rows > 0 && stride > INT64_MAX / 8 / rows);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
        bad_stride(out_stride, cols, rows) || width < 0 || width > kMostWidth ||
        (width > 0 && bad_stride(token_stride, width, rows)) || biases < 0 || biases > TF_TOPK_PENALTY_MAX_BIASES ||
        (biases > 0 && bad_stride(bias_stride, biases, rows)) ||
        (allowed && bad_stride(allowed_stride, ceil_div(cols, 32), rows)) || rows > INT32_MAX / ceil_div(cols, 1024) ||
        (out == logits && rows > 1 && out_stride != row_stride)) // rows of the one would be written over the other's
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
            for (bool hashed : {false, true})
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(name_for(d, hashed), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)table_bytes(hashed ? 2 * kHashed : kMostPlaces, hashed, true));
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
    a.chunks = (int32_t)ceil_div(cols, (int64_t)(kCopyThreads * kStep * 16) / (int64_t)size);
    // nothing to copy where the logits change in place without a mask
    a.copied = out != logits || allowed != nullptr;
    if (a.copied) e = launch(copy_for(dtype), rows * a.chunks, kCopyThreads, 0, a, stream);
    const bool asked = width > 0 && (repetition || presence || frequency);
    if (!asked) a.width = 0;
    const int64_t names = (int64_t)a.width + biases;
    if (e == cudaSuccess && names > 0) {
        a.hashed = names <= kHashed;
        a.shares = 1;
        a.places = kLeastPlaces;
        if (a.hashed) {
            while (a.places < 2 * names) a.places *= 2;
        } else {
            // as few CTAs as hold the columns, each of which reads all tokens, but one per SM
            while (a.shares * (int64_t)kMostPlaces < cols || (rows * a.shares < sm_count && a.shares < kMostShares))
                a.shares *= 2;
            while (a.places * (int64_t)a.shares < cols) a.places *= 2;
        }
        e = launch(name_for(dtype, a.hashed), rows * a.shares, kNameThreads,
                   table_bytes(a.places, a.hashed, biases > 0), a, stream);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}
