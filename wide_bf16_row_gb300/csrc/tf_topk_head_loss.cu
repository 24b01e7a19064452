// The head's loss and its gradient for GB300 (sm_103a): softmax cross entropy
// of an LM head's logits against one target column per row, without storing
// the logits.
//
// What is computed, for rows n, vocabulary columns v and dims d:
//   x[n][v]  = sum_d hidden[n][d] * weight[v][d]        (bf16 in, fp32 sum)
//   lse[n]   = log sum_v exp(x[n][v])
//   loss[n]  = lse[n] - x[n][target[n]]
// and, for a gradient g[n] of loss[n]:
//   G[n][v]  = g[n] * (exp(x[n][v] - lse[n]) - [v == target[n]])
//   d_hidden = G weight,   d_weight = G^T hidden.
// Rows whose target is ignored take no part.  The target's entry of G is
// g expm1(x_t - lse), from the logit that lse was made with (below).
//
// One kernel shape serves the four products: pair_product_kernel, persistent,
// a pair of CTAs (cluster of two, tcgen05.mma cta_group::2) per tile of 256
// rows x up to 256 columns.  Each CTA of the pair holds half of the tile's
// rows (M) and loads half of its columns (N); its 128 accumulator lanes are
// its rows.  Warp roles, per CTA:
//   warp 0     TMA producer: per ring stage one CTA's halves of A and B, 64
//              steps of the summed dimension K, 128-byte swizzle;
//   warp 1     TMEM allocation; in the leading CTA also the MMA issuer, into
//              one of two accumulators of 256 columns, so that the epilogue
//              of a tile overlaps the products of the next;
//   warps 2-9  epilogue, a thread per row and half of the tile's columns.
// The modes differ in the operands and the epilogue:
//   kLse   A = hidden, B = weight: per row and half tile the running maximum
//          and the sum of exp2, the target's column left out;
//   kProb  the same product, turned into G (bf16) for a piece of the
//          vocabulary;
//   kHidden  A = G, B = weight with K = the vocabulary (B is stored with N
//          contiguous): fp32 sums that grow from piece to piece;
//   kWeight  A = G^T, B = hidden with K = the rows (both stored with M and N
//          contiguous): the piece's rows of d_weight;
//   kGrads kHidden's tiles, then kWeight's, in one launch, so that the second
//          fill the last round of the first.
//
// The tensor cores truncate their running fp32 sums, which biases a logit of
// 12 by about -2.6e-5 at 2048 dims (measured against 64 bits; the fp32 FMA
// sum is unbiased).  In lse that is spread over many small logits, whose sums
// kLse keeps short (kPartSteps), but in loss it would be the target's alone, so
// the target's logit is summed by FMA in head_loss_rows_kernel and
//   loss = log(1 + exp(rest - x_t)),  rest = log sum over v != t of exp(x_v),
// which also keeps the digits of a loss near 0.  For the same reason p_t - 1 is
// not taken from the product's x_t, which is some 1e-5 away from the one in lse:
// of a row that is sure to 1e-4 nothing would be left.
//
// No wait is unbounded: every mbarrier wait gives up after kWaitLimit polls,
// records a fault code, and the CTA winds down.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "tf_topk.h"

int tf_topk_internal_fail_cuda(int cuda_error);
int tf_topk_internal_device(int *sm_count);

namespace {

constexpr int kTileRows = 256;                       // rows (M) of a pair's tile
constexpr int kTileCols = 256;                       // columns (N) of the widest tile
constexpr int kFewCols = 192;                        // of the widest tile of the loss with up to kHalf rows
constexpr int kHalf = 128;                           // one CTA's share of either
constexpr int kStepK = 64;                           // K per ring stage: one 128-byte swizzle row of bf16
constexpr uint32_t kShare = kHalf * kStepK * 2;      // 16 KB: one CTA's whole share of an operand per stage
constexpr int kMaxStages = 16;
constexpr uint32_t kRingBytes = 192 * 1024;
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 32 * (2 + kEpiWarps);
constexpr int kTmemCols = 2 * kTileCols;
constexpr int kChunk = 32;                           // accumulator columns an epilogue thread takes at a time
constexpr uint32_t kStagingWarp = 32 * kChunk * 4;   // an epilogue warp's outgoing chunk of fp32 (or two of bf16)
constexpr uint32_t kStagingBytes = kEpiWarps * kStagingWarp;
constexpr int kGroupRows = 16;                       // row tiles that share the sweep over the columns
// Polls of a wait: a second, for a poll of a barrier that does not complete
// suspends the warp for 3.9 us (measured).
#ifndef TF_TOPK_TEST_WAIT_TIMEOUT
constexpr uint32_t kWaitLimit = 1u << 18;
#else // test build (below): 16 ms
constexpr uint32_t kWaitLimit = 1u << 12;
#endif
constexpr uint32_t kFaultWait = 1;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLn2Rest = 7.35e-9f; // 1 / kLog2e (the float) less kLn2 (the float)

enum Mode { kLse, kProb, kHidden, kWeight, kGrads };

__device__ uint32_t g_head_loss_fault;

struct __align__(16) PairSmem {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;
};

// Rows that count, as the prepare kernel finds them.
struct RowHeader {
    int32_t count;
    float grad_scale; // largest finite |g|, or 1
    int32_t splits;   // shares of K that the hidden states' gradient is summed in
};

// What the epilogue needs of a packed row.
struct __align__(16) RowFacts {
    int32_t target;
    float lse2; // lse in powers of two
    float grad;
    float less_one; // of the target: p - 1
};

struct PairArgs {
    const RowHeader *header;  // null: every row counts, in its own place
    const RowFacts *facts;    // [count] of packed rows
    const void *target;       // int64 or int32 [rows], where rows are not packed
    int32_t target64;
    int32_t rows;             // all rows
    int32_t dim;
    int32_t vocab;
    int32_t begin, cols;      // the piece of the vocabulary [begin, begin + cols)
    int32_t width;            // columns of a tile
    int32_t stages;           // of the ring
    int32_t row_box;          // few rows: rows of A that both CTAs load, a multiple of 8
    int32_t slots;            // few rows: K steps of A, where all of it stays in shared memory, or 0
    int32_t pad_rows;         // row pitch of `partial`
    int32_t first;            // kHidden: the sums start here
    float2 *partial;          // kLse: [2 * column tiles][pad_rows]: reference exponent, sum; few rows: [2 or 4 * pairs]
};

// ---------------------------------------------------------------- PTX helpers

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}

// Address of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr(p)), "r"(rank));
    return r;
}

// Tells a barrier of the cluster that this warp has read its accumulator.
// Relaxed: what has to come before it are tensor memory loads, and their values
// are in registers by then (tcgen05.wait::ld), so that no later product can
// change them.  It rests on that, not on the memory model, in which the
// tcgen05.fence pair would want a release here.  A release at cluster scope
// would wait for the warp's stores to global memory as well: 2.5 us per tile
// (330 x 168 x 105859: 45 us with it, 38 without).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Bounded wait for the phase with this parity; gives up after kWaitLimit
// polls (recording the fault) or once another warp of this CTA has.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
{
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(saddr(bar)), "r"(parity)
                     : "memory");
        if (ok) return true;
        if (abort && *abort) return false;
    }
    atomicCAS(&g_head_loss_fault, 0u, kFaultWait);
    if (abort) *abort = 1;
    return false;
}

// Bounded wait of the wind-down: goes on whether or not the CTA gave up.
__device__ __forceinline__ bool mbar_drain(uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, nullptr); }

// As mbar_wait, by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
{
    const bool ok = mbar_wait(bar, parity, abort);
    return __all_sync(0xFFFFFFFFu, ok);
}

// Whether the phase with this parity has completed (no wait).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(saddr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// One lane of a converged warp, always the same.  The loops around TMA and
// MMA instructions run in the whole warp and only these instructions in the
// one lane: their operands then come from uniform registers (issued from a
// divergent lane, an MMA took 60 cycles and the 64-step loop 530, more than
// the products it issued).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// One box of a tensor map into this CTA's shared memory; its bytes count on
// the leading CTA's barrier.
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(saddr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// Shared-memory matrix descriptors of tiles written by TMA with the 128-byte
// swizzle (start address >> 4, leading byte offset at bit 16, stride byte
// offset at bit 32, version 1 at bit 46, swizzle mode 2 at bit 61).  K-major:
// eight 128-byte rows of 64 K steps are 1024 bytes apart (stride); the
// leading offset is not used.  MN-major: a 128-byte row holds 64 rows or
// columns of one K step, eight K steps are 1024 bytes apart (stride), and the
// next 64 rows or columns follow a whole box later (leading).
constexpr uint64_t kDescK = (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
constexpr uint64_t kDescMN =
    ((uint64_t)((kStepK * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);

__device__ __forceinline__ uint64_t desc_at(const void *p, uint64_t bits) { return bits | ((saddr(p) & 0x3FFFFu) >> 4); }

// Instruction descriptor of tcgen05.mma kind::f16: fp32 accumulator (bit 4),
// bf16 A and B (bits 7 and 10), A or B with M or N contiguous (bits 15 and
// 16), N / 8 at bit 17, M / 16 at bit 24.
__device__ __forceinline__ uint32_t instruction_desc(bool a_mn, bool b_mn, uint32_t n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((n >> 3) << 17) |
           ((uint32_t)(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// Arrive on this barrier in both CTAs of the pair once every tcgen05
// operation this thread issued before has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     saddr(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// This warp's 32 accumulator lanes (lane = thread), kChunk columns from
// `taddr`.  The wait stands in the same statement: until it is over nothing may
// touch the registers, not even to move or spill them.
__device__ __forceinline__ void tmem_take(uint32_t taddr, uint32_t (&r)[kChunk])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                   "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr)
                 : "memory");
}
// Sixteen columns added to what the thread has of them (fp32 bits).
__device__ __forceinline__ void tmem_add16(uint32_t taddr, uint32_t *to)
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) to[i] = __float_as_uint(__uint_as_float(to[i]) + __uint_as_float(r[i]));
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A warp's chunk of 32 rows goes out by TMA from shared memory: the warp
// writes its rows there (16-byte pieces swizzled as the tensor map expects,
// so that eight lanes meet eight bank groups), and one lane sends the box.
// (G of 3686 x 98592: 1062 us with 16-byte stores by row, 940 with 32-byte
// ones, 905 without any.)  The map cuts what lies past its extents.
__device__ __forceinline__ void send_box(const CUtensorMap *map, const void *box, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(saddr(box)), "r"(x), "r"(y)
                 : "memory");
}
// The same, added to what is there (fp32, in the L2).
__device__ __forceinline__ void add_box(const CUtensorMap *map, const void *box, int32_t x, int32_t y)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(saddr(box)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void box_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the last `kLeft` boxes of this thread have been read from shared memory.
template <int kLeft> __device__ __forceinline__ void box_read_wait()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void box_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// This lane's row of a 64-byte swizzled box: 32 bf16.
__device__ __forceinline__ void put_row_bf16(uint8_t *box, int lane, const uint32_t (&v)[kChunk / 2])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
// This lane's row of a 128-byte swizzled box: 32 fp32.
__device__ __forceinline__ void put_row_f32(uint8_t *box, int lane, const float (&v)[kChunk])
{
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

__device__ __forceinline__ int64_t target_of(const void *target, int target64, int row)
{
    return target64 ? static_cast<const int64_t *>(target)[row] : (int64_t)static_cast<const int32_t *>(target)[row];
}

// ---------------------------------------------------------------- the products

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Shares of K that the hidden states' gradient is summed in, `most` at most,
// so that its tiles come out in nearly whole rounds of the pairs; every share
// more costs its sums' traffic, taken as a fiftieth of a round.  One warp, a
// lane per candidate: kMostSplits at most, so that one tile (up to 256 rows and
// dims) keeps no more pairs busy.
constexpr int kMostSplits = 32;
__device__ __forceinline__ int best_splits(int row_tiles, int dim, int pairs, int most)
{
    const float per_share = __fdividef((float)row_tiles * (float)ceil_div(dim, kTileCols), (float)pairs); // of a round
    float cost = 3e38f;
    int best = most;
    const int s = (threadIdx.x & 31) + 1;
    if (s <= most) {
        cost = __fdividef(ceilf(per_share * (float)s - 1e-3f), (float)s) * (1.0f + 0.02f * (float)s);
        best = s;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, cost, d);
        const int os = __shfl_xor_sync(0xFFFFFFFFu, best, d);
        if (o < cost || (o == cost && os < best)) {
            cost = o;
            best = os;
        }
    }
    return best;
}

// A tile of the persistent schedule and its share [k0, k1) of the K steps.
struct Unit {
    int m, n, split, k0, k1;
};

template <int kMode> struct Shape {
    int m_tiles, n_tiles, k_steps, splits; // kGrads: the weight's
    int h_tiles, h_steps;                  // the hidden states' row tiles and K steps
    int64_t h_units;
    __device__ Shape(const PairArgs &a, int count)
    {
        const int row_tiles = max(1, ceil_div(count, kTileRows));
        splits = 1;
        h_tiles = h_steps = 0;
        h_units = 0;
        if (kMode == kLse || kMode == kProb) {
            m_tiles = row_tiles;
            n_tiles = ceil_div(a.cols, a.width);
            k_steps = ceil_div(a.dim, kStepK);
        } else {
            m_tiles = ceil_div(a.cols, kTileRows);
            n_tiles = ceil_div(a.dim, kTileCols);
            k_steps = max(1, ceil_div(count, kStepK));
            if (kMode != kWeight) {
                h_tiles = row_tiles;
                h_steps = ceil_div(a.cols, kStepK);
                splits = min(a.header->splits, h_steps);
                h_units = (int64_t)h_tiles * n_tiles * splits;
            }
        }
    }
    __device__ int64_t units() const { return h_units + (kMode == kHidden ? 0 : (int64_t)m_tiles * n_tiles); }
    // Whether a unit is a tile of d_weight.
    __device__ bool of_weight(int64_t u) const { return kMode == kWeight || (kMode == kGrads && u >= h_units); }
    __device__ Unit at(int64_t u) const { return units() <= INT32_MAX ? at_index((int32_t)u) : at_index(u); }

  private:
    template <typename I> __device__ Unit at_index(I u) const
    {
        Unit t;
        if (kMode == kHidden || (kMode == kGrads && u < (I)h_units)) {
            t.m = (int)(u % h_tiles);
            const I r = u / h_tiles;
            t.n = (int)(r % n_tiles);
            t.split = (int)(r / n_tiles);
            t.k0 = (int)((int64_t)h_steps * t.split / splits);
            t.k1 = (int)((int64_t)h_steps * (t.split + 1) / splits);
            return t;
        }
        // groups of kGroupRows row tiles; in a group the row tile moves
        // first, so that the pairs at work share the tiles of B
        u -= (I)h_units;
        int g = 0, in_group = m_tiles;
        I r = u;
        if (m_tiles > kGroupRows) {
            const I per_group = (I)kGroupRows * n_tiles;
            g = (int)(u / per_group);
            r = u - g * per_group;
            in_group = min(kGroupRows, m_tiles - g * kGroupRows);
        }
        t.m = g * kGroupRows + (in_group > 1 ? (int)(r % in_group) : 0);
        t.n = in_group > 1 ? (int)(r / in_group) : (int)r;
        t.split = 0;
        t.k0 = 0;
        t.k1 = k_steps;
        return t;
    }
};

// K steps [begin, end) of one tile, that many ring stages from `s` on, into
// accumulator `d`.  False when a wait gave up.
template <bool kAMN, bool kBMN>
__device__ __forceinline__ bool issue_tile(PairSmem &sm, uint32_t d, uint32_t idesc, int begin, int end, uint32_t &s,
                                           uint32_t &parity, uint32_t stages, const uint8_t *ring_a, uint32_t share_a, bool a_stays,
                                           const uint8_t *ring_b, uint32_t share_b, volatile uint32_t *abort)
{
    // 16 K steps: 32 bytes along a K-major row, 16 whole rows of an MN-major box
    constexpr uint64_t step_a = kAMN ? (16 * 128) >> 4 : 32 >> 4;
    constexpr uint64_t step_b = kBMN ? (16 * 128) >> 4 : 32 >> 4;
    bool ready = false;
    for (int k = begin; k < end; ++k) {
        if (!ready && !mbar_wait_warp(&sm.full[s], parity, abort)) return false;
        const uint32_t here = s;
        if (++s == stages) s = 0, parity ^= 1;
        const bool next = mbar_test(&sm.full[s], parity); // answered while the products are issued
        tc_fence_after();
        const uint64_t ad = desc_at(ring_a + (a_stays ? k : here) * share_a, kAMN ? kDescMN : kDescK);
        const uint64_t bd = desc_at(ring_b + here * share_b, kBMN ? kDescMN : kDescK);
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kStepK / 16; ++kk)
                mma_pair(d, ad + kk * step_a, bd + kk * step_b, idesc, k != begin || kk != 0);
            mma_commit_pair(&sm.empty[here]);
        }
        __syncwarp();
        ready = __all_sync(0xFFFFFFFFu, next);
    }
    return true;
}

// Rows of a product: any number, up to kHalf, and those where all their K
// steps stay in shared memory.
enum PairRows { kManyRows, kFewRows, kRowsStay };

// K steps of a tile that the tensor cores add up by themselves, in kLse; the
// epilogue adds such parts up, rounding to nearest.  The tensor cores cut off
// what an addition of 16 products leaves below the last place of its largest,
// always toward zero, and the error grows with the additions: one row's loss is
// off by 8.6e-7 of it at 2048 dims and by 14e-7 at 4096 in one sum, by 2.4e-7
// and 2.2e-7 in parts of 512 dims (1.6e-7 and 1.9e-7 by FMA throughout).  With
// few rows the parts cost little (15 x 2048 x 98592: 69.0 -> 71.0 us in a
// graph).  With many rows, whose errors differ, 1000 losses at 4096 dims are off
// by 6.1e-7 in one sum, no more than by FMA (6.4e-7), and the parts' 128 sums a
// thread keep the kernels before and after this one from the SM: 333 x 2048 x
// 32771 takes 39.0 us in parts of 1024 dims, 35.3 in one.
template <PairRows kRows> constexpr int kPartSteps = kRows == kManyRows ? 64 : 8;

// Parts that a tile's K steps are summed in, each in an accumulator of its own.
template <PairRows kRows, bool kParts> __device__ __forceinline__ int parts_of_sum(int steps)
{
    return kParts ? ceil_div(steps, kPartSteps<kRows>) : 1;
}

template <int kMode, PairRows kRows, bool kParts>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ CUtensorMap map_wa, const __grid_constant__ CUtensorMap map_wb,
                        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_wout,
                        PairArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    // Rows of A that are not loaded leave whatever the ring holds in their
    // lanes of the accumulator, which nothing reads; the MMA reads on from a
    // short share of A into what follows it in the ring.
    const int half_cols = kMode == kLse ? a.width / 2 : kHalf; // one CTA's share of B
    // (Whole shares have the ring's shape at compile time: the issuing thread
    // keeps up better, 615 against 631 us on 800 x 2048 x 248320.)
    constexpr bool kFew = kRows != kManyRows;
    const uint32_t share_a = kFew ? (uint32_t)a.row_box * kStepK * 2 : kShare;
    const uint32_t share_b = kFew ? (uint32_t)half_cols * kStepK * 2 : kShare;
    const uint32_t stages = kFew ? (uint32_t)a.stages : kRingBytes / (2 * kShare);
    constexpr bool stays = kRows == kRowsStay; // A is loaded with a pair's first tile only
    // Few rows: both CTAs load them, so that each has all columns of the tile
    // for them and the epilogue is shared; or the leading one alone, where the
    // stream of B is what counts (the loss of 15 x 2048 x 98592 takes 2.5 %
    // longer with two).
    constexpr bool both = kFew && (kMode != kLse || stays);
    uint8_t *ring_a = ring, *ring_b = ring + (stays ? (uint32_t)a.slots : stages) * share_a;
    uint8_t *staging = ring + kRingBytes; // 1024-byte aligned
    PairSmem &sm = *reinterpret_cast<PairSmem *>(staging + (kMode == kLse ? 0 : kStagingBytes));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = blockIdx.x & 1; // in the pair; rank 0 leads
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sm.tmem_base)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    grid_dependency_wait(); // the inputs may come from the kernel before on the stream
    if (kMode == kLse) grid_dependents_go(); // the rows' kernel may take its place beside this one

    const int count = a.header ? a.header->count : a.rows;
    const Shape<kMode> shape(a, count);
    const int64_t units = shape.units();
    volatile uint32_t *abort = &sm.abort;

    if (warp == 0) {
        // ---- TMA producer
        const uint32_t bytes_a = (!kFew || both ? 2 : 1) * share_a, bytes_b = 2 * (uint32_t)half_cols * kStepK * 2;
        const uint32_t full0 = peer_addr(&sm.full[0], 0); // the leading CTA's barriers
        uint32_t s = 0, turn = 0;                         // ring stage, times round the ring
        bool ok = true;
        for (int64_t u = pair; u < units && ok; u += pairs) {
            const Unit t = shape.at(u);
            const bool weight = shape.of_weight(u);
            const int row = t.m * kTileRows + (kFew ? 0 : (int)rank * kHalf);
            const int col = t.n * kTileCols + (int)rank * kHalf;
            const int voc = a.begin + t.n * a.width + (int)rank * half_cols;
            for (int k = t.k0; k < t.k1; ++k) {
                ok = *abort == 0 && (turn == 0 || mbar_wait(&sm.empty[s], (turn - 1) & 1, abort));
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (elect_one()) {
                    const bool new_a = !stays || u == pair, has_a = new_a && (!kFew || both || rank == 0);
                    if (rank == 0) mbar_expect_tx(&sm.full[s], new_a ? bytes_a + bytes_b : bytes_b);
                    const uint32_t bar = full0 + s * (uint32_t)sizeof(uint64_t);
                    uint8_t *da = ring_a + (stays ? k : s) * share_a, *db = ring_b + s * share_b;
                    const int kx = k * kStepK;
                    if (kMode == kLse || kMode == kProb) {
                        if (has_a) tma_load(da, &map_a, kx, row, bar);
                        tma_load(db, &map_b, kx, voc, bar);
                    } else if (!weight) {
                        if (has_a) tma_load(da, &map_a, kx, row, bar);
                        tma_load(db, &map_b, col, a.begin + kx, bar);
                        tma_load(db + kShare / 2, &map_b, col + 64, a.begin + kx, bar);
                    } else {
                        tma_load(da, &map_wa, row, kx, bar);
                        tma_load(da + kShare / 2, &map_wa, row + 64, kx, bar);
                        tma_load(db, &map_wb, col, kx, bar);
                        tma_load(db + kShare / 2, &map_wb, col + 64, kx, bar);
                    }
                }
                __syncwarp();
                if (++s == stages) s = 0, ++turn;
            }
        }
        // both CTAs' copies land before the pair leaves: the last fill of
        // each stage (the leader's barrier counts both CTAs' bytes).  Where one
        // does not, for a second, the others would not either.
        bool landed = rank == 0;
        for (uint32_t j = 0; j < stages && landed; ++j) {
            const uint32_t filled = j < s ? turn + 1 : turn; // times stage j was filled
            if (filled) landed = mbar_drain(&sm.full[j], (filled - 1) & 1);
        }
    } else if (warp == 1) {
        // ---- MMA issuer (the leading CTA's)
        if (rank == 0) {
            const uint32_t cols = (uint32_t)half_cols * 2;
            uint32_t s = 0, parity = 0, sum = 0;
            bool ok = true;
#ifdef TF_TOPK_TEST_WAIT_TIMEOUT
            ok = mbar_wait_warp(&sm.drain, 0, abort); // nothing completes it yet: the wait runs out
#endif
            for (int64_t u = pair; u < units && ok; u += pairs) {
                const Unit t = shape.at(u);
                const int steps = t.k1 - t.k0, parts = parts_of_sum<kRows, kParts>(steps);
                for (int part = 0; part < parts && ok; ++part, ++sum) {
                    const uint32_t buf = sum & 1, use = sum >> 1;
                    ok = use == 0 || mbar_wait_warp(&sm.acc_empty[buf], (use - 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * kTileCols;
                    const int begin = kParts ? part * kPartSteps<kRows> : 0;
                    const int end = kParts ? min(steps, begin + kPartSteps<kRows>) : steps;
                    if (kMode == kLse || kMode == kProb)
                        ok = issue_tile<false, false>(sm, d, instruction_desc(false, false, cols), begin, end, s, parity,
                                                      stages, ring_a, share_a, stays, ring_b, share_b, abort);
                    else if (!shape.of_weight(u))
                        ok = issue_tile<false, true>(sm, d, instruction_desc(false, true, cols), begin, end, s, parity,
                                                     stages, ring_a, share_a, false, ring_b, share_b, abort);
                    else
                        ok = issue_tile<true, true>(sm, d, instruction_desc(true, true, cols), begin, end, s, parity,
                                                    stages, ring_a, share_a, false, ring_b, share_b, abort);
                    if (!ok) break;
                    if (elect_one()) mma_commit_pair(&sm.acc_full[buf]);
                    __syncwarp();
                }
            }
            // every product is done before the TMEM is freed
            if (elect_one())
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 saddr(&sm.drain))
                             : "memory");
            __syncwarp();
            mbar_drain(&sm.drain, 0);
        }
    } else {
        // ---- epilogue
        const int q = warp & 3, h = (warp - 2) >> 2;
        const uint32_t acc_empty0 = peer_addr(&sm.acc_empty[0], 0), acc_empty1 = peer_addr(&sm.acc_empty[1], 0);
        uint8_t *box = staging + (warp - 2) * kStagingWarp; // this warp's
        uint32_t sent = 0;                                  // bf16 boxes alternate between its halves
        const auto send_bf16 = [&](const CUtensorMap *map, const uint32_t (&v)[kChunk / 2], int x, int y, bool any) {
            uint8_t *half = box + (sent & 1) * (kStagingWarp / 2);
            if (elect_one()) box_read_wait<1>();
            __syncwarp();
            put_row_bf16(half, lane, v);
            fence_async_proxy();
            __syncwarp();
            if (elect_one()) {
                if (any) send_box(map, half, x, y);
                box_commit();
            }
            __syncwarp();
            ++sent;
        };
        uint32_t done = 0; // accumulators taken
        // kLse: reference exponent (base 2), its logit, sum of exp2; with few
        // rows over all of the pair's tiles
        float ref = 0.0f, top = -INFINITY, sum = 0.0f;
        // few rows: the warps that have none (but for kProb's zeros) skip the tile
        const int first_row = (both ? 0 : (int)rank * kHalf) + 32 * q;
        const bool no_rows = kFew && kMode != kProb && first_row >= count;
        // a row's facts are fetched a tile ahead
        const auto row_of = [&](int m) { return m * kTileRows + first_row + lane; };
        // the share of a tile's columns that this warp takes, in whole chunks: a
        // half, or where both CTAs have the rows a quarter
        constexpr int parts = both ? 4 : 2;
        const int part = both ? 2 * h + (int)rank : h, all_chunks = half_cols / (kChunk / 2);
        const int first_chunk = all_chunks * part / parts, last_chunk = all_chunks * (part + 1) / parts;
        const auto facts_of = [&](int row) {
            RowFacts f = {-1, 0.0f, 0.0f, 0.0f};
            if ((kMode == kLse || kMode == kProb) && row < count) {
                if (a.facts) {
                    f = a.facts[row];
                } else {
                    const int64_t target = target_of(a.target, a.target64, row);
                    f.target = target >= 0 && target < a.vocab ? (int32_t)target : -1;
                }
            }
            return f;
        };
        // body(c, x) for the chunks of an accumulator (loading the next one
        // meanwhile costs more registers than it hides: 12 % slower tiles)
        const auto walk = [&](uint32_t taddr, int chunks, auto body) {
            for (int c = 0; c < chunks; ++c) {
                uint32_t r[kChunk];
                tmem_take(taddr + c * kChunk, r);
                float x[kChunk];
#pragma unroll
                for (int i = 0; i < kChunk; ++i) x[i] = __uint_as_float(r[i]);
                body(c, x);
            }
        };
        Unit t = {}, ahead = {};
        RowFacts facts = {}, facts_ahead = {};
        if (pair < units) {
            ahead = shape.at(pair);
            facts_ahead = facts_of(row_of(ahead.m));
        }
        // The next accumulator, once it is whole, and its return.
        const auto next_sum = [&]() {
            const bool ready = mbar_wait(&sm.acc_full[done & 1], (done >> 1) & 1, abort);
            if (!__all_sync(0xFFFFFFFFu, ready)) return false;
            tc_fence_after();
            return true;
        };
        const auto give_back = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(done & 1 ? acc_empty1 : acc_empty0);
            ++done;
        };
        for (int64_t u = pair; u < units; u += pairs) {
            t = ahead;
            facts = facts_ahead;
            const int row = row_of(t.m); // M index of this thread
            if (u + pairs < units) {
                ahead = shape.at(u + pairs);
                if (ahead.m != t.m) facts_ahead = facts_of(row_of(ahead.m));
            }
            if (!next_sum()) break;
            // the target's column of the piece
            const int at = facts.target >= a.begin && facts.target < a.begin + a.cols ? facts.target - a.begin : -1;
            const float lse2 = facts.lse2, g = kMode == kProb ? facts.grad / a.header->grad_scale : 0.0f;
            const uint32_t lanes = tmem + (done & 1) * kTileCols + ((uint32_t)(32 * q) << 16);
            // columns of the tile that this thread takes
            const int c0 = first_chunk * kChunk, chunks = no_rows ? 0 : last_chunk - first_chunk;
            // gradients: those that hold columns of them
            const int chunks_in_dim = min(chunks, ceil_div(max(0, a.dim - t.n * kTileCols - c0), kChunk));
            if (kMode == kGrads) { // boxes of the other kind may still be on their way out
                if (elect_one()) box_read_wait<0>();
                __syncwarp();
            }
            if constexpr (kMode == kLse) {
                if (!kFew) ref = 0.0f, top = -INFINITY, sum = 0.0f;
                const auto take = [&](int c, float (&x)[kChunk]) {
                    const int col = t.n * a.width + c0 + c * kChunk; // of the piece
                    const int left = a.cols - col;
                    if (left < kChunk)
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            if (i >= left) x[i] = -INFINITY;
                    const int hit = at - col;
                    if (__any_sync(0xFFFFFFFFu, (uint32_t)hit < (uint32_t)kChunk))
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            if (i == hit) x[i] = -INFINITY;
                    // four chains each: one of 32 steps is longer than the rest of the chunk
                    float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int i = 4; i < kChunk; ++i) m4[i & 3] = fmaxf(m4[i & 3], x[i]);
                    const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    if (m > top) {
                        // the reference of an infinite maximum is finite, so that inf and NaN show in the
                        // sum, and above all others, so that no part of the sum outdoes it
                        const float next = fminf(m * kLog2e, FLT_MAX);
                        sum *= top > -INFINITY ? exp2_fast(ref - next) : 1.0f;
                        ref = next;
                        top = m;
                    }
                    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) s4[i & 3] += exp2_fast(fmaf(x[i], kLog2e, -ref));
                    sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                };
                if constexpr (!kParts) {
                    walk(lanes + c0, chunks, take);
                    give_back();
                } else {
                    constexpr int most_chunks = (kFew && !both ? kFewCols : kTileCols) / kChunk / parts;
                    uint32_t sums[most_chunks][kChunk]; // fp32 bits
#pragma unroll
                    for (int c = 0; c < most_chunks; ++c)
                        if (c < chunks) tmem_take(lanes + c0 + c * kChunk, sums[c]);
                    give_back();
                    bool ok = true;
                    for (int piece = parts_of_sum<kRows, kParts>(t.k1 - t.k0); piece > 1; --piece) {
                        ok = next_sum();
                        if (!ok) break;
                        const uint32_t from = tmem + (done & 1) * kTileCols + ((uint32_t)(32 * q) << 16) + c0;
#pragma unroll
                        for (int c = 0; c < most_chunks; ++c)
                            if (c < chunks) {
                                tmem_add16(from + c * kChunk, &sums[c][0]);
                                tmem_add16(from + c * kChunk + 16, &sums[c][16]);
                            }
                        give_back();
                    }
                    if (!ok) break;
                    // rolled: the chunk's body four times over would be more
                    // code to fetch than the selections are to run
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        float x[kChunk];
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            uint32_t bits = sums[0][i];
#pragma unroll
                            for (int k = 1; k < most_chunks; ++k) bits = c == k ? sums[k][i] : bits;
                            x[i] = __uint_as_float(bits);
                        }
                        take(c, x);
                    }
                }
                if (row < count && !kFew)
                    a.partial[(size_t)(2 * t.n + h) * a.pad_rows + row] =
                        make_float2(top == -INFINITY ? -INFINITY : ref, sum);
            } else if (kMode == kProb) {
                // rows past the count are zeros up to the last K step of the
                // products over rows, and nothing reads those behind it
                const int end = max(1, ceil_div(count, kStepK)) * kStepK;
                walk(lanes + c0, row - lane < end ? chunks : 0, [&](int c, float (&x)[kChunk]) {
                    const int col = t.n * kTileCols + c0 + c * kChunk;
                    const int left = row < count ? a.cols - col : 0;
                    const int hit = at - col;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) x[i] = exp2_fast(fmaf(x[i], kLog2e, -lse2));
                    if (__any_sync(0xFFFFFFFFu, (uint32_t)hit < (uint32_t)kChunk))
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            x[i] = i == hit ? facts.less_one : x[i]; // (a conditional store costs 24 registers)
                    if (__any_sync(0xFFFFFFFFu, left < kChunk))
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) x[i] = i < left ? x[i] : 0.0f;
                    uint32_t out[kChunk / 2];
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i) out[i] = pack_bf16(x[2 * i] * g, x[2 * i + 1] * g);
                    send_bf16(&map_out, out, col, row - lane, true);
                });
            } else if (!shape.of_weight(u)) {
                walk(lanes + c0, chunks_in_dim, [&](int c, float (&x)[kChunk]) {
                    const int col = t.n * kTileCols + c0 + c * kChunk;
                    const bool any = row - lane < count; // rows past the count get sums nothing reads
                    if (elect_one()) box_read_wait<0>();
                    __syncwarp();
                    put_row_f32(box, lane, x);
                    fence_async_proxy();
                    __syncwarp();
                    if (elect_one() && any) {
                        const int y = t.split * a.pad_rows + row - lane;
                        if (a.first) send_box(&map_out, box, col, y);
                        else add_box(&map_out, box, col, y); // once per element and launch: the order is the pieces'
                        box_commit();
                    }
                    __syncwarp();
                });
            } else {
                const float scale = a.header->grad_scale;
                walk(lanes + c0, chunks_in_dim, [&](int c, float (&x)[kChunk]) {
                    const int col = t.n * kTileCols + c0 + c * kChunk;
                    uint32_t out[kChunk / 2];
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i) out[i] = pack_bf16(x[2 * i] * scale, x[2 * i + 1] * scale);
                    send_bf16(&map_wout, out, col, a.begin + row - lane, row - lane < a.cols);
                });
            }
            if constexpr (kMode != kLse) give_back();
        }
        if (kMode != kLse) box_wait(); // what this lane sent is written
        if (kMode == kLse && kFew) {
            const int row = first_row + lane;
            if (row < count)
                a.partial[(size_t)(parts * pair + part) * a.pad_rows + row] =
                    make_float2(top == -INFINITY ? -INFINITY : ref, sum);
        }
    }
    __syncwarp();
    if (kMode != kLse) grid_dependents_go();
    tc_fence_before();
    __syncthreads();
    // a pair that gave up may have copies in flight that no barrier of this
    // CTA counts: time for them to land (tens of times a copy's own)
    if (*abort)
        for (int i = 0; i < 64; ++i) __nanosleep(1000);
    cluster_sync(); // neither CTA leaves while the other may still reach its shared memory
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
    }
}

// ---------------------------------------------------------------- rows before and after

constexpr int kPrepareThreads = 1024;
constexpr int kPackRows = 4096; // rows whose order a CTA can hold

// A packed row: a copy of a hidden row, or zeros.
__device__ __forceinline__ void pack_row(__nv_bfloat16 *to, const __nv_bfloat16 *from, int dim, int thread, int threads)
{
    uint4 *dst = reinterpret_cast<uint4 *>(to);
    const uint4 *src = reinterpret_cast<const uint4 *>(from);
    for (int i = thread; i < dim / 8; i += threads) dst[i] = src ? src[i] : make_uint4(0, 0, 0, 0);
}

// A row's logit of one column by FMA, the same in lse and in the target's p - 1:
// 32 lanes' sums, added up with what each addition rounds away (x the sum, y the
// rest; in 64 bits a loss takes 1.6 us longer).  By a whole warp, the answer in
// every lane; without the two rows 0.
__device__ __forceinline__ float2 column_logit(const __nv_bfloat16 *hidden, const __nv_bfloat16 *weight, int dim, int lane)
{
    float dot = 0.0f;
    if (hidden) {
        const uint4 *hv = reinterpret_cast<const uint4 *>(hidden), *wv = reinterpret_cast<const uint4 *>(weight);
#pragma unroll 4
        for (int i = lane; i < dim / 8; i += 32) {
            const uint4 p = hv[i], w = wv[i];
            const uint32_t pa[4] = {p.x, p.y, p.z, p.w}, wa[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dot = fmaf(__uint_as_float(pa[k] << 16), __uint_as_float(wa[k] << 16), dot);
                dot = fmaf(__uint_as_float(pa[k] & 0xFFFF0000u), __uint_as_float(wa[k] & 0xFFFF0000u), dot);
            }
        }
    }
    float rest = 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, dot, d), more = __shfl_xor_sync(0xFFFFFFFFu, rest, d);
        const float sum = dot + other, part = sum - dot;
        rest += more + ((dot - (sum - part)) + (other - part)); // exact, of a finite sum
        dot = sum;
    }
    return make_float2(dot, fabsf(dot) < INFINITY ? rest : 0.0f);
}

// p - 1 of the packed rows' targets: a warp per row, neighbours in different
// CTAs, and few rows in those that copy none.
__device__ __forceinline__ void targets_less_one(const int32_t *order, int count, const void *target, int target64,
                                                 const float *lse, const __nv_bfloat16 *hidden, int64_t stride,
                                                 const __nv_bfloat16 *weight, int64_t weight_stride, int dim, RowFacts *facts)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    for (int j = (int)(threadIdx.x / 32 * gridDim.x + (gridDim.x - 1 - blockIdx.x)); j < count; j += (int)gridDim.x * warps) {
        const int r = order[j];
        const float l = lse[r];
        const float x = column_logit(hidden + (size_t)r * stride,
                                     weight + (size_t)target_of(target, target64, r) * weight_stride, dim, lane)
                            .x;
        if (lane == 0) facts[j].less_one = expm1f(x - l);
    }
}

// The rows that count, in their order (order[j] the row at place j and its
// facts, place[r] the row's place or -1), and the largest finite |g|, by
// which every g is divided before G is rounded to bf16: with one g for all
// rows (a mean) the target's entry of G is then exactly p - 1, and no g leaves
// bf16's range.  kCopy, up to kPackRows rows: every CTA finds the order for
// itself and copies its share of the rows, a launch less (2 us of 96 at
// 333x1032x32771; with more rows the scans would outweigh it and
// head_loss_gather_kernel copies); the first CTA writes the rest.  kGrad: the
// gradient's (the loss's has registers few enough to run beside the product).
template <bool kCopy, bool kGrad>
__global__ void __launch_bounds__(kPrepareThreads)
    head_loss_prepare_kernel(const void *target, int target64, int64_t ignore, const float *lse, const float *grad,
                             int rows, int vocab, int dim, int pairs, int most_splits, RowHeader *header,
                             int32_t *order, int32_t *place, RowFacts *facts, const __nv_bfloat16 *hidden,
                             int64_t stride, const __nv_bfloat16 *weight, int64_t weight_stride, int pitch,
                             __nv_bfloat16 *packed)
{
    __shared__ int32_t own_order[kCopy ? kPackRows : 1];
    __shared__ int warp_sum[32];
    __shared__ float warp_max[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    int base = 0;
    float top = 0.0f;
    for (int r0 = 0; r0 < rows; r0 += kPrepareThreads) {
        const int r = r0 + tid;
        bool counts = false;
        RowFacts fact = {-1, 0.0f, 0.0f, 0.0f};
        if (r < rows) {
            const int64_t t = target_of(target, target64, r);
            if (kGrad) {
                fact.lse2 = lse[r] * kLog2e;
                fact.grad = grad[r];
            }
            counts = t != ignore && t >= 0 && t < vocab;
            if (counts) {
                fact.target = (int32_t)t;
                if (fabsf(fact.grad) < INFINITY) top = fmaxf(top, fabsf(fact.grad));
            }
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, counts);
        if (lane == 0) warp_sum[warp] = __popc(mask);
        __syncthreads();
        int before = base, total = 0;
        for (int w = 0; w < 32; ++w) {
            const int n = warp_sum[w];
            if (w < warp) before += n;
            total += n;
        }
        const int at = before + __popc(mask & ((1u << lane) - 1u));
        if (kCopy && counts) own_order[at] = r;
        if (r < rows && blockIdx.x == 0) {
            place[r] = counts ? at : -1;
            if (counts) {
                if (!kCopy) order[at] = r;
                facts[at].target = fact.target; // (less_one: targets_less_one)
                facts[at].lse2 = fact.lse2;
                facts[at].grad = fact.grad;
            }
        }
        base += total;
        __syncthreads();
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    if (warp == 0 && blockIdx.x == 0) {
        top = warp_max[lane];
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const int splits = best_splits(max(1, ceil_div(base, kTileRows)), dim, pairs, most_splits);
        if (lane == 0) {
            header->count = base;
            header->grad_scale = top > 0.0f ? top : 1.0f;
            header->splits = splits;
        }
    }
    if (kCopy) { // 256 threads a row
        if (kGrad)
            targets_less_one(own_order, base, target, target64, lse, hidden, stride, weight, weight_stride, dim, facts);
        const int end = max(1, ceil_div(base, kTileRows)) * kTileRows, at_once = kPrepareThreads / 256;
        for (int j = blockIdx.x * at_once + tid / 256; j < end; j += gridDim.x * at_once)
            pack_row(packed + (size_t)j * pitch, j < base ? hidden + (size_t)own_order[j] * stride : nullptr, dim, tid & 255,
                     256);
    }
    grid_dependents_go();
}

// The hidden rows that count, packed, with zero rows up to the next whole
// tile (the products sum over whole K steps of rows), and, with `lse`, their
// targets' p - 1.
__global__ void __launch_bounds__(256)
    head_loss_gather_kernel(const __nv_bfloat16 *hidden, int64_t stride, int dim, const RowHeader *header,
                            const int32_t *order, const void *target, int target64, const float *lse,
                            const __nv_bfloat16 *weight, int64_t weight_stride, RowFacts *facts, int pitch,
                            __nv_bfloat16 *packed)
{
    grid_dependency_wait();
    const int count = header->count;
    if (lse) targets_less_one(order, count, target, target64, lse, hidden, stride, weight, weight_stride, dim, facts);
    const int end = max(1, ceil_div(count, kTileRows)) * kTileRows;
    for (int j = blockIdx.x; j < end; j += gridDim.x)
        pack_row(packed + (size_t)j * pitch, j < count ? hidden + (size_t)order[j] * stride : nullptr, dim, threadIdx.x,
                 blockDim.x);
    grid_dependents_go();
}

constexpr int kRowsThreads = 256;
constexpr int kRowsPerCta = 4; // neighbours of `partial` share its 32-byte sectors

// exp2 sums over two reference exponents; (-inf, 0) is none yet.  The floor
// keeps -inf - -inf away.
__device__ __forceinline__ float2 join(float2 p, float2 q)
{
    const float top = fmaxf(fmaxf(p.x, q.x), -FLT_MAX);
    return make_float2(fmaxf(p.x, q.x), p.y * exp2_fast(p.x - top) + q.y * exp2_fast(q.x - top));
}

// The rows' losses: four rows per CTA.  The target's logit by FMA (while the
// products still run), the partial sums of a row joined, and both into loss
// and lse.  (`partial`, and `sums` of the kernel below, change while the kernel
// may already run: no __restrict__, which would let their loads be taken for
// loads of constants and move across the wait.)
__global__ void __launch_bounds__(kRowsThreads)
    head_loss_rows_kernel(const float2 *partial, int parts, int pad_rows, const int32_t *place,
                          const __nv_bfloat16 *__restrict__ hidden, int64_t hidden_stride,
                          const __nv_bfloat16 *__restrict__ weight, int64_t weight_stride,
                          int dim, int vocab, const void *target, int target64, int64_t ignore, int rows, float *loss,
                          float *lse)
{
    __shared__ float2 part[kRowsThreads / 32][kRowsPerCta];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.x * kRowsPerCta;
    // warps 0-3 = row: the target's logit.  The kernel before let this one start
    // only once the kernels before it had ended, so the inputs are there.
    const int r = r0 + warp;
    const int64_t t = warp < kRowsPerCta && r < rows ? target_of(target, target64, r) : ignore;
    const bool counts = t != ignore && t >= 0 && t < vocab;
    const float2 dot = column_logit(counts ? hidden + (size_t)r * hidden_stride : nullptr,
                                    counts ? weight + (size_t)t * weight_stride : nullptr, dim, lane);
    grid_dependency_wait();
    {
        // thread = (row tid % 4, every 64th part)
        const int rr = r0 + (tid & 3);
        const int j = rr < rows ? (place ? place[rr] : rr) : -1;
        float2 mine = make_float2(-INFINITY, 0.0f);
        constexpr int kAhead = 8; // loads in flight
        for (int p = tid >> 2; j >= 0 && p < parts; p += kAhead * kRowsThreads / 4) {
            float2 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int q = p + i * (kRowsThreads / 4);
                v[i] = q < parts ? partial[(size_t)q * pad_rows + j] : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) mine = join(mine, v[i]);
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            const float2 other = make_float2(__shfl_xor_sync(0xFFFFFFFFu, mine.x, d), __shfl_xor_sync(0xFFFFFFFFu, mine.y, d));
            mine = join(mine, other);
        }
        if (lane < 4) part[warp][lane] = mine;
    }
    __syncthreads();
    if (warp < kRowsPerCta && r < rows && lane == 0) {
        if (t == ignore) {
            loss[r] = lse[r] = 0.0f;
        } else if (t < 0 || t >= vocab) {
            loss[r] = lse[r] = NAN;
        } else {
            float2 all = part[0][warp];
            for (int w = 1; w < kRowsThreads / 32; ++w) all = join(all, part[w][warp]);
            // rest, and rest - dot with what is large cancelled before the logarithm of the sum is added, so
            // that a loss has the digits of its own size
            const float more = log2f(all.y) * kLn2;
            float rest = fmaf(all.x, kLn2, more);
            float above = fmaf(all.x, kLn2, -dot.x) + fmaf(all.x, kLn2Rest, -dot.y) + more;
            // a vocabulary of one column leaves no other
            if (all.x == -INFINITY && all.y == 0.0f) rest = -INFINITY, above = -INFINITY - dot.x;
            const float tail = log1pf(expf(-fabsf(above)));
            loss[r] = isnan(above) ? above : fmaxf(above, 0.0f) + tail;
            lse[r] = isnan(above) ? rest + dot.x : fmaxf(rest, dot.x) + tail; // (both infinite: that infinity)
        }
    }
    grid_dependents_go();
}

// d_hidden: the shares' sums of a row added up, scaled back and rounded;
// zeros for the rows that do not count.  kGroups, up to 1024 columns: few
// columns have many shares, and several threads add up each column's
// (46 x 144 x 164754: 77 -> 74 us).
template <bool kGroups>
__global__ void __launch_bounds__(256)
    head_loss_hidden_kernel(const float *sums, int pad_rows, int dim, const RowHeader *header,
                            const int32_t *place, int rows, __nv_bfloat16 *d_hidden)
{
    __shared__ float4 part[2][kGroups ? 256 : 1];
    grid_dependency_wait();
    const float scale = header->grad_scale;
    const int splits = header->splits;
    const int vecs = dim / 8, tid = threadIdx.x;
    // every by-th share of eight columns of a packed row
    const auto sum = [&](int j, int i, int from, int by, float (&v)[8]) {
#pragma unroll 4
        for (int s = from; s < splits; s += by) {
            const float4 *src = reinterpret_cast<const float4 *>(sums + ((size_t)s * pad_rows + j) * dim) + 2 * i;
            const float4 p = src[0], q = src[1];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
            v[4] += q.x, v[5] += q.y, v[6] += q.z, v[7] += q.w;
        }
    };
    const auto put = [&](int r, int i, const float (&v)[8]) {
        reinterpret_cast<uint4 *>(d_hidden + (size_t)r * dim)[i] =
            make_uint4(pack_bf16(v[0] * scale, v[1] * scale), pack_bf16(v[2] * scale, v[3] * scale),
                       pack_bf16(v[4] * scale, v[5] * scale), pack_bf16(v[6] * scale, v[7] * scale));
    };
    if constexpr (!kGroups) {
        for (int r = blockIdx.x; r < rows; r += gridDim.x) {
            const int j = place[r];
            for (int i = tid; i < vecs; i += 256) {
                float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (j >= 0) sum(j, i, 0, 1, v);
                put(r, i, v);
            }
        }
    } else {
        const int groups = 256 / vecs, group = tid / vecs, i = tid - group * vecs;
        for (int r = blockIdx.x; r < rows; r += gridDim.x) {
            const int j = place[r];
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (j >= 0 && group < groups) sum(j, i, group, groups, v);
            part[0][tid] = make_float4(v[0], v[1], v[2], v[3]);
            part[1][tid] = make_float4(v[4], v[5], v[6], v[7]);
            __syncthreads();
            if (group == 0) {
                for (int g = 1; g < min(groups, splits); ++g) {
                    const float4 p = part[0][g * vecs + i], q = part[1][g * vecs + i];
                    v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
                    v[4] += q.x, v[5] += q.y, v[6] += q.z, v[7] += q.w;
                }
                put(r, i, v);
            }
            __syncthreads();
        }
    }
    grid_dependents_go();
}

// ---------------------------------------------------------------- host side

constexpr size_t kPairSmemBytes = 1024 + (size_t)kRingBytes + kStagingBytes + sizeof(PairSmem);
constexpr size_t kLseSmemBytes = kPairSmemBytes - kStagingBytes; // leaves an SM room for the rows' kernel
static_assert(kPairSmemBytes <= 227 * 1024, "the pair kernel's shared memory fits one CTA");

constexpr int kMaxDevices = 64;
struct LossDevice {
    std::atomic<bool> ready{false};
    int pairs = 0; // CTA pairs that fit the device at a time
};
LossDevice g_loss_dev[kMaxDevices];
std::mutex g_loss_mutex;
PFN_cuTensorMapEncodeTiled_v12000 g_loss_encode = nullptr;

template <int kMode> constexpr bool kHasFew = kMode != kWeight && kMode != kGrads;
template <int kMode> constexpr bool kHasStay = kMode == kLse || kMode == kProb;

template <int kMode, PairRows kRows> cudaError_t allow_smem_of()
{
    cudaError_t e = cudaFuncSetAttribute(pair_product_kernel<kMode, kRows, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmemBytes);
    if constexpr (kMode == kLse)
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(pair_product_kernel<kMode, kRows, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kPairSmemBytes);
    return e;
}

template <int kMode> cudaError_t allow_smem()
{
    cudaError_t e = allow_smem_of<kMode, kManyRows>();
    if constexpr (kHasFew<kMode>)
        if (e == cudaSuccess) e = allow_smem_of<kMode, kFewRows>();
    if constexpr (kHasStay<kMode>)
        if (e == cudaSuccess) e = allow_smem_of<kMode, kRowsStay>();
    return e;
}

// Per device, once: the kernels' shared memory limits, the pairs the device
// holds, and the driver's tensor-map encoder.
int loss_setup(int *pairs, int *sm_count)
{
    int st = tf_topk_internal_device(sm_count);
    if (st != TF_TOPK_OK) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
    LossDevice &d = g_loss_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_loss_mutex);
        if (!d.ready.load(std::memory_order_relaxed)) {
            e = allow_smem<kLse>();
            if (e == cudaSuccess) e = allow_smem<kProb>();
            if (e == cudaSuccess) e = allow_smem<kHidden>();
            if (e == cudaSuccess) e = allow_smem<kWeight>();
            if (e == cudaSuccess) e = allow_smem<kGrads>();
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(*sm_count / 2 * 2), 1, 1);
            cfg.blockDim = dim3(kPairThreads, 1, 1);
            cfg.dynamicSmemBytes = kPairSmemBytes; // kLse's is less
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, pair_product_kernel<kLse, kManyRows, true>, &cfg);
            if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
            d.pairs = n < 1 ? 1 : n;
            if (!g_loss_encode) {
                void *fn = nullptr;
                cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
                e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
                if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
                if (q != cudaDriverEntryPointSuccess || !fn) return TF_TOPK_ERR_DEVICE;
                g_loss_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
            }
            d.ready.store(true, std::memory_order_release);
        }
    }
    *pairs = d.pairs;
    return TF_TOPK_OK;
}

// A 2-D bf16 tensor map, boxes of 64 x box_rows with the 128-byte swizzle;
// coordinates past either extent read as zero.
bool encode_map(CUtensorMap *map, const void *p, int64_t inner, int64_t outer, int64_t stride, int box_rows)
{
    cuuint64_t gdim[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    cuuint64_t gstride[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {(cuuint32_t)kStepK, (cuuint32_t)box_rows};
    cuuint32_t estride[2] = {1, 1};
    return g_loss_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), gdim, gstride, box, estride,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of an output: boxes of kChunk x 32, bf16 (64-byte swizzle) or fp32
// (128-byte swizzle); what lies past either extent is not written.
bool encode_out(CUtensorMap *map, const void *p, bool f32, int64_t inner, int64_t outer)
{
    cuuint64_t gdim[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    cuuint64_t gstride[1] = {(cuuint64_t)inner * (f32 ? 4 : 2)};
    cuuint32_t box[2] = {(cuuint32_t)kChunk, 32};
    cuuint32_t estride[2] = {1, 1};
    return g_loss_encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void *>(p), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t config(int grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute *attr)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Tensor maps of a product: operands and output, and those of kGrads' second kind.
struct PairMaps {
    CUtensorMap a, b, wa, wb, out, wout;
};

// The ring of a product with up to kHalf rows: as many rows of A as there are
// (in eights), and the stages take what is left (15 x 2048 x 98592: 74 us, with
// whole shares of A 128).  Rows of few K steps stay beside the ring instead of
// coming again with every tile.
bool set_ring(PairArgs &a, int mode, int64_t rows)
{
    if (mode == kWeight || mode == kGrads || rows > kHalf) return false;
    a.row_box = (int32_t)((rows + 7) / 8 * 8);
    const int cols = mode == kHidden ? kHalf : a.width / 2;
    const uint32_t row = kStepK * 2;
    const int64_t steps = ((int64_t)a.dim + kStepK - 1) / kStepK, all = steps * a.row_box * row;
    const bool stays = mode != kHidden && all <= kRingBytes / 8;
    a.slots = stays ? (int32_t)steps : 0;
    const int fit = (int)(stays ? (kRingBytes - all) / (cols * row) : kRingBytes / ((a.row_box + cols) * row));
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    return true;
}

template <int kMode, PairRows kRows> auto product_kernel(int dim)
{
    if constexpr (kMode == kLse)
        if (dim > kPartSteps<kRows> * kStepK) return pair_product_kernel<kMode, kRows, true>;
    return pair_product_kernel<kMode, kRows, false>;
}

template <int kMode>
cudaError_t launch_product(const PairMaps &m, PairArgs &a, int64_t most_units, int pairs, cudaStream_t stream)
{
    const bool few = set_ring(a, kMode, a.rows);
    cudaLaunchAttribute attr[1];
    const int64_t n = most_units < pairs ? most_units : pairs;
    const cudaLaunchConfig_t cfg = config((int)(2 * n), kPairThreads, kMode == kLse ? kLseSmemBytes : kPairSmemBytes, stream, attr);
    auto kernel = product_kernel<kMode, kManyRows>(a.dim);
    if constexpr (kHasFew<kMode>)
        if (few) kernel = product_kernel<kMode, kFewRows>(a.dim);
    if constexpr (kHasStay<kMode>)
        if (few && a.slots) kernel = product_kernel<kMode, kRowsStay>(a.dim);
    return cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, m.wa, m.wb, m.out, m.wout, a);
}

// Row pitch of the packed hidden states: whole 128-byte lines, whatever dim.
int64_t packed_pitch(int64_t dim) { return (dim + kStepK - 1) / kStepK * kStepK; }

int64_t pad_rows_of(int64_t rows) { return (rows + kTileRows - 1) / kTileRows * kTileRows; }

// Carves a workspace into 256-byte aligned parts.
struct Carver {
    uintptr_t at;
    explicit Carver(const void *p) : at((reinterpret_cast<uintptr_t>(p) + 255) & ~(uintptr_t)255) {}
    template <typename T> T *take(int64_t n)
    {
        T *p = reinterpret_cast<T *>(at);
        at += ((size_t)n * sizeof(T) + 255) & ~(size_t)255;
        return p;
    }
};

// Columns of a tile for the forward product: the widest tile moves the
// fewest bytes through shared memory, a narrower one may fill the last round
// of the pairs better.  A round costs about its width plus 32 columns.  Of
// packed rows the host does not know how many count: all of them and half are
// weighed alike.  With few rows a thread of the epilogue then has fewer sums in
// its registers (15 x 2048 x 98592: 76.6 us with up to 256 columns, 75.2 with
// 192).
int tile_width(int64_t rows, int64_t vocab, int pairs)
{
    const int64_t m = pad_rows_of(rows) / kTileRows;
    int best = kTileCols;
    int64_t least = INT64_MAX;
    for (int w = rows <= kHalf ? kFewCols : kTileCols; w >= 64; w -= 64) {
        const int64_t tiles = (vocab + w - 1) / w;
        const int64_t rounds = (m * tiles + pairs - 1) / pairs + ((m + 1) / 2 * tiles + pairs - 1) / pairs;
        const int64_t cost = rounds * (w + 32);
        if (cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

// Rows the loss takes at a time: its workspace grows with them (16 bytes per
// row and tile), and so many fill the device hundreds of times over.
constexpr int64_t kLossRows = 16384;

struct LossSpace {
    RowHeader *header;
    int32_t *order, *place;
    RowFacts *facts;
    __nv_bfloat16 *packed;
    float2 *partial;
    size_t bytes;
};

// Rows are packed when they fill more than one row tile (then every ignored
// row saves its share of the product).
LossSpace loss_space(const void *p, int64_t rows, int64_t dim, int64_t parts)
{
    Carver c(p);
    LossSpace s = {};
    if (rows > kTileRows) {
        s.header = c.take<RowHeader>(1);
        s.order = c.take<int32_t>(rows);
        s.place = c.take<int32_t>(rows);
        s.facts = c.take<RowFacts>(rows);
        s.packed = c.take<__nv_bfloat16>(pad_rows_of(rows) * packed_pitch(dim));
    }
    s.partial = c.take<float2>(parts * pad_rows_of(rows));
    s.bytes = (size_t)(c.at - (reinterpret_cast<uintptr_t>(p))) + 256;
    return s;
}

// Parts of a row's sum: two halves per tile, or at most four quarters per pair
// with few rows.
int64_t sum_parts(int64_t rows, int64_t tiles, int pairs)
{
    return rows > kHalf ? 2 * tiles : 4 * (tiles < pairs ? tiles : pairs);
}

// Bytes of a workspace at `p` that serves every block of rows.
size_t loss_bytes(const void *p, int64_t rows, int64_t dim, int64_t vocab, int pairs)
{
    size_t most = 0;
    for (const int64_t n : {rows < kLossRows ? rows : kLossRows, rows % kLossRows}) {
        if (n == 0) continue;
        const int width = tile_width(n, vocab, pairs);
        const size_t bytes = loss_space(p, n, dim, sum_parts(n, (vocab + width - 1) / width, pairs)).bytes;
        most = bytes > most ? bytes : most;
    }
    return most;
}

struct GradSpace {
    RowHeader *header;
    int32_t *order, *place;
    RowFacts *facts;
    __nv_bfloat16 *packed;
    float *sums;
    __nv_bfloat16 *prob;
    int splits;
    int64_t piece; // columns of a piece
    size_t bytes;
};

constexpr int64_t kProbBytes = 256ll << 20; // G of a piece, where the caller has the room

// Shares the workspace holds sums for: few tiles want many, and from 16
// rounds on a share more no longer saves what its sums cost.
int most_splits(int64_t rows, int64_t dim, int pairs)
{
    const int64_t tiles = pad_rows_of(rows) / kTileRows * ((dim + kTileCols - 1) / kTileCols);
    const int64_t few = (2 * (int64_t)pairs + tiles - 1) / tiles, many = (16 * (int64_t)pairs + tiles - 1) / tiles;
    const int64_t s = few > 4 ? few : many < 4 ? many : 4;
    return (int)(s > kMostSplits ? kMostSplits : s);
}

GradSpace grad_space(const void *p, int64_t rows, int64_t dim, int64_t vocab, int pairs, bool hidden, int64_t piece)
{
    Carver c(p);
    GradSpace s = {};
    s.piece = piece;
    s.splits = most_splits(rows, dim, pairs);
    const int64_t pad = pad_rows_of(rows);
    s.header = c.take<RowHeader>(1);
    s.order = c.take<int32_t>(rows);
    s.place = c.take<int32_t>(rows);
    s.facts = c.take<RowFacts>(rows);
    s.packed = c.take<__nv_bfloat16>(pad * packed_pitch(dim));
    if (hidden) s.sums = c.take<float>((int64_t)s.splits * pad * dim);
    s.prob = c.take<__nv_bfloat16>(pad * piece);
    s.bytes = (size_t)(c.at - (reinterpret_cast<uintptr_t>(p))) + 256;
    return s;
}

int64_t whole_piece(int64_t vocab) { return (vocab + kTileCols - 1) / kTileCols * kTileCols; }

// The recommended columns of a piece: G of up to kProbBytes, at least one
// tile, and the width (from half of that on) at which the tiles of G come out
// in the fewest rounds of the pairs, a launch costing about as much as half a
// round.
int64_t good_piece(int64_t rows, int64_t vocab, int pairs)
{
    const int64_t row_tiles = pad_rows_of(rows) / kTileRows, all = whole_piece(vocab) / kTileCols;
    int64_t most = kProbBytes / (2 * pad_rows_of(rows)) / kTileCols;
    if (most < 1) most = 1;
    if (most >= all) return all * kTileCols; // one piece
    int64_t best = most;
    double least = 1e300;
    for (int64_t t = most; t >= 1 && 2 * t >= most; --t) {
        const int64_t whole = all / t, rest = all % t;
        const double cost = (double)(whole * ((row_tiles * t + pairs - 1) / pairs) + (row_tiles * rest + pairs - 1) / pairs) +
                            0.5 * (double)(whole + (rest > 0));
        if (cost < least) {
            least = cost;
            best = t;
        }
    }
    return best * kTileCols;
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool bad_shape(int64_t rows, int32_t dim, int64_t vocab)
{
    return rows < 0 || rows > TF_TOPK_HEAD_LOSS_MAX_ROWS || dim < 8 || dim % 8 != 0 || vocab < 1 ||
           vocab > (int64_t)INT32_MAX - 1024;
}

bool bad_stride(int64_t stride, int64_t dim, int64_t n)
{
    // 16-byte rows whose byte offsets stay below the tensor maps' 2^40
    return stride < dim || stride % 8 != 0 || stride >= (1ll << 39) || (n > 0 && stride > INT64_MAX / 4 / n);
}

// Finds and packs the rows that count (`lse`, `grad` null for the loss alone).
template <typename Space>
cudaError_t pack_rows(const Space &s, const void *hidden, int64_t stride, const void *weight, int64_t weight_stride,
                      int64_t rows, int32_t dim, int64_t vocab, const void *target, int32_t target_bytes,
                      int64_t ignore, const float *lse, const float *grad,
                      int pairs, int splits, int sms, cudaStream_t stream)
{
    const auto *from = static_cast<const __nv_bfloat16 *>(hidden), *head = static_cast<const __nv_bfloat16 *>(weight);
    const int pitch = (int)packed_pitch(dim), wide = target_bytes == 8;
    cudaLaunchAttribute attr[1];
    const auto prepare = [&](auto kernel, int64_t ctas) {
        const cudaLaunchConfig_t cfg = config((int)(ctas < sms ? ctas : sms), kPrepareThreads, 0, stream, attr);
        return cudaLaunchKernelEx(&cfg, kernel, target, wide, ignore, lse, grad, (int)rows, (int)vocab, (int)dim, pairs, splits,
                                  s.header, s.order, s.place, s.facts, from, stride, head, weight_stride, pitch, s.packed);
    };
    if (rows <= kPackRows)
        return prepare(grad ? head_loss_prepare_kernel<true, true> : head_loss_prepare_kernel<true, false>,
                       (pad_rows_of(rows) + 3) / 4);
    const cudaError_t e =
        prepare(grad ? head_loss_prepare_kernel<false, true> : head_loss_prepare_kernel<false, false>, 1);
    if (e != cudaSuccess) return e;
    const cudaLaunchConfig_t cfg = config((int)(rows < 4 * sms ? rows : 4 * sms), 256, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, head_loss_gather_kernel, from, stride, (int)dim, (const RowHeader *)s.header,
                              (const int32_t *)s.order, target, wide, lse, head, weight_stride, s.facts, pitch, s.packed);
}

// One block of rows of the loss (checked arguments).
int loss_of_rows(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride, int64_t rows,
                 int32_t dim, int64_t vocab, const void *target, int32_t target_bytes, int64_t ignore, void *workspace,
                 float *loss, float *lse, int pairs, int sms, cudaStream_t strm)
{
    const int width = tile_width(rows, vocab, pairs);
    const int64_t tiles = (vocab + width - 1) / width;
    const int64_t most_parts = sum_parts(rows, tiles, pairs);
    const LossSpace s = loss_space(workspace, rows, dim, most_parts);
    PairMaps m = {};
    const bool packed = s.packed != nullptr;
    const int box = rows <= kHalf ? (int)((rows + 7) / 8 * 8) : kHalf; // rows of A a CTA loads (set_ring)
    if (!encode_map(&m.a, packed ? s.packed : hidden, dim, packed ? pad_rows_of(rows) : rows,
                    packed ? packed_pitch(dim) : hidden_stride, box) ||
        !encode_map(&m.b, weight, dim, vocab, weight_stride, width / 2))
        return tf_topk_internal_fail_cuda((int)cudaErrorInvalidValue);
    cudaLaunchAttribute attr[1];
    cudaError_t e = cudaSuccess;
    if (packed)
        e = pack_rows(s, hidden, hidden_stride, weight, weight_stride, rows, dim, vocab, target, target_bytes, ignore,
                      nullptr, nullptr, pairs, 1, sms, strm);
    PairArgs a = {};
    a.header = s.header;
    a.facts = s.facts;
    a.target = target;
    a.target64 = target_bytes == 8;
    a.rows = (int32_t)rows;
    a.dim = dim;
    a.vocab = (int32_t)vocab;
    a.begin = 0;
    a.cols = (int32_t)vocab;
    a.width = width;
    a.pad_rows = (int32_t)pad_rows_of(rows);
    a.partial = s.partial;
    const int64_t units = tiles * (pad_rows_of(rows) / kTileRows);
    if (e == cudaSuccess) e = launch_product<kLse>(m, a, units, pairs, strm);
    const int parts = (int)(rows > kHalf || a.slots ? most_parts : most_parts / 2);
    const cudaLaunchConfig_t cfg =
        config((int)((rows + kRowsPerCta - 1) / kRowsPerCta), kRowsThreads, 0, strm, attr);
    if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, head_loss_rows_kernel, (const float2 *)s.partial,
                               parts, a.pad_rows, (const int32_t *)s.place, static_cast<const __nv_bfloat16 *>(hidden),
                               hidden_stride, static_cast<const __nv_bfloat16 *>(weight), weight_stride, (int)dim,
                               (int)vocab, target,
                               (int)(target_bytes == 8), ignore, (int)rows, loss, lse);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}

int run_loss(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride, int64_t rows,
             int32_t dim, int64_t vocab, const void *target, int32_t target_bytes, int64_t ignore, void *workspace,
             size_t workspace_bytes, float *loss, float *lse, void *stream)
{
    if (bad_shape(rows, dim, vocab) || bad_stride(hidden_stride, dim, rows) || bad_stride(weight_stride, dim, vocab))
        return TF_TOPK_ERR_SHAPE;
    if (rows == 0) return TF_TOPK_OK;
    if (target_bytes != 4 && target_bytes != 8) return TF_TOPK_ERR_ARG;
    if (!hidden || !weight || !target || !workspace || !loss || !lse) return TF_TOPK_ERR_NULL;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(target, (size_t)target_bytes) || !aligned(loss, 4) ||
        !aligned(lse, 4))
        return TF_TOPK_ERR_ALIGN;
    int pairs = 0, sms = 0;
    const int st = loss_setup(&pairs, &sms);
    if (st != TF_TOPK_OK) return st;
    if (loss_bytes(workspace, rows, dim, vocab, pairs) > workspace_bytes) return TF_TOPK_ERR_SCRATCH;
    for (int64_t r = 0; r < rows; r += kLossRows) {
        const int64_t n = rows - r < kLossRows ? rows - r : kLossRows;
        const int s = loss_of_rows(static_cast<const char *>(hidden) + (size_t)r * hidden_stride * 2, hidden_stride, weight,
                                   weight_stride, n, dim, vocab,
                                   static_cast<const char *>(target) + (size_t)r * target_bytes, target_bytes, ignore,
                                   workspace, loss + r, lse + r, pairs, sms, static_cast<cudaStream_t>(stream));
        if (s != TF_TOPK_OK) return s;
    }
    return TF_TOPK_OK;
}

int run_grad(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride, int64_t rows,
             int32_t dim, int64_t vocab, const void *target, int32_t target_bytes, int64_t ignore, const float *lse,
             const float *grad_loss, void *workspace, size_t workspace_bytes, void *d_hidden, void *d_weight,
             void *stream)
{
    if (bad_shape(rows, dim, vocab) || bad_stride(hidden_stride, dim, rows) || bad_stride(weight_stride, dim, vocab))
        return TF_TOPK_ERR_SHAPE;
    if (rows == 0) { // nothing flows to the weight
        if (!d_weight) return TF_TOPK_OK;
        if (!aligned(d_weight, 16)) return TF_TOPK_ERR_ALIGN;
        int sms = 0;
        const int st = tf_topk_internal_device(&sms);
        if (st != TF_TOPK_OK) return st;
        const cudaError_t e =
            cudaMemsetAsync(d_weight, 0, (size_t)vocab * dim * 2, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
    }
    if (target_bytes != 4 && target_bytes != 8) return TF_TOPK_ERR_ARG;
    if (!hidden || !weight || !target || !lse || !grad_loss || !workspace || (!d_hidden && !d_weight))
        return TF_TOPK_ERR_NULL;
    if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(d_hidden, 16) || !aligned(d_weight, 16) ||
        !aligned(target, (size_t)target_bytes) || !aligned(lse, 4) || !aligned(grad_loss, 4))
        return TF_TOPK_ERR_ALIGN;
    int pairs = 0, sms = 0;
    const int st = loss_setup(&pairs, &sms);
    if (st != TF_TOPK_OK) return st;
    // the widest pieces the workspace holds, up to the recommended ones
    int64_t piece = good_piece(rows, vocab, pairs);
    if (grad_space(workspace, rows, dim, vocab, pairs, d_hidden != nullptr, piece).bytes > workspace_bytes) {
        const size_t least = grad_space(workspace, rows, dim, vocab, pairs, d_hidden != nullptr, kTileCols).bytes;
        if (least > workspace_bytes) return TF_TOPK_ERR_SCRATCH;
        piece = kTileCols + (int64_t)((workspace_bytes - least) / (2 * (size_t)pad_rows_of(rows))) / kTileCols * kTileCols;
    }
    const GradSpace s = grad_space(workspace, rows, dim, vocab, pairs, d_hidden != nullptr, piece);
    const int64_t pad = pad_rows_of(rows);
    const cudaStream_t strm = static_cast<cudaStream_t>(stream);
    const int box = rows <= kHalf ? (int)((rows + 7) / 8 * 8) : kHalf; // rows of A a CTA loads (set_ring)
    PairMaps prob = {}, grads = {};
    if (!encode_map(&prob.a, s.packed, dim, pad, packed_pitch(dim), box) || !encode_map(&prob.b, weight, dim, vocab, weight_stride, kHalf) ||
        !encode_out(&prob.out, s.prob, false, piece, pad) ||
        (d_hidden && (!encode_map(&grads.a, s.prob, piece, pad, piece, box) ||
                      !encode_map(&grads.b, weight, dim, vocab, weight_stride, kStepK) ||
                      !encode_out(&grads.out, s.sums, true, dim, pad * s.splits))) ||
        (d_weight && (!encode_map(&grads.wa, s.prob, piece, pad, piece, kStepK) ||
                      !encode_map(&grads.wb, s.packed, dim, pad, packed_pitch(dim), kStepK) ||
                      !encode_out(&grads.wout, d_weight, false, dim, vocab))))
        return tf_topk_internal_fail_cuda((int)cudaErrorInvalidValue);
    // every share of the sums starts in the first piece, the widest
    const int64_t steps = ((vocab < piece ? vocab : piece) + kStepK - 1) / kStepK;
    const int splits = (int)(s.splits < steps ? s.splits : steps);
    cudaLaunchAttribute attr[1];
    cudaError_t e = pack_rows(s, hidden, hidden_stride, weight, weight_stride, rows, dim, vocab, target, target_bytes,
                              ignore, lse, grad_loss, pairs, splits, sms, strm);
    PairArgs a = {};
    a.header = s.header;
    a.facts = s.facts;
    a.target = target;
    a.target64 = target_bytes == 8;
    a.rows = (int32_t)rows;
    a.dim = dim;
    a.vocab = (int32_t)vocab;
    a.width = kTileCols;
    a.pad_rows = (int32_t)pad;
    const int64_t row_tiles = pad / kTileRows, dim_tiles = (dim + kTileCols - 1) / kTileCols;
    for (int64_t begin = 0; begin < vocab && e == cudaSuccess; begin += piece) {
        a.begin = (int32_t)begin;
        a.cols = (int32_t)(vocab - begin < piece ? vocab - begin : piece);
        a.first = begin == 0;
        const int64_t col_tiles = (a.cols + kTileCols - 1) / kTileCols;
        const int64_t hidden_units = row_tiles * dim_tiles * splits, weight_units = col_tiles * dim_tiles;
        e = launch_product<kProb>(prob, a, row_tiles * col_tiles, pairs, strm);
        if (e != cudaSuccess) break;
        if (d_hidden && d_weight && rows > kHalf) {
            e = launch_product<kGrads>(grads, a, hidden_units + weight_units, pairs, strm);
            continue;
        }
        if (d_hidden) e = launch_product<kHidden>(grads, a, hidden_units, pairs, strm);
        if (e == cudaSuccess && d_weight)
            e = launch_product<kWeight>(grads, a, weight_units, pairs, strm);
    }
    if (e == cudaSuccess && d_hidden) {
        const cudaLaunchConfig_t cfg = config((int)(rows < 8 * sms ? rows : 8 * sms), 256, 0, strm, attr);
        e = cudaLaunchKernelEx(&cfg, dim <= 1024 ? head_loss_hidden_kernel<true> : head_loss_hidden_kernel<false>,
                               (const float *)s.sums, a.pad_rows, (int)dim, (const RowHeader *)s.header,
                               (const int32_t *)s.place, (int)rows, static_cast<__nv_bfloat16 *>(d_hidden));
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}

} // namespace

// This file's fault word, read and cleared (tf_topk_device_fault reports it).
uint32_t tf_topk_internal_head_loss_fault_take()
{
    uint32_t f = 0;
    if (cudaMemcpyFromSymbol(&f, g_head_loss_fault, sizeof f) != cudaSuccess) return 0;
    if (f) {
        const uint32_t zero = 0;
        cudaMemcpyToSymbol(g_head_loss_fault, &zero, sizeof zero);
    }
    return f;
}

extern "C" {

int tf_topk_head_loss_bf16(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride,
                           int64_t rows, int32_t dim, int64_t vocab, const void *target, int32_t target_bytes,
                           int64_t ignore_index, void *workspace, size_t workspace_bytes, float *out_loss,
                           float *out_lse, void *stream)
{
    return run_loss(hidden, hidden_stride, weight, weight_stride, rows, dim, vocab, target, target_bytes, ignore_index,
                    workspace, workspace_bytes, out_loss, out_lse, stream);
}

size_t tf_topk_head_loss_bf16_workspace(int64_t rows, int32_t dim, int64_t vocab)
{
    int pairs = 0, sms = 0;
    if (rows < 1 || bad_shape(rows, dim, vocab) || loss_setup(&pairs, &sms) != TF_TOPK_OK) return 0;
    return loss_bytes(nullptr, rows, dim, vocab, pairs) + 256;
}

int tf_topk_head_loss_grad_bf16(const void *hidden, int64_t hidden_stride, const void *weight, int64_t weight_stride,
                                int64_t rows, int32_t dim, int64_t vocab, const void *target, int32_t target_bytes,
                                int64_t ignore_index, const float *lse, const float *grad_loss, void *workspace,
                                size_t workspace_bytes, void *out_grad_hidden, void *out_grad_weight, void *stream)
{
    return run_grad(hidden, hidden_stride, weight, weight_stride, rows, dim, vocab, target, target_bytes, ignore_index,
                    lse, grad_loss, workspace, workspace_bytes, out_grad_hidden, out_grad_weight, stream);
}

size_t tf_topk_head_loss_grad_bf16_workspace(int64_t rows, int32_t dim, int64_t vocab, int32_t least)
{
    int pairs = 0, sms = 0;
    if (rows < 1 || bad_shape(rows, dim, vocab) || loss_setup(&pairs, &sms) != TF_TOPK_OK) return 0;
    return grad_space(nullptr, rows, dim, vocab, pairs, true, least ? kTileCols : good_piece(rows, vocab, pairs)).bytes + 256;
}

} // extern "C"
