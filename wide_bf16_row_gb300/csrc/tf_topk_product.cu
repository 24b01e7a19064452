// Products in 8 bits for GB300 (sm_103a): rows of e4m3 values with a scale for
// each 128 of a row, times weights of e4m3 values with a scale for each block
// of 128 x 128; one matrix, or the experts' matrices over their sorted rows.
//
// What is computed, for a row r of group g, a column n and blocks b of 128 dims:
//   y[r][n] = sum_b scale[r][b] * weight_scale[g][n / 128][b]
//                   * sum_{d in b} q[r][d] * weight[g][n][d]
// A block's sum is the tensor cores' (fp32, 4 products of 32 steps); the sum
// over the blocks, with their scales, is fp32 FMA in registers, so that each
// block's scale is applied exactly where it belongs and the tensor cores'
// truncating additions reach over 128 dims only.
//
// Two kernels, both persistent over the tiles of all groups, found in a prefix
// sum over the groups that each CTA makes from the offsets:
//   product_wide_kernel  many rows per group, bound by the tensor cores: a pair
//       of CTAs (cluster of two, tcgen05.mma cta_group::2, kind::f8f6f4) per tile
//       of 256 rows x 256 or 128 columns; each CTA holds 128 of the rows and
//       loads half of the columns.
//   product_thin_kernel  few rows per group, bound by the weight's bytes: a CTA
//       per tile of up to 128 columns x up to 64 rows, with the weight as the
//       MMA's A, so that its 128 lanes are columns and a block's sums of 16 rows
//       are 16 accumulator columns, quickly taken.
// Warp roles, per CTA: a TMA producer (per ring stage a block of 128 dims of rows
// and columns, 128-byte swizzle), an MMA issuer (a block into one of several
// accumulators in tensor memory), and warps that take each block's sums from
// there, scale and add them.
//
// No wait is unbounded: every mbarrier wait gives up after kWaitLimit polls,
// records a fault code, and the CTA winds down.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "tf_topk.h"

int tf_topk_internal_fail_cuda(int cuda_error);
int tf_topk_internal_device(int *sm_count);

namespace {

constexpr int kTileRows = 256;            // wide: rows (M) of a pair's tile
constexpr int kHalf = 128;                // wide: one CTA's; thin: columns (M) of a tile at most
constexpr int kBlock = TF_TOPK_FP8_BLOCK; // dims of a scale, and of a ring stage: one 128-byte swizzle row
constexpr int kMaxWidth = 256;
constexpr uint32_t kShare = kHalf * kBlock; // 16 KB: 128 rows or columns of a block
constexpr int kStages = 4;                // wide: of the ring
constexpr uint32_t kWideStage = 2 * kShare;
constexpr int kRowBox = 16;               // rows of a small box
constexpr int kThinRows = 64;             // thin: rows of a tile at most
// Rows per group on average up to which the thin kernel takes a product of several
// groups (one group: kThinRows).  Both (us, thin / wide, 128 experts, 2048 x 1536):
// 4 rows 62/81, 16 66/91, 32 79/93, 48 99/99, 64 116/102 (routed; groups of more than 64
// read their weight twice); one matrix 2048 x 98592: 16 rows 36/54, 48 40/56, 64 43/55.
// Half of all rows at one of the 128: 2048 rows 75/98, 6144 98/103, and over the limit
// 8192 108/106.  The columns are not looked at, and with few of them the two meet
// earlier: 8 groups of 48 rows 14.7/12.8 (4096 columns 15.2/21.7), one matrix of 64 rows
// 7168 x 8192 43/30 (7168 x 24576 44/59).
constexpr int kThinMostRows = 48;
constexpr uint32_t kWideRing = kStages * kWideStage, kThinRing = 92 * 1024;
constexpr int kThinMostStages = kThinRing / (kShare + kRowBox * kBlock); // with the fewest rows a tile has
constexpr int kThinCtas = 2; // of an SM: while one waits for its loads the other's products run
constexpr int kMaxGroups = TF_TOPK_ROUTE_MAX_EXPERTS;
constexpr int kEpiWarps = 8;
// A warpgroup for TMA and MMA and two that scale.  Those hold 128 sums a
// thread, so registers move over to them: 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kWideThreads = 32 * (4 + kEpiWarps);
constexpr int kFrontRegs = 72, kEpiRegs = 216;
constexpr int kWideTmem = 2 * kMaxWidth;
constexpr int kChunk = 16;       // accumulator columns a thread takes at a time
constexpr uint32_t kBoxBytes = 4096; // wide: 32 rows x 128 bytes on their way out
constexpr uint32_t kStagingWarp = 2 * kBoxBytes, kStagingBytes = kEpiWarps * kStagingWarp;
constexpr int kTurnCols = 32;    // columns a warp turns round at a time, where the result's rows are no whole 16 bytes
constexpr int kTurnPitch = kTurnCols + 1;
static_assert(32 * kTurnPitch * 4 <= kStagingWarp, "the turned columns fit");
constexpr int kGroupRows = 16;   // row tiles that share the sweep over the columns
constexpr int kThinEpiWarps = 8; // two for each 32 columns, which share the rows
constexpr int kThinThreads = 32 * (2 + kThinEpiWarps);
constexpr int kThinAccs = 4;     // accumulators
constexpr int kThinTmem = kThinAccs * kThinRows;
constexpr int kScaleBlocks = 16; // thin: blocks whose scales are fetched at a time
constexpr uint32_t kAll = 0xFFFFFFFFu;
// Polls of a wait: a second, for a poll of a barrier that does not complete
// suspends the warp for 3.9 us.
#ifndef TF_TOPK_TEST_WAIT_TIMEOUT
constexpr uint32_t kWaitLimit = 1u << 18;
#else // test build: 16 ms
constexpr uint32_t kWaitLimit = 1u << 12;
#endif
constexpr uint32_t kFaultWait = 1;

__device__ uint32_t g_product_fault;

using Pair = unsigned long long; // of fp32

// The groups' tiles, as every CTA makes them for itself.
struct Groups {
    int32_t warp_sum[32];
    int32_t begin[kMaxGroups + 1]; // a group's first row; [groups] is the end of the last
    int32_t tiles[kMaxGroups + 1]; // tiles of the groups before
};

struct __align__(16) WideSmem {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;
    Groups groups;
};

struct __align__(16) ThinSmem {
    float scale[2][kScaleBlocks][kThinRows];
    float weight_scale[2][kScaleBlocks][2];
    uint64_t full[kThinMostStages], empty[kThinMostStages];
    uint64_t acc_full[kThinAccs], acc_empty[kThinAccs];
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;
    Groups groups;
};

struct ProductArgs {
    const float *scale;        // [rows][blocks]
    const float *weight_scale; // [groups][column blocks][blocks]
    const int32_t *offsets;    // null: one group of all rows
    void *out;
    int32_t rows, cols, groups, blocks, col_blocks, col_tiles;
    int32_t width; // columns of a tile
    int32_t tile_rows; // thin: rows of a tile
    int32_t stages; // thin: of the ring
    int32_t boxes; // wide: the result's rows are whole 16 bytes and go out by TMA
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
// change them; nothing else is handed over.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// As mbar_arrive_cluster, to a barrier of this CTA.
__device__ __forceinline__ void mbar_arrive_own(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}

// Bounded wait for the phase with this parity; gives up after kWaitLimit
// polls (recording the fault) or once another warp of this CTA has.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
{
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(saddr(bar)), "r"(parity)
                     : "memory");
        if (ok) return true;
        if (abort && *abort) return false;
    }
    atomicCAS(&g_product_fault, 0u, kFaultWait);
    if (abort) *abort = 1;
    return false;
}

// As mbar_wait, by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
{
    const bool ok = mbar_wait(bar, parity, abort);
    return __all_sync(kAll, ok);
}

// One lane of a converged warp, always the same: the operands of the TMA and
// MMA instructions it issues come from uniform registers.
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

// Shared-memory matrix descriptor of a K-major tile written by TMA with the
// 128-byte swizzle: start address >> 4, eight rows of 128 bytes 1024 bytes
// apart (stride byte offset at bit 32), version 1 at bit 46, swizzle mode 2 at
// bit 61.
constexpr uint64_t kDescK = (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);

__device__ __forceinline__ uint64_t desc_at(const void *p) { return kDescK | ((saddr(p) & 0x3FFFFu) >> 4); }

// Instruction descriptor of tcgen05.mma kind::f8f6f4: fp32 accumulator (bit
// 4), e4m3 A and B (0 at bits 7 and 10), both K-major, N / 8 at bit 17, M / 16
// at bit 24.
__device__ __forceinline__ uint32_t instruction_desc(uint32_t m, uint32_t n)
{
    return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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

// The same within one CTA.
__device__ __forceinline__ void tma_load_own(void *dst, const CUtensorMap *map, int32_t x, int32_t y, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(saddr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(saddr(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_own(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}
__device__ __forceinline__ void mma_commit_own(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// This warp's 32 accumulator lanes (lane = thread), kChunk columns from
// `taddr`.  The wait stands in the same statement: until it is over nothing may
// touch the registers, not even to move or spill them.
__device__ __forceinline__ void tmem_take(uint32_t taddr, uint32_t (&r)[kChunk])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void put(float *to, float x) { *to = x; }
__device__ __forceinline__ void put(__half *to, float x) { *to = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16 *to, float x) { *to = __float2bfloat16_rn(x); }

__device__ __forceinline__ void tmem_take8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Two fp32 sums in a register pair: one instruction for two FMAs.
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
    return p;
}
__device__ __forceinline__ Pair pair_of(float x) { return pair_of(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float pair_at(Pair p, int i) { return __uint_as_float((uint32_t)(p >> (32 * i))); }
__device__ __forceinline__ void fma_pair(Pair &sum, Pair a, Pair b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(a), "l"(b));
}
__device__ __forceinline__ Pair mul_pair(Pair a, Pair b)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
// Boxes on their way out: from shared memory to the result, cut at its extents.
__device__ __forceinline__ void send_box(const CUtensorMap *map, const void *box, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(saddr(box)), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void box_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void box_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void box_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- the tiles

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Tile {
    int group, row, end, col; // first row and the group's end, first column
};

// What find_groups makes, for offsets that run backwards (no order has them), by one
// thread: an offset below an earlier one counts as that one (an empty group), so
// that a row belongs to one group at most, and there are no more tiles than the host
// has held against 32 bits.  A call of its own: inlined it took registers from the
// sums (16384 x 2048 x 128: 11.3 to 12.4 us).
__device__ __noinline__ void find_groups_in_turn(Groups &s, const int32_t *offsets, int groups, int rows, int col_tiles,
                                                 int tile_rows)
{
    if (threadIdx.x == 0) {
        int edge = 0, tiles = 0;
        for (int g = 0; g <= groups; ++g) {
            s.begin[g] = edge, s.tiles[g] = tiles;
            const int next = g < groups ? max(edge, min(offsets[g + 1], rows)) : edge;
            tiles += ceil_div(next - edge, tile_rows) * col_tiles;
            edge = next;
        }
    }
}

// The groups' first rows and the tiles before each, by the whole CTA, four
// groups a thread (256 threads and more) or more of them; offsets out of range are
// held to it.
template <int kThreads> __device__ __forceinline__ void find_groups(Groups &s, const ProductArgs &a, int tile_rows)
{
    constexpr int kEach = (kMaxGroups + 1 + kThreads - 1) / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = tid * kEach;
    int n[kEach], sum = 0;
    bool back = false;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = first + i;
        n[i] = 0;
        if (g < a.groups) {
            const int lo = g == 0 ? 0 : min(max(a.offsets[g], 0), a.rows);
            const int hi = a.offsets ? min(max(a.offsets[g + 1], 0), a.rows) : a.rows;
            n[i] = hi > lo ? ceil_div(hi - lo, tile_rows) * a.col_tiles : 0;
            back |= hi < lo;
            s.begin[g] = lo;
            if (g == a.groups - 1) s.begin[a.groups] = hi;
        }
        sum += n[i];
    }
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) s.warp_sum[warp] = upto;
    if (__syncthreads_or(back)) {
        find_groups_in_turn(s, a.offsets, a.groups, a.rows, a.col_tiles, tile_rows);
        return;
    }
    int before = upto - sum;
    for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (first + i <= a.groups) s.tiles[first + i] = before;
        before += n[i];
    }
}

// The tile with this number, by a whole warp.  The group is the last with no
// more tiles before it: 32 boundaries at a time, in two steps.
__device__ __forceinline__ Tile tile_at(const Groups &s, const ProductArgs &a, int u, int tile_rows, int width)
{
    const int lane = threadIdx.x & 31;
    int g = (lane + 1) * 32;
    const int block = __popc(__ballot_sync(kAll, g <= a.groups && s.tiles[min(g, a.groups)] <= u));
    g = block * 32 + lane + 1;
    const int group = block * 32 + __popc(__ballot_sync(kAll, g <= a.groups && s.tiles[min(g, a.groups)] <= u));
    Tile t;
    t.group = group;
    t.end = s.begin[group + 1];
    const int begin = s.begin[group], all = ceil_div(t.end - begin, tile_rows);
    // sweeps of kGroupRows row tiles; in a sweep the row tile moves first, so
    // that the CTAs at work share the weight's tiles
    int r = u - s.tiles[group], sweep = 0, m_tiles = all;
    if (all > kGroupRows) {
        sweep = r / (kGroupRows * a.col_tiles);
        r -= sweep * kGroupRows * a.col_tiles;
        m_tiles = min(kGroupRows, all - sweep * kGroupRows);
    }
    const int n = m_tiles > 1 ? r / m_tiles : r;
    t.row = begin + (sweep * kGroupRows + r - n * m_tiles) * tile_rows;
    t.col = n * width;
    return t;
}

// Rows behind the last group become zeros; thread `me` of `all`.
template <typename Out>
__device__ __forceinline__ void zero_unused(const ProductArgs &a, int used, int64_t me, int64_t all)
{
    Out *out = static_cast<Out *>(a.out);
    const int64_t from = (int64_t)used * a.cols, to = (int64_t)a.rows * a.cols;
    constexpr int kEach = 16 / sizeof(Out);
    const int64_t lead = ((16 - (reinterpret_cast<uintptr_t>(out + from) & 15)) & 15) / sizeof(Out);
    const int64_t whole = min(to, from + lead), vecs = (to - whole) / kEach;
    for (int64_t i = me; i < vecs; i += all) reinterpret_cast<uint4 *>(out + whole)[i] = make_uint4(0, 0, 0, 0);
    if (me < kEach) {
        if (from + me < whole) put(out + from + me, 0.0f);
        if (whole + vecs * kEach + me < to) put(out + whole + vecs * kEach + me, 0.0f);
    }
}

// A warp's finished sums, a row per thread.  Whole slices of 32 rows go out as
// boxes, which the warp does not wait for (with 32-byte stores of its own a
// thread held up the next tile: 463 us for experts 16384 x 2048 x 1536, k 8,
// against 411); a group's last rows by themselves; and where rows are no whole 16 bytes
// the warp turns 32 columns at a time round in shared memory, so that lanes next
// to each other write columns next to each other.
template <typename Out, int kCols>
__device__ __forceinline__ void put_sums(const ProductArgs &a, const CUtensorMap *map, const Pair (&sum)[kCols / 2],
                                         uint8_t *staging, int row0, int end, int col0)
{
    const int lane = threadIdx.x & 31;
    Out *out = static_cast<Out *>(a.out);
    constexpr int kEach = 16 / sizeof(Out), kBoxCols = 128 / sizeof(Out);
    const auto piece = [&](int c) { // kEach columns from c on
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(Out) == 4)
                v[i] = __float_as_uint(pair_at(sum[(c + i) / 2], i & 1));
            else
                v[i] = pack2(pair_at(sum[c / 2 + i], 0), pair_at(sum[c / 2 + i], 1), Out());
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    };
    if (a.boxes && row0 + 32 <= end) {
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 2 * kBoxCols) { // two boxes at a time
            if (elect_one()) box_read_wait();
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + b * kBoxCols < kCols)
                        *reinterpret_cast<uint4 *>(staging + b * kBoxBytes + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            piece(c0 + b * kBoxCols + j * kEach);
            fence_async_proxy();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (c0 + b * kBoxCols < kCols && col0 + c0 + b * kBoxCols < a.cols)
                        send_box(map, staging + b * kBoxBytes, col0 + c0 + b * kBoxCols, row0);
                box_commit();
            }
            __syncwarp();
        }
        return;
    }
    if (a.boxes) {
        Out *to = out + (int64_t)(row0 + lane) * a.cols + col0;
#pragma unroll
        for (int c = 0; c < kCols; c += kEach)
            if (row0 + lane < end && col0 + c < a.cols) *reinterpret_cast<uint4 *>(to + c) = piece(c); // cols: whole pieces
        return;
    }
    float *turn = reinterpret_cast<float *>(staging);
#pragma unroll
    for (int c = 0; c < kCols; c += kTurnCols) {
#pragma unroll
        for (int i = 0; i < kTurnCols; ++i) turn[lane * kTurnPitch + i] = pair_at(sum[(c + i) / 2], i & 1);
        __syncwarp();
        const int col = col0 + c + lane;
        Out *to = out + (int64_t)row0 * a.cols + col;
        const int rows = col < a.cols ? min(32, end - row0) : 0;
#pragma unroll 8
        for (int r = 0; r < 32; ++r)
            if (r < rows) put(to + (int64_t)r * a.cols, turn[r * kTurnPitch + lane]);
        __syncwarp();
    }
}

template <typename Out, int kWidth>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    product_wide_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_few,
                        const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_out,
                        const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *staging = ring + kWideRing; // 1024-byte aligned
    WideSmem &sm = *reinterpret_cast<WideSmem *>(staging + kStagingBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = blockIdx.x & 1; // in the pair; rank 0 leads
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    constexpr int kShareCols = kWidth / 2; // a CTA loads

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
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
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sm.tmem_base)),
                     "n"(kWideTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait(); // the inputs may come from the kernel before on the stream
    tc_fence_before();
    find_groups<kWideThreads>(sm.groups, a, kTileRows);
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int units = sm.groups.tiles[a.groups];
    volatile uint32_t *abort = &sm.abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFrontRegs));
        if (warp == 0) {
            // ---- TMA producer
            const uint32_t full0 = peer_addr(&sm.full[0], 0); // the leading CTA's barriers
            uint32_t s = 0, turn = 0;                         // ring stage, times round the ring
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const Tile t = tile_at(sm.groups, a, u, kTileRows, kWidth);
                const int left = t.end - t.row;
                const bool few = left <= kRowBox, both = left > kHalf, has_rows = rank == 0 || both;
                const uint32_t bytes = (few ? kRowBox * kBlock : both ? 2 * kShare : kShare) + kWidth * kBlock;
                const int wrow = t.group * a.cols + t.col + (int)rank * kShareCols;
                for (int b = 0; b < a.blocks; ++b) {
                    ok = turn == 0 || mbar_wait_warp(&sm.empty[s], (turn - 1) & 1, abort);
                    if (!ok) break;
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(&sm.full[s], bytes);
                        const uint32_t bar = full0 + s * (uint32_t)sizeof(uint64_t);
                        uint8_t *at = ring + s * kWideStage;
                        if (has_rows) tma_load(at, few ? &map_few : &map_q, b * kBlock, t.row + (int)rank * kHalf, bar);
                        tma_load(at + kShare, &map_w, b * kBlock, wrow, bar);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, ++turn;
                }
            }
            // both CTAs' copies land before the pair leaves: the last fill of
            // each stage (the leader's barrier counts both CTAs' bytes)
            bool landed = rank == 0;
            for (uint32_t j = 0; j < kStages && landed; ++j) {
                const uint32_t filled = j < s ? turn + 1 : turn; // times stage j was filled
                if (filled) landed = mbar_wait(&sm.full[j], (filled - 1) & 1, nullptr);
            }
        } else if (warp == 1) {
            // ---- MMA issuer (the leading CTA's)
            if (rank == 0) {
                const uint32_t idesc = instruction_desc(kTileRows, kWidth);
                uint32_t s = 0, parity = 0, sum = 0;
                bool ok = true;
#ifdef TF_TOPK_TEST_WAIT_TIMEOUT
                ok = mbar_wait_warp(&sm.drain, 0, abort); // nothing completes it yet: the wait runs out
#endif
                for (int u = pair; u < units && ok; u += pairs) {
                    for (int b = 0; b < a.blocks; ++b, ++sum) {
                        const uint32_t buf = sum & 1, use = sum >> 1;
                        ok = (use == 0 || mbar_wait_warp(&sm.acc_empty[buf], (use - 1) & 1, abort)) &&
                             mbar_wait_warp(&sm.full[s], parity, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = desc_at(ring + s * kWideStage), bd = desc_at(ring + s * kWideStage + kShare);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < kBlock / 32; ++k) // 32 steps: 32 bytes along a row
                                mma_pair(tmem + buf * kMaxWidth, ad + k * 2, bd + k * 2, idesc, k != 0);
                            mma_commit_pair(&sm.empty[s]);
                            mma_commit_pair(&sm.acc_full[buf]);
                        }
                        __syncwarp();
                        if (++s == kStages) s = 0, parity ^= 1;
                    }
                }
                // every product is done before the TMEM is freed
                if (elect_one())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                     saddr(&sm.drain))
                                 : "memory");
                __syncwarp();
                mbar_wait(&sm.drain, 0, nullptr);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // ---- scaling and sums
        constexpr int kCols = kWidth / (kEpiWarps / 4); // of a thread
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t empty0 = peer_addr(&sm.acc_empty[0], 0), empty1 = peer_addr(&sm.acc_empty[1], 0);
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + h * kCols;
        uint32_t done = 0; // accumulators taken
        bool ok = true;
        for (int u = pair; u < units && ok; u += pairs) {
            const Tile t = tile_at(sm.groups, a, u, kTileRows, kWidth);
            const int row0 = t.row + (int)rank * kHalf + 32 * q, col0 = t.col + h * kCols;
            const bool has_rows = row0 < t.end;
            // A row's scales and the columns' are fetched four blocks ahead, along the
            // row: a sector holds those of eight blocks.  (Two ahead, or with the
            // scales block by block so that a warp reads whole lines, every block
            // waited: 208 us for 8192 x 7168 x 4096 against 214 and 327; through shared
            // memory 265.)
            const float *rs = a.scale + (int64_t)min(row0 + lane, a.rows - 1) * a.blocks;
            const float *ws = a.weight_scale +
                              ((int64_t)t.group * a.col_blocks + min(col0 / kBlock, a.col_blocks - 1)) * a.blocks;
            float r0 = rs[0], w0 = ws[0], r1 = 0.0f, w1 = 0.0f, r2 = 0.0f, w2 = 0.0f, r3 = 0.0f, w3 = 0.0f;
            if (a.blocks > 1) r1 = rs[1], w1 = ws[1];
            if (a.blocks > 2) r2 = rs[2], w2 = ws[2];
            if (a.blocks > 3) r3 = rs[3], w3 = ws[3];
            Pair sum[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = 0;
            for (int b = 0; b < a.blocks; ++b, ++done) {
                const uint32_t buf = done & 1;
                const Pair f = pair_of(r0 * w0);
                r0 = r1, w0 = w1, r1 = r2, w1 = w2, r2 = r3, w2 = w3;
                if (b + 4 < a.blocks) r3 = rs[b + 4], w3 = ws[b + 4];
                ok = mbar_wait_warp(&sm.acc_full[buf], (done >> 1) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                if (has_rows) {
#pragma unroll
                    for (int c = 0; c < kCols; c += kChunk) {
                        uint32_t x[kChunk];
                        tmem_take(lanes + buf * kMaxWidth + c, x);
#pragma unroll
                        for (int i = 0; i < kChunk; i += 2) fma_pair(sum[(c + i) / 2], f, pair_of(x[i], x[i + 1]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(buf ? empty1 : empty0);
            }
            if (ok && has_rows)
                put_sums<Out, kCols>(a, &map_out, sum, staging + (warp - 4) * kStagingWarp, row0, t.end, col0);
        }
        if (elect_one()) box_wait();
        __syncwarp();
        zero_unused<Out>(a, sm.groups.begin[a.groups], (int64_t)blockIdx.x * (32 * kEpiWarps) + tid - 128,
                         (int64_t)gridDim.x * (32 * kEpiWarps));
    }
    __syncwarp();
    grid_dependents_go();
    tc_fence_before();
    __syncthreads();
    // a pair that gave up may have copies in flight that no barrier of this
    // CTA counts: time for them to land (tens of times a copy's own)
    if (*abort)
        for (int i = 0; i < 64; ++i) __nanosleep(1000);
    cluster_sync(); // neither CTA leaves while the other may still reach its shared memory
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kWideTmem) : "memory");
    }
}

// ---------------------------------------------------------------- few rows

__device__ __forceinline__ void copy4_async(float *to, const float *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(saddr(to)), "l"(from) : "memory");
}

template <typename Out>
__global__ void __launch_bounds__(kThinThreads, kThinCtas)
    product_thin_kernel(const __grid_constant__ CUtensorMap map_rows, const __grid_constant__ CUtensorMap map_w,
                        const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    ThinSmem &sm = *reinterpret_cast<ThinSmem *>(ring + kThinRing);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < kThinMostStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kThinAccs; ++b) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], kThinEpiWarps);
        }
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_rows) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sm.tmem_base)),
                     "n"(kThinTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait(); // the inputs may come from the kernel before on the stream
    tc_fence_before();
    find_groups<kThinThreads>(sm.groups, a, a.tile_rows);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int units = sm.groups.tiles[a.groups], ctas = gridDim.x;
    volatile uint32_t *abort = &sm.abort;
    const auto boxes_of = [&](const Tile &t) { return ceil_div(min(t.end - t.row, a.tile_rows), kRowBox); };
    const uint32_t stages = a.stages, stage = kShare + a.tile_rows * kBlock;

    if (warp == 0) {
        // ---- TMA producer
        uint32_t s = 0, turn = 0; // ring stage, times round the ring
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += ctas) {
            const Tile t = tile_at(sm.groups, a, u, a.tile_rows, a.width);
            const int boxes = boxes_of(t), wrow = t.group * a.cols + t.col;
            const uint32_t bytes = (uint32_t)(a.width + boxes * kRowBox) * kBlock;
            for (int b = 0; b < a.blocks; ++b) {
                ok = turn == 0 || mbar_wait_warp(&sm.empty[s], (turn - 1) & 1, abort);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.full[s], bytes);
                    uint8_t *at = ring + s * stage;
                    tma_load_own(at, &map_w, b * kBlock, wrow, &sm.full[s]);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_own(at + kShare + i * kRowBox * kBlock, &map_rows, b * kBlock, t.row + i * kRowBox,
                                     &sm.full[s]);
                }
                __syncwarp();
                if (++s == stages) s = 0, ++turn;
            }
        }
        // the copies land before the CTA leaves: the last fill of each stage
        bool landed = true;
        for (uint32_t j = 0; j < stages && landed; ++j) {
            const uint32_t filled = j < s ? turn + 1 : turn; // times stage j was filled
            if (filled) landed = mbar_wait(&sm.full[j], (filled - 1) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ---- MMA issuer
        uint32_t s = 0, parity = 0, sum = 0;
        bool ok = true;
#ifdef TF_TOPK_TEST_WAIT_TIMEOUT
        ok = mbar_wait_warp(&sm.drain, 0, abort); // nothing completes it yet: the wait runs out
#endif
        for (int u = blockIdx.x; u < units && ok; u += ctas) {
            const int boxes = boxes_of(tile_at(sm.groups, a, u, a.tile_rows, a.width));
            const uint32_t idesc = instruction_desc(kHalf, boxes * kRowBox);
            for (int b = 0; b < a.blocks; ++b, ++sum) {
                const uint32_t buf = sum % kThinAccs, use = sum / kThinAccs;
                ok = (use == 0 || mbar_wait_warp(&sm.acc_empty[buf], (use - 1) & 1, abort)) &&
                     mbar_wait_warp(&sm.full[s], parity, abort);
                if (!ok) break;
                tc_fence_after();
                const uint64_t ad = desc_at(ring + s * stage), bd = desc_at(ring + s * stage + kShare);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k) // 32 steps: 32 bytes along a row
                        mma_own(tmem + buf * kThinRows, ad + k * 2, bd + k * 2, idesc, k != 0);
                    mma_commit_own(&sm.empty[s]);
                    mma_commit_own(&sm.acc_full[buf]);
                }
                __syncwarp();
                if (++s == stages) s = 0, parity ^= 1;
            }
        }
        // every product is done before the TMEM is freed
        if (elect_one()) mma_commit_own(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, nullptr);
    } else {
        // ---- scaling and sums: two threads per column, with eight of each sixteen
        // rows.  A wait that gives up leaves out what it waited for, not the
        // barriers of these warps.
        constexpr int kMine = kRowBox / 2;
        const int q = warp & 3, h = (warp - 2) >> 2, me = tid - 64;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + h * kMine;
        Out *out = static_cast<Out *>(a.out);
        // The scales of kScaleBlocks blocks at a time, for these threads
        // together: fetched while the ones before are used, from one tile into the next.
        int next_u = blockIdx.x, next_b = 0, fetched = 0;
        Tile next = {};
        if (next_u < units) next = tile_at(sm.groups, a, next_u, a.tile_rows, a.width);
        const auto fetch = [&] {
            if (next_u < units) {
                constexpr int kShares = 32 * kThinEpiWarps / kThinRows, kEach = kScaleBlocks / kShares;
                const int buf = fetched & 1, row = me % kThinRows, i0 = me / kThinRows * kEach;
                if (row < min(next.end - next.row, a.tile_rows)) {
                    const float *from = a.scale + (int64_t)(next.row + row) * a.blocks + next_b;
#pragma unroll
                    for (int i = i0; i < i0 + kEach; ++i)
                        if (next_b + i < a.blocks) copy4_async(&sm.scale[buf][i][row], from + i);
                }
                if (me < 2 * kScaleBlocks) {
                    const int i = me >> 1, block = min(next.col / kBlock + (me & 1), a.col_blocks - 1);
                    if (next_b + i < a.blocks)
                        copy4_async(&sm.weight_scale[buf][i][me & 1],
                                    a.weight_scale + ((int64_t)next.group * a.col_blocks + block) * a.blocks + next_b + i);
                }
                next_b += kScaleBlocks;
                if (next_b >= a.blocks) {
                    next_b = 0;
                    next_u += ctas;
                    if (next_u < units) next = tile_at(sm.groups, a, next_u, a.tile_rows, a.width);
                }
            }
            ++fetched;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch();
        uint32_t done = 0; // accumulators taken
        int used = 0;      // fetches used
        bool ok = true;
        for (int u = blockIdx.x; u < units; u += ctas) {
            const Tile t = tile_at(sm.groups, a, u, a.tile_rows, a.width);
            const int boxes = boxes_of(t), rows = min(t.end - t.row, a.tile_rows);
            const int col = t.col + 32 * q + lane;
            const int side = min(col / kBlock - t.col / kBlock, 1);
            const bool in = 32 * q + lane < a.width && col < a.cols;
            Pair sum[kThinRows / kRowBox][kMine / 2];
#pragma unroll
            for (int c = 0; c < kThinRows / kRowBox; ++c)
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i) sum[c][i] = 0;
            for (int b0 = 0; b0 < a.blocks; b0 += kScaleBlocks, ++used) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kThinEpiWarps) : "memory");
                fetch();
                const int blocks = min(kScaleBlocks, a.blocks - b0), from = used & 1;
                for (int b = 0; b < blocks && ok; ++b, ++done) {
                    const uint32_t buf = done % kThinAccs;
                    const Pair w = pair_of(sm.weight_scale[from][b][side]);
                    ok = mbar_wait_warp(&sm.acc_full[buf], (done / kThinAccs) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kThinRows / kRowBox; ++c) {
                        if (c >= boxes) break;
                        const ulonglong2 *f =
                            reinterpret_cast<const ulonglong2 *>(&sm.scale[from][b][c * kRowBox + h * kMine]);
                        const ulonglong2 f0 = f[0], f1 = f[1];
                        uint32_t x[kMine];
                        tmem_take8(lanes + buf * kThinRows + c * kRowBox, x);
                        fma_pair(sum[c][0], mul_pair(w, f0.x), pair_of(x[0], x[1]));
                        fma_pair(sum[c][1], mul_pair(w, f0.y), pair_of(x[2], x[3]));
                        fma_pair(sum[c][2], mul_pair(w, f1.x), pair_of(x[4], x[5]));
                        fma_pair(sum[c][3], mul_pair(w, f1.y), pair_of(x[6], x[7]));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_own(&sm.acc_empty[buf]);
                }
            }
            if (!ok || !in) continue;
            Out *to = out + (int64_t)t.row * a.cols + col;
#pragma unroll
            for (int c = 0; c < kThinRows / kRowBox; ++c)
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int r = c * kRowBox + h * kMine + i;
                    if (r < rows) put(to + (int64_t)r * a.cols, pair_at(sum[c][i / 2], i & 1));
                }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        zero_unused<Out>(a, sm.groups.begin[a.groups], (int64_t)blockIdx.x * (32 * kThinEpiWarps) + me,
                         (int64_t)gridDim.x * (32 * kThinEpiWarps));
    }
    __syncwarp();
    grid_dependents_go();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kThinTmem) : "memory");
    }
}

// ---------------------------------------------------------------- host side

constexpr size_t kWideSmem = 1024 + kWideRing + kStagingBytes + sizeof(WideSmem);
constexpr size_t kThinSmem = 1024 + kThinRing + sizeof(ThinSmem);
static_assert(kWideSmem <= 227 * 1024 && kThinCtas * (kThinSmem + 1024) <= 228 * 1024,
              "the kernels' shared memory fits an SM");

constexpr int kMaxDevices = 64;
struct ProductDevice {
    std::atomic<bool> ready{false};
    int pairs = 0; // CTA pairs that fit the device at a time
};
ProductDevice g_product_dev[kMaxDevices];
std::mutex g_product_mutex;
PFN_cuTensorMapEncodeTiled_v12000 g_product_encode = nullptr;

using WideKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, ProductArgs);
using ThinKernel = void (*)(CUtensorMap, CUtensorMap, ProductArgs);

WideKernel wide_kernel(int32_t dtype, int width)
{
    if (dtype == TF_TOPK_DTYPE_F32) return width == 256 ? product_wide_kernel<float, 256> : product_wide_kernel<float, 128>;
    if (dtype == TF_TOPK_DTYPE_F16) return width == 256 ? product_wide_kernel<__half, 256> : product_wide_kernel<__half, 128>;
    return width == 256 ? product_wide_kernel<__nv_bfloat16, 256> : product_wide_kernel<__nv_bfloat16, 128>;
}

ThinKernel thin_kernel(int32_t dtype)
{
    return dtype == TF_TOPK_DTYPE_F32   ? product_thin_kernel<float>
           : dtype == TF_TOPK_DTYPE_F16 ? product_thin_kernel<__half>
                                        : product_thin_kernel<__nv_bfloat16>;
}

// Per device, once: the kernels' shared memory limits, the CTA pairs the device
// holds at a time, and the driver's tensor-map encoder.
int product_setup(int *pairs, int *sm_count)
{
    const int st = tf_topk_internal_device(sm_count);
    if (st != TF_TOPK_OK) return st;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
    if (dev >= kMaxDevices) return TF_TOPK_ERR_DEVICE;
    ProductDevice &d = g_product_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_product_mutex);
        if (!d.ready.load(std::memory_order_relaxed)) {
            const auto allow = [&](const void *kernel, size_t bytes) {
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
            };
            for (int32_t dtype : {TF_TOPK_DTYPE_BF16, TF_TOPK_DTYPE_F16, TF_TOPK_DTYPE_F32}) {
                for (int width : {128, 256}) allow((const void *)wide_kernel(dtype, width), kWideSmem);
                allow((const void *)thin_kernel(dtype), kThinSmem);
            }
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(*sm_count / 2 * 2), 1, 1);
            cfg.blockDim = dim3(kWideThreads, 1, 1);
            cfg.dynamicSmemBytes = kWideSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, wide_kernel(TF_TOPK_DTYPE_BF16, 256), &cfg);
            if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
            d.pairs = n < 1 ? 1 : n;
            if (!g_product_encode) {
                void *fn = nullptr;
                cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
                e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
                if (e != cudaSuccess) return tf_topk_internal_fail_cuda((int)e);
                if (q != cudaDriverEntryPointSuccess || !fn) return TF_TOPK_ERR_DEVICE;
                g_product_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
            }
            d.ready.store(true, std::memory_order_release);
        }
    }
    *pairs = d.pairs;
    return TF_TOPK_OK;
}

// A map of packed rows of bytes, boxes of 128 x box_rows with the 128-byte
// swizzle; coordinates past either extent read as zero.
bool encode_map(CUtensorMap *map, const void *p, int64_t inner, int64_t outer, int box_rows)
{
    cuuint64_t gdim[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    cuuint64_t gstride[1] = {(cuuint64_t)inner};
    cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows};
    cuuint32_t estride[2] = {1, 1};
    return g_product_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), gdim, gstride, box, estride,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of the result: boxes of 128 bytes x 32 rows with the 128-byte swizzle.
bool encode_out(CUtensorMap *map, const void *p, int32_t dtype, int64_t cols, int64_t rows)
{
    const size_t size = dtype == TF_TOPK_DTYPE_F32 ? 4 : 2;
    cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t gstride[1] = {(cuuint64_t)cols * size};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32};
    cuuint32_t estride[2] = {1, 1};
    return g_product_encode(map,
                            dtype == TF_TOPK_DTYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                            : dtype == TF_TOPK_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            2, const_cast<void *>(p), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Tiles there can be: a group's last one may be short, and groups without rows have none.
int64_t most_units(int64_t rows, int64_t groups, int64_t tile_rows, int64_t col_tiles)
{
    return (rows / tile_rows + (rows < groups ? rows : groups)) * col_tiles;
}

// Columns of a thin tile: as narrow as they can be without more rounds of the
// CTAs, in sixteens, from 32 on, so that the rounds come out whole (with a row
// in every group; the device knows the groups' rows, the host does not).
int thin_width(int64_t groups, int64_t cols, int ctas)
{
    const int64_t rounds = (groups * ((cols + kHalf - 1) / kHalf) + ctas - 1) / ctas;
    const int64_t tiles = rounds * ctas / groups; // of a group
    const int64_t width = ((cols + tiles - 1) / tiles + 15) / 16 * 16;
    return width < 32 ? 32 : width > kHalf ? kHalf : (int)width;
}

// Rows of a thin tile: all there can be, or for several groups what four times
// the average needs, in sixteens: a group beyond reads its weight again, from
// the L2, and rows that are not there take room from the ring.  (Twice, four and eight
// times, us, 128 groups of 2048 x 1536: 1024 rows, half of them of one group, 77, 72
// and 71, evenly 67, 67 and 66; 512 rows, nine tenths of eight groups, 45, 45 and 42.)
int thin_rows(int64_t rows, int64_t groups)
{
    const int64_t want = groups == 1 ? rows : (4 * rows + groups - 1) / groups;
    const int64_t tile = ((want < rows ? want : rows) + kRowBox - 1) / kRowBox * kRowBox;
    return tile < kThinRows ? (int)tile : kThinRows;
}

cudaLaunchConfig_t config(int64_t grid, int threads, size_t smem, void *stream, cudaLaunchAttribute *attr)
{
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

} // namespace

// This file's fault word, read and cleared (tf_topk_device_fault reports it).
uint32_t tf_topk_internal_product_fault_take()
{
    uint32_t f = 0;
    if (cudaMemcpyFromSymbol(&f, g_product_fault, sizeof f) != cudaSuccess) return 0;
    if (f) {
        const uint32_t zero = 0;
        cudaMemcpyToSymbol(g_product_fault, &zero, sizeof zero);
    }
    return f;
}

extern "C" int tf_topk_product_fp8(const void *q, const float *scale, int64_t rows, int32_t dim, const void *weight,
                                   const float *weight_scale, int64_t cols, int32_t groups, const int32_t *offsets,
                                   int32_t dtype, void *out, void *stream)
{
    if (dtype != TF_TOPK_DTYPE_BF16 && dtype != TF_TOPK_DTYPE_F16 && dtype != TF_TOPK_DTYPE_F32)
        return TF_TOPK_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX - kTileRows || dim < 16 || dim > (1 << 30) || dim % 16 != 0 ||
        cols < 1 || groups < 1 ||
        groups > kMaxGroups || (!offsets && groups != 1) || cols > (INT32_MAX - 1024) / groups ||
        most_units(rows, groups, kRowBox, (cols + 31) / 32) > INT32_MAX / 2)
        return TF_TOPK_ERR_SHAPE;
    if (rows == 0) return TF_TOPK_OK;
    if (!q || !scale || !weight || !weight_scale || !out) return TF_TOPK_ERR_NULL;
    const size_t size = dtype == TF_TOPK_DTYPE_F32 ? 4 : 2;
    if (!aligned(q, 16) || !aligned(weight, 16) || !aligned(scale, 4) || !aligned(weight_scale, 4) ||
        !aligned(offsets, 4) || !aligned(out, size))
        return TF_TOPK_ERR_ALIGN;
    int pairs = 0, sms = 0;
    const int st = product_setup(&pairs, &sms);
    if (st != TF_TOPK_OK) return st;
    ProductArgs a;
    a.scale = scale;
    a.weight_scale = weight_scale;
    a.offsets = offsets;
    a.out = out;
    a.rows = (int32_t)rows;
    a.cols = (int32_t)cols;
    a.groups = groups;
    a.blocks = (dim + kBlock - 1) / kBlock;
    a.col_blocks = (int32_t)((cols + kBlock - 1) / kBlock);
    a.boxes = aligned(out, 16) && (size_t)cols * size % 16 == 0;
    const int64_t active = rows < groups ? rows : groups; // groups that may have rows
    const bool thin = rows <= active * (active == 1 ? kThinRows : kThinMostRows);
    a.width = thin ? thin_width(active, cols, kThinCtas * sms) : cols <= kHalf ? 128 : 256;
    a.tile_rows = thin ? thin_rows(rows, active) : kTileRows;
    a.stages = (int32_t)(kThinRing / (kShare + a.tile_rows * kBlock)); // thin
    a.col_tiles = (int32_t)((cols + a.width - 1) / a.width);
    CUtensorMap map_q, map_few, map_w, map_out = {};
    if (!encode_map(&map_few, q, dim, rows, kRowBox) || (!thin && !encode_map(&map_q, q, dim, rows, kHalf)) ||
        !encode_map(&map_w, weight, dim, (int64_t)groups * cols, thin ? a.width : a.width / 2) ||
        (!thin && a.boxes && !encode_out(&map_out, out, dtype, cols, rows)))
        return tf_topk_internal_fail_cuda((int)cudaErrorInvalidValue);
    cudaLaunchAttribute attr[1];
    cudaError_t e;
    if (thin) {
        const int64_t units = most_units(rows, groups, a.tile_rows, a.col_tiles);
        const cudaLaunchConfig_t cfg =
            config(units < kThinCtas * sms ? units : kThinCtas * sms, kThinThreads, kThinSmem, stream, attr);
        e = cudaLaunchKernelEx(&cfg, thin_kernel(dtype), map_few, map_w, a);
    } else {
        const int64_t units = most_units(rows, groups, kTileRows, a.col_tiles);
        const cudaLaunchConfig_t cfg = config(2 * (units < pairs ? units : pairs), kWideThreads, kWideSmem, stream, attr);
        e = cudaLaunchKernelEx(&cfg, wide_kernel(dtype, a.width), map_q, map_few, map_w, map_out, a);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TF_TOPK_OK : tf_topk_internal_fail_cuda((int)e);
}
