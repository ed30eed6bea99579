// Sparse MLA attention over selected blocks (pages of 64 positions) of bf16 latent rows, on
// pairs of CTAs; and the form for every other cache: the blocks' positions written out for
// the attention over single rows.
//
// The mathematics: for query t, head h and the positions S of its blocks, those up to its own,
//     logit_s = scale * q[t,h] . row_s[0:576],  out = sum_s softmax(logit)_s row_s[0:512],
//     lse = log sum_s exp(logit_s).
//
// What bounds it: a row is 1152 bytes and 278,528 flop for 128 heads, 242 flop per byte
// (this card's measured rates: 289), so for one query a block HBM and the tensor cores are
// about even, and where queries share rows the tensor cores.  The rows of a block lie one after
// the other in the cache: a 64 x 64 box of a tensor map is an operand atom as the tensor cores
// read it, so what attn.cu's producer warps gather row by row a thread asks the TMA for, several
// atoms a request (with one atom each the requests paced the loads: a chunk 800 us, 780), and
// nothing but the softmax is left for warps to do.
//
// As in attn_e2m1.cu the two CTAs of a cluster split the heads (64 each) and issue pair MMAs
// (cta_group::2, M = 128): each supplies half of the B operand, so the logits are computed
// once.  A tile is two blocks.  For Q K^T a CTA brings its own block in full, nine atoms: X =
// dims [0, 256), Y = dims [256, 512), R = rope; for P V both need block 0 at one offset and
// block 1 at another, each its own value dims: rank 0 (block 0, dims [0, 256)) has them in X
// and lets the TMA put block 1's over Y, dead once Q K^T is complete, rank 1 (block 1, dims
// [256, 512)) has them in Y and takes block 0's over X.  P of block 0 goes into R, dead as well, P
// of block 1 into a buffer of its own.  P V leaves atoms 0, 1, 4 and 5 first, and the loads of the
// tile after next begin there.  36 + 16 MMAs a tile: 1152 + 1024 clocks.
//   shared memory: Q 72 KB | stage 0, 72 KB | stage 1 | P of block 1, 8 KB | maxima, barriers
//   TMEM: logits [0,64) [64,128), O [256,512).  An N-wide accumulator of a pair MMA takes N/2
//   columns: lanes 0-63 are the CTA's heads for the first half of N, lanes 64-127 for the second.
//
// A block that reaches past the query's position is masked in the logits, and its rows behind
// the position, which may hold anything, are zeroed in shared memory before P V: 0 * NaN is
// not 0.  A tile's missing second block is a box outside the tensor map, which reads as zeros.
//
// P goes to bf16, the type of V: at most 2^-8 of a weight, half a step; what normalises the output is
// the sum of the unrounded weights, the one the log-sum-exp takes.  m, a running bound of the
// logits, is set by the first tile and moves only when it grows by more than 2^64: bf16 and fp32
// have the exponents for it, and O is hardly ever rescaled.
//
// Work.  An item is a slice of the blocks (few queries: joined by attn_combine) of 128 heads
// of a query; the clusters that fit the GPU at once share the items out, and tiles, buffers and
// phases are counted through a cluster's items, so that the next item's rows, query and first
// logits are on their way during the last softmax and the output.
//
// Warps.  0 finds the items' blocks (entries 32 at a time, those that select something moved
// together) and loads own blocks; 1 loads the other block's values and the queries; 2 issues Q
// K^T, 3 P V (rank 0 for both CTAs).  What both CTAs load for an MMA is counted on a barrier of the
// leader's (passing on an arrival took 500 clocks).  4-19 are softmax and output, a thread 16 logits.
//
// Measured (32 blocks a query, 128 heads): 785 us for a chunk of 2048 queries, 1490 TFLOP/s of the
// 1926 measured (85 % of what the card holds over seconds: clocks fall to 1.8 GHz); 37.5 us for 64
// queries, 10.2 for one (16 slices and their merge).  A tile takes 2900 clocks in the middle of a chunk
// where its MMAs need 2176: shared memory moves 360 KB for it (240 for operands, 104 from the TMA, 16
// of P), 2880 clocks of its 128 bytes a clock.  64 queries read their 151 MB at 6 TB/s once under way
// (8 us are launch, dependent loads and output); asking the L2 for blocks two tiles ahead takes 38 us,
// one tile 38, three 41, six 47, not asking 41.5.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "pair_mma.cuh"

DSA_DEFINE_STATUS_WORD(attn_block)

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleM = 64.0f;   // growth of m that is let pass, log2 units

constexpr int kHeads = 64;            // heads per CTA
constexpr int kPage = 64;
constexpr int kDqk = 576, kDv = 512;
constexpr int kAtom = 64 * 128;       // bytes of a [64 rows x 64 dims] atom
constexpr int kStage = 9 * kAtom;
constexpr int kWarpOwn = 0, kWarpOther = 1, kWarpQk = 2, kWarpPv = 3, kWarpSoft = 4;
constexpr int kParts = 4;             // threads that share a (head, block)'s logits
constexpr int kCols = kPage / kParts; // logits a thread
constexpr int kSoftWarps = 4 * kParts;
static_assert(kParts == 4, "a thread's 64 columns of O are one atom of the output");
constexpr int kThreads = 32 * (kWarpSoft + kSoftWarps);
constexpr int kAhead = 2;             // tiles that the L2 is asked for a block before its load

constexpr int kOffQ = 0;
constexpr int kOffStage = kOffQ + 9 * kAtom;              // [2]
constexpr int kOffP1 = kOffStage + 2 * kStage;            // P of block 1
constexpr int kOffMax = kOffP1 + kAtom;                   // float [2][2 kParts][32]: of 32 heads' threads each
constexpr int kOffInfo = kOffMax + 2 * 2 * kParts * 32 * 4;   // int4 [4]: what a tile is, by tile number mod 4
constexpr int kOffOk = kOffInfo + 4 * 16;                 // int [kSoftWarps]
constexpr int kOffBar = kOffOk + kSoftWarps * 4;
// What a tile is, in info: x flags, y the other block's first cache row, z and w how many rows of
// blocks 0 and 1 count.  Written before the tile's loads, that is when the first half of P V of the
// tile two before is complete; the tile four before, whose place it takes, has long been passed.
constexpr int kFirst = 1, kLast = 2, kEnd = 4;            // of its item; last of all
constexpr int kNumBars = 24;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kUsed = kOffMisc + 16;
constexpr int kSmemBytes = 232448;
constexpr int kSlack = kSmemBytes - kUsed;                // for re-aligning the base to 1024 bytes
static_assert(kSlack >= 128 && kOffBar % 8 == 0 && kOffInfo % 16 == 0, "shared memory layout");

constexpr uint32_t kColO = 256;
constexpr uint32_t kIdescQK = make_idesc(kFmtBF16, kFmtBF16, false, false, 128, 128);
constexpr uint32_t kIdescPV = make_idesc(kFmtBF16, kFmtBF16, false, true, 128, 256);

struct BlockParams {
  SeqArgs seq;
  MlaArgs a;                // idx: [T, K] blocks
  int32_t n_split;          // slices per query
  int32_t per_split;        // entries per slice, an even number
  int32_t head_blocks;      // blocks of 128 heads
  int32_t items;            // T * head_blocks * n_split, shared out among the clusters
  // [n_split, T, H, 512] (n_split > 1), bf16 as attn.cu's for the same merge: 2^-8 of a partial at most.  Of the
  // output, root of the mean square: 0.0021 of it off without slices (P and the output's own rounding, which
  // alone is 0.0017), 0.0022 (one query of 32 blocks) to 0.0025 (7 of 13) with them.
  uint16_t* ws_o;
  float* ws_lse;            // [n_split, T, H]
  uint64_t wait_limit_ns;
  uint32_t dbg_withhold;
  Divisor split, heads;     // by n_split, head_blocks
  float scale_log2;         // softmax scale * log2 e
  uint32_t page_bytes;      // of a block from its first row to its last row's end; 0: rows too far apart to ask for it whole
};

// Whether a wait must end (1): another thread of the CTA gave up, or the wait has been going
// on for longer than the limit (which this sets the flags for).  Else when it must.
__device__ __noinline__ uint64_t wait_until(volatile int* abort_flag, uint64_t until, uint64_t limit_ns) {
  if (*abort_flag) return 1;
  const uint64_t now = globaltimer_ns();
  if (until == 0) return now + limit_ns;
  if (now < until) return until;
  atomicOr(&g_status_attn_block, kDevTimeout);
  *abort_flag = 1;
  return 1;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  const uint32_t addr = smem_u32(bar);
  uint64_t until = 0;
  for (uint32_t it = 1; !mbar_try_wait(addr, parity); ++it)
    if ((it & 63u) == 0u && (until = wait_until(abort_flag, until, limit_ns)) == 1) return false;
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_block_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap2,
                      const __grid_constant__ CUtensorMap kmap1, const __grid_constant__ CUtensorMap omap,
                      BlockParams p) {
  grid_dep_launch();   // the kernel after waits for this grid before it reads what this grid writes
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (sm - sm_raw > kSlack) {   // the same in both CTAs: their shared windows have one layout
    if (threadIdx.x == 0) atomicOr(&g_status_attn_block, kDevConfig);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  // Barriers in pairs belong to a tile's stage or logit buffer: nothing comes to one for the
  // tile after next before its waiters have passed it for this one.  What both CTAs load for an
  // MMA is counted on one barrier of the leader, which issues it.
  uint64_t* ifull = bars;         // [2] what the tile is has been written
  uint64_t* own = bars + 2;       // [2][2] leader: own blocks landed in both CTAs, atoms 0, 1, 4, 5 and the rest
  uint64_t* pvhalf = bars + 6;    // [2] P V complete as far as atoms 0, 1, 4, 5 go
  uint64_t* oth = bars + 8;       // [2] leader: the other blocks' values landed in both CTAs
  uint64_t* othpart = bars + 10;  // [2] they have landed in this CTA (tiles with rows to zero only)
  uint64_t* sfull = bars + 12;    // [2] Q K^T complete: logits there, half of the stage and its rope atom dead
  uint64_t* sfree = bars + 14;    // [2] leader: logits read, both CTAs
  uint64_t* pvdone = bars + 16;   // [2] P V complete: the tile's stage and P free
  uint64_t* edone = bars + 18;    // [2] an item's output has left the stage of its last tile
  // A pair too: the warps of block 0 write P without waiting for P V of the tile before, so some may
  // arrive for a tile while others have yet to for the one before it; for the one after it none can,
  // whose loads wait for this one's P V.
  uint64_t* pfull = bars + 20;    // [2] leader: P written and rows zeroed, both CTAs
  uint64_t* qfull = bars + 22;    // leader: an item's query has come, both CTAs
  uint64_t* drain = bars + 23;    // every MMA complete (teardown)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const volatile int* info = reinterpret_cast<const volatile int*>(sm + kOffInfo);
  const uint64_t wlim = p.wait_limit_ns;
  const int N = p.a.K, H = p.a.H;

  // Work items, one after the other, the clusters in turn: a slice of 128 heads of a query, the
  // last query first (longest causal history).
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto slice_of = [&](int item) -> int { return item - p.split(item) * p.n_split; };
  auto query_of = [&](int item) -> int { return p.seq.T - 1 - p.heads(p.split(item)); };
  auto head_of = [&](int item) -> int {   // this CTA's first head
    const int i = p.split(item);
    return (i - p.heads(i) * p.head_blocks) * 128 + static_cast<int>(rank) * kHeads;
  };

  if (warp == kWarpOwn && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&own[2 * i], 1);
      mbar_init(&own[2 * i + 1], 1);
      mbar_init(&pvhalf[i], 1);
      mbar_init(&oth[i], 2);
      mbar_init(&othpart[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 2 * kSoftWarps);
      mbar_init(&pvdone[i], 1);
      mbar_init(&edone[i], kSoftWarps);
      mbar_init(&pfull[i], 2 * kSoftWarps);
    }
    mbar_init(qfull, 1);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpOther && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap2);
    tma_prefetch_desc(&kmap1);
  }
  __syncwarp();
  if (warp == kWarpQk) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(misc)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_arrive();
  grid_dep_wait();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem0 = misc[0];
  // Whether a tile holds rows behind its query's position, which have to be zeroed.
  auto zeroes = [](const int4& what) -> bool { return ((what.z | what.w) & (kPage - 1)) != 0; };
  auto wait = [&](uint64_t* bar, int use) -> bool {   // the whole warp
    return __all_sync(0xffffffffu, wait_bar(bar, use & 1, abort_flag, wlim));
  };

  if (warp == kWarpOwn) {
    // ------------------------------------------------ the items' blocks, own blocks
    const int none = static_cast<int>(p.seq.cache_rows);   // a box from here on reads as zeros
    int item = first, e0 = 0, e1 = 0, qp = 0, b = 0;
    bool fresh = false;      // the open item has given no blocks yet
    uint32_t bad = 0;
    // the next blocks: lane l holds the first cache row of block l of cnt, and how many rows of it count
    int n_row = 0, n_rows = 0, n_cnt = 0;
    bool n_there = false, n_first = false;
    int opened = -1, fresh_at = -1;   // entries from fresh_at on, loaded already
    auto load_blk = [&](int it, int e) -> int {
      return e + lane < e1 ? __ldg(p.a.idx + static_cast<int64_t>(query_of(it)) * N + e + lane) : -1;
    };
    auto next_blocks = [&]() {
      n_there = false;
      n_cnt = 0;
      for (;;) {
        if (e0 >= e1) {
          if (fresh) break;   // an item that selects nothing: one tile of no rows
          if (item >= p.items) return;
          const int t = query_of(item);
          e0 = slice_of(item) * p.per_split;
          e1 = min(N, e0 + p.per_split);
          opened = load_blk(item, e0);   // its first entries, beside the query's position and sequence
          qp = __ldg(p.seq.q_pos + t);
          b = __ldg(p.seq.q_seq + t);
          if (qp < 0 || qp >= p.seq.max_ctx || b < 0 || b >= p.seq.B) {
            bad |= kDevBadPos;
            e1 = e0;
          }
          fresh = true;
          fresh_at = e0;
          item += step;
          continue;
        }
        int blk = fresh_at == e0 ? opened : load_blk(item - step, e0);   // (item has moved on)
        fresh_at = -1;
        e0 += 32;
        if (blk > (qp >> 6)) {
          bad |= kDevBadIndex;
          blk = -1;
        }
        int page = blk >= 0 ? __ldg(p.seq.block_table + static_cast<int64_t>(b) * p.seq.bt_stride + blk) : -1;
        if (blk >= 0 && (page < 0 || page >= p.seq.n_pages)) {
          bad |= kDevBadIndex;
          page = -1;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
        if (mask == 0) continue;
        n_cnt = __popc(mask);
        n_row = page * kPage;
        n_rows = min(kPage, qp + 1 - blk * kPage);
        if (mask & (mask + 1)) {   // holes: lane l takes the l-th that selects something
          const int src = static_cast<int>(__fns(mask, 0, lane + 1)) & 31;
          n_row = __shfl_sync(0xffffffffu, n_row, src);
          n_rows = __shfl_sync(0xffffffffu, n_rows, src);
        }
        break;
      }
      n_first = fresh;
      fresh = false;
      n_there = true;
    };
    int j = 0, ended = 0;        // tiles; items that have ended before tile j - 1
    int last1 = 0, last2 = 0;    // whether tiles j - 1 and j - 2 ended an item
    bool ok = true, half_issued = false;
    next_blocks();
    while (ok && n_there) {
      const int row = n_row, rows = n_rows, cnt = n_cnt, tiles = max(1, (n_cnt + 1) >> 1);
      const bool starts = n_first;
      // the next blocks are looked up behind two tiles under way, before the last tile: whether it
      // ends the item depends on them
      const int ahead = min(2, tiles - 1);
      for (int k = 0; k < tiles; ++k, ++j) {
        if (k == ahead) next_blocks();
        const int row0 = __shfl_sync(0xffffffffu, row, (2 * k) & 31), row1 = __shfl_sync(0xffffffffu, row, (2 * k + 1) & 31);
        const int c0 = __shfl_sync(0xffffffffu, rows, (2 * k) & 31), c1 = __shfl_sync(0xffffffffu, rows, (2 * k + 1) & 31);
        const bool has0 = 2 * k < cnt, has1 = 2 * k + 1 < cnt;
        const bool last = k == tiles - 1 && (!n_there || n_first);
        const int flags = (starts && k == 0 ? kFirst : 0) | (last ? kLast | (n_there ? 0 : kEnd) : 0);
        if (j >= 2) {
          // (an item's output leaves through the stage of its last tile)
          if (last2) ok = wait(&edone[ended & 1], ended >> 1);
          ended += last2;
          if (ok) ok = wait(&pvhalf[j & 1], (j >> 1) - 1);
          if (!ok) break;
        }
        last2 = last1;
        last1 = last ? 1 : 0;
        const int at0 = has0 ? row0 : none, at1 = has1 ? row1 : none, at = rank ? at1 : at0;
        uint8_t* dst = sm + kOffStage + (j & 1) * kStage;
        uint64_t* bar = &own[2 * (j & 1)];
        if (lane == 0) {
          *reinterpret_cast<int4*>(sm + kOffInfo + (j & 3) * 16) =
              make_int4(flags, rank ? at0 : at1, has0 ? c0 : 0, has1 ? c1 : 0);
          if (!(p.dbg_withhold && j == 0)) mbar_arrive(&ifull[j & 1]);
          if (rank == 0) mbar_arrive_expect_tx(bar, 2 * 4 * kAtom);
          tma_load_atoms_pair(dst, &kmap2, leader_addr(bar), at, 0);
          tma_load_atoms_pair(dst + 4 * kAtom, &kmap2, leader_addr(bar), at, 4);
        }
        __syncwarp();
        if (j >= 2) ok = wait(&pvdone[j & 1], (j >> 1) - 1);
        if (!ok) {
          half_issued = true;
          break;
        }
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(bar + 1, 2 * 5 * kAtom);
          tma_load_atoms_pair(dst + 2 * kAtom, &kmap2, leader_addr(bar + 1), at, 2);
          tma_load_atoms_pair(dst + 6 * kAtom, &kmap2, leader_addr(bar + 1), at, 6);
          tma_load_atoms_pair(dst + 8 * kAtom, &kmap1, leader_addr(bar + 1), at, 8);
        }
        // the L2 is asked for the own block of a tile some tiles on
        if (p.page_bytes > 0) {
          const int e = 2 * (k + kAhead) + static_cast<int>(rank);
          const int from = __shfl_sync(0xffffffffu, row, e & 31);
          if (lane == 0 && e < cnt)
            prefetch_l2_bulk(static_cast<const uint8_t*>(p.a.kv) + static_cast<int64_t>(from) * p.a.row_bytes, p.page_bytes);
        }
        __syncwarp();
      }
    }
    if (bad) atomicOr(&g_status_attn_block, bad);
    // the last copies, of both CTAs, have landed before either leaves
    for (int k = max(0, j - 2); k < j && rank == 0; ++k)
      for (int i = 0; i < 2; ++i) mbar_drain(&own[2 * (k & 1) + i], (k >> 1) & 1, &g_status_attn_block, wlim);
    if (half_issued && rank == 0) mbar_drain(&own[2 * (j & 1)], (j >> 1) & 1, &g_status_attn_block, wlim);
  } else if (warp == kWarpOther) {
    // ------------------------------------------------ queries, the other block's values
    auto query_row = [&](int item) -> int { return query_of(item) * H + head_of(item); };   // < 2^31
    auto load_query = [&](int item) {
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(qfull, 2 * 9 * kAtom);
        const uint32_t bar = leader_addr(qfull);
        const int row = query_row(item);
        // heads beyond H: the next token's, or zeros; nothing is written of them
#pragma unroll
        for (int k3 = 0; k3 < 3; ++k3) tma_load_atoms_pair(sm + kOffQ + 3 * k3 * kAtom, &qmap, bar, row, 3 * k3);
        // the L2 is asked for the query after it
        const int next = item + step;
        if (next < p.items) {
          const int64_t from = query_row(next), rows = min(static_cast<int64_t>(kHeads), static_cast<int64_t>(p.seq.T) * H - from);
          if (rows > 0)
            prefetch_l2_bulk(static_cast<const uint8_t*>(p.a.q) + from * (kDqk * 2), static_cast<uint32_t>(rows) * (kDqk * 2));
        }
      }
      __syncwarp();
    };
    int item = first, g = 0, queries = 1;
    int parts[2] = {0, 0};   // tiles with rows to zero, of either stage
    load_query(item);
    for (bool more = true; more; ++g) {
      const int st = g & 1;
      if (!wait(&ifull[st], g >> 1) || !wait(&sfull[st], g >> 1)) break;
      const int4 what = *reinterpret_cast<const int4*>(sm + kOffInfo + (g & 3) * 16);
      more = !(what.x & kEnd);
      const bool zero = zeroes(what);
      if (lane == 0) {
        uint32_t bar = leader_addr(&oth[st]);
        if (zero) {   // the copies are waited for in their own CTA
          mbar_arrive_expect_tx(&othpart[st], 4 * kAtom);
          bar = smem_u32(&othpart[st]);
        } else if (rank == 0) {
          mbar_arrive_expect_tx(&oth[st], 2 * 4 * kAtom);
          mbar_arrive(&oth[st]);
        }
        uint8_t* dst = sm + kOffStage + st * kStage + (rank ? 0 : 4) * kAtom;
        tma_load_atoms_pair(dst, &kmap2, bar, what.y, rank ? 4 : 0);
        tma_load_atoms_pair(dst + 2 * kAtom, &kmap2, bar, what.y, rank ? 6 : 2);
      }
      __syncwarp();
      if ((what.x & (kLast | kEnd)) == kLast) {   // Q K^T of the item's last tile is complete
        item += step;
        load_query(item);
        ++queries;
      }
      if (zero) {
        if (!wait(&othpart[st], parts[st]++)) {
          ++g;
          break;
        }
        if (lane == 0) arrive_pair(leader_addr(&oth[st]));
        __syncwarp();
      }
    }
    for (int st = 0; st < 2; ++st)
      if (parts[st]) mbar_drain(&othpart[st], (parts[st] - 1) & 1, &g_status_attn_block, wlim);
    if (rank == 0) {
      for (int k = max(0, g - 2); k < g; ++k) mbar_drain(&oth[k & 1], (k >> 1) & 1, &g_status_attn_block, wlim);
      mbar_drain(qfull, (queries - 1) & 1, &g_status_attn_block, wlim);
    }
  } else if (warp == kWarpQk) {
    const uint64_t dq = make_sdesc(smem_u32(sm + kOffQ), 16, 1024, kLayoutSw128);
    const uint64_t dk0 = make_sdesc(smem_u32(sm + kOffStage), 16, 1024, kLayoutSw128);
    int n = 0;   // items
    bool ok = rank == 0, more = true;
#pragma unroll 1
    for (int g = 0; ok && more; ++g) {
      const int sb = g & 1;
      ok = wait(&ifull[sb], g >> 1);
      if (!ok) break;
      const int flags = info[(g & 3) * 4];
      more = !(flags & kEnd);
      if (flags & kFirst) ok = wait(qfull, n++);
      if (ok && g >= 2) ok = wait(&sfree[sb], (g >> 1) - 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem0 + sb * 64;
      const uint64_t dk = dk0 + static_cast<uint64_t>((sb * kStage) >> 4);
      auto multiply = [&](int a) {   // 64 dims
        const uint64_t off = static_cast<uint64_t>((a * kAtom) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_pair(d, dq + off + 2 * kk, dk + off + 2 * kk, kIdescQK, static_cast<uint32_t>(a | kk));
      };
#pragma unroll
      for (int i = 0; ok && i < 2; ++i) {   // atoms 0, 1, 4, 5, then 2, 3, 6, 7, 8
        ok = wait(&own[2 * sb + i], g >> 1);
        if (ok && elect_one()) {
          multiply(2 * i);
          multiply(2 * i + 1);
          multiply(2 * i + 4);
          multiply(2 * i + 5);
          if (i == 1) {
            multiply(8);
            commit_pair(&sfull[sb]);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp == kWarpPv) {
    const uint64_t dv0 = make_sdesc(smem_u32(sm + kOffStage), kAtom, 1024, kLayoutSw128);
    const uint64_t dp0 = make_sdesc(smem_u32(sm + kOffStage + 8 * kAtom), 16, 1024, kLayoutSw128);
    const uint64_t dp1 = make_sdesc(smem_u32(sm + kOffP1), 16, 1024, kLayoutSw128);
    bool ok = rank == 0, more = true;
#pragma unroll 1
    for (int g = 0; ok && more; ++g) {
      const int sb = g & 1;
      ok = wait(&ifull[sb], g >> 1);
      if (!ok) break;
      const int flags = info[(g & 3) * 4];
      more = !(flags & kEnd);
      ok = wait(&oth[sb], g >> 1) && wait(&pfull[sb], g >> 1);
      if (!ok) break;
      tc_fence_after();
      fence_proxy_async_smem();
      if (elect_one()) {
        const uint64_t st = static_cast<uint64_t>((sb * kStage) >> 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // value atoms 2 (q / 2), block q & 1
          const uint64_t da = (q & 1) ? dp1 : dp0 + st;
          const uint64_t db = dv0 + st + static_cast<uint64_t>((((q & 1) * 4 + (q >> 1) * 2) * kAtom) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_pair(tmem0 + kColO + (q >> 1) * 128, da + 2 * kk, db + 128 * kk, kIdescPV,
                      static_cast<uint32_t>((~flags & kFirst) | (q & 1) | kk));
          if (q == 1) commit_pair(&pvhalf[sb]);
        }
        commit_pair(&pvdone[sb]);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------ softmax and output
    const int sw = warp - kWarpSoft;
    const int quarter = warp & 3;
    const int hl = (quarter & 1) * 32 + lane;   // head within the CTA
    const int half = quarter >> 1;              // block of the tile; of the output: half of the value dims
    const int part = sw >> 2;                   // this thread's rows [kCols part, kCols part + kCols)
    const int rq = half * kParts + part;
    const uint32_t tmem = tmem0 + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = p.scale_log2;
    const uint32_t head_bar = 2 + (quarter & 1);   // the threads of 32 heads
    constexpr uint32_t kHeadThreads = 64 * kParts;
    float* xmax = reinterpret_cast<float*>(sm + kOffMax) + (quarter & 1) * (2 * kParts * 32) + lane;   // [2 kParts][32]
    volatile int* oks = reinterpret_cast<volatile int*>(sm + kOffOk);
    const uint32_t prow0 = smem_u32(sm + (half ? kOffP1 : kOffStage + 8 * kAtom)) + static_cast<uint32_t>(hl * 128);
    const uint32_t pstep = half ? 0u : static_cast<uint32_t>(kStage);   // block 0: the stage's rope atom
    bool ok = true;
    int j = 0, done = 0;   // tiles, items whose output has left
    bool stored = false;   // an item's output is on its way
    int parts0 = 0, parts1 = 0;   // tiles with rows to zero, of either stage
#pragma unroll 1
    for (int item = first; item < p.items; item += step) {
      float m = -INFINITY, l = 0.f;
      bool last = false, stop = false;
#pragma unroll 1
      for (; !last; ++j) {
        const int st = j & 1;
        ok = ok && wait(&ifull[st], j >> 1) && wait(&sfull[st], j >> 1);
        if (stored) {   // the last item's output has left its stage (seldom still to be waited for: loads went before it)
          if (lane == 0) {
            bulk_wait_read();
            mbar_arrive(&edone[done & 1]);
          }
          __syncwarp();
          ++done;
          stored = false;
        }
        tc_fence_after();
        const uint32_t stage = smem_u32(sm + kOffStage) + static_cast<uint32_t>(st * kStage);
        float x[kCols];
        float mx = -INFINITY;
        if (ok) {
          uint32_t s[kCols];
          tmem_ld16(tmem + st * 64 + part * kCols, s);
          const int4 what = *reinterpret_cast<const int4*>(sm + kOffInfo + (j & 3) * 16);
          last = (what.x & kLast) != 0;
          const int mine = (half ? what.w : what.z) - part * kCols;   // of this thread's rows that count
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_pair(leader_addr(&sfree[st]));   // the logit buffer has been read
#pragma unroll
          for (int i = 0; i < kCols; i += 2)
            mul2(x[i], x[i + 1], __uint_as_float(s[i]), __uint_as_float(s[i + 1]), sl2, sl2);
          if (mine < kCols) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) x[i] = i < mine ? x[i] : -INFINITY;
          }
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kCols; i += 2) mq[(i >> 1) & 3] = fmax3(mq[(i >> 1) & 3], x[i], x[i + 1]);
          mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
          // rows behind the query's position: nothing of them may reach O
          if (zeroes(what)) {
            ok = wait(&othpart[st], st ? parts1++ : parts0++);
            if (ok) {
#pragma unroll 1
              for (int blk = 0; blk < 2; ++blk) {
                const int from = blk ? what.w : what.z;
                if (from == 0) continue;   // not there: zeros already
                for (int i = sw * 32 + lane; i < (kPage - from) * 32; i += kSoftWarps * 32)
                  st_shared_v4(stage + (blk * 4 + ((i >> 3) & 3)) * kAtom + (from + (i >> 5)) * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
              }
            }
          }
        }
        // The threads of a head share m, and their warps leave together when one has given up.  One
        // barrier tells whether any of them has to let m grow (the first tile, and seldom after);
        // only then do they exchange their maxima.
        const bool grow = named_bar_or(head_bar, kHeadThreads, !ok || mx > m + kRescaleM);
        if (grow) {
          // O may have to be rescaled: P V of the tile before is complete
          const bool pv_ok = !(j >= 1 && ok) || wait(&pvdone[(j - 1) & 1], (j - 1) >> 1);
          ok = ok && pv_ok;
          xmax[rq * 32] = mx;
          if (lane == 0) oks[sw] = ok ? 1 : 0;
          named_bar_sync(head_bar, kHeadThreads);
#pragma unroll
          for (int k = 0; k < 2 * kParts; ++k) mx = fmaxf(mx, xmax[k * 32]);
          // the warps whose number is as odd as this one's
#pragma unroll
          for (int k = 0; k < 2 * kParts; ++k) ok = ok && oks[2 * k + (sw & 1)] != 0;
          named_bar_sync(head_bar, kHeadThreads);
          if (!ok) {
            stop = true;
            break;
          }
          const bool need = mx > m + kRescaleM;
          if (__any_sync(0xffffffffu, need && m > -INFINITY)) {   // (m of -inf: nothing in O yet)
            tc_fence_after();
            const float f = need && m > -INFINITY ? exp2f(m - mx) : 1.f;
#pragma unroll 1
            for (int cc = 0; cc < 256 / kParts / 16; ++cc) {   // this thread's share of the columns
              uint32_t o[16];
              const uint32_t at = tmem + kColO + part * (256 / kParts) + cc * 16;
              tmem_ld16(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(at, o);
            }
            tmem_st_wait();
          }
          if (need) {
            l *= exp2f(m - mx);
            m = mx;
          }
        }
        const float msub = (m == -INFINITY) ? 0.f : m;
        const uint32_t prow = prow0 + (j & 1) * pstep;
        float se[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) {
          float d0, d1;
          add2(d0, d1, x[2 * k], x[2 * k + 1], -msub, -msub);
          const float p0 = fast_exp2(d0), p1 = fast_exp2(d1);
          add2(se[2 * (k & 1)], se[2 * (k & 1) + 1], se[2 * (k & 1)], se[2 * (k & 1) + 1], p0, p1);
          pk[k] = pack_bf16x2(p0, p1);
        }
        // P of block 1 has one buffer: P V of the tile before is complete
        if (half && j >= 1) ok = wait(&pvdone[(j - 1) & 1], (j - 1) >> 1);
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c)
          st_shared_v4(prow + static_cast<uint32_t>(((part * (kCols / 8) + c) ^ (hl & 7)) << 4), pk[4 * c], pk[4 * c + 1],
                       pk[4 * c + 2], pk[4 * c + 3]);
        l += (se[0] + se[1]) + (se[2] + se[3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(leader_addr(&pfull[j & 1]));
      }
      if (stop) break;
      // ---- the output: O / l, log-sum-exp
      ok = ok && wait(&pvdone[(j - 1) & 1], (j - 1) >> 1);
      // the sums of a head's threads
      xmax[rq * 32] = l;
      named_bar_sync(head_bar, kHeadThreads);
      l = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * kParts; ++k) l += xmax[k * 32];
      named_bar_sync(head_bar, kHeadThreads);
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;   // l may be NaN
        const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        const int t = query_of(item), h0 = head_of(item) + (quarter & 1) * 32;
        // through the last tile's stage, which P V has left and the loads leave alone till edone: the
        // warp's 32 heads x 64 dims, half an atom, as a box of a TMA store
        uint8_t* out = sm + kOffStage + ((j - 1) & 1) * kStage + (half * 4 + part) * kAtom + (quarter & 1) * 4096;
        const uint32_t stg = smem_u32(out) + lane * 128;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t o[32];
          tmem_ld32(tmem + kColO + part * 64 + hf * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared_v4(stg + (((hf * 4 + k) ^ (lane & 7)) << 4),
                         pack_bf16x2(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                         pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        const int row = (p.n_split > 1 ? slice_of(item) * p.seq.T : 0) + t;
        if (lane == 0 && h0 < H) tma_store_heads(&omap, out, h0, row, half * 4 + part);
        if (rq == 0 && h0 + lane < H) {
          const int64_t at = static_cast<int64_t>(row) * H + h0 + lane;
          if (p.n_split > 1)
            p.ws_lse[at] = lse;
          else if (p.a.lse)
            p.a.lse[at] = lse;
        }
        if (lane == 0) bulk_commit();
      }
      __syncwarp();
      stored = true;
    }
    if (lane == 0) bulk_wait();
    __syncwarp();
  }

  // Every MMA has finished in both CTAs before either releases its TMEM or leaves (after
  // an abort some may still be running).
  if (rank == 0 && (warp == kWarpQk || warp == kWarpPv)) {
    if (elect_one()) commit_pair(drain);
    __syncwarp();
  }
  if (warp == kWarpQk) mbar_drain(drain, 0, &g_status_attn_block, p.wait_limit_ns);
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (warp == kWarpQk) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem0), "r"(512u) : "memory");
  }
}

// Blocks to positions, ascending within a block; -1 for what is masked.
__global__ void __launch_bounds__(256) expand_blocks_kernel(SeqArgs seq, const int32_t* blocks, int32_t N, int32_t* idx) {
  grid_dep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, per = static_cast<int64_t>(N) * seq.page_size;
  const int64_t t = i / per;
  if (t >= seq.T) return;
  const int k = static_cast<int>(i - t * per), j = k / seq.page_size, inside = k - j * seq.page_size;
  const int qp = __ldg(seq.q_pos + t);
  const int blk = __ldg(blocks + t * N + j);
  int pos = -1;
  if (blk >= 0 && qp >= 0 && qp < seq.max_ctx) {   // a bad position is flagged by the attention
    if (blk > qp / seq.page_size) {
      if (inside == 0) atomicOr(&g_status_attn_block, kDevBadIndex);
    } else if (inside <= qp - blk * seq.page_size) {   // (the sum could pass 2^31)
      pos = blk * seq.page_size + inside;
    }
  }
  idx[i] = pos;
}

// Clusters that the current device holds at once (its SMs need not pair up everywhere), asked once.
int resident_clusters(int num_sms) {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return std::max(1, num_sms / 2);
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  const void* kernel = reinterpret_cast<const void*>(attn_block_kernel);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(2, num_sms & ~1)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (ensure_smem_limit(kernel, kSmemBytes, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
    static_cast<void>(cudaGetLastError());
    return std::max(1, num_sms / 2);
  }
  cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Slices per query: a cluster for each while the GPU holds them all at once, a slice at least one
// tile, or two where more than 32 slices would hold one each: their merge costs what it saves.
// Measured with other numbers of slices (us, 32 blocks a query, this rule's first): 1 query 16 slices
// 10.2, 8 11.0, 1 29.4; 4 queries 8 slices 11.7, 16 13.2, 4 14.1; 16 queries 4 slices 21.0, 2 23.8, 8
// 24.0; 38 queries 2 slices 31.2, 1 34.4, 3 38.7; 40 queries 1 slice 34.5, 2 45.8; 64 queries 1 slice
// 37.3, 2 48.3; 80 queries 1 slice 55.1, 2 63.4; 1 query of 128 blocks 32 slices 11.9, 64 15.3, 16 14.4.
int choose_split(const SeqArgs& seq, const MlaArgs& a, int num_sms) {
  const int64_t tiles = (a.K + 1) / 2;
  const int64_t clusters = std::max<int64_t>(1, static_cast<int64_t>(seq.T) * ((a.H + 127) / 128));
  const int64_t held = std::max<int64_t>(1, resident_clusters(num_sms) / clusters);
  if (tiles <= held && clusters * tiles > 32) return static_cast<int>((tiles + 1) / 2);
  return static_cast<int>(std::min(tiles, held));
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Whether the blocks are boxes of a tensor map: bf16 rows of the tensor-core path's dims in pages of 64.
bool boxes(const SeqArgs& seq, const MlaArgs& a) {
  return a.kind == MlaKind::kBF16 && a.d_latent == kDv && a.d_rope == kDqk - kDv && seq.page_size == kPage &&
         a.row_bytes % 16 == 0;
}

}  // namespace

bool attn_block_positions(const SeqArgs& seq, const MlaArgs& a) { return !boxes(seq, a); }

size_t attn_block_workspace_bytes(const SeqArgs& seq, const MlaArgs& a, int num_sms) {
  if (seq.T == 0) return 0;
  if (!boxes(seq, a)) {
    MlaArgs rows = a;
    rows.K = a.K * seq.page_size;
    return align256(static_cast<size_t>(seq.T) * rows.K * sizeof(int32_t)) + attn_workspace_bytes(seq, rows, num_sms);
  }
  const int split = choose_split(seq, a, num_sms);
  if (split <= 1) return 0;
  return align256(static_cast<size_t>(split) * seq.T * a.H * kDv * sizeof(uint16_t)) +
         align256(static_cast<size_t>(split) * seq.T * a.H * sizeof(float));
}

cudaError_t launch_attn_block(const SeqArgs& seq, const MlaArgs& a, void* workspace, size_t ws_bytes,
                              const LaunchEnv& env, std::string* plan, bool* unsupported, std::string* why) {
  *unsupported = false;
  if (seq.T == 0) {
    *plan += "attn_block[empty]";
    return cudaSuccess;
  }
  if (!boxes(seq, a)) {
    MlaArgs rows = a;
    rows.K = a.K * seq.page_size;
    int32_t* idx = static_cast<int32_t*>(workspace);
    rows.idx = idx;
    const size_t used = align256(static_cast<size_t>(seq.T) * rows.K * sizeof(int32_t));
    const int64_t n = static_cast<int64_t>(seq.T) * rows.K;
    const cudaError_t e = launch_kernel(expand_blocks_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0,
                                        env.stream, true, 1, seq, a.idx, a.K, idx);
    if (e != cudaSuccess) return e;
    *plan += "expand_blocks -> ";
    return launch_attn(seq, rows, static_cast<char*>(workspace) + used, ws_bytes - used, env, plan, unsupported, why);
  }
  int split = choose_split(seq, a, env.num_sms);
  if (split > 1 && (workspace == nullptr || ws_bytes < attn_block_workspace_bytes(seq, a, env.num_sms)))
    split = 1;   // no room for partials: one slice per query
  const int tiles = (a.K + 1) / 2;
  const int per = (tiles + split - 1) / split * 2;
  split = (a.K + per - 1) / per;   // every slice non-empty
  const int head_blocks = (a.H + 127) / 128;
  const int64_t items = static_cast<int64_t>(seq.T) * head_blocks * split;
  if (items > 0x3FFFFFFFll || static_cast<int64_t>(seq.T) * a.H > 0x7FFFFF00ll) return cudaErrorInvalidConfiguration;
  BlockParams p{seq,     a,       split,        per, head_blocks,    static_cast<int32_t>(items),
                nullptr, nullptr, kWaitLimitNs, 0u,  Divisor(split), Divisor(head_blocks),
                a.softmax_scale * kLog2e,
                a.row_bytes <= 2 * kDqk + 128 ? static_cast<uint32_t>((kPage - 1) * a.row_bytes + 2 * kDqk) : 0u};
  debug_wait_state(&p.wait_limit_ns, &p.dbg_withhold);
  if (split > 1) {
    p.ws_o = static_cast<uint16_t*>(workspace);
    p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        align256(static_cast<size_t>(split) * seq.T * a.H * kDv * sizeof(uint16_t)));
  }
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(attn_block_kernel), kSmemBytes, env.device);
  if (e != cudaSuccess) return e;
  alignas(64) CUtensorMap qmap, kmap2, kmap1, omap;   // boxes of three atoms of 64 heads, of two and one of 64 cache rows, of one of 32 heads of the output
  std::string reason;
  const uint64_t rows = static_cast<uint64_t>(seq.cache_rows), row_bytes = static_cast<uint64_t>(a.row_bytes);
  if (!encode_tmap_atoms(&qmap, a.q, 9, static_cast<uint64_t>(seq.T) * a.H, kDqk * 2, kHeads, 3, &reason) ||
      !encode_tmap_atoms(&kmap2, a.kv, 9, rows, row_bytes, kPage, 2, &reason) ||
      !encode_tmap_atoms(&kmap1, a.kv, 9, rows, row_bytes, kPage, 1, &reason) ||
      !encode_tmap_heads(&omap, split > 1 ? static_cast<const void*>(p.ws_o) : a.out, 8, static_cast<uint64_t>(a.H),
                         static_cast<uint64_t>(split) * seq.T, 32, &reason)) {
    *unsupported = true;
    *why = "block attention: " + reason;
    return cudaSuccess;
  }
  const int64_t grid = 2 * std::min<int64_t>(items, resident_clusters(env.num_sms));
  e = launch_kernel(attn_block_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, env.stream, true,
                    2, qmap, kmap2, kmap1, omap, p);
  if (e != cudaSuccess) return e;
  char buf[96];
  snprintf(buf, sizeof(buf), "attn_block<bf16>[split=%d,grid=%lld]", split, static_cast<long long>(grid));
  *plan += buf;
  if (split > 1) {
    e = launch_attn_combine(p.ws_o, p.ws_lse, split, seq.T, a.H, a.out, a.lse, env);
    if (e != cudaSuccess) return e;
    *plan += "+attn_combine";
  }
  return cudaGetLastError();
}

}  // namespace dsa
