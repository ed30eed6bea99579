// Sparse MLA attention over 4-bit latent rows (DSA_E2M1, latent_e2m1.cuh), on pairs of CTAs.
//
// The mathematics is attn.cu's: for query t, head h and its selected rows S,
//     logit_s = scale * q[t,h] . row_s[0:576],  out = sum_s softmax(logit)_s row_s[0:512],
//     lse = log sum_s exp(logit_s),
// with row_s the values the codes stand for, code * block scale * row scale.
//
// What bounds it: a row is 432 bytes and 278,528 flop for 128 heads, 645 flop per
// byte, so the tensor cores (284 flop per byte at this card's measured rates).  O of
// one query, 128 heads x 512 fp32, fills a whole TMEM, so one CTA cannot hold it
// beside the logits.  attn.cu gives each of two CTAs half of the value dims and lets
// both compute all logits, 1.53 times the flops.  Here the two CTAs of a cluster
// split the heads and issue pair MMAs (cta_group::2, M = 128: 64 heads each, at the
// full rate of 8192 flop per SM and clock): each CTA supplies half of the B operand,
// so the logits are computed once and each CTA widens
//     its own 64 rows of a 128-row tile in full (for Q K^T), and
//     its own half of the value dims of the other CTA's 64 rows (for P V),
// 26 % fewer values than all rows of both.  Nothing is exchanged between the CTAs but
// barrier arrivals.  36 + 16 MMAs a tile: 1152 + 1024 clocks, 2176 per 128 rows.
//
// Types.  code * block scale has at most six significant bits and lies in
// [2^-10, 2688]: exact in f16, and two instructions per pair of values (a convert and
// a half product) where bf16 takes five; eight codes cost a warp 12.9 clocks of issue
// against 26.2, and the widening was what the kernel waited for.  So the latent part
// runs in f16: the query's latent part as q * 2^-a with the head's largest magnitude
// in [2^14, 2^15) (exact for values down to 2^-32 of it), the rope part in bf16 into
// logits of its own, and the row scale, in fp32, where the two meet:
//     x = (latent logit * 2^a) * row scale + rope logit.
// P is f16 as well and carries the row scale: P = 2^(x c - m) * row scale * 2^(m - g),
// c = scale * log2 e, with m a running bound of x c and g one of x c + log2 |row scale|, less
// 7.  Both move only when they grow: m by more than 2^64 (l is fp32), g when P would pass
// 2^15.  So P of the row whose weight times row scale is largest is 2^7 or more (2^4 where
// a cheaper bound may be taken, of row scales within 2^3 of one another), and what P loses under
// f16's normal range, 2^-25 each, is 2^-29 of that row's weight times row scale at most: an output is
// off by 2^-29 max_s(p_s |row scale_s|) sum_s |v_s / row scale_s| for it, p the normalised weights.
// f16 rounds P by 2^-11 of itself, an eighth of bf16's, so the sum that normalises
// the output is that of the unrounded weights, the one the log-sum-exp takes too.
//
// A stage (72 KB, two of them) holds a tile: nine [64 rows x 64 dims] atoms, 128-byte
// swizzle, the same bytes read K-major by Q K^T (rows = N) and MN-major by P V (rows =
// K).  For Q K^T the CTA's own rows: X = dims [0, 256), Y = dims [256, 512), R = rope.
// For P V both CTAs need rows 0-63 at one offset and rows 64-127 at another, each with
// its own value dims: rank 0 (rows 0-63, dims [0, 256)) has them in X already and
// overwrites Y, dead once Q K^T is complete, with rows 64-127; rank 1 (rows 64-127,
// dims [256, 512)) has them in Y and overwrites X with rows 0-63.  P of tile rows 0-63
// goes into R (dead as well), P of rows 64-127 into a buffer of its own.  (Buffers of their
// own for keys and values write and load a third more, and the load/store pipe is what is
// nearest its limit.)
//   shared memory: Q 72 KB | stage 0 | stage 1 | P, rows 64-127 8 KB | row scales, rows, masks, barriers
//   TMEM: latent logits [0,64) [64,128), rope logits [128,192) [192,256), O [256,512).  An
//   N-wide accumulator of a pair MMA takes N/2 columns: lanes 0-63 are the CTA's heads
//   for the first half of N, lanes 64-127 the same heads for the second.
//
// Work.  An item is a row slice (few queries: joined by attn_combine) of 128 heads of a
// query; the clusters that fit the GPU at once share the items out.  Tiles are counted through a
// cluster's items, so the next item's rows, codes and first logits are on their way during
// the last softmax and the output (with a cluster for each item 1290 us instead of 1177).
// Tiles at an item's end that select nothing -- a context shorter than K -- are left out: the
// row warps look for the last selected entry when they open an item and say with every tile
// whether it is its item's first or last (400 queries on a context of 400, K = 2048: 88 us, 273
// with all tiles).
//
// Warps.  0-15 producers, four own and four other rows of a tile each, whichever can go on
// (in a fixed order the other rows wait for Q K^T of rows just written: 1496 us); codes, scales
// and rope are loaded into registers a tile ahead, right after the registers' last use, a
// row's whole 256 or 128 bytes by neighbouring lanes (32-byte pieces of eight rows took three
// times as long).  16 Q K^T and 17 P V (rank 0 issues for both CTAs).  18 and 19 find the
// tiles' cache rows, row scales and masks, two tiles ahead.  20-27 turn the query, which the
// TMA brings once Q K^T of the item before is complete, into f16; then softmax, a thread
// one head and 32 of the tile's rows; the four threads of a head agree on m and g through
// shared memory, when one of them has to let them grow.  Registers are dealt out by
// setmaxnreg, so that no role spills: 224 KB of shared memory leave almost nothing of the L1,
// and a spilled word comes back from the L2 (60 spilled bytes cost 1 %).  The code is kept small
// (rolled loops, short waits): with 98 KB of it every role ran from a cold instruction cache.
//
// Measured (2048 selected rows, 128 heads): 1115 us for 2048 queries, 1047 TFLOP/s of the
// 1926 measured; 55.3 us for 64 (one cluster a query: 128 of 152 SMs), 11.6 us for one (a
// tile each for 16 clusters: latencies).  A tile takes 4300 clocks where its MMAs need 2176: two
// are in flight, each a chain own rows - Q K^T - other rows - P V, and the links slow one another
// (of the loop's clocks the load/store pipe has a wavefront in 71 %, tensor operands are read
// in 45 %, issue slots are taken in 49 %).
// The 48-row kernel of attn.cu's kind, which widens every row in both CTAs: 2171, 100 and 11.7.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "latent_e2m1.cuh"
#include "pair_mma.cuh"

DSA_DEFINE_STATUS_WORD(attn_e2m1)

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleM = 64.0f;                       // growth of m that is let pass, log2 units
constexpr float kPStart = 7.0f, kPMost = 15.0f;          // log2 of the bound of P: when g is set, at most
constexpr float kAlike = 3.0f;                           // spread of a tile's row scales, log2, that the bound may pass over

constexpr int kHeads = 64;            // heads per CTA
constexpr int kTile = 128;            // selected rows per tile
constexpr int kOwn = 64;              // of which this CTA's own
constexpr int kDqk = 576, kDv = 512;
constexpr int kAtom = 64 * 128;       // bytes of a [64 rows x 64 dims] atom
constexpr int kStage = 9 * kAtom;
constexpr int kProducers = 16;
constexpr int kWarpQk = 16, kWarpPv = 17, kWarpRows = 18, kWarpSoft = 20;
constexpr int kThreads = 896;
// registers a thread: 72 at launch (7 groups of 4 warps, 504 in all), then
constexpr int kRegsProducer = 56, kRegsMma = 72, kRegsSoft = 104;
static_assert(4 * kRegsProducer + kRegsMma + 2 * kRegsSoft <= 7 * 72, "register split");

constexpr int kOffQ = 0;
constexpr int kOffStage = kOffQ + 9 * kAtom;             // [2]
constexpr int kOffP1 = kOffStage + 2 * kStage;           // P of tile rows 64-127
constexpr int kOffScale = kOffP1 + kAtom;                 // float [2][128] row scales
constexpr int kOffRows = kOffScale + 2 * kTile * 4;      // int [2][128] cache rows, -1 for none
constexpr int kOffSum = kOffRows + 2 * kTile * 4;        // for 32 heads each: float [2][32]
constexpr int kOffMask = kOffSum + 2 * kHeads * 4;       // uint32 [2][4] valid rows
constexpr int kOffRmax = kOffMask + 32;                  // float [2][2][2] largest, smallest row scale but 0 of a tile's halves
constexpr int kOffOk = kOffRmax + 32;                    // int [8 softmax warps]
constexpr int kOffExp = kOffOk + 32;                     // int8 [64 heads] a
constexpr int kOffInfo = kOffExp + kHeads;               // uint8 [8] what a tile is (tile number mod 8)
constexpr int kOffBar = kOffInfo + 8;
// what a tile is: written before its rows are given out; the warps that read it are fewer than
// eight tiles apart (rows of tile g + 2 wait for Q K^T of g - 1 and so for P V of g - 3)
constexpr uint32_t kFirst = 1, kLast = 2, kEnd = 4, kThere = 8;   // of its item; last of all; a tile at all
constexpr int kNumBars = 25;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kUsed = kOffMisc + 16;
constexpr int kSmemBytes = 232448;
constexpr int kSlack = kSmemBytes - kUsed;               // for re-aligning the base to 1024 bytes
static_assert(kSlack >= 128, "shared memory budget");

constexpr uint32_t kColRope = 128, kColO = 256;
constexpr uint32_t kFmtF16 = 0;
constexpr uint32_t kIdescLatent = make_idesc(kFmtF16, kFmtF16, false, false, 128, 128);
constexpr uint32_t kIdescRope = make_idesc(kFmtBF16, kFmtBF16, false, false, 128, 128);
constexpr uint32_t kIdescPV = make_idesc(kFmtF16, kFmtF16, false, true, 128, 256);

struct PairParams {
  SeqArgs seq;
  MlaArgs a;
  int32_t n_split;          // row slices per query
  int32_t rows_per_split;   // a multiple of kTile
  int32_t head_blocks;      // blocks of 128 heads
  int32_t items;            // T * head_blocks * n_split, shared out among the clusters
  // Partials (n_split > 1), each normalised by its own sum, in bf16 as attn.cu's are: 2^-8 of a partial besides the
  // output's own rounding, where more than one slice is taken (relative error of the outputs 0.0021 instead of
  // 0.0016 for one query).  A choice: in fp32 one query takes 13.0 us instead of 11.5, 16 queries 25.9
  // instead of 22.0; in f16 with an exponent for every 128 dims 12.4 and 22.9.
  uint16_t* ws_o;           // [n_split, T, H, 512]
  float* ws_lse;            // [n_split, T, H]
  uint64_t wait_limit_ns;
  uint32_t dbg_withhold;
  Divisor page, split, heads;   // by the page size, n_split, head_blocks
  float scale_log2;         // |softmax scale| * log2 e; tiny for 0, so that it leaves a masked logit at -inf
  uint32_t early_query;     // the query was complete before the kernel before this one let it launch
};

// Whether a wait must end (1): another thread of the CTA gave up, or the wait has been going
// on for longer than the limit (which this sets the flags for).  Else when it must.
__device__ __noinline__ uint64_t wait_until(volatile int* abort_flag, uint64_t until, uint64_t limit_ns) {
  if (*abort_flag) return 1;
  const uint64_t now = globaltimer_ns();
  if (until == 0) return now + limit_ns;
  if (now < until) return until;
  atomicOr(&g_status_attn_e2m1, kDevTimeout);
  *abort_flag = 1;
  return 1;
}
// Bounded wait for a phase of `bar`.  Short on purpose: fourteen copies of it, and the
// kernel's code has to stay in the instruction cache.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  const uint32_t addr = smem_u32(bar);
  uint64_t until = 0;
  for (uint32_t it = 1; !mbar_try_wait(addr, parity); ++it)
    if ((it & 63u) == 0u && (until = wait_until(abort_flag, until, limit_ns)) == 1) return false;
  return true;
}

// Sixteen codes (8 bytes) times their E4M3 block scale -> sixteen halves, exact.
__device__ __forceinline__ void widen_codes(uint2 u, uint32_t scale_code, uint32_t (&o)[8]) {
  const __half2_raw sr = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>((scale_code & 0xFFu) * 0x0101u), __NV_E4M3);
  const __half2 s = *reinterpret_cast<const __half2*>(&sr);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t h[4];
    e2m1x8_to_half2x4(w ? u.y : u.x, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), s);
      o[4 * w + i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_e2m1_kernel(const __grid_constant__ CUtensorMap qmap, PairParams p) {
  grid_dep_launch();   // the kernel after waits for this grid before it reads what this grid writes
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (sm - sm_raw > kSlack) {   // the same in both CTAs: their shared windows have one layout
    if (threadIdx.x == 0) atomicOr(&g_status_attn_e2m1, kDevConfig);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  // Barriers in pairs belong to a tile's stage or logit buffer: nothing comes to one for the
  // tile after next before its waiter has passed it for this one.
  uint64_t* ownfull = bars;       // [2] leader: both CTAs' own rows written
  uint64_t* othfull = bars + 2;   // [2] leader: the other CTA's rows written, in both
  uint64_t* pvdone = bars + 4;    // [2] P V complete: the tile's stage and P free
  uint64_t* sfree = bars + 6;     // [2] leader: logits read, both CTAs
  uint64_t* sfull = bars + 8;     // [2] Q K^T complete: logits there, half of the stage and its rope atom dead
  uint64_t* mfull = bars + 10;    // [2] row scales and mask of a tile written
  uint64_t* mfree = bars + 12;    // [2] and read
  uint64_t* rfull = bars + 14;    // [2] cache rows of a tile written
  uint64_t* rfree = bars + 16;    // [2] and read
  uint64_t* qstaged = bars + 18;  // this CTA's query staged
  uint64_t* qfull = bars + 19;    // leader: both CTAs' queries staged and their a read
  uint64_t* pfull = bars + 20;    // leader: P written, both CTAs (one buffer: P V of the tile before is complete)
  uint64_t* drain = bars + 21;    // every MMA complete (teardown)
  volatile uint8_t* info = sm + kOffInfo;
  uint64_t* edone = bars + 22;    // [2] an item's output has left the stage of its last tile
  uint64_t* qraw = bars + 24;     // an item's query has come
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* fetched = abort_flag + 1;   // the number of the cluster's item whose query was fetched last
  const uint64_t wlim = p.wait_limit_ns;
  const int K = p.a.K, H = p.a.H;

  // Work items, one after the other, the clusters in turn: a row slice of 128 heads of a query,
  // the last query first (longest causal history).  Tiles, buffers and phases are counted
  // through all of a cluster's items, so that the next item's rows and codes are fetched, its
  // keys written and multiplied while this one's last tile is in its softmax.
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto slice_of = [&](int item) -> int { return item - p.split(item) * p.n_split; };
  auto query_of = [&](int item) -> int { return p.seq.T - 1 - p.heads(p.split(item)); };
  auto head_of = [&](int item) -> int {   // this CTA's first head
    const int i = p.split(item);
    return (i - p.heads(i) * p.head_blocks) * 128 + static_cast<int>(rank) * kHeads;
  };

  auto row_of = [&](int item) -> int { return query_of(item) * H + head_of(item); };   // < 2^31
  // Fetches an item's query, 64 heads as they are (heads beyond H: the next token's, or zeros; nothing
  // is written of them), into its nine swizzled atoms; one thread.
  auto load_query = [&](int row) {
    mbar_arrive_expect_tx(qraw, 9 * kAtom);
#pragma unroll 1
    for (int a = 0; a < 9; ++a) tma_load_2d(sm + kOffQ + a * kAtom, &qmap, qraw, a * 64, row);
  };

  // Warps set out as soon as they can: only what reaches the other CTA, the barriers or TMEM
  // comes after cluster_wait.
  if (warp == kWarpRows && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfree[i], 16);
      mbar_init(&ownfull[i], 2 * kProducers);
      mbar_init(&othfull[i], 2 * kProducers);
      mbar_init(&sfull[i], 1);
      mbar_init(&edone[i], 8);
      mbar_init(&pvdone[i], 1);
      mbar_init(&mfull[i], 2);
      mbar_init(&mfree[i], 8);
      mbar_init(&rfull[i], 2);
      mbar_init(&rfree[i], kProducers);
    }
    mbar_init(pfull, 16);
    mbar_init(drain, 2);
    mbar_init(qstaged, 8);
    mbar_init(qraw, 1);
    mbar_init(qfull, 16);
    *abort_flag = 0;
    *fetched = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == kWarpQk) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(misc)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_arrive();
  if (!p.early_query) grid_dep_wait();

  const uint8_t* kv = static_cast<const uint8_t*>(p.a.kv);
  const uint32_t row_bytes = static_cast<uint32_t>(p.a.row_bytes);   // < 2^31, the host sees to that
  if (warp < kProducers) {
    // ------------------------------------------------ producers
    const int32_t* rows_sm = reinterpret_cast<const int32_t*>(sm + kOffRows);
    shrink_registers<kRegsProducer>();
    cluster_wait();
    const int sub = lane >> 4, blk = lane & 15, l8 = lane >> 3, b8 = lane & 7;
    // In registers.  Own: codes of block `lane` of the warp's four own rows; scale word and
    // rope chunk b8 of row l8.  Other: codes of block blk of this CTA's value dims of rows
    // 2 k + sub of four; scale word lane & 3 of row (lane / 4) & 3.  A row that selects nothing reads
    // row 0 with scales of zero: its logits are masked, and its values must not be row 0's
    // own, which could be anything, NaN among it.
    uint2 kcode[4], vcode[2];
    uint32_t ksc, vsc;
    bool khave, vhave;
    uint4 rope;
    int krow[5], vrow[3];   // the next tile's cache rows
    auto at_row = [&](int row) { return kv + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * row_bytes; };
    auto rows_k = [&](int j) {
      const int32_t* r = rows_sm + (j & 1) * kTile + rank * kOwn + warp * 4;
      const int4 r4 = *reinterpret_cast<const int4*>(r);
      krow[0] = r4.x, krow[1] = r4.y, krow[2] = r4.z, krow[3] = r4.w;
      krow[4] = r[l8];
    };
    auto fetch_k = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) kcode[i] = __ldg(reinterpret_cast<const uint2*>(at_row(krow[i])) + lane);
      const uint8_t* rp = at_row(krow[4]);
      ksc = __ldg(reinterpret_cast<const uint32_t*>(rp + kE2m1Scales) + b8);
      rope = __ldg(reinterpret_cast<const uint4*>(rp + kE2m1Rope) + b8);
      khave = krow[4] >= 0;
    };
    auto rows_v = [&](int j) {
      const int32_t* r = rows_sm + (j & 1) * kTile + (rank ^ 1u) * kOwn + warp * 4;
      vrow[0] = r[sub], vrow[1] = r[2 + sub], vrow[2] = r[(lane >> 2) & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&rfree[j & 1]);   // both have been read
    };
    auto fetch_v = [&]() {
#pragma unroll
      for (int k = 0; k < 2; ++k) vcode[k] = __ldg(reinterpret_cast<const uint2*>(at_row(vrow[k])) + rank * 16 + blk);
      vsc = __ldg(reinterpret_cast<const uint32_t*>(at_row(vrow[2]) + kE2m1Scales) + rank * 4 + (lane & 3));
      vhave = vrow[2] >= 0;
    };
    // Block b of a row goes to chunks 2 (b & 3), 2 (b & 3) + 1 of its atom, swizzled by the row.
    // Lanes of odd atoms take their second half first: eight lanes then cover all banks.
    const bool flip = (lane >> 2) & 1;
    auto put = [&](uint32_t at, uint2 c, uint32_t scale_word, int byte) {
      uint32_t o[8];
      widen_codes(flip ? make_uint2(c.y, c.x) : c, scale_word >> (8 * byte), o);
      st_shared_v4(at, o[0], o[1], o[2], o[3]);
      st_shared_v4(at ^ 16u, o[4], o[5], o[6], o[7]);
    };
    // rows 4 w + i: the swizzle of rows 4-7 of eight
    const uint32_t chunk = static_cast<uint32_t>(((2 * (lane & 3) + (flip ? 1 : 0)) << 4) ^ ((warp & 1) << 6));
    const uint32_t stage0 = smem_u32(sm + kOffStage) + static_cast<uint32_t>(warp * 512);
    const uint32_t kdst = stage0 + static_cast<uint32_t>((lane >> 2) * kAtom) + chunk;
    const uint32_t vdst = stage0 + static_cast<uint32_t>(((rank ^ 1u) * 4 + (blk >> 2)) * kAtom + sub * 128) +
                          (chunk ^ static_cast<uint32_t>(sub << 4));
    const uint32_t rdst = stage0 + static_cast<uint32_t>(8 * kAtom + l8 * 128 + (((b8 ^ l8) << 4) ^ ((warp & 1) << 6)));
    auto wait = [&](uint64_t* bar, int use) -> bool {
      return __all_sync(0xffffffffu, wait_bar(bar, use & 1, abort_flag, wlim));
    };
    // Own rows of tile a once P V of a - 2 has freed the stage, the other CTA's rows of tile b
    // over the half of the stage that is dead once Q K^T of b is complete, whichever can go on.
    // The next tile's row numbers are read before the writes, its codes loaded right after.
    if (wait(&rfull[0], 0)) {
      rows_k(0);
      rows_v(0);
      fetch_k();
      fetch_v();
      // Own rows of tile a take the stage of a - 2: free once P V of that is complete or, when that
      // was an item's last tile, once the item's output, which goes through the stage, has been
      // written.  what: of tiles a, a - 1 and a - 2, four bits each.
      int a = 0, b = 0, item_n = 0;
      uint32_t what = info[0], idle = 0;
      bool more_own = true, end_b = (what & kEnd) != 0;   // end_b: of tile b
      auto own_free = [&]() -> bool {
        if (a < 2) return true;
        return (what >> 8) & kLast ? mbar_test(&edone[item_n & 1], (item_n >> 1) & 1)
                                   : mbar_test(&pvdone[a & 1], ((a >> 1) - 1) & 1);
      };
      uint64_t until = 0;
#pragma unroll 1
      while (true) {
        if (b < a && __all_sync(0xffffffffu, mbar_test(&sfull[b & 1], (b >> 1) & 1))) {
          const uint32_t at = vdst + static_cast<uint32_t>((b & 1) * kStage);
          const bool last = end_b;
          if (!last) {
            end_b = (info[(b + 1) & 7] & kEnd) != 0;
            rows_v(b + 1);   // rfull of b + 1: seen for own rows of b
          }
          vsc = vhave ? vsc : 0u;
          uint32_t w[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) w[k] = __shfl_sync(0xffffffffu, vsc, (2 * k + sub) * 4 + (blk >> 2));
#pragma unroll
          for (int k = 0; k < 2; ++k) put((at ^ (2 * k << 4)) + k * 256, vcode[k], w[k], lane & 3);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_pair(leader_addr(&othfull[b & 1]));
          if (last) break;
          fetch_v();
          ++b;
        } else if (more_own && __all_sync(0xffffffffu, own_free())) {
          const uint32_t st = static_cast<uint32_t>((a & 1) * kStage);
          if ((what >> 8) & kLast) ++item_n;   // a < 2: no such tile
          more_own = !(what & kEnd);
          what <<= 4;
          if (more_own) {
            if (!wait(&rfull[(a + 1) & 1], (a + 1) >> 1)) break;
            rows_k(a + 1);
            what |= info[(a + 1) & 7];
          }
          ksc = khave ? ksc : 0u;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = __shfl_sync(0xffffffffu, ksc, i * 8 + (lane >> 2));
#pragma unroll
          for (int i = 0; i < 4; ++i) put(((kdst + st) ^ (i << 4)) + i * 128, kcode[i], w[i], lane & 3);
          st_shared_v4(rdst + st, rope.x, rope.y, rope.z, rope.w);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && !(p.dbg_withhold && warp == 0 && a == 0)) arrive_pair(leader_addr(&ownfull[a & 1]));
          if (more_own) fetch_k();
          ++a;
        } else {
          __nanosleep(160);
          if ((++idle & 31u) == 0u) {
            until = wait_until(abort_flag, until, wlim);
            if (__any_sync(0xffffffffu, until == 1)) break;
          }
          continue;
        }
        until = 0;
      }
    }
  } else if (warp < kWarpSoft) {
    shrink_registers<kRegsMma>();
    if (warp >= kWarpRows) {
      // ------------------------------------------------ the tiles' rows, row scales and masks
      if (warp == kWarpRows && lane == 0) load_query(row_of(first));   // its thread made the barrier
      __syncwarp();
      if (p.early_query) grid_dep_wait();   // the selected indices come from the kernel before
      // Tile row 32 k + lane from wrow on, k = 0, 1.  A selected entry's way to its row, a tile's
      // time between the steps: the position, its page id, the cache row, the row's scale.
      int pos[2], pos1[2], page[2], row1[2];
      float rs1[2];
      uint32_t sc1[2];   // its last four block scales
#pragma unroll
      for (int k = 0; k < 2; ++k) pos[k] = pos1[k] = page[k] = row1[k] = -1;
      // the tile that load_pos comes to next: entries [gi0, gi1) of the open item are left; the
      // query's position and sequence, and what the tile is, go with it from step to step
      int item = first, gi0 = 0, gi1 = 0, qp1 = 0, b1 = 0;
      uint32_t what1 = 0, what = 0;
      const int32_t* idx = nullptr;
      uint32_t bad = 0;
      const int wrow = (warp - kWarpRows) * 64;
      auto load_pos = [&]() {
        what1 = 0;
        if (gi0 >= gi1 && item < p.items) {
          const int t = query_of(item);
          gi0 = slice_of(item) * p.rows_per_split;
          gi1 = min(K, gi0 + p.rows_per_split);
          idx = p.a.idx + static_cast<int64_t>(t) * K;
          qp1 = __ldg(p.seq.q_pos + t);
          b1 = __ldg(p.seq.q_seq + t);
          item += step;
          what1 = kFirst;
        }
        if (what1 & kFirst) {
          // tiles at the end that select nothing (a context shorter than K) are left out, all but the
          // item's first: the last 128 entries, then 512 at a time towards the first
          const int top = gi1;   // most often the last tile's entries settle it
          for (int e = top; e > gi0 + kTile;) {
            const int from = max(gi0, e - (e == top ? kTile : 512));
            int last = -1;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int i = from + k * 32 + lane;
              if (i < e && __ldg(idx + i) >= 0) last = i;
            }
            last = __reduce_max_sync(0xffffffffu, last);
            gi1 = max(last + 1, min(gi1, gi0 + kTile));
            e = last >= 0 ? 0 : from;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = gi0 + wrow + k * 32 + lane;
          pos1[k] = i < gi1 ? __ldg(idx + i) : -1;
        }
        if (gi0 < gi1) what1 |= kThere | (gi0 + kTile >= gi1 ? kLast | (item >= p.items ? kEnd : 0u) : 0u);
        gi0 += kTile;
      };
      auto load_page = [&]() {   // of pos <- pos1
        what = what1;
        int qp = qp1, b = b1;
        if (qp < 0 || qp >= p.seq.max_ctx || b < 0 || b >= p.seq.B) {
          bad |= kDevBadPos;
          qp = -1;
          b = 0;
        }
        const int32_t* bt = p.seq.block_table + static_cast<int64_t>(b) * p.seq.bt_stride;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          pos[k] = pos1[k];
          if (pos[k] > qp) {
            bad |= kDevBadIndex;
            pos[k] = -1;
          }
          page[k] = pos[k] >= 0 ? __ldg(bt + p.page(pos[k])) : -1;
        }
      };
      auto row_at = [&](int row) { return kv + static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * row_bytes; };
      auto load_scale = [&]() {   // row1, rs1, sc1 of pos, page
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool good = page[k] >= 0 && page[k] < p.seq.n_pages;
          if (pos[k] >= 0 && !good) bad |= kDevBadIndex;
          row1[k] = good ? (page[k] - p.page(pos[k])) * p.seq.page_size + pos[k] : -1;   // < cache_rows < 2^31
          const uint8_t* rp = row_at(row1[k]);
          rs1[k] = __ldg(reinterpret_cast<const float*>(rp + kE2m1RowScale));
          sc1[k] = __ldg(reinterpret_cast<const uint32_t*>(rp + kE2m1RowScale) - 1);
        }
      };
      // step j: scales and mask of tile j - 1 and rows of tile j given out, pages of j + 1 and
      // positions of j + 2 loaded; steps -2 and -1 only load
      uint32_t given = 0;   // what tile j - 1 is
#pragma unroll 1
      for (int j = -2;; ++j) {
        asm volatile("" : "+r"(j));   // one copy of the loop's code
        if (j == 0) cluster_wait();
        const int st = j & 1;
        if (given) {
          if (j >= 3 &&
              !__all_sync(0xffffffffu, wait_bar(&mfree[st ^ 1], (((j - 1) >> 1) - 1) & 1, abort_flag, wlim)))
            break;
          uint32_t rmax = 0u, rmin = 0x7F800000u;   // magnitudes' bits, in the order of the magnitudes
          uint32_t mask[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mine = row1[k] >= 0 ? rs1[k] : 0.f;
            // A row whose block scales are all zero has no values, and its row scale (1, where the writer has
            // stored it) must not stand for any: it takes part with 0.  Seldom more than a look at four scales
            // (64 queries 55.3 us, 54.3 without it; the chunk the same).
            constexpr uint32_t kAbs = 0x7F7F7F7Fu;
            const bool look = row1[k] >= 0 && (sc1[k] & kAbs) == 0u;
            if (__any_sync(0xffffffffu, look) && look) {
              const uint4* sp = reinterpret_cast<const uint4*>(row_at(row1[k]) + kE2m1Scales);
              const uint4 a = __ldg(sp), c = __ldg(sp + 1);
              if (((a.x | a.y | a.z | a.w | c.x | c.y | c.z | c.w) & kAbs) == 0u) mine = 0.f;
            }
            const uint32_t bits = __float_as_uint(mine) & 0x7FFFFFFFu;
            rmax = max(rmax, bits);
            rmin = min(rmin, bits ? bits : rmin);
            mask[k] = __ballot_sync(0xffffffffu, row1[k] >= 0);
            reinterpret_cast<float*>(sm + kOffScale)[(st ^ 1) * kTile + wrow + k * 32 + lane] = mine;
          }
          rmax = __reduce_max_sync(0xffffffffu, rmax);
          rmin = __reduce_min_sync(0xffffffffu, rmin);
          if (lane == 0) {
            *reinterpret_cast<uint2*>(sm + kOffMask + (st ^ 1) * 16 + wrow / 8) = make_uint2(mask[0], mask[1]);
            *reinterpret_cast<uint2*>(sm + kOffRmax + (st ^ 1) * 16 + wrow / 8) = make_uint2(rmax, rmin);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&mfull[st ^ 1]);
          if (given & kEnd) break;
        }
        given = j >= 0 ? what : 0u;
        if (j >= 0 && !given) break;   // not before the end
        if (given) {
          if (j >= 2 && !__all_sync(0xffffffffu, wait_bar(&rfree[st], ((j >> 1) - 1) & 1, abort_flag, wlim))) break;
          load_scale();
#pragma unroll
          for (int k = 0; k < 2; ++k)
            reinterpret_cast<int32_t*>(sm + kOffRows)[st * kTile + wrow + k * 32 + lane] = row1[k];
          if (warp == kWarpRows && lane == 0) info[j & 7] = static_cast<uint8_t>(given);
          __syncwarp();
          if (lane == 0) mbar_arrive(&rfull[st]);
        }
        load_page();
        load_pos();
      }
      if (bad) atomicOr(&g_status_attn_e2m1, bad);
    } else if (warp == kWarpQk) {
      cluster_wait();
      tc_fence_after();
      const uint32_t tmem = misc[0];
      const uint64_t dq = make_sdesc(smem_u32(sm + kOffQ), 16, 1024, kLayoutSw128);
      const uint64_t dk0 = make_sdesc(smem_u32(sm + kOffStage), 16, 1024, kLayoutSw128);
      int n = 0;   // items
      bool ok = rank == 0, more = true;
#pragma unroll 1
      for (int g = 0; ok && more; ++g) {
        const int sb = g & 1;
        // the keys are there, the logit buffer is free and the query is the item's
        ok = __all_sync(0xffffffffu, wait_bar(&ownfull[sb], (g >> 1) & 1, abort_flag, wlim));
        if (!ok) break;
        const uint32_t what = info[g & 7];
        more = !(what & kEnd);
        if (g >= 2) ok = __all_sync(0xffffffffu, wait_bar(&sfree[sb], ((g >> 1) - 1) & 1, abort_flag, wlim));
        if (ok && (what & kFirst)) ok = __all_sync(0xffffffffu, wait_bar(qfull, n++ & 1, abort_flag, wlim));
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();
        if (elect_one()) {
          const uint32_t d = tmem + sb * 64;
          const uint64_t dk = dk0 + static_cast<uint64_t>((sb * kStage) >> 4);
#pragma unroll 1
          for (int a = 0; a < 8; ++a) {   // 64 dims a turn
            const uint64_t off = static_cast<uint64_t>((a * kAtom) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_pair(d, dq + off + 2 * kk, dk + off + 2 * kk, kIdescLatent, static_cast<uint32_t>(a | kk));
          }
          constexpr uint64_t off = (8 * kAtom) >> 4;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_pair(d + kColRope, dq + off + 2 * kk, dk + off + 2 * kk, kIdescRope, static_cast<uint32_t>(kk));
          commit_pair(&sfull[sb]);
        }
        __syncwarp();
      }
    } else if (warp == kWarpPv) {
      cluster_wait();
      tc_fence_after();
      const uint32_t tmem = misc[0];
      const uint64_t dv0 = make_sdesc(smem_u32(sm + kOffStage), kAtom, 1024, kLayoutSw128);
      const uint64_t dp0 = make_sdesc(smem_u32(sm + kOffStage + 8 * kAtom), 16, 1024, kLayoutSw128);
      const uint64_t dp1 = make_sdesc(smem_u32(sm + kOffP1), 16, 1024, kLayoutSw128);
      bool ok = rank == 0, more = true;
#pragma unroll 1
      for (int g = 0; ok && more; ++g) {
        ok = __all_sync(0xffffffffu, wait_bar(&othfull[g & 1], (g >> 1) & 1, abort_flag, wlim));
        const uint32_t what = info[g & 7];
        more = !(what & kEnd);
        if (ok) ok = __all_sync(0xffffffffu, wait_bar(pfull, g & 1, abort_flag, wlim));
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();
        if (elect_one()) {
          const uint64_t st = static_cast<uint64_t>(((g & 1) * kStage) >> 4);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {   // value atoms 2 (q / 2), tile rows [64 (q & 1), 64 (q & 1) + 64)
            const uint64_t da = (q & 1) ? dp1 : dp0 + st;
            const uint64_t db = dv0 + st + static_cast<uint64_t>((((q & 1) * 4 + (q >> 1) * 2) * kAtom) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_pair(tmem + kColO + (q >> 1) * 128, da + 2 * kk, db + 128 * kk, kIdescPV,
                        static_cast<uint32_t>((~what & kFirst) | (q & 1) | kk));
          }
          commit_pair(&pvdone[g & 1]);
        }
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------ softmax and epilogue
    grow_registers<kRegsSoft>();
    const int quarter = warp & 3;
    const int hl = (quarter & 1) * 32 + lane;   // head within the CTA
    const int half = quarter >> 1;              // tile rows [64 half, 64 half + 64), of which
    const int part32 = (warp - kWarpSoft) >> 2; // this thread's [32 part32, 32 part32 + 32)
    const int rq = half * 2 + part32;           // row quarter of the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    const uint32_t head_bar = 2 + (quarter & 1);   // the 128 threads of 32 heads
    // where the four threads of a head exchange sums, and maxima: [2][4 row quarters][32], in that part
    // of the P buffer that these threads write (P V of the tile before is complete, this tile's P not begun)
    float* sums = reinterpret_cast<float*>(sm + kOffSum + (quarter & 1) * 256) + lane;
    float* xmax = reinterpret_cast<float*>(sm + kOffP1 + (quarter & 1) * 4096) + lane;
    volatile int* oks = reinterpret_cast<volatile int*>(sm + kOffOk);
    const volatile float* scale_range = reinterpret_cast<const volatile float*>(sm + kOffRmax);
    const volatile uint32_t* masks = reinterpret_cast<const volatile uint32_t*>(sm + kOffMask);
    const uint32_t prow0 = smem_u32(sm + (half ? kOffP1 : kOffStage + 8 * kAtom)) + static_cast<uint32_t>(hl * 128);
    const uint32_t pstep = half ? 0u : static_cast<uint32_t>(kStage);   // rows 0-63: the stage's rope atom
    // The query: eight heads a warp, their latent part turned in place into f16 with a power of
    // two per head.  Loops, not straight code: this runs once an item, from
    // a cold instruction cache.
    const uint32_t qsm = smem_u32(sm + kOffQ);
    auto stage_query = [&](int n, bool& ok) {
      const int w8 = (warp - kWarpSoft) * 8;
      ok = __all_sync(0xffffffffu, wait_bar(qraw, n & 1, abort_flag, wlim)) && ok;
      // head lane & 7, atoms 2 (lane / 8) and the next
      const int h = lane & 7;
      const uint32_t at = qsm + static_cast<uint32_t>((lane >> 3) * 2 * kAtom + (w8 + h) * 128);
      auto chunk_at = [&](int c) { return static_cast<uint32_t>((c >> 3) * kAtom + (((c ^ h) & 7) << 4)); };
      __nv_bfloat162 mx = __float2bfloat162_rn(0.f);
#pragma unroll 4
      for (int c = 0; c < 16; ++c) {
        const uint4 v = ld_shared_v4(at + chunk_at(c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = __hmax2(mx, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
      }
      float amax = fmaxf(__low2float(mx), __high2float(mx));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
      // floor(log2 amax) - 14 from the exponent's bits; a subnormal maximum is small enough for the clamp
      const int e = amax > 0.f ? max(-110, min(113, static_cast<int>(__float_as_uint(amax) >> 23) - 141)) : 0;
      // the maximum is taken over unscaled logits: a negative scale turns the query round
      const uint32_t flip = p.a.softmax_scale < 0.f ? 0x80008000u : 0u;
      const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23 | (flip & 0x80000000u));   // +-2^-e
      if (lane < 8) reinterpret_cast<int8_t*>(sm + kOffExp)[w8 + h] = static_cast<int8_t>(e);
#pragma unroll 1
      for (int c4 = 0; c4 < 16; c4 += 8) {   // eight loads, then eight stores
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = ld_shared_v4(at + chunk_at(c4 + k));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 q2 =
                __floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
            o[i] = *reinterpret_cast<const uint32_t*>(&q2);
          }
          st_shared_v4(at + chunk_at(c4 + k), o[0], o[1], o[2], o[3]);
        }
      }
      if (flip) {   // the rope part: chunks lane / 8 and that plus four of the eight
#pragma unroll 1
        for (int c = lane >> 3; c < 8; c += 4) {
          const uint32_t a = qsm + static_cast<uint32_t>(8 * kAtom + (w8 + h) * 128 + ((c ^ h) << 4));
          const uint4 v = ld_shared_v4(a);
          st_shared_v4(a, v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    // Tells the CTA's softmax warps that the query is staged, waits for all of them, fetches this
    // thread's 2^a and lets the leader multiply.
    auto query_exp = [&](int n, bool& ok) -> float {
      if (lane == 0) mbar_arrive(qstaged);
      ok = __all_sync(0xffffffffu, wait_bar(qstaged, n & 1, abort_flag, wlim)) && ok;
      const int e = reinterpret_cast<const volatile int8_t*>(sm + kOffExp)[hl];
      const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      __syncwarp();
      if (lane == 0) arrive_pair(leader_addr(qfull));
      return f;
    };
    // Turn by turn: the next item's query is staged (Q K^T of the last tile is complete), the
    // last item's output written, the next item's tiles taken.
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = misc[0] + lane_off;
    bool ok = true;
    float m = -INFINITY, g = -INFINITY, l = 0.f, qexp = 0.f;
    int gt = 0, n = 0, done = 0;   // tiles, items staged and done
#pragma unroll 1
    for (int item = first;; item += step) {
      const bool more = item < p.items;
      if (more) {
        stage_query(n, ok);
        qexp = query_exp(n++, ok);
      }
      if (item != first) {
        const int last = item - step;
        ok = __all_sync(0xffffffffu, ok && wait_bar(&pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1, abort_flag, wlim));
        // the sums of a head's four threads
        if (rq >= 2) sums[(rq - 2) * 32] = l;
        named_bar_sync(head_bar, 128);
        if (rq < 2) sums[rq * 32] += l;
        named_bar_sync(head_bar, 128);
        l = sums[0] + sums[32];
        if (ok) {
          tc_fence_after();
          // O holds sum p rs 2^(m - g) v over l = sum p
          const float inv = l == 0.f ? 0.f : exp2f(fminf(fmaxf(g - m, -126.f), 126.f)) / l;   // l may be NaN
          const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          const int t = query_of(last), h0 = head_of(last);
          const int heads = min(32, H - (h0 + (quarter & 1) * 32));   // of this warp's 32 that exist
          const bool part = p.n_split > 1;
          const int64_t head0 =
              (static_cast<int64_t>(part ? slice_of(last) : 0) * p.seq.T + t) * H + h0 + (quarter & 1) * 32;
          uint8_t* out = reinterpret_cast<uint8_t*>(part ? p.ws_o : static_cast<uint16_t*>(p.a.out)) +
                         (head0 * kDv + half * 256 + part32 * 128) * 2;
          // through the last tile's stage, which P V has left and the producers leave alone till edone:
          // a thread holds one head's values, and neighbouring lanes should store a head's
          const uint32_t stg = smem_u32(sm + kOffStage) + ((gt - 1) & 1) * kStage + (warp - kWarpSoft) * 4096;
          if (heads > 0) {
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {
#pragma unroll 1
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t o[32];
                tmem_ld32(tmem + kColO + part32 * 128 + cc * 64 + hf * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  st_shared_v4(stg + lane * 128 + (((hf * 4 + k) ^ (lane & 7)) << 4),
                               pack_bf16x2(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv),
                               pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv),
                               pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv),
                               pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv));
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int row = i * 4 + (lane >> 3), c4 = lane & 7;
                const uint4 v = ld_shared_v4(stg + row * 128 + ((c4 ^ (row & 7)) << 4));
                if (row < heads)
                  *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * kDv * 2 + cc * 128 + c4 * 16) = v;
              }
              __syncwarp();
            }
            if (rq == 0 && lane < heads) {
              if (part)
                p.ws_lse[head0 + lane] = lse;
              else if (p.a.lse)
                p.a.lse[head0 + lane] = lse;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&edone[done++ & 1]);
      }
      if (!more) break;
      const int next_row = row_of(min(item + step, p.items - 1));
      bool last_tile = false, stop = false;
      m = g = -INFINITY;
      l = 0.f;
#pragma unroll 1
      for (; !last_tile; ++gt) {
        const int j = gt, st = j & 1;
        ok = ok && wait_bar(&mfull[st], (j >> 1) & 1, abort_flag, wlim) &&
             wait_bar(&sfull[st], (j >> 1) & 1, abort_flag, wlim);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        // Q K^T of the item's last tile is complete: the next item's query may come
        if (ok && warp == kWarpSoft && (info[j & 7] & (kLast | kEnd)) == kLast) {
          if (lane == 0) {
            load_query(next_row);
            *fetched = n;
          }
          __syncwarp();
        }
        const uint32_t scales = smem_u32(sm + kOffScale) + static_cast<uint32_t>((st * kTile + rq * 32) * 4);
        float x[32];
        float mx = -INFINITY, rmax = 0.f;
        if (ok) {
          // x = latent * 2^a * row scale + rope, -inf for rows that select nothing
          uint32_t s0[32];
          tmem_ld32(tmem + st * 64 + part32 * 32, s0);
          {
            uint32_t s1[32];
            tmem_ld32(tmem + kColRope + st * 64 + part32 * 32, s1);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(s1[i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_pair(leader_addr(&sfree[st]));   // the logit buffer has been read
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const uint4 rs = ld_shared_v4(scales + static_cast<uint32_t>(i * 4));
            float t0, t1, t2, t3;
            mul2(t0, t1, __uint_as_float(s0[i]), __uint_as_float(s0[i + 1]), qexp, qexp);
            mul2(t2, t3, __uint_as_float(s0[i + 2]), __uint_as_float(s0[i + 3]), qexp, qexp);
            fma2(x[i], x[i + 1], t0, t1, __uint_as_float(rs.x), __uint_as_float(rs.y));
            fma2(x[i + 2], x[i + 3], t2, t3, __uint_as_float(rs.z), __uint_as_float(rs.w));
          }
          last_tile = (info[j & 7] & kLast) != 0;
          const uint32_t vmask = masks[st * 4 + rq];
          if (vmask != ~0u) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = ((vmask >> i) & 1u) ? x[i] : -INFINITY;
          }
          rmax = fmaxf(scale_range[4 * st], scale_range[4 * st + 2]);
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2) mq[(i >> 1) & 3] = fmax3(mq[(i >> 1) & 3], x[i], x[i + 1]);
          mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sl2;
        }
        // The four threads of a head share m and g, and their warps leave together when one
        // has given up.  One barrier tells the 128 threads of 32 heads whether any of them has
        // to let m or g grow; only then (the first tile, and seldom after) do they exchange
        // their maxima.  For g the sum of two maxima, a bound, tells when to look.
        const float lrmax = __log2f(rmax);
        const bool grow = named_bar_or(head_bar, 128, !ok || mx > m + kRescaleM || mx + lrmax > g + kPMost);
        // P has one buffer and O may have to be rescaled: P V of the tile before is complete
        bool pv_ok = true;
        if (j >= 1 && ok) pv_ok = wait_bar(&pvdone[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, wlim);
        if (grow) {
          // What P is bounded by.  Where the tile's row scales are much alike the sum of the two maxima, too large by
          // their spread at most; else the largest weight times row scale of one row, or a row of large scale
          // and no weight would take the others' P under f16's range.  (The latter for every tile that comes here:
          // one query 11.9 us instead of 11.5, the chunk 1129 instead of 1115.)
          const bool alike = rmax <= exp2f(kAlike) * fminf(scale_range[4 * st + 1], scale_range[4 * st + 3]);
          float wx = mx + lrmax;
          if (!alike) {
            wx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const uint4 rs = ld_shared_v4(scales + static_cast<uint32_t>(i * 4));
              wx = fmax3(wx, fmaf(x[i], sl2, __log2f(fabsf(__uint_as_float(rs.x)))),
                         fmaf(x[i + 1], sl2, __log2f(fabsf(__uint_as_float(rs.y)))));
              wx = fmax3(wx, fmaf(x[i + 2], sl2, __log2f(fabsf(__uint_as_float(rs.z)))),
                         fmaf(x[i + 3], sl2, __log2f(fabsf(__uint_as_float(rs.w)))));
            }
          }
          xmax[rq * 32] = mx;
          xmax[128 + rq * 32] = wx;
          if (lane == 0) oks[warp - kWarpSoft] = ok ? 1 : 0;
          named_bar_sync(head_bar, 128);
#pragma unroll
          for (int k = 1; k < 4; ++k) {
            mx = fmaxf(mx, xmax[(rq ^ k) * 32]);
            wx = fmaxf(wx, xmax[128 + (rq ^ k) * 32]);
          }
          // the four warps: those whose number is as odd as this one's
#pragma unroll
          for (int k = 0; k < 4; ++k) ok = ok && oks[2 * k + (warp & 1)] != 0;
          named_bar_sync(head_bar, 128);
          if (!ok) {
            stop = true;
            break;
          }
          const float gx = wx - kPStart;
          const bool need_m = mx > m + kRescaleM, need_g = wx > g + kPMost;
          // (g of -inf: nothing in O yet)
          if (__any_sync(0xffffffffu, need_g && g > -INFINITY)) {
            tc_fence_after();
            const float f = need_g && g > -INFINITY ? exp2f(g - gx) : 1.f;
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {   // this thread's half of the columns
              uint32_t o[16];
              const uint32_t at = tmem + kColO + part32 * 128 + cc * 16;
              tmem_ld16(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(at, o);
            }
            tmem_st_wait();
          }
          if (need_g) g = gx;
          if (need_m) {
            l *= exp2f(m - mx);
            m = mx;
          }
        }
        ok = __all_sync(0xffffffffu, pv_ok);
        const float msub = (m == -INFINITY) ? 0.f : m;
        // 2^(m - g), kept finite and nonzero
        const float gain = (g == -INFINITY) ? 1.f : exp2f(fminf(fmaxf(msub - g, -126.f), 126.f));
        const uint32_t prow = prow0 + (j & 1) * pstep;
        float se[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = 8 * c + 4 * q;
            const uint4 rs = ld_shared_v4(scales + static_cast<uint32_t>(i * 4));
            const float r[4] = {__uint_as_float(rs.x), __uint_as_float(rs.y), __uint_as_float(rs.z),
                                __uint_as_float(rs.w)};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              float d0 = -msub, d1 = -msub;
              fma2(d0, d1, x[i + k], x[i + k + 1], sl2, sl2);
              const float p0 = fast_exp2(d0), p1 = fast_exp2(d1);
              add2(se[k], se[k + 1], se[k], se[k + 1], p0, p1);
              float w0, w1;
              mul2(w0, w1, p0, p1, gain, gain);
              mul2(w0, w1, w0, w1, r[k], r[k + 1]);
              const __half2 h = __floats2half2_rn(w0, w1);
              pk[2 * q + (k >> 1)] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          st_shared_v4(prow + static_cast<uint32_t>(((part32 * 4 + c) ^ (hl & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        l += (se[0] + se[1]) + (se[2] + se[3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_pair(leader_addr(pfull));
          mbar_arrive(&mfree[st]);
        }
      }
      if (stop) break;
    }
  }

  // The last query fetched has come (after an abort it may not have been waited for).
  if (warp == kWarpSoft) mbar_drain(qraw, *fetched & 1, &g_status_attn_e2m1, p.wait_limit_ns);
  // Every MMA has finished in both CTAs before either releases its TMEM or leaves (after
  // an abort some may still be running).
  if (rank == 0 && (warp == kWarpQk || warp == kWarpPv)) {
    if (elect_one()) commit_pair(drain);
    __syncwarp();
  }
  if (warp == kWarpQk) mbar_drain(drain, 0, &g_status_attn_e2m1, p.wait_limit_ns);
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (warp == kWarpQk) {
    tc_fence_after();
    const uint32_t tmem = misc[0];
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Clusters that the current device holds at once (its SMs need not pair up everywhere), asked once.
int resident_clusters(int num_sms) {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return std::max(1, num_sms / 2);
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  const void* kernel = reinterpret_cast<const void*>(attn_e2m1_kernel);
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

// Row slices per query: one cluster for each while the GPU holds them all at once, a
// slice at least one tile.  Measured with other numbers of slices (us, 2048 rows a query, this
// rule's first): 1 query 16 slices 11.7, 8 14.0, 1 43.7; 16 queries 4 slices 22.7, 3 27.2, 8 28.5,
// 1 47.6; 38 queries 2 slices 37.7, 4 41.7, 1 54.5; 40 queries 1 slice 54.4, 2 63.4, 3 53.1; 64
// queries 1 slice 55.6, 2 66.6, 3 70.0; 80 queries 1 slice 102, 2 93.5, 4 91.6; 160 queries 1 slice
// 151, 2 155.  An item costs its query's staging, its output and a share of the merge besides its
// tiles, so slices that fill the last clusters gain 10 % at 77 to 100 queries and lose elsewhere.
int choose_split(const SeqArgs& seq, const MlaArgs& a, int num_sms) {
  const int tiles = (a.K + kTile - 1) / kTile;
  const int64_t clusters = static_cast<int64_t>(seq.T) * ((a.H + 127) / 128);
  return static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(tiles, resident_clusters(num_sms) / std::max<int64_t>(1, clusters))));
}

}  // namespace

size_t attn_e2m1_workspace_bytes(const SeqArgs& seq, const MlaArgs& a, int num_sms) {
  if (seq.T == 0) return 0;
  const int split = choose_split(seq, a, num_sms);
  if (split <= 1) return 0;
  const size_t o = static_cast<size_t>(split) * seq.T * a.H * kDv * sizeof(uint16_t);
  const size_t l = static_cast<size_t>(split) * seq.T * a.H * sizeof(float);
  return ((o + 255) / 256) * 256 + ((l + 255) / 256) * 256;
}

cudaError_t launch_attn_e2m1(const SeqArgs& seq, const MlaArgs& a, void* workspace, size_t ws_bytes,
                             const LaunchEnv& env, std::string* plan) {
  int split = choose_split(seq, a, env.num_sms);
  if (split > 1 && (workspace == nullptr || ws_bytes < attn_e2m1_workspace_bytes(seq, a, env.num_sms)))
    split = 1;   // no room for partials: one slice per query
  const int tiles = (a.K + kTile - 1) / kTile;
  const int rps = (tiles + split - 1) / split * kTile;
  split = (a.K + rps - 1) / rps;   // every slice non-empty
  const int head_blocks = (a.H + 127) / 128;
  const int64_t items = static_cast<int64_t>(seq.T) * head_blocks * split;
  if (items > 0x3FFFFFFFll) return cudaErrorInvalidConfiguration;
  float scale_log2 = std::fabs(a.softmax_scale) * kLog2e;
  if (scale_log2 < 1e-30f) scale_log2 = 1e-30f;   // NaN stays
  PairParams p{seq,     a,  split,        rps,  head_blocks, static_cast<int32_t>(items),
               nullptr, nullptr, kWaitLimitNs, 0u, Divisor(seq.page_size), Divisor(split), Divisor(head_blocks),
               scale_log2, env.chained ? 1u : 0u};
  debug_wait_state(&p.wait_limit_ns, &p.dbg_withhold);
  if (split > 1) {
    const size_t o = static_cast<size_t>(split) * seq.T * a.H * kDv * sizeof(uint16_t);
    p.ws_o = static_cast<uint16_t*>(workspace);
    p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((o + 255) / 256) * 256);
  }
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(attn_e2m1_kernel), kSmemBytes, env.device);
  if (e != cudaSuccess) return e;
  alignas(64) CUtensorMap qmap;   // the queries' heads as rows; boxes of 64 dims of 64 heads
  std::string why;
  if (static_cast<int64_t>(seq.T) * a.H > 0x7FFFFF00ll ||
      !encode_tmap_2d(&qmap, a.q, 2, kDqk, static_cast<uint64_t>(seq.T) * a.H, kDqk * 2, 64, kHeads, &why))
    return cudaErrorInvalidValue;
  const int64_t grid = 2 * std::min<int64_t>(items, resident_clusters(env.num_sms));
  e = launch_kernel(attn_e2m1_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, env.stream, true,
                    2, qmap, p);
  if (e != cudaSuccess) return e;
  char buf[96];
  snprintf(buf, sizeof(buf), "attn_tc<e2m1x128>[split=%d,grid=%lld]", split, static_cast<long long>(grid));
  *plan += buf;
  if (split > 1) {
    e = launch_attn_combine(p.ws_o, p.ws_lse, split, seq.T, a.H, a.out, a.lse, env);
    if (e != cudaSuccess) return e;
    *plan += "+attn_combine";
  }
  return cudaGetLastError();
}

}  // namespace dsa
