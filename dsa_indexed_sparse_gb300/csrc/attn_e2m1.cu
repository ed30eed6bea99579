// Sparse MLA attention over 4-bit latent rows (DSA_E2M1, latent_e2m1.cuh), on pairs of CTAs.
//
// The mathematics is attn.cu's: for query t, head h and its selected rows S,
//     logit_s = scale * q[t,h] . row_s[0:576],  out = sum_s softmax(logit)_s row_s[0:512],
//     lse = log sum_s exp(logit_s),
// with row_s the values the codes stand for, widened to bf16 (code * block scale *
// row scale: at most six significant bits, so exact for a power-of-two row scale).
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
// c = scale * log2 e, with m a running bound of x c and g one of x c + log2(row
// scale).  Both move only when they grow, m by more than 2^64 (l is fp32) and g by
// more than 2^14 (P stays below 2^15; what falls under f16's 2^-24 is 2^-38 of it).
// f16 rounds P by 2^-12 of itself, an eighth of bf16's, so the sum that normalises
// the output is that of the unrounded weights, the one the log-sum-exp takes too.
//
// A stage (72 KB, two of them) holds a tile: nine [64 rows x 64 dims] atoms, 128-byte
// swizzle, the same bytes read K-major by Q K^T (rows = N) and MN-major by P V (rows =
// K).  For Q K^T the CTA's own rows: X = dims [0, 256), Y = dims [256, 512), R = rope.
// For P V both CTAs need rows 0-63 at one offset and rows 64-127 at another, each with
// its own value dims: rank 0 (rows 0-63, dims [0, 256)) has them in X already and
// overwrites Y, dead once Q K^T is complete, with rows 64-127; rank 1 (rows 64-127,
// dims [256, 512)) has them in Y and overwrites X with rows 0-63.  P of tile rows 0-63
// goes into R (dead as well), P of rows 64-127 into a buffer of its own.
//   shared memory: Q 72 KB | stage 0 | stage 1 | P, rows 64-127 8 KB | row scales, masks, barriers
//   TMEM: latent logits [0,64) [64,128), rope logits [128,192) [192,256), O [256,512).  An
//   N-wide accumulator of a pair MMA takes N/2 columns: lanes 0-63 are the CTA's heads
//   for the first half of N, lanes 64-127 the same heads for the second.
//
// Warps: 0-7 producers, eight own and eight of the other CTA's rows each.  Their codes,
// scales and rope are loaded into registers a tile ahead.  Turn by turn: the other
// CTA's rows of tile j once Q K^T_j is complete (beside the softmax), the own rows of
// tile j + 1 once P V_{j-1} has freed its stage (beside Q K^T_j + 1 of the other
// stage).  8 Q K^T and 9 P V (rank 0 issues for both CTAs).  10-17 softmax: a thread
// owns one head and 32 of the tile's rows, the four threads of a head agree on m and g
// through shared memory.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "latent_e2m1.cuh"

DSA_DEFINE_STATUS_WORD(attn_e2m1)

namespace dsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleM = 64.0f, kRescaleG = 14.0f;   // growth of m and g that is let pass, log2 units

constexpr int kHeads = 64;            // heads per CTA
constexpr int kTile = 128;            // selected rows per tile
constexpr int kOwn = 64;              // of which this CTA's own
constexpr int kDqk = 576, kDv = 512;
constexpr int kAtom = 64 * 128;       // bytes of a [64 rows x 64 dims] atom
constexpr int kStageBytes = 9 * kAtom;
constexpr int kRopeAtom = 8 * kAtom;  // offset of the rope atom (P of rows 0-63 later) in a stage
constexpr int kProducers = 8;
constexpr int kWarpQk = 8, kWarpPv = 9, kWarpSoft = 10;
constexpr int kThreads = 576;

constexpr int kOffQ = 0;
constexpr int kOffStage = 9 * kAtom;
constexpr int kOffP1 = kOffStage + 2 * kStageBytes;
constexpr int kOffScale = kOffP1 + kAtom;                // float [2 stages][128] row scales
constexpr int kOffMask = kOffScale + 2 * kTile * 4;      // uint64 [2 stages][2 halves of the tile]
constexpr int kOffRmax = kOffMask + 64;                  // float [2 stages][8] largest row scale of a warp's rows
constexpr int kOffQexp = kOffRmax + 64;                  // float [64] the heads' 2^a
constexpr int kOffOk = kOffQexp + kHeads * 4;            // int [2][8 softmax warps]
constexpr int kOffBar = kOffOk + 64;
constexpr int kNumBars = 16;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffMax = kOffMisc + 16;                   // float [4 row quarters][64 heads]
constexpr int kUsed = kOffMax + 4 * kHeads * 4;
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
  uint16_t* ws_o;           // [n_split, T, H, 512] bf16 partials (n_split > 1), each normalised by its own sum
  float* ws_lse;            // [n_split, T, H]
  uint64_t wait_limit_ns;
  uint32_t dbg_withhold;
  uint32_t early_query;     // the query was complete before the kernel before this one let it launch
};

// ------------------------------------------------------------------ pair instructions
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `bar` in the leader CTA (rank 0) of the cluster.
__device__ __forceinline__ uint32_t leader_addr(const uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
// Arrival on a barrier of either CTA.  At CTA scope: what the arrival announces -- rows,
// P and logits read -- lies in this CTA's own shared memory and TMEM and is handed to
// the tensor cores by the proxy and tcgen05 fences before it.  A release at cluster
// scope waited for the warp's global loads as well: 4000 clocks a tile.
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  return mbar_wait(bar, parity, &g_status_attn_e2m1, abort_flag, limit_ns);
}
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival on `bar` of both CTAs when every MMA issued so far by this thread is complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
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

// Writes block `blk` (16 dims) of row r into the atoms at `region`: chunks 2 blk and
// 2 blk + 1 of 16 bytes, at their swizzled places.  Lanes of odd atoms write their
// second chunk first: eight lanes then cover all banks.
__device__ __forceinline__ void store_block(uint32_t region, int r, int blk, const uint32_t (&o)[8]) {
  const uint32_t base = region + static_cast<uint32_t>((blk >> 2) * kAtom + r * 128);
  const int c = (blk & 3) * 2, flip = (blk >> 2) & 1;
  const uint32_t a0 = base + static_cast<uint32_t>(((c + flip) ^ (r & 7)) << 4);
  const uint32_t a1 = base + static_cast<uint32_t>(((c + 1 - flip) ^ (r & 7)) << 4);
  st_shared_v4(a0, flip ? o[4] : o[0], flip ? o[5] : o[1], flip ? o[6] : o[2], flip ? o[7] : o[3]);
  st_shared_v4(a1, flip ? o[0] : o[4], flip ? o[1] : o[5], flip ? o[2] : o[6], flip ? o[3] : o[7]);
}

__global__ void __launch_bounds__(kThreads, 1) attn_e2m1_kernel(PairParams p) {
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
  uint64_t* full = bars;          // [2] leader: own rows of both CTAs in the stage
  uint64_t* vfull = bars + 2;     // [2] leader: the other CTA's rows in the stage, both CTAs
  uint64_t* pfull = bars + 4;     // [2] leader: P written, both CTAs
  uint64_t* sfree = bars + 6;     // [2] leader: logits read, both CTAs
  uint64_t* sfull = bars + 8;     // [2] Q K^T complete
  uint64_t* empty = bars + 10;    // [2] P V complete
  uint64_t* mfull = bars + 12;    // [2] row masks of the stage written
  uint64_t* drain = bars + 14;    // every MMA complete (teardown)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const uint64_t wlim = p.wait_limit_ns;

  int item = blockIdx.x >> 1;
  const int split = item % p.n_split;
  item /= p.n_split;
  const int hb = item % p.head_blocks;
  const int t = p.seq.T - 1 - item / p.head_blocks;   // last query first (longest causal history)
  const int K = p.a.K, H = p.a.H;
  const int r0 = split * p.rows_per_split;
  const int r1 = min(K, r0 + p.rows_per_split);
  const int ntiles = (r1 - r0 + kTile - 1) / kTile;
  const int h0 = hb * 128 + static_cast<int>(rank) * kHeads;   // this CTA's first head

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 2 * kProducers);
      mbar_init(&vfull[i], 2 * kProducers);
      mbar_init(&pfull[i], 16);
      mbar_init(&sfree[i], 16);
      mbar_init(&sfull[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&mfull[i], kProducers);
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpQk) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(misc)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the leader's barriers and both CTAs' TMEM exist before anyone arrives or multiplies
  tc_fence_after();
  const uint32_t tmem = misc[0];

  if (!p.early_query) grid_dep_wait();
  int qp = __ldg(p.seq.q_pos + t);
  int b = __ldg(p.seq.q_seq + t);
  if (qp < 0 || qp >= p.seq.max_ctx || b < 0 || b >= p.seq.B) {
    if (threadIdx.x == 0) atomicOr(&g_status_attn_e2m1, kDevBadPos);
    qp = -1;
    b = 0;
  }
  const uint8_t* kv = static_cast<const uint8_t*>(p.a.kv);
  const int64_t row_bytes = p.a.row_bytes;
  const int32_t* bt = p.seq.block_table + static_cast<int64_t>(b) * p.seq.bt_stride;
  const int32_t* idx = p.a.idx + static_cast<int64_t>(t) * K;
  // A selected entry's way to its row, a tile's worth of time between the steps: the
  // position (load_pos), its page id (load_page), the cache row or -1 (row_of).
  const int page_size = p.seq.page_size;
  auto load_page = [&](int pos) -> int {
    if (pos > qp) atomicOr(&g_status_attn_e2m1, kDevBadIndex);
    return (pos >= 0 && pos <= qp) ? __ldg(bt + pos / page_size) : -1;
  };
  auto row_of = [&](int pos, int page) -> int {
    if (pos < 0 || pos > qp) return -1;
    if (page < 0 || page >= p.seq.n_pages) {
      atomicOr(&g_status_attn_e2m1, kDevBadIndex);
      return -1;
    }
    return page * page_size + pos % page_size;   // < cache_rows < 2^31
  };

  // The query: warps 0-15 four heads each, eight lanes a head, lane c of them chunk c of
  // every atom.  The latent part becomes f16 with its own power of two per head.
  if (warp < kHeads / 4) {
    const int hl = warp * 4 + (lane >> 3), c = lane & 7;
    const bool have = h0 + hl < H;
    const uint4* qg = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.a.q) +
                                                     (static_cast<int64_t>(t) * H + h0 + hl) * kDqk) + c;
    uint4 v[9];
#pragma unroll
    for (int a = 0; a < 9; ++a) v[a] = have ? __ldg(qg + 8 * a) : make_uint4(0u, 0u, 0u, 0u);
    __nv_bfloat162 mx = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = __hmax2(mx, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    }
    float amax = fmaxf(__low2float(mx), __high2float(mx));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = amax > 0.f ? max(-110, min(113, ilogbf(amax) - 14)) : 0;
    // the maximum is taken over unscaled logits: a negative scale turns the query round
    const bool negate = p.a.softmax_scale < 0.f;
    const float f = ldexpf(negate ? -1.f : 1.f, -e);
    const uint32_t flip = negate ? 0x80008000u : 0u;
    if (c == 0) reinterpret_cast<float*>(sm + kOffQexp)[hl] = ldexpf(1.f, e);
    const uint32_t dst = smem_u32(sm + kOffQ) + static_cast<uint32_t>(hl * 128 + ((c ^ (hl & 7)) << 4));
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 q2 = __floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
        o[i] = *reinterpret_cast<const uint32_t*>(&q2);
      }
      st_shared_v4(dst + static_cast<uint32_t>(a * kAtom), o[0], o[1], o[2], o[3]);
    }
    st_shared_v4(dst + static_cast<uint32_t>(8 * kAtom), v[8].x ^ flip, v[8].y ^ flip, v[8].z ^ flip, v[8].w ^ flip);
    fence_proxy_async_smem();
  }
  __syncthreads();
  // both CTAs' queries must be there before the leader multiplies: the softmax warps'
  // first arrivals on sfree say so
  if (warp >= kWarpSoft && lane == 0) {
    arrive_pair(leader_addr(&sfree[0]));
    arrive_pair(leader_addr(&sfree[1]));
  }

  if (warp < kProducers) {
    // ------------------------------------------------ producers
    if (p.early_query) grid_dep_wait();   // the selected indices come from the kernel before
    // lanes 0-7 look after own rows [8 w, 8 w + 8) of the tile, lanes 8-15 after the other CTA's
    const int tile_row = (static_cast<int>(rank ^ static_cast<uint32_t>(lane >> 3)) & 1) * kOwn + warp * 8 + (lane & 7);
    const int sub = lane >> 4, blk = lane & 15;
    const uint32_t region = rank == 0 ? 4 * kAtom : 0;   // of the other CTA's rows: Y in rank 0, X in rank 1
    auto load_pos = [&](int j) -> int {
      const int gi = r0 + j * kTile + tile_row;
      return (lane < 16 && j < ntiles && gi < r1) ? __ldg(idx + gi) : -1;
    };
    // Own rows: codes of block `lane`; scale bytes as words, word lane & 7 of rows lane / 8
    // and lane / 8 + 4; rope chunk lane & 7 of the same rows.  Other rows: codes of block blk
    // (of this CTA's value dims) of rows 2 k + sub; scale word lane & 3 of row lane / 4.  A
    // row that selects nothing reads row 0, with scales and rope values of zero.
    uint2 code[8], pcode[4];
    uint32_t sc[2], psc = 0u;
    uint4 rope[2];
    float rs = 0.f;
    uint32_t valid = 0u;   // of tile `my_row`: bits 0-7 own, 8-15 other
    auto fetch_own = [&](int my_row) {
      valid = __ballot_sync(0xffffffffu, my_row >= 0);
      const int safe = max(my_row, 0);
      int row[8], row2[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = __shfl_sync(0xffffffffu, safe, i);
#pragma unroll
      for (int k = 0; k < 2; ++k) row2[k] = __shfl_sync(0xffffffffu, safe, (lane >> 3) + 4 * k);
#pragma unroll
      for (int i = 0; i < 8; ++i) code[i] = __ldg(reinterpret_cast<const uint2*>(kv + row[i] * row_bytes) + lane);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint8_t* rp = kv + row2[k] * row_bytes;
        sc[k] = __ldg(reinterpret_cast<const uint32_t*>(rp + kE2m1Scales) + (lane & 7));
        rope[k] = __ldg(reinterpret_cast<const uint4*>(rp + kE2m1Rope) + (lane & 7));
      }
      rs = __ldg(reinterpret_cast<const float*>(kv + safe * row_bytes + kE2m1RowScale));
    };
    uint32_t pvalid = 0u;
    auto fetch_other = [&](int my_row) {
      pvalid = __ballot_sync(0xffffffffu, my_row >= 0) >> 8;
      const int safe = max(my_row, 0);
      int row[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) row[k] = __shfl_sync(0xffffffffu, safe, 8 + 2 * k + sub);
      const int row1 = __shfl_sync(0xffffffffu, safe, 8 + (lane >> 2));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        pcode[k] = __ldg(reinterpret_cast<const uint2*>(kv + row[k] * row_bytes) + rank * 16 + blk);
      psc = __ldg(reinterpret_cast<const uint32_t*>(kv + row1 * row_bytes + kE2m1Scales) + rank * 4 + (lane & 3));
    };
    // Own rows into the stage, and the row scales and masks of all sixteen rows beside it.
    auto write_own = [&](int j) {
      const int st = j & 1;
      const uint32_t stage = smem_u32(sm + kOffStage + st * kStageBytes);
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) sc[k] = ((valid >> ((lane >> 3) + 4 * k)) & 1u) ? sc[k] : 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __shfl_sync(0xffffffffu, sc[i >> 2], (i & 3) * 8 + (lane >> 2));
      const float my_rs = ((valid >> lane) & 1u) ? rs : 0.f;
      if (lane < 16) reinterpret_cast<float*>(sm + kOffScale)[st * kTile + tile_row] = my_rs;
      float rmax = lane < 16 ? my_rs : 0.f;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, o));
      if (lane == 0) {
        reinterpret_cast<float*>(sm + kOffRmax)[st * 8 + warp] = rmax;
        (sm + kOffMask + st * 16 + rank * 8)[warp] = static_cast<uint8_t>(valid);
        (sm + kOffMask + st * 16 + (rank ^ 1u) * 8)[warp] = static_cast<uint8_t>(valid >> 8);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t o[8];
        widen_codes(code[i], w[i] >> (8 * (lane & 3)), o);
        store_block(stage, warp * 8 + i, lane, o);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = warp * 8 + (lane >> 3) + 4 * k;
        const uint32_t keep = ((valid >> ((lane >> 3) + 4 * k)) & 1u) ? 0xFFFFFFFFu : 0u;
        st_shared_v4(stage + static_cast<uint32_t>(kRopeAtom + r * 128 + (((lane & 7) ^ (r & 7)) << 4)), rope[k].x & keep,
                     rope[k].y & keep, rope[k].z & keep, rope[k].w & keep);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&mfull[st]);
        if (!(p.dbg_withhold && warp == 0 && j == 0)) arrive_pair(leader_addr(&full[st]));
      }
    };
    auto write_other = [&](int j) {
      const int st = j & 1;
      const uint32_t dst = smem_u32(sm + kOffStage + st * kStageBytes) + region;
      psc = ((pvalid >> (lane >> 2)) & 1u) ? psc : 0u;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __shfl_sync(0xffffffffu, psc, (2 * k + sub) * 4 + (blk >> 2));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t o[8];
        widen_codes(pcode[k], w[k] >> (8 * (blk & 3)), o);
        store_block(dst, warp * 8 + 2 * k + sub, blk, o);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_pair(leader_addr(&vfull[st]));
    };
    // Steps -1, 0, 1, ...: at step j the other CTA's rows of tile j, then the own rows of
    // tile j + 1; own registers hold tile j + 1 and take tile j + 2, the other rows' hold
    // tile j and take tile j + 1.  row1 / row2: rows of tiles j + 1 and j + 2.
    int row1 = -1, row2;
    int pos3, page3;
    {
      const int pos0 = load_pos(0), pos1 = load_pos(1);
      pos3 = load_pos(2);
      const int page0 = load_page(pos0), page1 = load_page(pos1);
      page3 = load_page(pos3);
      row1 = row_of(pos0, page0);
      row2 = row_of(pos1, page1);
    }
    fetch_own(row1);
    int pos4 = load_pos(3);
#pragma unroll 1
    for (int j = -1; j < ntiles; ++j) {
      if (j >= 0) {
        // Q K^T has read the rows that these replace
        const bool ok = wait_bar(&sfull[j & 1], (j >> 1) & 1, abort_flag, wlim);
        if (!__all_sync(0xffffffffu, ok)) break;
        write_other(j);
      }
      if (j + 1 < ntiles) {
        fetch_other(row1);
        if (j >= 1) {
          const bool ok = wait_bar(&empty[(j + 1) & 1], ((j - 1) >> 1) & 1, abort_flag, wlim);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        write_own(j + 1);
        fetch_own(row2);
      }
      row1 = row2;
      row2 = row_of(pos3, page3);
      pos3 = pos4;
      page3 = load_page(pos3);
      pos4 = load_pos(j + 5);
    }
  } else if (warp == kWarpQk) {
    if (rank == 0) {
      const uint64_t dq = make_sdesc(smem_u32(sm + kOffQ), 16, 1024, kLayoutSw128);
      const uint64_t dk0 = make_sdesc(smem_u32(sm + kOffStage), 16, 1024, kLayoutSw128);
      for (int j = 0; j < ntiles; ++j) {
        const int st = j & 1;
        // the logit buffer is free (the first phase: the queries are staged) and the tile has landed
        if (!__all_sync(0xffffffffu, wait_bar(&sfree[st], (j >> 1) & 1, abort_flag, wlim))) break;
        if (!__all_sync(0xffffffffu, wait_bar(&full[st], (j >> 1) & 1, abort_flag, wlim))) break;
        tc_fence_after();
        fence_proxy_async_smem();
        if (elect_one()) {
          const uint64_t dk = dk0 + static_cast<uint64_t>((st * kStageBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < kDqk / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4);
            if (kk < kDv / 16)
              umma_pair(tmem + st * 64, dq + off, dk + off, kIdescLatent, kk > 0 ? 1u : 0u);
            else
              umma_pair(tmem + kColRope + st * 64, dq + off, dk + off, kIdescRope, kk > kDv / 16 ? 1u : 0u);
          }
          commit_pair(&sfull[st]);
        }
        __syncwarp();
      }
    }
  } else if (warp == kWarpPv) {
    if (rank == 0) {
      const uint64_t dv0 = make_sdesc(smem_u32(sm + kOffStage), kAtom, 1024, kLayoutSw128);
      const uint64_t dp0 = make_sdesc(smem_u32(sm + kOffStage + kRopeAtom), 16, 1024, kLayoutSw128);
      const uint64_t dp1 = make_sdesc(smem_u32(sm + kOffP1), 16, 1024, kLayoutSw128);
      for (int j = 0; j < ntiles; ++j) {
        const int st = j & 1;
        if (!__all_sync(0xffffffffu, wait_bar(&vfull[st], (j >> 1) & 1, abort_flag, wlim))) break;
        if (!__all_sync(0xffffffffu, wait_bar(&pfull[st], (j >> 1) & 1, abort_flag, wlim))) break;
        tc_fence_after();
        fence_proxy_async_smem();
        if (elect_one()) {
          const uint64_t so = static_cast<uint64_t>((st * kStageBytes) >> 4);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              const uint64_t da = (kk < 4 ? dp0 + so : dp1) + static_cast<uint64_t>(((kk & 3) * 32) >> 4);
              // rows 16 kk ..: X holds tile rows 0-63, Y rows 64-127; value atoms 2 q, 2 q + 1
              const uint64_t db = dv0 + so + static_cast<uint64_t>(((kk >> 2) * 4 * kAtom + q * 2 * kAtom + (kk & 3) * 2048) >> 4);
              umma_pair(tmem + kColO + q * 128, da, db, kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
            }
          }
          commit_pair(&empty[st]);
        }
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------ softmax and epilogue
    const int quarter = warp & 3;
    const int hl = (quarter & 1) * 32 + lane;   // head within the CTA
    const int half = quarter >> 1;              // tile rows [64 half, 64 half + 64), of which
    const int part32 = (warp - kWarpSoft) >> 2; // this thread's [32 part32, 32 part32 + 32)
    const int rq = half * 2 + part32;           // row quarter of the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // a scale of 0 becomes a tiny one, so that it leaves a masked logit at -inf
    const float sl2 = fmaxf(fabsf(p.a.softmax_scale) * kLog2e, 1e-30f);
    const uint32_t head_bar = 2 + (quarter & 1), read_bar = 4 + (quarter & 1);   // the 128 threads of 32 heads
    float* xmax = reinterpret_cast<float*>(sm + kOffMax);
    volatile int* oks = reinterpret_cast<volatile int*>(sm + kOffOk);
    const volatile uint32_t* masks = reinterpret_cast<const volatile uint32_t*>(sm + kOffMask);
    const uint32_t sfree_leader0 = leader_addr(&sfree[0]), sfree_leader1 = leader_addr(&sfree[1]);
    const uint32_t pfull_leader0 = leader_addr(&pfull[0]), pfull_leader1 = leader_addr(&pfull[1]);
    const float qexp = reinterpret_cast<const float*>(sm + kOffQexp)[hl];
    float m = -INFINITY, g = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      const int st = j & 1;
      ok = wait_bar(&mfull[st], (j >> 1) & 1, abort_flag, wlim) &&
           wait_bar(&sfull[st], (j >> 1) & 1, abort_flag, wlim);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t scales = smem_u32(sm + kOffScale) + static_cast<uint32_t>((st * kTile + rq * 32) * 4);
      float x[32];
      float mx = -INFINITY, rmax = 0.f;
      if (ok) {
        uint32_t s0[32], s1[32];
        tmem_ld32(tmem + lane_off + st * 64 + part32 * 32, s0);
        tmem_ld32(tmem + lane_off + kColRope + st * 64 + part32 * 32, s1);
        const uint32_t vmask = masks[st * 4 + rq];
        const float* rmaxs = reinterpret_cast<const float*>(sm + kOffRmax) + st * 8;
#pragma unroll
        for (int i = 0; i < kProducers; ++i) rmax = fmaxf(rmax, rmaxs[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const uint4 rs = ld_shared_v4(scales + static_cast<uint32_t>(i * 4));
          float t0, t1, t2, t3;
          mul2(t0, t1, __uint_as_float(s0[i]), __uint_as_float(s0[i + 1]), qexp, qexp);
          mul2(t2, t3, __uint_as_float(s0[i + 2]), __uint_as_float(s0[i + 3]), qexp, qexp);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[i + k] = __uint_as_float(s1[i + k]);
          fma2(x[i], x[i + 1], t0, t1, __uint_as_float(rs.x), __uint_as_float(rs.y));
          fma2(x[i + 2], x[i + 3], t2, t3, __uint_as_float(rs.z), __uint_as_float(rs.w));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(st ? sfree_leader1 : sfree_leader0);
        if (vmask != ~0u) {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = ((vmask >> i) & 1u) ? x[i] : -INFINITY;
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; i += 2) mq[(i >> 1) & 3] = fmax3(mq[(i >> 1) & 3], x[i], x[i + 1]);
        mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sl2;
      }
      // The four threads of a head take the largest maximum, and their warps leave together
      // when one has given up.  There is room for one buffer: the last tile's entries have
      // been read once all four warps have arrived on read_bar.
      if (j >= 1) named_bar_sync(read_bar, 256);
      xmax[rq * kHeads + hl] = mx;
      if (lane == 0) oks[st * 8 + warp - kWarpSoft] = ok ? 1 : 0;
      named_bar_sync(head_bar, 128);
#pragma unroll
      for (int k = 1; k < 4; ++k) mx = fmaxf(mx, xmax[(rq ^ k) * kHeads + hl]);
      // the four warps: quarters with this one's low bit, both row halves of each
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (((k + kWarpSoft) & 1) == (quarter & 1)) ok = ok && oks[st * 8 + k] != 0;
      named_bar_arrive(read_bar, 256);
      if (!ok) break;
      const float gx = mx + __log2f(rmax);
      const bool need_m = mx > m + kRescaleM, need_g = gx > g + kRescaleG;
      if (j >= 1 && __any_sync(0xffffffffu, need_g)) {
        // O is rescaled: P V of the tile before must have written it
        ok = wait_bar(&empty[st ^ 1], ((j - 1) >> 1) & 1, abort_flag, wlim);
        tc_fence_after();
        const float f = need_g ? exp2f(g - gx) : 1.f;
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {   // this thread's half of the columns
          uint32_t o[16];
          tmem_ld16(tmem + lane_off + kColO + part32 * 128 + cc * 16, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st16(tmem + lane_off + kColO + part32 * 128 + cc * 16, o);
        }
        tmem_st_wait();
      }
      if (need_g) g = gx;
      if (need_m) {
        l *= exp2f(m - mx);
        m = mx;
      }
      const float msub = (m == -INFINITY) ? 0.f : m;
      // 2^(m - g), kept finite and nonzero
      const float gain = (g == -INFINITY) ? 1.f : exp2f(fminf(fmaxf(msub - g, -126.f), 126.f));
      // P of tile rows 64-127 has one buffer: P V of the tile before must have read it
      if (half == 1 && j >= 1) ok = ok && wait_bar(&empty[st ^ 1], ((j - 1) >> 1) & 1, abort_flag, wlim);
      const uint32_t prow = smem_u32(half == 0 ? sm + kOffStage + st * kStageBytes + kRopeAtom : sm + kOffP1) +
                            static_cast<uint32_t>(hl * 128);
      float se[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = 8 * c + 4 * q;
          const uint4 rs = ld_shared_v4(scales + static_cast<uint32_t>(i * 4));
          const float r[4] = {__uint_as_float(rs.x), __uint_as_float(rs.y), __uint_as_float(rs.z), __uint_as_float(rs.w)};
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
      if (lane == 0) arrive_pair(st ? pfull_leader1 : pfull_leader0);
    }
    const int last = ntiles - 1;
    if (ok) ok = wait_bar(&empty[last & 1], (last >> 1) & 1, abort_flag, wlim);
    ok = __all_sync(0xffffffffu, ok);
    // the sums of a head's four threads
    named_bar_sync(head_bar, 128);
    xmax[rq * kHeads + hl] = l;
    named_bar_sync(head_bar, 128);
#pragma unroll
    for (int k = 1; k < 4; ++k) l += xmax[(rq ^ k) * kHeads + hl];
    if (ok) {
      tc_fence_after();
      // O holds sum p rs 2^(m - g) v over l = sum p
      const float inv = l > 0.f ? exp2f(fminf(fmaxf(g - m, -126.f), 126.f)) / l : 0.f;
      const float lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      const int heads = min(32, H - (h0 + (quarter & 1) * 32));   // of this warp's 32 that exist
      const bool part = p.n_split > 1;
      const int64_t head0 = (static_cast<int64_t>(part ? split : 0) * p.seq.T + t) * H + h0 + (quarter & 1) * 32;
      uint8_t* out = reinterpret_cast<uint8_t*>(part ? p.ws_o : static_cast<uint16_t*>(p.a.out)) +
                     (head0 * kDv + half * 256 + part32 * 128) * 2;
      const uint32_t stg = smem_u32(sm + kOffStage) + (warp - kWarpSoft) * 4096;   // all MMAs are complete
      if (heads > 0) {
#pragma unroll 1
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t o0[32], o1[32];
          tmem_ld32(tmem + lane_off + kColO + part32 * 128 + cc * 64, o0);
          tmem_ld32(tmem + lane_off + kColO + part32 * 128 + cc * 64 + 32, o1);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            st_shared_v4(stg + lane * 128 + ((k ^ (lane & 7)) << 4),
                         pack_bf16x2(__uint_as_float(o0[8 * k]) * inv, __uint_as_float(o0[8 * k + 1]) * inv),
                         pack_bf16x2(__uint_as_float(o0[8 * k + 2]) * inv, __uint_as_float(o0[8 * k + 3]) * inv),
                         pack_bf16x2(__uint_as_float(o0[8 * k + 4]) * inv, __uint_as_float(o0[8 * k + 5]) * inv),
                         pack_bf16x2(__uint_as_float(o0[8 * k + 6]) * inv, __uint_as_float(o0[8 * k + 7]) * inv));
            st_shared_v4(stg + lane * 128 + (((k + 4) ^ (lane & 7)) << 4),
                         pack_bf16x2(__uint_as_float(o1[8 * k]) * inv, __uint_as_float(o1[8 * k + 1]) * inv),
                         pack_bf16x2(__uint_as_float(o1[8 * k + 2]) * inv, __uint_as_float(o1[8 * k + 3]) * inv),
                         pack_bf16x2(__uint_as_float(o1[8 * k + 4]) * inv, __uint_as_float(o1[8 * k + 5]) * inv),
                         pack_bf16x2(__uint_as_float(o1[8 * k + 6]) * inv, __uint_as_float(o1[8 * k + 7]) * inv));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3), c4 = lane & 7;
            const uint4 v = ld_shared_v4(stg + row * 128 + ((c4 ^ (row & 7)) << 4));
            if (row < heads) *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * kDv * 2 + cc * 128 + c4 * 16) = v;
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
  }

  // Every MMA has finished in both CTAs before either releases its TMEM or leaves (after
  // an abort some may still be running).
  if (rank == 0 && (warp == kWarpQk || warp == kWarpPv)) {
    if (elect_one()) commit_pair(drain);
    __syncwarp();
  }
  if (warp == kWarpQk) mbar_drain(drain, 0, &g_status_attn_e2m1, wlim);
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == kWarpQk) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Row slices per query: one cluster for each while the GPU holds them all at once, a
// slice at least one tile.
int choose_split(const SeqArgs& seq, const MlaArgs& a, int num_sms) {
  const int tiles = (a.K + kTile - 1) / kTile;
  const int64_t clusters = static_cast<int64_t>(seq.T) * ((a.H + 127) / 128);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tiles, (num_sms / 2) / std::max<int64_t>(1, clusters))));
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
  PairParams p{seq, a, split, rps, (a.H + 127) / 128, nullptr, nullptr, kWaitLimitNs, 0u, env.chained ? 1u : 0u};
  debug_wait_state(&p.wait_limit_ns, &p.dbg_withhold);
  if (split > 1) {
    const size_t o = static_cast<size_t>(split) * seq.T * a.H * kDv * sizeof(uint16_t);
    p.ws_o = static_cast<uint16_t*>(workspace);
    p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((o + 255) / 256) * 256);
  }
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(attn_e2m1_kernel), kSmemBytes, env.device);
  if (e != cudaSuccess) return e;
  const int64_t grid = 2ll * seq.T * p.head_blocks * split;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  e = launch_kernel(attn_e2m1_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, env.stream, true, 2, p);
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
