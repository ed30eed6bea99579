// Per-query choice of blocks (pages) by the best index score in each.
//
// For query t at position p the candidates are the blocks 0 .. p / page_size; a block's key is
// the largest of the scores of its positions up to p, and the N best are taken, the first and
// the last few always, ties to the lower block, written in ascending order, -1 behind them.
// The indexer ("Large Language Model Inference Acceleration in Practice", section 1.2) is the
// cheap score; a page is the block because its cache rows lie together.
//
// What bounds it: four bytes a score, read once; for few queries the latencies of one load and
// of the choice among a few hundred keys.  A query is one CTA, or a cluster of them that read
// a part of its scores each and write their blocks' keys into the first one's shared memory.
//
// Scores to keys (pages of 64): a warp takes 16 blocks, eight 16-byte loads a lane, two blocks
// a load; the maxima of 16 lanes are then exchanged so that each lane goes on with half of
// its values: eight shuffles for 16 blocks instead of 64.
//
// The choice, among the blocks that are not taken in any case: a histogram of eight bits of key
// minus smallest key, from the highest bit that their range has on (scores of one query share
// their first bits, and atomics on few bins would wait for one another), says which bin holds the
// last key to take; the bin's keys are looked at again by their next eight bits until all of them
// are taken or one key is left.  Of keys equal to it the first ones are taken.
#include <algorithm>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "topk_select.cuh"

DSA_DEFINE_STATUS_WORD(block_topk)

namespace dsa {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxBlocks = 32768;   // keys of a query in shared memory
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;          // of a histogram: eight bits

struct BlockTopkArgs {
  const float* scores;
  int64_t ld;
  const int32_t* q_pos;
  int32_t T, max_ctx, page_size, N, n_first, n_last;
  int32_t* out;
};

template <bool kPage64>
__global__ void __launch_bounds__(kMaxThreads, 2) block_topk_kernel(BlockTopkArgs a) {
  grid_dep_wait();
  grid_dep_launch();   // the kernel after waits for this grid before it reads the blocks
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t bins[4][kBins];
  __shared__ uint32_t red[2][32];
  __shared__ uint32_t pick[2][3];   // of a pass: digit, keys above its bin, keys in it
  const int CL = static_cast<int>(cl_size()), rank = static_cast<int>(cl_rank());
  const int t = a.T - 1 - static_cast<int>(blockIdx.x) / CL;   // longest causal histories first
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  int qp = __ldg(a.q_pos + t);
  if (qp < 0 || qp >= a.max_ctx) {
    if (tid == 0 && rank == 0) atomicOr(&g_status_block_topk, kDevBadPos);
    qp = -1;   // no block: all -1
  }
  const int n_tok = qp + 1, N = a.N;
  const int n = kPage64 ? (n_tok + 63) >> 6 : (n_tok > 0 ? qp / a.page_size + 1 : 0);
  int32_t* out = a.out + static_cast<int64_t>(t) * N;
  if (n <= N) {   // cluster-uniform
    for (int i = rank * nt + tid; i < N; i += CL * nt) out[i] = i < n ? i : -1;
    return;
  }
  // ---- this CTA's blocks [lo, hi) to keys in the first CTA
  const float* row = a.scores + static_cast<int64_t>(t) * a.ld;
  const uint32_t dst = CL > 1 ? cl_map(smem_u32(keys), 0) : 0u;
  for (int i = tid; i < 4 * kBins; i += nt) (&bins[0][0])[i] = 0u;
  auto put = [&](int blk, float best) {
    const uint32_t k = order_key(fmaxf(best, -INFINITY));   // (a NaN only where there is nothing else)
    if (CL > 1)
      cl_store(dst + static_cast<uint32_t>(blk) * 4u, k);
    else
      keys[blk] = k;
  };
  if (CL > 1) {   // every CTA of the cluster runs before one writes into another
    cl_arrive();
    cl_wait();
  }
  const int slice = ((n + CL - 1) / CL + 15) & ~15;
  const int lo = min(n, rank * slice), hi = min(n, lo + slice);
  if constexpr (kPage64) {
    for (int b0 = lo + warp * 16; b0 < hi; b0 += (nt >> 5) * 16) {
      float v[8];
      const int pos0 = b0 * 64 + (lane >> 4) * 64 + (lane & 15) * 4;
      float4 f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pos = pos0 + i * 128;
        f[i] = pos < n_tok ? __ldg(reinterpret_cast<const float4*>(row + pos))
                           : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int left = n_tok - (pos0 + i * 128);   // of these four, behind the query's position: not scores
        if (left < 4) {
          if (left < 2) f[i].y = -INFINITY;
          if (left < 3) f[i].z = -INFINITY;
          f[i].w = -INFINITY;
        }
        v[i] = fmaxf(fmaxf(f[i].x, f[i].y), fmaxf(f[i].z, f[i].w));
      }
#pragma unroll
      for (int o = 8, half = 4; o >= 2; o >>= 1, half >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
          v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
      }
      v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
      const int blk = b0 + 2 * (((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1)) + (lane >> 4);
      if (!(lane & 1) && blk < hi) put(blk, v[0]);
    }
  } else {
    for (int blk = lo + warp; blk < hi; blk += nt >> 5) {
      float best = -INFINITY;
      const int start = blk * a.page_size;
      // what is left is counted, not positions: the one a step behind the last may pass 2^31
      const float* at = row + start + lane;
#pragma unroll 4
      for (int left = (blk == n - 1 ? n_tok - start : a.page_size) - lane; left > 0; left -= 32, at += 32) best = fmaxf(best, __ldg(at));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      if (lane == 0) put(blk, best);
    }
  }
  if (CL > 1) {
    cl_arrive();
    cl_wait();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the last key to take: T, an offset from the smallest key
  auto forced = [&](int i) -> bool { return i < a.n_first || i >= n - a.n_last; };   // n > N: no block twice
  uint32_t rem = static_cast<uint32_t>(N - a.n_first - a.n_last);   // of the others
  const bool some = rem > 0;
  uint32_t base = 0u, T = 0u;
  bool exact = false;   // all keys from T on are taken; else those above, and `rem` equal ones
  if (some) {
    uint32_t lo_key = 0xFFFFFFFFu, hi_key = 0u;
    for (int i = tid; i < n; i += nt) {
      if (forced(i)) continue;
      lo_key = min(lo_key, keys[i]);
      hi_key = max(hi_key, keys[i]);
    }
    lo_key = __reduce_min_sync(0xffffffffu, lo_key);
    hi_key = __reduce_max_sync(0xffffffffu, hi_key);
    if (lane == 0) red[0][warp] = lo_key, red[1][warp] = hi_key;
    __syncthreads();
    const bool has = lane < (nt >> 5);
    base = __reduce_min_sync(0xffffffffu, has ? red[0][lane] : 0xFFFFFFFFu);
    const uint32_t range = __reduce_max_sync(0xffffffffu, has ? red[1][lane] : 0u) - base;
    int shift = 32 - __clz(static_cast<int>(range));   // bits that are not settled
    for (int pass = 0; shift > 0 && !exact; ++pass) {
      const int above = shift, bits = min(8, shift);
      shift -= bits;
      for (int i = tid; i < n; i += nt) {
        const uint32_t d = keys[i] - base;
        if (!forced(i) && (pass == 0 || (d >> above) == (T >> above))) atomicAdd(&bins[pass][(d >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      if (warp == 0) {   // lane l: bins 255 - 8 l and the seven below
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += c[k] = bins[pass][kBins - 1 - (8 * lane + k)];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += u;
        }
        uint32_t before = incl - sum;
        if (before < rem && incl >= rem) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (before < rem && before + c[k] >= rem) {
              pick[pass & 1][0] = static_cast<uint32_t>(kBins - 1 - (8 * lane + k));
              pick[pass & 1][1] = before;
              pick[pass & 1][2] = c[k];
              before = rem;   // found
            } else {
              before += c[k];
            }
          }
        }
      }
      __syncthreads();
      T |= pick[pass & 1][0] << shift;
      rem -= pick[pass & 1][1];
      exact = pick[pass & 1][2] == rem;
    }
  }
  // ---- what is taken, in ascending order
  const int equal_most = static_cast<int>(rem);
  int o = 0, equals = 0;   // written, equal ones met, in the chunks before
  for (int i0 = 0; i0 < n; i0 += nt) {
    const int i = i0 + tid;
    bool take = i < n && forced(i), same = false;
    if (i < n && some && !take) {
      const uint32_t d = keys[i] - base;
      take = d > T || (exact && d == T);
      same = !exact && d == T;
    }
    const uint32_t gt = __ballot_sync(0xffffffffu, take), eq = __ballot_sync(0xffffffffu, same);
    __syncthreads();
    if (lane == 0) red[0][warp] = static_cast<uint32_t>(__popc(gt) | (__popc(eq) << 16));
    __syncthreads();
    const uint32_t v = lane < (nt >> 5) ? red[0][lane] : 0u;
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u), all = __reduce_add_sync(0xffffffffu, v);
    const uint32_t lt = (1u << lane) - 1u;
    const int eq_before = equals + static_cast<int>(before >> 16) + __popc(eq & lt);
    const int gt_before = static_cast<int>(before & 0xFFFFu) + __popc(gt & lt);
    // of the equal ones before this key in the chunk, those that are taken
    const int eq_taken = min(eq_before, equal_most) - min(equals, equal_most);
    if (take || (same && eq_before < equal_most)) out[o + gt_before + eq_taken] = i;
    const int eq_all = equals + static_cast<int>(all >> 16);
    o += static_cast<int>(all & 0xFFFFu) + min(eq_all, equal_most) - min(equals, equal_most);
    equals = eq_all;
  }
}

}  // namespace

cudaError_t launch_block_topk(const SeqArgs& seq, const float* scores, int64_t ld, int32_t N, int32_t n_first,
                              int32_t n_last, int32_t* out, const LaunchEnv& env, std::string* plan, bool* unsupported,
                              std::string* why) {
  *unsupported = false;
  const int64_t blocks = (static_cast<int64_t>(seq.max_ctx) + seq.page_size - 1) / seq.page_size;
  if (blocks > kMaxBlocks) {
    *unsupported = true;
    *why = "block top-k: more than 32768 blocks of max_ctx";
    return cudaSuccess;
  }
  if (seq.T == 0) {
    *plan += "block_topk[empty]";
    return cudaSuccess;
  }
  const bool page64 = seq.page_size == 64;
  void (*kernel)(BlockTopkArgs) = page64 ? block_topk_kernel<true> : block_topk_kernel<false>;
  const cudaError_t ae = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kMaxBlocks * 4, env.device);
  if (ae != cudaSuccess) return ae;
  // Few queries: as many CTAs a query as the GPU holds at once, 128 blocks each at least.  One query of 32768
  // scores takes 4.5 us (4.9 with one CTA), one of 131072 6.4 (12.3 with two CTAs).
  const int want = std::max(1, env.num_sms / seq.T), feed = static_cast<int>(std::max<int64_t>(1, blocks / 128));
  const int cl = std::max(1, std::min(kMaxCluster, std::min(want, feed)));
  // Many queries: small CTAs, whose loads and choices overlap on an SM.  4096 queries of 16384 scores take
  // 46.4 us with 64 threads, 48.3 with 128, 51.9 with 256, 72 with 512; 2048 of 4096 8.2, 9.4, 15.3 and
  // 27.9; 1024 of 65536 60.2, 47.0, 48.9 and 54.2.
  const int threads = static_cast<int64_t>(seq.T) * cl > 2 * env.num_sms ? (blocks > 512 ? 128 : 64) : kMaxThreads;
  const BlockTopkArgs a{scores, ld, seq.q_pos, seq.T, seq.max_ctx, seq.page_size, N, n_first, n_last, out};
  const cudaError_t e = launch_kernel(kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(seq.T) * cl)), dim3(threads),
                                      static_cast<size_t>(blocks) * 4, env.stream, true, cl, a);
  char buf[96];
  snprintf(buf, sizeof(buf), "block_topk[cluster=%d,threads=%d]", cl, threads);
  *plan += buf;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
