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
// The choice: the largest key bits that N keys reach, bit by bit from the top, with a count over
// the CTA for each (one barrier that counts, where a thread holds one key); it ends early when
// exactly N keys do.  Keys above are taken, of those equal to it the first ones.
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

struct BlockTopkArgs {
  const float* scores;
  int64_t ld;
  const int32_t* q_pos;
  int32_t T, max_ctx, page_size, N, n_first, n_last;
  int32_t* out;
};

// A block's key: above all others where it is taken in any case; -inf for scores of nothing but
// NaN (the maximum of a NaN and a number is the number).
__device__ __forceinline__ uint32_t block_key(const BlockTopkArgs& a, int blk, int n, float best) {
  return blk < a.n_first || blk >= n - a.n_last ? 0xFFFFFFFFu : order_key(fmaxf(best, -INFINITY));
}

// Sum over the CTA of a value per thread; red: one word per warp, of two sets taken in turn.
__device__ __forceinline__ int block_count(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0);
}

template <bool kPage64>
__global__ void __launch_bounds__(kMaxThreads) block_topk_kernel(BlockTopkArgs a) {
  grid_dep_wait();
  grid_dep_launch();   // the kernel after waits for this grid before it reads the blocks
  extern __shared__ uint32_t keys[];
  __shared__ int red[2][32];
  const int CL = static_cast<int>(cl_size()), rank = static_cast<int>(cl_rank());
  const int t = a.T - 1 - static_cast<int>(blockIdx.x) / CL;   // longest causal histories first
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  int qp = __ldg(a.q_pos + t);
  if (qp < 0 || qp >= a.max_ctx) {
    if (tid == 0 && rank == 0) atomicOr(&g_status_block_topk, kDevBadPos);
    qp = -1;   // no block: all -1
  }
  const int n_tok = qp + 1, N = a.N;
  const int n = kPage64 ? (n_tok + 63) >> 6 : (n_tok + a.page_size - 1) / a.page_size;
  int32_t* out = a.out + static_cast<int64_t>(t) * N;
  if (n <= N) {   // cluster-uniform
    for (int i = rank * nt + tid; i < N; i += CL * nt) out[i] = i < n ? i : -1;
    return;
  }
  // ---- this CTA's blocks [lo, hi) to keys in the first CTA
  const float* row = a.scores + static_cast<int64_t>(t) * a.ld;
  const uint32_t dst = CL > 1 ? cl_map(smem_u32(keys), 0) : 0u;
  auto put = [&](int blk, float best) {
    const uint32_t k = block_key(a, blk, n, best);
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
      const int end = min(n_tok, (blk + 1) * a.page_size);
      for (int pos = blk * a.page_size + lane; pos < end; pos += 32) best = fmaxf(best, __ldg(row + pos));
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

  // ---- the largest bits that N keys reach
  const bool one = n <= nt;   // one key a thread
  const uint32_t mine = tid < n ? keys[tid] : 0u;
  uint32_t best = 0u;
  int reach = n, set = 0;
  for (int b = 31; b >= 0 && reach != N; --b) {
    const uint32_t cand = best | (1u << b);
    int c;
    if (one) {
      c = __syncthreads_count(tid < n && mine >= cand);
    } else {
      c = 0;
      for (int i = tid; i < n; i += nt) c += keys[i] >= cand ? 1 : 0;
      c = block_count(c, red[set]);
      set ^= 1;
    }
    if (c >= N) {
      best = cand;
      reach = c;
    }
  }
  // ---- keys above it, and of the keys equal to it so many that there are N, in ascending order
  int above = N;
  if (reach != N) {   // best is a key: some equal ones are left out
    int c = 0;
    for (int i = tid; i < n; i += nt) c += keys[i] > best ? 1 : 0;
    above = block_count(c, red[set]);
    set ^= 1;
  }
  const int equal_most = reach == N ? n : N - above;
  int o = 0, equals = 0;   // written, equal ones met, in the chunks before
  for (int i0 = 0; i0 < n; i0 += nt) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? keys[i] : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, i < n && k > best), eq = __ballot_sync(0xffffffffu, i < n && k == best);
    __syncthreads();
    if (lane == 0) red[0][warp] = __popc(gt) | (__popc(eq) << 16);
    __syncthreads();
    const int v = lane < (nt >> 5) ? red[0][lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0), all = __reduce_add_sync(0xffffffffu, v);
    const uint32_t lt = (1u << lane) - 1u;
    const int eq_before = equals + (before >> 16) + __popc(eq & lt);
    const int gt_before = (before & 0xFFFF) + __popc(gt & lt);
    // of the equal ones before this key in the chunk, those that are taken
    const int eq_taken = min(eq_before, equal_most) - min(equals, equal_most);
    if (((gt >> lane) & 1u) || (((eq >> lane) & 1u) && eq_before < equal_most)) out[o + gt_before + eq_taken] = i;
    o += (all & 0xFFFF) + min(equals + (all >> 16), equal_most) - min(equals, equal_most);
    equals += all >> 16;
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
  // few queries: as many CTAs a query as the GPU holds at once, 128 blocks each at least
  const int want = std::max(1, env.num_sms / seq.T), feed = static_cast<int>(std::max<int64_t>(1, blocks / 128));
  const int cl = std::max(1, std::min(kMaxCluster, std::min(want, feed)));
  const int threads = seq.T * cl > 2 * env.num_sms ? 256 : kMaxThreads;
  const BlockTopkArgs a{scores, ld, seq.q_pos, seq.T, seq.max_ctx, seq.page_size, N, n_first, n_last, out};
  const cudaError_t e = launch_kernel(kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(seq.T) * cl)), dim3(threads),
                                      static_cast<size_t>(blocks) * 4, env.stream, true, cl, a);
  char buf[96];
  snprintf(buf, sizeof(buf), "block_topk[cluster=%d,threads=%d]", cl, threads);
  *plan += buf;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dsa
