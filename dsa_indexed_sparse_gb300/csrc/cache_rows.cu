// Cache rows with rotary positions: the writers that rotate a new token's rope
// part on the way into the paged caches, the 4-bit latent writer, and the reader
// that gives cached rows back as values.
//
// "Large Language Model Inference Acceleration in Practice", section 3.2 (the
// indexer prolog updates the key cache) and section 4 (layered quantisation of
// the KV cache).  Formats, quantisation rules and addressing are those of
// cache_append.cu (one warp per token, the cache row of position q_pos[t] of
// sequence q_seq[t] through the page table); the 4-bit row is described in
// latent_e2m1.cuh.  The rotation is formed in fp32 and rounded once, to the
// type that the cache holds it in (index keys: by their quantisation).
//
// All of these move a few hundred bytes to a few kilobytes per token and compute
// next to nothing: the time is the latency of a launch and of the chain position
// -> page -> row for a few tokens, and the bytes for many.  Writing 8192 bf16 rows
// takes 3.7 us (5.2 TB/s; 4.5 with the values loaded after the chain), 64 4-bit rows or
// 333 read ones 2 us; reading 65,536 4-bit rows into bf16 19.7 us (5.3 TB/s).  After a writer the
// next kernel may launch as soon as a block has waited for the kernel before: it waits
// for this grid before it reads a cache (and a query that it stages earlier was complete
// by then).  Not so after the reader, whose output may be anything, a query among it.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <type_traits>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "latent_e2m1.cuh"
#include "rope.cuh"

DSA_DEFINE_STATUS_WORD(rows)

namespace dsa {
namespace {

constexpr int kRowWarps = 8;
constexpr int kReadRows = 2;        // rows a warp reads at once, of many
constexpr int kReadWarps = 4;       // warps per block then
constexpr int kIndexWarps = 4;      // index-key writer: a 4 KB row of fp32 values per warp in shared memory

// Cache row of token t, or -1 (flagged) when its position or page is invalid.
__device__ __forceinline__ int64_t token_row(const SeqArgs& seq, int t, int* pos) {
  const int qp = __ldg(seq.q_pos + t), b = __ldg(seq.q_seq + t);
  *pos = qp;
  if (qp < 0 || qp >= seq.max_ctx || b < 0 || b >= seq.B) {
    atomicOr(&g_status_rows, kDevBadPos);
    return -1;
  }
  return phys_row(seq.block_table + static_cast<int64_t>(b) * seq.bt_stride, qp, seq.page_size, seq.n_pages,
                  &g_status_rows);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ uint32_t e4m3_code(float v) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint32_t e4m3_code2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint32_t e4m3_code4(float a, float b, float c, float d) {
  return e4m3_code2(a, b) | (e4m3_code2(c, d) << 16);
}
// floor(log2 amax) - kTop clamped to [-127, 127]; -127 for 0: the shared exponent of blocks
// of codes whose largest number has exponent kTop (8 for E4M3, 2 for E2M1).
template <int kTop = 8>
__device__ __forceinline__ int mx_exponent(float amax) {
  if (!(amax > 0.f)) return -127;
  return max(-127, min(127, ilogbf(amax) - kTop));
}

// Pair i of a row of rope values as they are given (loaded) or held (stored).
template <bool kF32>
__device__ __forceinline__ float2 load_pair(const RopeArgs& rope, int pairs, const void* src, int i) {
  const int e0 = rope.half ? i : 2 * i, e1 = rope.half ? i + pairs : 2 * i + 1;
  if constexpr (kF32) {
    const float* s = static_cast<const float*>(src);
    return make_float2(__ldg(s + e0), __ldg(s + e1));
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(src);
    if (rope.half) return make_float2(bf16_bits_to_float(__ldg(s + e0)), bf16_bits_to_float(__ldg(s + e1)));
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
}
template <bool kF32>
__device__ __forceinline__ void store_pair(const RopeArgs& rope, int pairs, uint8_t* dst, int i, float2 v) {
  const int e0 = rope.half ? i : 2 * i, e1 = rope.half ? i + pairs : 2 * i + 1;
  if constexpr (kF32) {
    reinterpret_cast<float*>(dst)[e0] = v.x;
    reinterpret_cast<float*>(dst)[e1] = v.y;
  } else {
    const uint32_t y = pack_bf16x2(v.x, v.y);
    if (rope.half) {
      reinterpret_cast<uint16_t*>(dst)[e0] = static_cast<uint16_t>(y & 0xFFFFu);
      reinterpret_cast<uint16_t*>(dst)[e1] = static_cast<uint16_t>(y >> 16);
    } else {
      reinterpret_cast<uint32_t*>(dst)[i] = y;
    }
  }
}

// A token's rope values, pair i of lane i % 32: the first pair of each lane is loaded
// before the token's position is known, the rotation and the stores follow.
template <bool kF32>
struct RopeRow {
  float2 v;
  uint64_t turns;
  __device__ __forceinline__ void load(const RopeArgs& rope, int d_rope, const void* src, int lane) {
    if (lane < d_rope / 2) {
      v = load_pair<kF32>(rope, d_rope / 2, src, lane);
      turns = __ldg(rope.turns + lane);
    }
  }
  __device__ __forceinline__ void write(const RopeArgs& rope, int d_rope, const void* src, int pos, uint8_t* dst,
                                        int lane) const {
    const int pairs = d_rope / 2;
    if (lane < pairs)
      store_pair<kF32>(rope, pairs, dst, lane, rope_pair(v.x, v.y, rope_cos_sin(turns, pos, rope.magnitude)));
    for (int i = lane + 32; i < pairs; i += 32) {
      const float2 u = load_pair<kF32>(rope, pairs, src, i);
      store_pair<kF32>(rope, pairs, dst, i, rope_pair(u.x, u.y, rope_cos_sin(__ldg(rope.turns + i), pos, rope.magnitude)));
    }
  }
};

// Sixteen bf16 values from two 16-byte words.
__device__ __forceinline__ void widen16(uint4 a, uint4 b, float (&v)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The quantised latent part of a row: lane l holds dims [16 l, 16 l + 16).
template <MlaKind kKind>
__device__ __forceinline__ void write_latent(const float (&v)[16], uint8_t* dst, int lane) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
  if constexpr (kKind == MlaKind::kE2M1) {
    const int e = e2m1_row_exponent(warp_max(amax));
    const float p = ldexpf(1.f, -e);   // x p: the power-of-two quotient, exact
    const uint32_t sc = e4m3_code(__fdiv_rn(amax * p, 6.f));
    const float s = e4m3_to_float(static_cast<uint8_t>(sc));
    uint32_t w[2] = {0u, 0u};
    if (s > 0.f) {
      // The quotients by s, which has four significant bits, of values with eight: one that is not
      // half way between two codes differs from there by 2^-8 of itself at least, so the product
      // with the rounded reciprocal, rounded to f16 (2^-11), falls on the same side, and one
      // that is half way comes out so.  (With a division for each
      // value writing and reading 16,384 rows took 17.9 us, so 15.7.)
      const float r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 q = __half22float2(__floats2half2_rn(v[2 * i] * p * r, v[2 * i + 1] * p * r));
        w[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(q, __NV_E2M1, cudaRoundNearest)) << (8 * (i & 3));
      }
    }
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
    dst[kE2m1Scales + lane] = static_cast<uint8_t>(sc);
    if (lane < 4) reinterpret_cast<float*>(dst + kE2m1RowScale)[lane] = lane == 0 ? ldexpf(1.f, e) : 0.f;
  } else {
    float q[16];
    if constexpr (kKind == MlaKind::kFP8Row) {
      amax = warp_max(amax);
      const float scale = e4m3_scale(amax);
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(v[i], scale);
      if (lane < 4) reinterpret_cast<float*>(dst + 512)[lane] = lane == 0 ? scale : 0.f;
    } else {   // one power-of-two scale per 128 dims: tile lane / 8
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = mx_exponent(amax);
      const float p = ldexpf(1.f, -e);   // representable: -e is in [-127, 127]
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = v[i] * p;
      if ((lane & 7) == 0) reinterpret_cast<float*>(dst + 512)[lane >> 3] = ldexpf(1.f, e);
    }
    reinterpret_cast<uint4*>(dst)[lane] =
        make_uint4(e4m3_code4(q[0], q[1], q[2], q[3]), e4m3_code4(q[4], q[5], q[6], q[7]),
                   e4m3_code4(q[8], q[9], q[10], q[11]), e4m3_code4(q[12], q[13], q[14], q[15]));
  }
}

struct LatentWriteArgs {
  RopeArgs rope;            // turns == nullptr: the rope part is copied
  const uint8_t* latent;    // [T] rows of d_latent values
  int64_t latent_stride;    // bytes
  const uint8_t* k_rope;    // [T] rows of d_rope values
  int64_t rope_stride;      // bytes
  uint8_t* cache;
  int64_t row_bytes;
  int32_t d_latent, d_rope;
};

// What does not depend on the token's cache row is loaded before the row is looked up.
template <MlaKind kKind>
__global__ void __launch_bounds__(kRowWarps * 32) latent_write_kernel(SeqArgs seq, LatentWriteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tw = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (tw >= seq.T) return;
  const int t = static_cast<int>(tw);
  const uint4* src = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
  const uint8_t* rsrc = a.k_rope + t * a.rope_stride;
  constexpr bool kF32 = kKind == MlaKind::kF32;
  RopeRow<kF32> rr;
  if (a.rope.turns) rr.load(a.rope, a.d_rope, rsrc, lane);
  if constexpr (kF32 || kKind == MlaKind::kBF16) {
    constexpr int kAhead = kF32 ? 4 : 2;   // words a lane: 512 values
    const int words = a.d_latent * (kF32 ? 4 : 2) / 16;
    uint4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (lane + 32 * k < words) u[k] = __ldg(src + lane + 32 * k);
    int pos;
    const int64_t row = token_row(seq, t, &pos);
    if (row < 0) return;
    uint4* dst = reinterpret_cast<uint4*>(a.cache + row * a.row_bytes);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (lane + 32 * k < words) dst[lane + 32 * k] = u[k];
    for (int c = lane + 32 * kAhead; c < words; c += 32) dst[c] = __ldg(src + c);
    rr.write(a.rope, a.d_rope, rsrc, pos, reinterpret_cast<uint8_t*>(dst + words), lane);
  } else {
    const uint4 u0 = __ldg(src + 2 * lane), u1 = __ldg(src + 2 * lane + 1);
    int pos;
    const int64_t row = token_row(seq, t, &pos);
    if (row < 0) return;
    uint8_t* dst = a.cache + row * a.row_bytes;
    float v[16];
    widen16(u0, u1, v);
    write_latent<kKind>(v, dst, lane);
    uint8_t* rdst = dst + (kKind == MlaKind::kE2M1 ? kE2m1Rope : 528);
    if (a.rope.turns)
      rr.write(a.rope, 64, rsrc, pos, rdst, lane);
    else if (lane < 8)
      reinterpret_cast<uint4*>(rdst)[lane] = __ldg(reinterpret_cast<const uint4*>(rsrc) + lane);
  }
}

// Index keys: the row in shared memory as fp32 values, dims [off, off + d_rot)
// rotated there, then quantised as cache_append.cu does.
struct IndexWriteArgs {
  RopeArgs rope;
  int32_t D, off;
  const uint8_t* k_new;
  int64_t stride;           // bytes
  uint8_t* k_cache;
  void* k_scale;            // fp32 [rows], or E8M0 uint8 [rows, D / 32]
};

template <bool kBf16In, IndexKind kKind>
__global__ void __launch_bounds__(kIndexWarps * 32) index_write_kernel(SeqArgs seq, IndexWriteArgs a) {
  __shared__ __align__(16) float rows[kIndexWarps][1024];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tw = static_cast<int64_t>(blockIdx.x) * kIndexWarps + warp;
  if (tw >= seq.T) return;
  const int t = static_cast<int>(tw);
  const int nq = a.D / 4;
  float4* v4 = reinterpret_cast<float4*>(rows[warp]);
  const uint8_t* src = a.k_new + t * a.stride;
  for (int c = lane; c < nq; c += 32) {
    if constexpr (kBf16In) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(src) + c);
      v4[c] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                          __uint_as_float(u.y & 0xFFFF0000u));
    } else {
      v4[c] = __ldg(reinterpret_cast<const float4*>(src) + c);
    }
  }
  int pos;
  const int64_t row = token_row(seq, t, &pos);
  if (row < 0) return;
  __syncwarp();
  float* v = rows[warp] + a.off;
  const int pairs = a.rope.d_rot / 2;
  for (int i = lane; i < pairs; i += 32) {
    const int e0 = a.rope.half ? i : 2 * i, e1 = a.rope.half ? i + pairs : 2 * i + 1;
    const float2 w = rope_cos_sin(__ldg(a.rope.turns + i), pos, a.rope.magnitude);
    const float2 y = rope_pair(v[e0], v[e1], w);
    v[e0] = y.x;
    v[e1] = y.y;
  }
  __syncwarp();
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.k_cache + row * a.D);
  if constexpr (kKind == IndexKind::kMx8 || kKind == IndexKind::kMx4) {
    constexpr bool kFp4 = kKind == IndexKind::kMx4;
    // blocks of 32 values: the 4-value chunks of 8 consecutive lanes (nq is a multiple of 8)
    for (int c0 = 0; c0 < nq; c0 += 32) {
      const int c = c0 + lane;
      const float4 f = c < nq ? v4[c] : make_float4(0.f, 0.f, 0.f, 0.f);
      float amax = fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w)));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = kFp4 ? mx_exponent<2>(amax) : mx_exponent<8>(amax);
      const float p = ldexpf(1.f, -e);
      if (c < nq) {
        if constexpr (kFp4) {
          const uint32_t lo = __nv_cvt_float2_to_fp4x2(make_float2(f.x * p, f.y * p), __NV_E2M1, cudaRoundNearest);
          const uint32_t hi = __nv_cvt_float2_to_fp4x2(make_float2(f.z * p, f.w * p), __NV_E2M1, cudaRoundNearest);
          reinterpret_cast<uint16_t*>(a.k_cache + row * (a.D / 2))[c] = static_cast<uint16_t>(lo | (hi << 8));
        } else {
          dst[c] = e4m3_code4(f.x * p, f.y * p, f.z * p, f.w * p);
        }
        if ((lane & 7) == 0) static_cast<uint8_t*>(a.k_scale)[row * (a.D / 32) + c / 8] = static_cast<uint8_t>(e + 127);
      }
    }
  } else {
    float amax = 0.f;
    for (int c = lane; c < nq; c += 32) {
      const float4 f = v4[c];
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
    }
    amax = warp_max(amax);
    const float scale = e4m3_scale(amax);
    for (int c = lane; c < nq; c += 32) {
      const float4 f = v4[c];
      dst[c] = e4m3_code4(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale), __fdiv_rn(f.z, scale), __fdiv_rn(f.w, scale));
    }
    if (lane == 0) static_cast<float*>(a.k_scale)[row] = scale;
  }
}

// ------------------------------------------------------------------ reading
struct LatentReadArgs {
  const uint8_t* cache;
  int64_t row_bytes;
  uint8_t* out;
  int64_t out_stride;       // bytes
  int32_t d_latent, d_rope;
};

// V consecutive values to an output row, in 16-byte stores (8 bytes for four bf16).
template <bool kF32Out, int V>
__device__ __forceinline__ void store_values(uint8_t* dst, int i, const float (&v)[V]) {
  if constexpr (kF32Out) {
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(dst) + i + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(dst) + i) = make_uint2(w[0], w[1]);
  }
}

// A warp reads kRows tokens' rows: their places in the cache are looked up by its
// first lanes at once, then every row's loads are under way before the first store.
// A lane takes as many values as fill a 16-byte store, neighbouring lanes
// neighbouring values.
template <MlaKind kKind, bool kF32Out, int kRows>
__global__ void __launch_bounds__(kRowWarps * 32) latent_read_kernel(SeqArgs seq, LatentReadArgs a) {
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp) * kRows;
  if (t0 >= seq.T) return;
  int pos;
  const int64_t mine = lane < kRows && t0 + lane < seq.T ? token_row(seq, static_cast<int>(t0) + lane, &pos) : -1;
  int64_t row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) row[r] = __shfl_sync(0xffffffffu, mine, r);
  uint8_t* out = a.out + t0 * a.out_stride;
  if constexpr (kKind == MlaKind::kF32 || kKind == MlaKind::kBF16) {
    constexpr bool kBf16In = kKind == MlaKind::kBF16;
    constexpr int V = kBf16In && !kF32Out ? 8 : 4;
    using Word = std::conditional_t<kBf16In && kF32Out, uint2, uint4>;   // V values
    const int n = (a.d_latent + a.d_rope) / V;
    for (int c = lane; c < n; c += 32) {
      Word u[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (row[r] >= 0) u[r] = __ldg(reinterpret_cast<const Word*>(a.cache + row[r] * a.row_bytes) + c);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (row[r] < 0) continue;
        uint8_t* dst = out + r * a.out_stride;
        if constexpr (kBf16In != kF32Out) {   // the same type
          reinterpret_cast<Word*>(dst)[c] = u[r];
        } else if constexpr (kBf16In) {
          const float v[4] = {__uint_as_float(u[r].x << 16), __uint_as_float(u[r].x & 0xFFFF0000u),
                              __uint_as_float(u[r].y << 16), __uint_as_float(u[r].y & 0xFFFF0000u)};
          store_values<kF32Out>(dst, 4 * c, v);
        } else {
          const float v[4] = {__uint_as_float(u[r].x), __uint_as_float(u[r].y), __uint_as_float(u[r].z),
                              __uint_as_float(u[r].w)};
          store_values<kF32Out>(dst, 4 * c, v);
        }
      }
    }
  } else {
    constexpr int V = kF32Out ? 4 : 8, kSteps = 512 / (32 * V);
    constexpr bool kE2 = kKind == MlaKind::kE2M1;
    // codes of values [V c, V c + V), c = lane + 32 k, and their scales
    uint32_t code[kRows][kSteps][kE2 ? 1 : V / 4];
    float scale[kRows][kKind == MlaKind::kFP8Row ? 1 : kSteps];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row[r] < 0) continue;
      const uint8_t* src = a.cache + row[r] * a.row_bytes;
      const float rs = kKind == MlaKind::kFP8Tile ? 1.f : __ldg(reinterpret_cast<const float*>(src + (kE2 ? kE2m1RowScale : 512)));
      if constexpr (kKind == MlaKind::kFP8Row) scale[r][0] = rs;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int c = lane + 32 * k;
        if constexpr (kE2) {
          if constexpr (V == 8)
            code[r][k][0] = __ldg(reinterpret_cast<const uint32_t*>(src) + c);
          else
            code[r][k][0] = __ldg(reinterpret_cast<const uint16_t*>(src) + c);
          scale[r][k] = e4m3_to_float(__ldg(src + kE2m1Scales + c * V / 16)) * rs;
        } else {
          if constexpr (V == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(src) + c);
            code[r][k][0] = u.x;
            code[r][k][1] = u.y;
          } else {
            code[r][k][0] = __ldg(reinterpret_cast<const uint32_t*>(src) + c);
          }
          if constexpr (kKind == MlaKind::kFP8Tile) scale[r][k] = __ldg(reinterpret_cast<const float*>(src + 512) + c * V / 128);
        }
      }
    }
    // the 64 rope values: eight lanes a row
    const int rl = lane >> 3, r8 = lane & 7;
    const int64_t rrow = __shfl_sync(0xffffffffu, mine, rl);   // -1 beyond kRows
    uint4 rope = make_uint4(0u, 0u, 0u, 0u);
    if (rrow >= 0) rope = __ldg(reinterpret_cast<const uint4*>(a.cache + rrow * a.row_bytes + (kE2 ? kE2m1Rope : 528)) + r8);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row[r] < 0) continue;
      uint8_t* dst = out + r * a.out_stride;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const float s = scale[r][kKind == MlaKind::kFP8Row ? 0 : k];
        float v[V];
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          float2 p;
          if constexpr (kE2)
            p = e2m1x2_to_float2((code[r][k][0] >> (4 * i)) & 0xFFu);
          else
            p = e4m3x2_to_float2(static_cast<uint16_t>(code[r][k][i >> 2] >> (8 * (i & 3))));
          v[i] = p.x * s;
          v[i + 1] = p.y * s;
        }
        store_values<kF32Out>(dst, V * (lane + 32 * k), v);
      }
    }
    if (rrow >= 0) {
      uint8_t* dst = out + rl * a.out_stride;
      if constexpr (kF32Out) {
        const float v[8] = {__uint_as_float(rope.x << 16), __uint_as_float(rope.x & 0xFFFF0000u),
                            __uint_as_float(rope.y << 16), __uint_as_float(rope.y & 0xFFFF0000u),
                            __uint_as_float(rope.z << 16), __uint_as_float(rope.z & 0xFFFF0000u),
                            __uint_as_float(rope.w << 16), __uint_as_float(rope.w & 0xFFFF0000u)};
        store_values<true>(dst, 512 + 8 * r8, v);
      } else {
        reinterpret_cast<uint4*>(dst)[64 + r8] = rope;
      }
    }
  }
}

// Warps per block: one for a few tokens (they spread over the SMs), up to kRowWarps.
int row_warps(int T, int num_sms) {
  int w = kRowWarps;
  while (w > 1 && (static_cast<int64_t>(T) + w - 1) / w < num_sms) w /= 2;
  return w;
}

}  // namespace

cudaError_t launch_latent_write(const SeqArgs& seq, const MlaArgs& a, const RopeArgs& rope, const void* latent,
                                int64_t latent_stride, const void* k_rope, int64_t rope_stride, void* kv_cache,
                                const LaunchEnv& env, std::string* plan) {
  if (seq.T == 0) {
    *plan += "latent_append[empty]";
    return cudaSuccess;
  }
  const LatentWriteArgs w{rope, static_cast<const uint8_t*>(latent), latent_stride, static_cast<const uint8_t*>(k_rope),
                          rope_stride, static_cast<uint8_t*>(kv_cache), a.row_bytes, a.d_latent, a.d_rope};
  const int warps = row_warps(seq.T, env.num_sms);
  const dim3 grid((static_cast<int64_t>(seq.T) + warps - 1) / warps), block(warps * 32);
  *plan += rope.turns ? "latent_append_rope<" : "latent_append<";
#define DSA_WRITE_GO(KIND, NAME)  \
  *plan += NAME ">";              \
  return launch_kernel(latent_write_kernel<KIND>, grid, block, 0, env.stream, true, 1, seq, w)
  switch (a.kind) {
    case MlaKind::kF32: DSA_WRITE_GO(MlaKind::kF32, "f32");
    case MlaKind::kBF16: DSA_WRITE_GO(MlaKind::kBF16, "bf16");
    case MlaKind::kFP8Row: DSA_WRITE_GO(MlaKind::kFP8Row, "fp8_row");
    case MlaKind::kFP8Tile: DSA_WRITE_GO(MlaKind::kFP8Tile, "fp8_tile128");
    case MlaKind::kE2M1: DSA_WRITE_GO(MlaKind::kE2M1, "e2m1");
  }
#undef DSA_WRITE_GO
  return cudaErrorInvalidValue;
}

cudaError_t launch_index_write(const SeqArgs& seq, const RopeArgs& rope, int32_t D, int32_t off, bool bf16_in, IndexKind kind,
                               const void* k_new, int64_t stride, uint8_t* k_cache, void* k_scale,
                               const LaunchEnv& env, std::string* plan) {
  if (seq.T == 0) {
    *plan += "index_append_rope[empty]";
    return cudaSuccess;
  }
  const IndexWriteArgs a{rope, D, off, static_cast<const uint8_t*>(k_new), stride, k_cache, k_scale};
  const dim3 grid((static_cast<int64_t>(seq.T) + kIndexWarps - 1) / kIndexWarps), block(kIndexWarps * 32);
  *plan += kind == IndexKind::kMx4 ? "index_append_rope<mxfp4," : (kind == IndexKind::kMx8 ? "index_append_rope<mx," : "index_append_rope<e4m3,");
  *plan += bf16_in ? "bf16>" : "f32>";
#define DSA_INDEX_GO(KIND)                                                                                         \
  return bf16_in ? launch_kernel(index_write_kernel<true, KIND>, grid, block, 0, env.stream, true, 1, seq, a)     \
                 : launch_kernel(index_write_kernel<false, KIND>, grid, block, 0, env.stream, true, 1, seq, a)
  if (kind == IndexKind::kMx4) DSA_INDEX_GO(IndexKind::kMx4);
  if (kind == IndexKind::kMx8) DSA_INDEX_GO(IndexKind::kMx8);
  DSA_INDEX_GO(IndexKind::kE4M3);
#undef DSA_INDEX_GO
}

cudaError_t launch_latent_read(const SeqArgs& seq, const MlaArgs& a, const void* kv_cache, bool f32_out, void* out,
                               int64_t out_stride, const LaunchEnv& env, std::string* plan) {
  if (seq.T == 0) {
    *plan += "latent_read[empty]";
    return cudaSuccess;
  }
  const LatentReadArgs r{static_cast<const uint8_t*>(kv_cache), a.row_bytes, static_cast<uint8_t*>(out), out_stride,
                         a.d_latent, a.d_rope};
  // Two rows a warp once there is a row for every warp that the GPU holds: 65,536 4-bit
  // rows take 19.7 us, 22.0 with one, 20.5 with three, 21.3 with four, 20.3 in blocks of eight
  // warps.  Fewer rows take no longer with a warp each, and spread further.
  const bool many = seq.T > env.num_sms * 64;
  const int warps = many ? kReadWarps : row_warps(seq.T, env.num_sms), per_block = warps * (many ? kReadRows : 1);
  const dim3 grid((static_cast<int64_t>(seq.T) + per_block - 1) / per_block), block(warps * 32);
  *plan += "latent_read<";
#define DSA_READ_LAUNCH(KIND, F32, ROWS) \
  launch_kernel(latent_read_kernel<KIND, F32, ROWS>, grid, block, 0, env.stream, true, 1, seq, r)
#define DSA_READ_GO(KIND, NAME)                                                                     \
  *plan += f32_out ? NAME ",f32>" : NAME ",bf16>";                                                  \
  if (many) return f32_out ? DSA_READ_LAUNCH(KIND, true, kReadRows) : DSA_READ_LAUNCH(KIND, false, kReadRows); \
  return f32_out ? DSA_READ_LAUNCH(KIND, true, 1) : DSA_READ_LAUNCH(KIND, false, 1)
  switch (a.kind) {
    case MlaKind::kF32: DSA_READ_GO(MlaKind::kF32, "f32");
    case MlaKind::kBF16: DSA_READ_GO(MlaKind::kBF16, "bf16");
    case MlaKind::kFP8Row: DSA_READ_GO(MlaKind::kFP8Row, "fp8_row");
    case MlaKind::kFP8Tile: DSA_READ_GO(MlaKind::kFP8Tile, "fp8_tile128");
    case MlaKind::kE2M1: DSA_READ_GO(MlaKind::kE2M1, "e2m1");
  }
#undef DSA_READ_GO
#undef DSA_READ_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace dsa
