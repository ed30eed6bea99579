// Index vectors as codes and scales: the writer of MXFP4 keys, the quantiser of query
// heads (E4M3, MXFP8, MXFP4), and the reader that gives cached keys back as values.
//
// "Large Language Model Inference Acceleration in Practice", section 3.2 (the indexer
// prolog: query quantisation, key-cache update) and section 4 (layered quantisation);
// "Day0 Inference Adaptation and Performance Optimization for Kimi K3.1 Pro", section
// 4.  MXFP4 (OCP Microscaling): a block b of 32 values gets the exponent
//     x_b = floor(log2 max |v|) - 2      (2: the exponent of E2M1's largest number, 6)
// clamped to [-127, 127], -127 for a block of zeros, stored as the byte x_b + 127, and
//     code_i = the E2M1 number nearest to v_i * 2^-x_b, ties to the even code, at most 6.
// The quotient is a product with a power of two and one rounding: whatever order it is
// done in, the same bits come out.  MXFP8 is the same with 8 and E4M3 (448), E4M3 with
// one fp32 scale a vector is cache_append.cu's rule.
//
// A vector of 128 bf16 values is 256 bytes in and 68 out, with a compare, a product and
// a convert per value: memory bounds it, and for few vectors the latency of a launch
// and, in the cache, of position -> page -> row.  So a thread takes 16 neighbouring values
// (whole sectors in, 8 or 16 bytes out), two threads a block's exponent (one shuffle), and
// a vector's threads are neighbours whatever its length: nothing is staged.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "latent_e2m1.cuh"
#include "pair_mma.cuh"

DSA_DEFINE_STATUS_WORD(index_keys)

namespace dsa {
namespace {

constexpr int kBlockThreads = 128;   // at most, in whole vectors (the E4M3 reader: up to twice that for the longest)
constexpr int kVals = 16;            // values a thread

// Cache row of token t, or -1 (flagged) when its position or page is invalid.
__device__ __forceinline__ int64_t token_row(const SeqArgs& seq, const Divisor& by_page, int t) {
  const int qp = __ldg(seq.q_pos + t), b = __ldg(seq.q_seq + t);
  if (qp < 0 || qp >= seq.max_ctx || b < 0 || b >= seq.B) {
    atomicOr(&g_status_index_keys, kDevBadPos);
    return -1;
  }
  const int blk = by_page(qp);
  const int page = __ldg(seq.block_table + static_cast<int64_t>(b) * seq.bt_stride + blk);
  if (page < 0 || page >= seq.n_pages) {
    atomicOr(&g_status_index_keys, kDevBadIndex);
    return -1;
  }
  return static_cast<int64_t>(page) * seq.page_size + (qp - blk * seq.page_size);
}

// Values [0, kVals) from src on.
template <bool kBf16In>
__device__ __forceinline__ void load_values(const uint8_t* src, float (&v)[kVals]) {
#pragma unroll
  for (int k = 0; k < kVals * (kBf16In ? 2 : 4) / 16; ++k) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + k);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBf16In) {
        v[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        v[4 * k + i] = __uint_as_float(w[i]);
      }
    }
  }
}

struct QuantizeArgs {
  int64_t rows;             // vectors
  int32_t H, D;             // vector r is head r % H of token r / H
  const uint8_t* src;
  int64_t stride_t, stride_h;   // bytes
  uint8_t* codes;           // [rows, D] or, MXFP4, [rows, D / 2]
  void* scale;              // E8M0 uint8 [rows, D / 32], or fp32 [rows] (E4M3)
  Divisor per, page;        // by the threads a vector (E4M3: unused), by the page size (cache only)
  bool packed;              // heads follow on one another across tokens
};

// Blocks of 32 values with a power-of-two scale.  kCache: vector t goes to the cache row of token t.
template <bool kBf16In, bool kFp4, bool kCache>
__global__ void __launch_bounds__(kBlockThreads) quantize_mx_kernel(SeqArgs seq, QuantizeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int per = a.D / kVals;   // threads a vector, an even number
  const int local = a.per(static_cast<int>(threadIdx.x)), c = static_cast<int>(threadIdx.x) - local * per;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * a.per(static_cast<int>(blockDim.x)) + local;
  if (r >= a.rows) return;
  const int64_t t = kCache ? r : (a.packed ? 0 : r / a.H);
  float v[kVals];
  load_values<kBf16In>(a.src + t * a.stride_t + (kCache ? 0 : (r - t * a.H) * a.stride_h) + c * (kVals * (kBf16In ? 2 : 4)), v);
  const int64_t row = kCache ? token_row(seq, a.page, static_cast<int>(t)) : r;
  if (row < 0) return;   // all threads of the vector
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kVals; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = fmaxf(amax, __shfl_xor_sync(3u << (threadIdx.x & 30u), amax, 1));   // the block's two threads
  // the exponent's byte from amax's own, which is 0 for subnormal numbers: too small for any but the byte 0
  const uint32_t e = static_cast<uint32_t>(max(0, static_cast<int>(__float_as_uint(amax) >> 23) - (kFp4 ? 2 : 8)));
  const float p = __uint_as_float((254u - e) << 23);   // 2^-(e - 127)
  uint32_t w[kVals / 4] = {};
#pragma unroll
  for (int i = 0; i < kVals; i += 2) {
    float x, y;
    mul2(x, y, v[i], v[i + 1], p, p);
    if constexpr (kFp4)
      w[i / 8] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(x, y), __NV_E2M1, cudaRoundNearest)) << (4 * (i & 7));
    else
      w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3)) << (8 * (i & 3));
  }
  if constexpr (kFp4)
    reinterpret_cast<uint2*>(a.codes + row * (a.D / 2))[c] = make_uint2(w[0], w[1]);
  else
    reinterpret_cast<uint4*>(a.codes + row * a.D)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  if ((c & 1) == 0) static_cast<uint8_t*>(a.scale)[row * (a.D / 32) + c / 2] = static_cast<uint8_t>(e);
}

// One fp32 scale a vector (E4M3): a warp a vector, four values a lane at a time.
constexpr int kRowWarps = 4;
template <bool kBf16In>
__global__ void __launch_bounds__(kRowWarps * 32) quantize_row_kernel(QuantizeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.rows) return;
  const int64_t t = r / a.H;
  const uint8_t* src = a.src + t * a.stride_t + (r - t * a.H) * a.stride_h;
  auto load = [&](int c) -> float4 {
    if constexpr (kBf16In) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(src) + c);
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xFFFF0000u));
    } else {
      return __ldg(reinterpret_cast<const float4*>(src) + c);
    }
  };
  const int nq = a.D / 4;
  float amax = 0.f;
  for (int c = lane; c < nq; c += 32) {
    const float4 f = load(c);
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = e4m3_scale(amax);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.codes + r * a.D);
  for (int c = lane; c < nq; c += 32) {   // the second look comes from the L1
    const float4 f = load(c);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale)), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.z, scale), __fdiv_rn(f.w, scale)), __NV_SATFINITE,
                                                 __NV_E4M3);
    dst[c] = lo | (hi << 16);
  }
  if (lane == 0) static_cast<float*>(a.scale)[r] = scale;
}

struct IndexReadArgs {
  int32_t D;
  const uint8_t* codes;
  const void* scale;
  uint8_t* out;
  int64_t out_stride;       // bytes
  Divisor per, page;        // by the threads a key, by the page size
};

template <IndexKind kKind, bool kF32Out>
__global__ void __launch_bounds__(2 * kBlockThreads) index_read_kernel(SeqArgs seq, IndexReadArgs a) {
  grid_dep_wait();
  constexpr bool kMx = kKind != IndexKind::kE4M3;
  constexpr int V = kMx ? kVals : 4;   // values a thread
  const int per = a.D / V;
  const int local = a.per(static_cast<int>(threadIdx.x)), c = static_cast<int>(threadIdx.x) - local * per;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * a.per(static_cast<int>(blockDim.x)) + local;
  if (t >= seq.T) return;
  const int64_t row = token_row(seq, a.page, static_cast<int>(t));
  if (row < 0) return;
  float v[V];
  float s;
  if constexpr (kMx)
    s = e8m0_to_float(__ldg(static_cast<const uint8_t*>(a.scale) + row * (a.D / 32) + c / 2));
  else
    s = a.scale ? __ldg(static_cast<const float*>(a.scale) + row) : 1.f;
  if constexpr (kKind == IndexKind::kMx4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(a.codes + row * (a.D / 2)) + c);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = e2m1x2_to_float2(((i < 4 ? u.x : u.y) >> (8 * (i & 3))) & 0xFFu);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  } else {
    uint32_t w[V / 4];
    if constexpr (kMx) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(a.codes + row * a.D) + c);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(a.codes + row * a.D) + c);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = e4m3x2_to_float2(static_cast<uint16_t>((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] *= s;
  uint8_t* dst = a.out + t * a.out_stride + c * V * (kF32Out ? 4 : 2);
  if constexpr (kF32Out) {
#pragma unroll
    for (int i = 0; i < V; i += 4) reinterpret_cast<float4*>(dst)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (kMx) {
#pragma unroll
    for (int i = 0; i < V; i += 8)
      reinterpret_cast<uint4*>(dst)[i / 8] = make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                                        pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
  } else {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// Whole vectors of `per` threads a block: as many as make kBlockThreads threads.
int block_vectors(int per) { return std::max(1, kBlockThreads / per); }

template <bool kFp4, bool kCache>
cudaError_t launch_mx(const SeqArgs& seq, const QuantizeArgs& a, bool bf16_in, const LaunchEnv& env) {
  const int per = a.D / kVals, n = block_vectors(per);
  const dim3 grid(static_cast<unsigned>((a.rows + n - 1) / n)), block(static_cast<unsigned>(n * per));
  return bf16_in ? launch_kernel(quantize_mx_kernel<true, kFp4, kCache>, grid, block, 0, env.stream, true, 1, seq, a)
                 : launch_kernel(quantize_mx_kernel<false, kFp4, kCache>, grid, block, 0, env.stream, true, 1, seq, a);
}

}  // namespace

cudaError_t launch_index_append_mx4(const SeqArgs& seq, int32_t D, bool bf16_in, const void* k_new, uint8_t* k_cache,
                                    uint8_t* k_exp, const LaunchEnv& env, std::string* plan) {
  if (seq.T == 0) {
    *plan += "index_append[empty]";
    return cudaSuccess;
  }
  const QuantizeArgs a{seq.T, 1, D, static_cast<const uint8_t*>(k_new), static_cast<int64_t>(D) * (bf16_in ? 2 : 4), 0,
                       k_cache, k_exp, Divisor(D / kVals), Divisor(seq.page_size), true};
  *plan += bf16_in ? "index_append<mxfp4,bf16>" : "index_append<mxfp4,f32>";
  return launch_mx<true, true>(seq, a, bf16_in, env);
}

cudaError_t launch_query_quantize(int64_t T, int32_t H, int32_t D, bool bf16_in, IndexKind kind, const void* q,
                                  int64_t stride_t, int64_t stride_h, uint8_t* codes, void* scale, const LaunchEnv& env,
                                  std::string* plan) {
  if (T == 0 || H == 0) {
    *plan += "query_quantize[empty]";
    return cudaSuccess;
  }
  const QuantizeArgs a{T * H, H, D, static_cast<const uint8_t*>(q), stride_t, stride_h, codes, scale,
                       Divisor(std::max(1, D / kVals)), Divisor(1), T == 1 || stride_t == H * stride_h};
  *plan += kind == IndexKind::kMx4 ? "query_quantize<mxfp4," : (kind == IndexKind::kMx8 ? "query_quantize<mxfp8," : "query_quantize<e4m3,");
  *plan += bf16_in ? "bf16>" : "f32>";
  const SeqArgs none{};
  if (kind == IndexKind::kMx4) return launch_mx<true, false>(none, a, bf16_in, env);
  if (kind == IndexKind::kMx8) return launch_mx<false, false>(none, a, bf16_in, env);
  const dim3 grid(static_cast<unsigned>((a.rows + kRowWarps - 1) / kRowWarps)), block(kRowWarps * 32);
  return bf16_in ? launch_kernel(quantize_row_kernel<true>, grid, block, 0, env.stream, true, 1, a)
                 : launch_kernel(quantize_row_kernel<false>, grid, block, 0, env.stream, true, 1, a);
}

cudaError_t launch_index_read(const SeqArgs& seq, IndexKind kind, int32_t D, const void* codes, const void* scale,
                              bool f32_out, void* out, int64_t out_stride, const LaunchEnv& env, std::string* plan) {
  if (seq.T == 0) {
    *plan += "index_read[empty]";
    return cudaSuccess;
  }
  const int per = D / (kind == IndexKind::kE4M3 ? 4 : kVals), n = block_vectors(per);
  const IndexReadArgs a{D, static_cast<const uint8_t*>(codes), scale, static_cast<uint8_t*>(out), out_stride, Divisor(per),
                        Divisor(seq.page_size)};
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(seq.T) + n - 1) / n)), block(static_cast<unsigned>(n * per));
#define DSA_READ_GO(KIND, NAME)                                                                                   \
  *plan += f32_out ? "index_read<" NAME ",f32>" : "index_read<" NAME ",bf16>";                                    \
  return f32_out ? launch_kernel(index_read_kernel<KIND, true>, grid, block, 0, env.stream, true, 1, seq, a)      \
                 : launch_kernel(index_read_kernel<KIND, false>, grid, block, 0, env.stream, true, 1, seq, a)
  switch (kind) {
    case IndexKind::kE4M3: DSA_READ_GO(IndexKind::kE4M3, "e4m3");
    case IndexKind::kMx8: DSA_READ_GO(IndexKind::kMx8, "mxfp8");
    case IndexKind::kMx4: DSA_READ_GO(IndexKind::kMx4, "mxfp4");
    case IndexKind::kF32: break;
  }
#undef DSA_READ_GO
  return cudaErrorInvalidValue;
}

}  // namespace dsa
