// Rotary positions on query heads (any strided part of a head), and the host
// side of the rotation: frequencies with their scalings for long contexts.
//
// The latent attention's keys and queries carry a rope part next to the latent
// part (the 64 rope dims of the cached rows: "Large Language Model Inference
// Acceleration in Practice", section 1.2), and the cache writers rotate the keys
// (cache_rows.cu); this is the query's side.  Pair (a, b) at position p becomes
//     (a cos - b sin, a sin + b cos),  cos and sin of the pair's angle, times a factor m;
// the inverse takes -sin (the transposed matrix: the gradient of the rotation).
//
// The work is one read and one write per value: the memory bounds it, and for a few
// tokens the launch.  A thread owns one 16-byte vector position within a head
// (interleaved pairs; two vectors, one per half, for the half layout) and walks over
// heads, so the block's cosines and sines -- one evaluation per (token, pair), in
// shared memory -- are fetched once per thread and token.  One token of 128 heads
// takes 1.7 us, 333 of 64 fp32 heads 2.4 us (4.5 TB/s, from the L2).
// The kernels do not let the next kernel launch early: the attention stages its
// query before it waits for the kernel before it, and the query is what these write.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "rope.cuh"

namespace dsa {
namespace {

// Threads of a block: 84 us for 16,384 tokens of 128 heads of 64 bf16 values (6.4 TB/s), 102
// with blocks of 256, which keep fewer loads under way at the seams between blocks; 85 with 64.
constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 256;     // d_rot <= 512; a block of the scalar kernel holds a token's pairs at least

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;       // values per 16 bytes
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { static_cast<float*>(p)[i] = v; }
  static __device__ __forceinline__ void unpack(uint4 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
  static __device__ __forceinline__ void unpack(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};

struct RopeKernelArgs {
  RopeArgs rope;
  const int32_t* pos;
  const void* x;
  void* out;
  int64_t x_st, x_sh, o_st, o_sh;   // strides of tokens and heads, in elements
  int32_t T, H;
  int32_t tokens;                   // tokens per block (1 unless a whole token is less than a block)
  int32_t heads;                    // heads per block
  int32_t units;                    // thread positions within a head
  float sign;                       // -1: inverse
};

// The cosines and sines of the block's tokens: cs[token * pairs + pair].
__device__ __forceinline__ void block_cos_sin(const RopeKernelArgs& a, int t0, int nt, float2* cs) {
  const int pairs = a.rope.d_rot / 2;
  for (int i = threadIdx.x; i < nt * pairs; i += blockDim.x) {
    const int tl = i / pairs;
    float2 v = rope_cos_sin(__ldg(a.rope.turns + (i - tl * pairs)), __ldg(a.pos + t0 + tl), a.rope.magnitude);
    v.y *= a.sign;
    cs[i] = v;
  }
  __syncthreads();
}

// kOneHead: every cosine is used once, so each thread forms its own, without the shared
// memory and its barrier (262,144 tokens of one 64-wide bf16 head: 27.0 us; 25.2 against 36.7
// through it before the quarter turns were split off).
template <typename T, bool kHalf, bool kOneHead>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(RopeKernelArgs a) {
  extern __shared__ float2 cs[];
  grid_dep_wait();
  constexpr int V = Elem<T>::kVec;
  constexpr int P = kHalf ? V : V / 2;   // pairs per thread and row
  const int t0 = blockIdx.x * a.tokens, h0 = blockIdx.y * a.heads;
  const int nt = min(a.tokens, a.T - t0), nh = min(a.heads, a.H - h0);
  const int slot = threadIdx.x / a.units, unit = threadIdx.x - slot * a.units;
  const int slots = blockDim.x / a.units;
  const int pairs = a.rope.d_rot / 2;
  const int e0 = unit * V, e1 = e0 + pairs;   // first elements of the thread's vector(s) (e1: half layout)
  const T* x = static_cast<const T*>(a.x);
  T* o = static_cast<T*>(a.out);
  // kBatch rows' loads before their stores: x may be out, so the compiler keeps
  // a load behind every earlier store.  The first batch is under way while the
  // cosines and sines are formed.
  constexpr int kBatch = kHalf ? 4 : 8;
  uint4 u0[kBatch], u1[kHalf ? kBatch : 1];
  int pos[kOneHead ? kBatch : 1];
  uint64_t turns[kOneHead ? P : 1];
  auto load = [&](int r0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * slots;
      if (r < nt * nh) {
        const int tl = a.tokens == 1 ? 0 : r / nh;
        const T* xr = x + (t0 + tl) * a.x_st + (h0 + r - tl * nh) * a.x_sh;
        u0[b] = *reinterpret_cast<const uint4*>(xr + e0);
        if constexpr (kHalf) u1[b] = *reinterpret_cast<const uint4*>(xr + e1);
        if constexpr (kOneHead) pos[b] = __ldg(a.pos + t0 + tl);
      }
    }
  };
  load(slot);
  if constexpr (kOneHead) {
#pragma unroll
    for (int i = 0; i < P; ++i) turns[i] = __ldg(a.rope.turns + unit * P + i);
  } else {
    block_cos_sin(a, t0, nt, cs);
  }
  float2 w[P];
  int tw = -1;
  for (int r0 = slot; r0 < nt * nh;) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * slots;
      if (r >= nt * nh) break;
      const int tl = a.tokens == 1 ? 0 : r / nh;
      T* orow = o + (t0 + tl) * a.o_st + (h0 + r - tl * nh) * a.o_sh;
      if constexpr (kOneHead) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          w[i] = rope_cos_sin(turns[i], pos[b], a.rope.magnitude);
          w[i].y *= a.sign;
        }
      } else if (tl != tw) {
        tw = tl;
#pragma unroll
        for (int i = 0; i < P; ++i) w[i] = cs[tl * pairs + unit * P + i];
      }
      float v0[V], v1[V], y0[V], y1[V];
      Elem<T>::unpack(u0[b], v0);
      if constexpr (kHalf) {
        Elem<T>::unpack(u1[b], v1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 y = rope_pair(v0[i], v1[i], w[i]);
          y0[i] = y.x;
          y1[i] = y.y;
        }
        *reinterpret_cast<uint4*>(orow + e1) = Elem<T>::pack(y1);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 y = rope_pair(v0[2 * i], v0[2 * i + 1], w[i]);
          y0[2 * i] = y.x;
          y0[2 * i + 1] = y.y;
        }
      }
      *reinterpret_cast<uint4*>(orow + e0) = Elem<T>::pack(y0);
    }
    r0 += slots * kBatch;
    load(r0);
  }
}

// Any strides and sizes: one pair per thread position.
template <typename T>
__global__ void __launch_bounds__(kRopeMaxPairs) rope_scalar_kernel(RopeKernelArgs a) {
  extern __shared__ float2 cs[];
  grid_dep_wait();
  const int t0 = blockIdx.x * a.tokens, h0 = blockIdx.y * a.heads;
  const int nt = min(a.tokens, a.T - t0), nh = min(a.heads, a.H - h0);
  const int slot = threadIdx.x / a.units, pair = threadIdx.x - slot * a.units;
  const int slots = blockDim.x / a.units;
  block_cos_sin(a, t0, nt, cs);
  const int pairs = a.rope.d_rot / 2;
  const int e0 = a.rope.half ? pair : 2 * pair, e1 = a.rope.half ? pair + pairs : 2 * pair + 1;
  for (int r = slot; r < nt * nh; r += slots) {
    const int tl = r / nh, h = h0 + r - tl * nh;
    const int64_t xi = (t0 + tl) * a.x_st + h * a.x_sh, oi = (t0 + tl) * a.o_st + h * a.o_sh;
    const float u = Elem<T>::load(a.x, xi + e0), v = Elem<T>::load(a.x, xi + e1);
    const float2 y = rope_pair(u, v, cs[tl * pairs + pair]);
    Elem<T>::store(a.out, oi + e0, y.x);
    Elem<T>::store(a.out, oi + e1, y.y);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& rope, int32_t T, int32_t H, const int32_t* pos, bool bf16, const void* x,
                        int64_t x_st, int64_t x_sh, void* out, int64_t o_st, int64_t o_sh, bool inverse,
                        const LaunchEnv& env, std::string* plan) {
  if (T == 0 || H == 0) {
    *plan += "rope[empty]";
    return cudaSuccess;
  }
  const int vec = bf16 ? 8 : 4, pairs = rope.d_rot / 2;
  // 16-byte vectors need whole vectors of values (of each half), and every row on a 16-byte boundary
  const bool aligned = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
                       (rope.half ? pairs : rope.d_rot) % vec == 0 && (T == 1 || (x_st % vec == 0 && o_st % vec == 0)) &&
                       (H == 1 || (x_sh % vec == 0 && o_sh % vec == 0));
  RopeKernelArgs a{rope, pos, x, out, x_st, x_sh, o_st, o_sh, T, H, 1, H, 0, inverse ? -1.f : 1.f};
  a.units = aligned ? (rope.half ? pairs : rope.d_rot) / vec : pairs;
  const int slots = std::max(1, kRopeThreads / a.units);
  // A block takes up to eight rows a thread, four of two vectors in the half layout -- as many
  // as a thread loads at once (99.5 us for 16,384 x 128 bf16 heads with eight, 83.6 with four);
  // the cosines are fetched once per thread and token -- fewer while the blocks do not fill
  // the GPU twice: part of one token's heads, or the heads of several tokens.
  int rows = rope.half && aligned ? 4 : 8;
  while (rows > 1 && static_cast<int64_t>(T) * H < 2ll * env.num_sms * slots * rows) rows /= 2;
  if (H > slots * rows)
    a.heads = slots * rows;
  else
    a.tokens = std::max(1, std::min({slots * rows / H, T, kRopeMaxPairs * 8 / pairs}));
  const dim3 grid((static_cast<int64_t>(T) + a.tokens - 1) / a.tokens, (H + a.heads - 1) / a.heads), block(a.units * slots);
  const bool one = aligned && H == 1;
  const size_t smem = one ? 0 : static_cast<size_t>(a.tokens) * pairs * sizeof(float2);
  *plan += aligned ? (rope.half ? "rope_vec<half," : "rope_vec<interleaved,") : "rope_scalar<";
  *plan += bf16 ? "bf16>" : "f32>";
#define DSA_ROPE_GO(K) launch_kernel(K, grid, block, smem, env.stream, true, 1, a)
  if (!aligned) return bf16 ? DSA_ROPE_GO(rope_scalar_kernel<__nv_bfloat16>) : DSA_ROPE_GO(rope_scalar_kernel<float>);
#define DSA_ROPE_VEC(T, HALF) \
  (one ? DSA_ROPE_GO((rope_vec_kernel<T, HALF, true>)) : DSA_ROPE_GO((rope_vec_kernel<T, HALF, false>)))
  if (rope.half) return bf16 ? DSA_ROPE_VEC(__nv_bfloat16, true) : DSA_ROPE_VEC(float, true);
  return bf16 ? DSA_ROPE_VEC(__nv_bfloat16, false) : DSA_ROPE_VEC(float, false);
#undef DSA_ROPE_VEC
#undef DSA_ROPE_GO
}

// Frequencies on the host, in double.  theta^(-2 i / d) per pair; LINEAR divides
// every frequency by the factor; NTK raises the base so that the slowest pair is
// slowed by the factor and the fastest kept; YARN blends the kept and the divided
// frequency by a ramp over the pairs between those that turn beta_fast and
// beta_slow times within original_ctx positions, with a factor of
// 0.1 ln(factor) + 1 on cosine and sine.
void rope_turns(int32_t d_rot, double theta, int scaling, double factor, double original_ctx, double beta_fast,
                double beta_slow, uint64_t* turns, float* magnitude) {
  const double two_pi = 6.283185307179586476925286766559;
  const int n = d_rot / 2;
  const double base = scaling == DSA_ROPE_NTK ? theta * std::pow(factor, d_rot / (d_rot - 2.0)) : theta;
  double lo = 0.0, hi = 1.0;
  if (scaling == DSA_ROPE_YARN) {
    auto pair_turning = [&](double turns_in_ctx) {
      return d_rot * std::log(original_ctx / (turns_in_ctx * two_pi)) / (2.0 * std::log(theta));
    };
    lo = std::max(std::floor(pair_turning(beta_fast)), 0.0);
    hi = std::min(std::ceil(pair_turning(beta_slow)), d_rot - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(base, -2.0 * i / d_rot);
    if (scaling == DSA_ROPE_LINEAR) f /= factor;
    if (scaling == DSA_ROPE_YARN) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    const double u = f / two_pi, frac = u - std::floor(u);
    turns[i] = static_cast<uint64_t>(std::ldexp(frac, 64));   // frac < 1 - 2^-53: below 2^64
  }
  *magnitude = scaling == DSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
}

}  // namespace dsa
