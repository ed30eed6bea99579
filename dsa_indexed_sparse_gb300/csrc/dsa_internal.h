// Host-side interface between the C-ABI facade (api.cu) and the kernel
// translation units.  Plain structs passed by value to the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dsa.h"

#include <string>
#include <utility>

namespace dsa {

// Counts of n in d, the last one short; of 0 <= n < 2^31, without a sum that passes 2^31.
__host__ __device__ constexpr int div_up(int n, int d) {
  return static_cast<int>((static_cast<uint32_t>(n) + static_cast<uint32_t>(d) - 1u) / static_cast<uint32_t>(d));
}

struct SeqArgs {
  int32_t B, T, max_ctx, q_per_seq;
  const int32_t* q_seq;
  const int32_t* q_pos;
  const int32_t* block_table;
  int32_t bt_stride, page_size;
  int64_t cache_rows;
  int64_t n_pages;  // cache_rows / page_size
};

// fp32 values; E4M3 codes with an fp32 scale a vector; E4M3 or E2M1 codes with an E8M0 scale per 32 values
enum class IndexKind { kF32 = 0, kE4M3 = 1, kMx8 = 2, kMx4 = 3 };

struct IndexerArgs {
  int32_t H_I, D_I;
  IndexKind kind;
  const void* q;
  const void* q_scale;  // fp32 [T, H_I] (may be null) or uint8 [T, H_I, D_I/32] (kMx8, kMx4)
  const float* w;
  const void* k;
  const void* k_scale;  // fp32 [rows] (may be null) or uint8 [rows, D_I/32] (kMx8, kMx4)
  float* scores;
  int64_t ld;
};

// kFP8Tile: scale per 128 latent dims; kE2M1: 4-bit codes, scale per 16 dims and per row
enum class MlaKind { kF32 = 0, kBF16 = 1, kFP8Row = 2, kFP8Tile = 3, kE2M1 = 4 };

struct MlaArgs {
  int32_t H, d_latent, d_rope;
  MlaKind kind;
  const void* q;
  const void* kv;
  int64_t row_bytes;
  float softmax_scale;
  const int32_t* idx;
  int32_t K;
  void* out;
  float* lse;  // may be null
};

struct LaunchEnv {
  cudaStream_t stream;
  int num_sms;
  int device;
  bool chained = false;   // decode step: the call's kernels before this one do not write the attention's query
};

// Each launcher validates kernel-specific limits, enqueues its kernels and
// appends a short description of what it launched to *plan.  Returns
// cudaSuccess or the launch error; `unsupported` is set (and nothing launched)
// when no kernel covers the arguments.

// Lightning indexer.
cudaError_t launch_indexer(const SeqArgs& seq, const IndexerArgs& a, const LaunchEnv& env,
                           std::string* plan, bool* unsupported, std::string* why);

// Fused decode plan: indexer scores kept in shared memory and the Top-K selected
// in the same kernel (clusters of CTAs per query); writes idx [T, K] only.  Sets
// *unsupported (and launches nothing) when the arguments call for the chained plan.
cudaError_t launch_decode_fused(const SeqArgs& seq, const IndexerArgs& a, int32_t K, int32_t* idx,
                                const LaunchEnv& env, std::string* plan, bool* unsupported, std::string* why);

// Top-K.
cudaError_t launch_topk(const SeqArgs& seq, const float* scores, int64_t ld, int32_t K,
                        int32_t* idx, const LaunchEnv& env, std::string* plan);

// Sparse MLA attention.  workspace may be null (ws_bytes 0).
size_t attn_workspace_bytes(const SeqArgs& seq, const MlaArgs& a, int num_sms);
cudaError_t launch_attn(const SeqArgs& seq, const MlaArgs& a, void* workspace, size_t ws_bytes,
                        const LaunchEnv& env, std::string* plan, bool* unsupported,
                        std::string* why);

// Attention over 4-bit rows (attn_e2m1.cu), any head count; and the merge of row
// slices' partial results, bf16 [n_split, T, H, 512] and their LSE.
size_t attn_e2m1_workspace_bytes(const SeqArgs& seq, const MlaArgs& a, int num_sms);
cudaError_t launch_attn_e2m1(const SeqArgs& seq, const MlaArgs& a, void* workspace, size_t ws_bytes,
                             const LaunchEnv& env, std::string* plan);
cudaError_t launch_attn_combine(const uint16_t* ws_o, const float* ws_lse, int n_split, int T, int H, void* out,
                                float* lse_out, const LaunchEnv& env);

// Blocks by the best score in each, and the attention over blocks (a.idx: [T, a.K] blocks).
// The workspace may be null (ws_bytes 0) unless attn_block_positions: then the blocks' positions
// are written into it for launch_attn.
cudaError_t launch_block_topk(const SeqArgs& seq, const float* scores, int64_t ld, int32_t N, int32_t n_first,
                              int32_t n_last, int32_t* out, const LaunchEnv& env, std::string* plan, bool* unsupported,
                              std::string* why);
bool attn_block_positions(const SeqArgs& seq, const MlaArgs& a);
size_t attn_block_workspace_bytes(const SeqArgs& seq, const MlaArgs& a, int num_sms);
cudaError_t launch_attn_block(const SeqArgs& seq, const MlaArgs& a, void* workspace, size_t ws_bytes,
                              const LaunchEnv& env, std::string* plan, bool* unsupported, std::string* why);

// Launches a kernel, when `pdl` with programmatic stream serialization (it
// may launch while the previous kernel on the stream is finishing; every
// kernel of this library waits for its predecessor with griddepcontrol.wait
// before reading anything), and when cluster > 1 as clusters of `cluster` CTAs
// along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                          bool pdl, int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The indexer prolog (projections, key normalisation, quantisation, key append).
struct PrologArgs {
  int32_t d_model, d_q, H_I;
  const void* x;        // bf16 [T, d_model]
  const void* x_q;      // bf16 [T, d_q]
  const void* w_q;      // bf16 [H_I * 128, d_q]
  const void* w_k;      // bf16 [128, d_model]
  const void* w_w;      // bf16 [H_I, d_model]
  const float* gamma;   // [128]
  const float* beta;    // [128]
  uint8_t* q_codes;     // [T, H_I, 128]
  float* q_scale;       // [T, H_I]
  float* w;             // [T, H_I]
  uint8_t* k_cache;     // [cache_rows, 128]
  float* k_scale;       // [cache_rows]
};
size_t prolog_workspace_bytes(int T, int H_I, int d_model, int d_q, int num_sms);
cudaError_t launch_prolog(const SeqArgs& seq, const PrologArgs& a, void* workspace, const LaunchEnv& env,
                          std::string* plan, bool* unsupported, std::string* why);

// Cache writers (the new tokens' index keys / latent rows into the paged caches).
cudaError_t launch_index_append(const SeqArgs& seq, int32_t D, bool bf16_in, const void* k_new, uint8_t* k_cache,
                                float* k_scale, const LaunchEnv& env, std::string* plan);
cudaError_t launch_index_append_mx(const SeqArgs& seq, int32_t D, bool bf16_in, const void* k_new, uint8_t* k_cache,
                                   uint8_t* k_exp, const LaunchEnv& env, std::string* plan);
cudaError_t launch_latent_append(const SeqArgs& seq, const MlaArgs& a, const void* kv_new, void* kv_cache,
                                 const LaunchEnv& env, std::string* plan);

// Rotary positions (rope.cuh holds RopeArgs): strided heads, and the host side's frequencies.
struct RopeArgs;
cudaError_t launch_rope(const RopeArgs& rope, int32_t T, int32_t H, const int32_t* pos, bool bf16, const void* x,
                        int64_t x_st, int64_t x_sh, void* out, int64_t o_st, int64_t o_sh, bool inverse,
                        const LaunchEnv& env, std::string* plan);
void rope_turns(int32_t d_rot, double theta, int scaling, double factor, double original_ctx, double beta_fast,
                double beta_slow, uint64_t* turns, float* magnitude);

// Cache writers that rotate (rope.turns null: the rope part is copied) and the
// cache reader.  Strides in bytes.
cudaError_t launch_latent_write(const SeqArgs& seq, const MlaArgs& a, const RopeArgs& rope, const void* latent,
                                int64_t latent_stride, const void* k_rope, int64_t rope_stride, void* kv_cache,
                                const LaunchEnv& env, std::string* plan);
cudaError_t launch_index_write(const SeqArgs& seq, const RopeArgs& rope, int32_t D, int32_t off, bool bf16_in, IndexKind kind,
                               const void* k_new, int64_t stride, uint8_t* k_cache, void* k_scale,
                               const LaunchEnv& env, std::string* plan);
cudaError_t launch_latent_read(const SeqArgs& seq, const MlaArgs& a, const void* kv_cache, bool f32_out, void* out,
                               int64_t out_stride, const LaunchEnv& env, std::string* plan);

// MXFP4 index keys, query heads to codes and scales (kind: kE4M3, kMx8, kMx4), and the
// reader of cached index keys.  Strides in bytes.
cudaError_t launch_index_append_mx4(const SeqArgs& seq, int32_t D, bool bf16_in, const void* k_new, uint8_t* k_cache,
                                    uint8_t* k_exp, const LaunchEnv& env, std::string* plan);
cudaError_t launch_query_quantize(int64_t T, int32_t H, int32_t D, bool bf16_in, IndexKind kind, const void* q,
                                  int64_t stride_t, int64_t stride_h, uint8_t* codes, void* scale, const LaunchEnv& env,
                                  std::string* plan);
cudaError_t launch_index_read(const SeqArgs& seq, IndexKind kind, int32_t D, const void* codes, const void* scale,
                              bool f32_out, void* out, int64_t out_stride, const LaunchEnv& env, std::string* plan);

// Sets the text dsa_last_error() returns on the calling thread.
void set_last_error(const std::string& msg);

// Raises `kernel`'s dynamic shared-memory limit to `bytes` on `device` (which
// must be current), once per (kernel, device); later calls return the first
// call's result.  Thread-safe.
cudaError_t ensure_smem_limit(const void* kernel, int bytes, int device);
// Whether one cluster of `cl` CTAs of `kernel` (`threads` threads, `smem` bytes of
// dynamic shared memory each) can be resident on `device`; the occupancy query is
// made once per distinct argument set (and allows non-portable sizes above 8).
bool cluster_fits(const void* kernel, int device, int cl, int threads, size_t smem);

// The failure-detection testing aid (dsa_debug_withhold_arrival): the wait
// bound the kernels use and whether the attention producer withholds an arrival.
void debug_wait_state(uint64_t* wait_limit_ns, uint32_t* withhold);

// Scratch bytes dsa_decode_step needs for these descriptors on the current
// device, with the status (and dsa_last_error text) dsa_decode_step itself
// would return for a bad descriptor.
dsa_status_t decode_workspace_need(const dsa_seq_desc_t* seq, const dsa_mla_desc_t* mla, int32_t K, size_t* need);

// Tensor-map encoder (driver entry point, resolved once).
bool encode_tmap_2d_u8(void* tmap_out, const void* base, uint64_t inner, uint64_t rows,
                       uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_rows,
                       std::string* why);
// Same for 1- or 2-byte elements (inner / box_inner counted in elements); the swizzle is
// that of the box's row, 128 or 64 bytes.
bool encode_tmap_2d(void* tmap_out, const void* base, int elem_bytes, uint64_t inner, uint64_t rows,
                    uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_rows, std::string* why);
// Rows of `atoms` * 64 16-bit values as operand atoms: coordinates (0, row, atom), a box 64
// values x box_rows rows x box_atoms atoms, which lands as so many [box_rows x 128 bytes] atoms
// one behind the other, 128-byte swizzle.
bool encode_tmap_atoms(void* tmap_out, const void* base, uint32_t atoms, uint64_t rows, uint64_t row_stride_bytes,
                       uint32_t box_rows, uint32_t box_atoms, std::string* why);
// Packed [tokens, heads, atoms * 64] 16-bit values in the same way, coordinates (0, head, token,
// atom): a box is 64 values x box_heads heads of one token, one atom, and ends at the token's last head.
bool encode_tmap_heads(void* tmap_out, const void* base, uint32_t atoms, uint64_t heads, uint64_t tokens,
                       uint32_t box_heads, std::string* why);

}  // namespace dsa

// Per-translation-unit device status words (read and clear; 0xFFFFFFFF on error).
uint32_t dsa_status_read_clear_indexer();
uint32_t dsa_status_read_clear_topk();
uint32_t dsa_status_read_clear_attn();
uint32_t dsa_status_read_clear_cache();
uint32_t dsa_status_read_clear_prolog();
uint32_t dsa_status_read_clear_rows();
uint32_t dsa_status_read_clear_attn_e2m1();
uint32_t dsa_status_read_clear_index_keys();
uint32_t dsa_status_read_clear_attn_block();
uint32_t dsa_status_read_clear_block_topk();
