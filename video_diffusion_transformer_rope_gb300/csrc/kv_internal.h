// Internal interface between the C-ABI front end of the paged-cache and cross-attention calls
// (kv_capi.cu) and their kernels.  Not part of the public API.
#pragma once
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "vdx_internal.h"

namespace vdx {

// Error-word bits of these kernels (bits 0-2 are the self-attention's).
constexpr unsigned kErrPage = 8u;       // a page index outside the cache
constexpr unsigned kErrLength = 16u;    // a length or row range past its bound
constexpr unsigned kErrPosition = 32u;  // a token outside the position grid or its page table

// Append: one problem, validated.  Strides in elements.
struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  long long q_row, q_head, k_row, k_head, v_row, v_head, q_out_row, q_out_head;
  long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  const int* cu;
  const int* kv_len;
  const int* pos_offset;      // of causal_block > 0; nullptr: 0
  const int* table;
  long long table_stride;
  const void* q_norm;         // nullptr: no norm
  const void* k_norm;
  float eps;
  int rows, S, Hq, Hkv;       // Hq = 0: no q
  int P, num_pages, max_pages;
  int T, Hg, Wg;
  int half_t, half_h;         // rotary pairs of the t and h axes (the rest turn with w)
  // Turns per position of each channel pair as a 64-bit fixed-point fraction: omega / 2 pi mod 1.
  uint64_t turn[64];
};
cudaError_t launch_append(const AppendParams& p, int d, int dtype, int sms, cudaStream_t stream);

// Attention over a paged cache (table != nullptr) or over dense keys (one "page" of P = M tokens
// per batch entry).  Rows: sequence s owns tokens cu[s] .. cu[s+1]-1 of one packed q, or, with
// cu == nullptr, N tokens of its own batch entry.
struct KvParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;                  // [.., token, Hq, d] contiguous
  float* lse;                 // nullptr, or [lse_b][Hq][N]
  long long q_b, q_t, q_h;
  long long k_p, k_t, k_h, v_p, v_t, v_h;
  const int* cu;
  const int* kv_len;          // nullptr: P keys
  const int* pos_offset;      // of causal_block > 0; nullptr: 0
  const int* table;
  long long table_stride;
  int max_pages, num_pages, P;
  int S, N, Hq, Hkv, g;       // N: tokens per batch entry, or packed rows in all
  int max_q, max_kv;
  int causal_block;
  float scale_log2;           // scale * log2(e)
  // The plan (plan_attention): row blocks per (sequence, kv head) and key splits.
  int rows_kernel;            // 1: few rows per kv head (attn_rows.cu), 0: tiles (attn_tiles_sm103.cu)
  // A kv head's rows are its sequence's (token, query head of the group) pairs, token-major:
  // row R is token R / g, head hk * g + R % g.  Block blk owns rows blk * block_rows and up.
  int block_rows;
  int nblk, nsplit;
  int cluster;                // rows kernel: the splits are the CTAs of a cluster, which join them themselves
  int box_rows;               // tile kernel: keys of a partial copy box (8 to 64); 0: tiles end with their page
  int split_keys;             // keys (rows kernel) or key tiles (tile kernel) per split
  float* part_o;              // [unit][split][block_rows][d], unit = (s * Hkv + hk) * nblk + blk
  float2* part_ml;            // [unit][split][block_rows]: running maximum (log2 units) and sum
};

// Opt a kernel in to `bytes` of dynamic shared memory, once per device (a process-wide property of the
// function; asking again on every call costs a microsecond of host time).  `done`: the kernel's own flags.
template <typename Kernel>
inline cudaError_t allow_shared(Kernel* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// Fill the plan for `sms` multiprocessors; returns the workspace bytes it needs.
size_t plan_attention(KvParams* p, int d, int sms);

cudaError_t launch_attn_rows(const KvParams& p, int d, int dtype, cudaStream_t stream);
cudaError_t launch_attn_tiles(const KvParams& p, int d, int dtype, EncodeTiledFn encode, int sms,
                              cudaStream_t stream, const char** what);
cudaError_t launch_attn_combine(const KvParams& p, int d, int dtype, cudaStream_t stream);

// Read and reset the error words of these translation units (synchronous).
cudaError_t read_and_clear_error_word_append(unsigned int* word);
cudaError_t read_and_clear_error_word_rows(unsigned int* word);
cudaError_t read_and_clear_error_word_tiles(unsigned int* word);

// cuTensorMapEncodeTiled, looked up once (vdx_capi.cu).  Sets vdx_last_error on failure.
bool encode_tiled_fn(EncodeTiledFn* fn);

}  // namespace vdx
