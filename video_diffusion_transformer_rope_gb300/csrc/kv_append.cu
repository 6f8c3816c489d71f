// Appending a chunk of new tokens to a paged key/value cache: per-head RMS norm of q and k,
// 3D rotary positions, the write of k and v through the page table and of the rotated q, in one
// pass (after the vidax page, "vidax: A Unified JAX Framework for Video Generative Models on
// Accelerator Meshes", §2 "3D RoPE, 3D VAEs, and flash attention", for the rotation).
//
// For a row x of d channels:  x' = x * rsqrt(mean(x^2) + eps) * w,  then pairs (2i, 2i+1) turn by
// pos_axis(i) * theta^(-2j/S).  d/8 lanes hold one (token, head) row, 16 bytes each; the norm is
// a shuffle sum over them.
//
// Bound: DRAM (each element is read once and written once; ~10 flops).  A block takes kTok
// tokens.  The cosines and sines of a token are shared by all its heads, so the block's threads
// first work them out once per (token, pair) into shared memory, with the token's destination;
// then the (token, head) rows are walked by groups of d/8 lanes, kUnroll rows in flight per lane.
//
// Angles: a double product loses nothing here but FP64 units are scarce; instead the turn per
// position, omega / 2 pi mod 1, is a 64-bit fixed-point fraction, so pos * turn mod 2^64 is the
// angle reduced exactly for any position, and its top 32 bits feed sincospi (error < 2^-32 turns
// before the function's own).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_common.cuh"

namespace vdx {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <typename T, int D, int kTok>
__global__ void __launch_bounds__(kThreads)
kv_append(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;                 // lanes per (token, head) row
  constexpr int kGroups = kThreads / kLanes;
  __shared__ float2 cs[kTok][D / 2];
  __shared__ long long s_kdst[kTok], s_vdst[kTok];   // cache offsets (elements); < 0: not written
  __shared__ long long s_pos[kTok];                  // grid token; < 0: row skipped
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * kTok;

  for (int j = tid >> 5; j < kTok; j += kThreads / 32) {     // one warp per token
    const int r = row0 + j;
    long long pos = -1, kd = -1, vd = -1;
    if (r < p.rows) {
      const int s = find_sequence(p.cu, p.S, r);
      const int begin = __ldg(p.cu + s), end = __ldg(p.cu + s + 1);
      if (r >= begin && r < end) {
        const long long c = static_cast<long long>(__ldg(p.kv_len + s)) - (end - begin) + (r - begin);
        const long long at = c + (p.pos_offset ? __ldg(p.pos_offset + s) : 0);
        if (c < 0 || c >= static_cast<long long>(p.max_pages) * p.P || at < 0 ||
            at >= static_cast<long long>(p.T) * p.Hg * p.Wg) {
          if ((tid & 31) == 0) atomicOr(&g_error_word, kErrPosition);
        } else {
          pos = at;
          const int pg = static_cast<int>(c / p.P), slot = static_cast<int>(c - static_cast<long long>(pg) * p.P);
          const int page = __ldg(p.table + s * p.table_stride + pg);
          if (page < 0 || page >= p.num_pages) {
            if ((tid & 31) == 0) atomicOr(&g_error_word, kErrPage);
          } else {
            kd = page * p.kc_page + slot * p.kc_token;
            vd = page * p.vc_page + slot * p.vc_token;
          }
        }
      }
    }
    if ((tid & 31) == 0) {
      s_pos[j] = pos;
      s_kdst[j] = kd;
      s_vdst[j] = vd;
    }
  }
  __syncthreads();
  for (int i = tid; i < kTok * (D / 2); i += kThreads) {
    const int j = i / (D / 2), pr = i % (D / 2);
    const long long pos = s_pos[j];
    if (pos < 0) continue;
    const unsigned area = static_cast<unsigned>(p.Hg) * static_cast<unsigned>(p.Wg);
    const unsigned long long frame = static_cast<unsigned long long>(pos) / area;
    const unsigned rest = static_cast<unsigned>(pos - frame * area);
    const unsigned long long x = pr < p.half_t ? frame
                                 : (pr < p.half_t + p.half_h ? rest / static_cast<unsigned>(p.Wg)
                                                             : rest % static_cast<unsigned>(p.Wg));
    const int hi = static_cast<int>((x * p.turn[pr]) >> 32);          // turns in [-1/2, 1/2) * 2^32
    float sn, cn;
    sincospif(static_cast<float>(hi) * 0x1p-31f, &sn, &cn);
    cs[j][pr] = make_float2(cn, sn);
  }
  __syncthreads();

  const int lane = tid % kLanes;
  const int heads = p.Hq + 2 * p.Hkv;
  const int units = kTok * heads;
  const int stride = kGroups * gridDim.y;
  float wq[8], wk[8];
  load8<T>(p.q_norm, lane, wq);
  load8<T>(p.k_norm, lane, wk);
  for (int u0 = blockIdx.y * kGroups + tid / kLanes; u0 < units; u0 += stride * kUnroll) {
    uint4 x[kUnroll];
    T* dst[kUnroll];
    int kind[kUnroll];                          // 0 q, 1 k, 2 v, < 0 nothing
    int tok[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const int u = u0 + e * stride;
      kind[e] = -1;
      dst[e] = nullptr;
      tok[e] = 0;
      x[e] = make_uint4(0u, 0u, 0u, 0u);
      if (u >= units) continue;
      const int j = u / heads, h = u - j * heads;
      const long long r = row0 + j;
      tok[e] = j;
      const T* src = nullptr;
      if (s_pos[j] < 0) continue;
      if (h < p.Hq) {
        kind[e] = 0;
        src = static_cast<const T*>(p.q) + r * p.q_row + h * p.q_head;
        dst[e] = static_cast<T*>(p.q_out) + r * p.q_out_row + h * p.q_out_head;
      } else if (s_kdst[j] >= 0) {
        const int hk = h - p.Hq;
        if (hk < p.Hkv) {
          kind[e] = 1;
          src = static_cast<const T*>(p.k) + r * p.k_row + hk * p.k_head;
          dst[e] = static_cast<T*>(p.k_cache) + s_kdst[j] + hk * p.kc_head;
        } else {
          kind[e] = 2;
          src = static_cast<const T*>(p.v) + r * p.v_row + (hk - p.Hkv) * p.v_head;
          dst[e] = static_cast<T*>(p.v_cache) + s_vdst[j] + (hk - p.Hkv) * p.vc_head;
        }
      }
      if (kind[e] >= 0) x[e] = *(reinterpret_cast<const uint4*>(src) + lane);
    }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      // every lane of the warp takes part in the shuffles, whatever its row is
      float f[8];
      unpack8<T>(x[e], f);
      const bool is_q = kind[e] == 0;
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (kind[e] < 0) continue;
      uint4 y = x[e];
      if (kind[e] < 2) {
        if (is_q ? p.q_norm != nullptr : p.k_norm != nullptr) {
          const float inv = rsqrtf(sq * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * (is_q ? wq[i] : wk[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = cs[tok[e]][lane * 4 + i];
          const float a = f[2 * i], b = f[2 * i + 1];
          f[2 * i] = fmaf(a, c.x, -b * c.y);
          f[2 * i + 1] = fmaf(a, c.y, b * c.x);
        }
        y = pack8<T>(f);
      }
      *(reinterpret_cast<uint4*>(dst[e]) + lane) = y;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  constexpr int kTok = 4;
  const int heads = p.Hq + 2 * p.Hkv;
  // Few tokens: split the heads over blocks too, until the device is covered or a block's
  // groups have one row each.
  const int blocks = (p.rows + kTok - 1) / kTok;
  int ny = 1;
  const int most = (kTok * heads + kGroups - 1) / kGroups;
  while (ny < most && static_cast<long long>(blocks) * ny < 304) ny *= 2;
  if (ny > most) ny = most;
  kv_append<T, D, kTok><<<dim3(blocks, ny), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int d, int dtype, cudaStream_t stream) {
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, stream) : launch<__nv_bfloat16, 64>(p, stream);
  return d == 128 ? launch<__half, 128>(p, stream) : launch<__half, 64>(p, stream);
}

cudaError_t read_and_clear_error_word_append(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
