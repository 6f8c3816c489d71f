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
// then the (token, head) rows are walked by groups of d/8 lanes, kUnroll rows in flight per lane (6.2 TB/s
// of reads and writes, 92 % of a plain copy's: 21600 tokens of 3 x 40 heads, 1.33 GB, 212 us; 3120 tokens of
// 3 x 12 heads, 58 MB, 12.4 us, of which 2.8 are what 8 tokens take).
//
// Angles: FP64 units are scarce, so the turn per position, omega / 2 pi mod 1, is a 64-bit fixed-point
// fraction and pos * turn mod 2^64 the reduced angle, with no error of its own: what is left is the turn's
// (worked out by the host in double: 2.3e-17 turns at most over usual sections and thetas, times the position:
// 2^-26 turns at 5e8) and the conversion of the top 32 bits to a float of 24 for sincospi (2^-26 turns, 1e-7 radians).
//
// Arithmetic is fp32 and rounds once, to the call's type (half a step: 2^-8 of the value in bf16,
// 2^-11 in fp16): q and k leave as the cache and the attention calls hold them.  The self-attention, which rotates
// within one call, keeps bf16 inputs in fp16 instead: on the same 264 tokens its largest error against 64 bits
// is 1.5e-3 in out and 1.6e-4 in lse, through the cache 3.0e-3 and 1.0e-3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_common.cuh"

namespace vdx {
namespace {

constexpr int kThreads = 128;
constexpr int kResident = 9;        // blocks that a multiprocessor holds at least (56 registers a thread)
// Rows that each group has in flight in a block of kTok tokens.  Small blocks and few rows in flight waste
// little where the heads do not divide by a batch of rows, and leave registers for more blocks: 3 rows of
// 128 threads and 4 tokens a block take 14.0 us for 3120 tokens of 3 x 12 heads and 215 us for 21600 of
// 3 x 40; 4 rows of 256 threads and 8 tokens 17.5 and 220 us; 8 rows 24 and 303 us.
template <int kTok>
constexpr int kRowsInFlight = kTok > 2 ? 3 : 1;

// The (token, head) rows of one tensor of a block's tokens, walked by groups of d/8 lanes, kUnroll
// loads in flight per lane.  One instance per kind (0 q, 1 k, 2 v), so a row carries no choices: with
// everything in one loop the selects and 64-bit addresses cost as much issue time as the memory
// takes (281 against 240 us for 21600 tokens of 3 x 40 heads).
template <typename T, int D, int kTok, int kKind>
struct RowWalk {
  static constexpr int kUnroll = kRowsInFlight<kTok>;
  const T* src;
  T* dst;                      // base of q_out or the cache
  long long src_row, src_head, dst_head, dst_row;
  int heads, step, rows;
  int j, h;                    // token and head of the next row
  uint4 weights;               // this lane's 8 of the norm's, if there is one
  uint4 x[kUnroll];
  int tok[kUnroll], head[kUnroll];      // tok < 0: past the block's rows
  __device__ __forceinline__ void init(const AppendParams& p, int row0) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    heads = kKind == 0 ? p.Hq : p.Hkv;
    src = static_cast<const T*>(kKind == 0 ? p.q : (kKind == 1 ? p.k : p.v)) + lane * 8;
    dst = static_cast<T*>(kKind == 0 ? p.q_out : (kKind == 1 ? p.k_cache : p.v_cache)) + lane * 8;
    src_row = kKind == 0 ? p.q_row : (kKind == 1 ? p.k_row : p.v_row);
    src_head = kKind == 0 ? p.q_head : (kKind == 1 ? p.k_head : p.v_head);
    dst_head = kKind == 0 ? p.q_out_head : (kKind == 1 ? p.kc_head : p.vc_head);
    dst_row = p.q_out_row;
    const void* norm = kKind == 0 ? p.q_norm : p.k_norm;
    weights = make_uint4(0u, 0u, 0u, 0u);
    if (kKind < 2 && norm) weights = load_b128(static_cast<const T*>(norm) + lane * 8);
    src += row0 * src_row;
    if (kKind == 0) dst += row0 * dst_row;
    rows = heads > 0 ? min(kTok, p.rows - row0) : 0;
    step = (kThreads / kLanes) * gridDim.y;
    j = 0;
    h = blockIdx.y * (kThreads / kLanes) + threadIdx.x / kLanes;
    wrap();
  }
  __device__ __forceinline__ void wrap() {
    while (h >= heads && j < rows) {
      h -= heads;
      ++j;
    }
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      tok[e] = j < rows ? j : -1;
      head[e] = h;
      x[e] = make_uint4(0u, 0u, 0u, 0u);
      if (j < rows) x[e] = load_b128(src + j * src_row + h * src_head);
      h += step;
      wrap();
    }
  }
  // The whole warp decides: its groups' rows run out at different times, and the norm's shuffles
  // take every lane.
  __device__ __forceinline__ bool more() const { return __any_sync(0xffffffffu, tok[0] >= 0); }
  // at[t]: where token t goes (an offset in the cache; q: a grid token), negative: nowhere.
  __device__ __forceinline__ void finish(const AppendParams& p, const float2 (*cs)[D / 2], const long long* at, bool norm) {
    const int lane = threadIdx.x % (D / 8);
    float w[8];
    if (kKind < 2) unpack8<T>(weights, w);
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      uint4 y = x[e];
      const int t = max(tok[e], 0);
      if (kKind < 2) {
        float f[8];
        unpack8<T>(x[e], f);
        if (norm) {
          float sq = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
#pragma unroll
          for (int o = D / 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
          const float inv = rsqrtf(sq * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= inv * w[i];
        }
        const float4* c4 = reinterpret_cast<const float4*>(&cs[t][lane * 4]);
        const float4 c01 = c4[0], c23 = c4[1];
        const float cn[4] = {c01.x, c01.z, c23.x, c23.z}, sn[4] = {c01.y, c01.w, c23.y, c23.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = f[2 * i], v = f[2 * i + 1];
          f[2 * i] = fmaf(u, cn[i], -v * sn[i]);
          f[2 * i + 1] = fmaf(u, sn[i], v * cn[i]);
        }
        y = pack8<T>(f);
      }
      if (tok[e] < 0 || at[t] < 0) continue;
      T* to = dst + (kKind == 0 ? t * dst_row : at[t]) + head[e] * dst_head;
      // 16 bytes a lane, in no order among rows: two rows for one slot leave pieces of both.  The next call
      // reads it: no streaming hint.
      *reinterpret_cast<uint4*>(to) = y;
    }
  }
};

template <typename T, int D, int kTok, int kKind>
__device__ __forceinline__ void append_rows(const AppendParams& p, int row0) {
  __shared__ __align__(16) float2 cs[kTok][D / 2];
  __shared__ long long s_at[kTok];    // where each token goes: cache offset, or grid token for q; < 0: nowhere
  __shared__ int s_axis[kTok][3];     // its (t, h, w)
  const int tid = threadIdx.x;
  RowWalk<T, D, kTok, kKind> rows;
  rows.init(p, row0);
  rows.load();

  for (int j = tid >> 5; j < kTok; j += kThreads / 32) {     // one warp per token
    const int r = row0 + j;
    long long at = -1;
    int frame = 0, row = 0, col = 0;
    if (r < p.rows) {
      const int s = find_sequence(p.cu, p.S, r);
      const int begin = load_i32(p.cu + s), end = load_i32(p.cu + s + 1);
      if (begin < 0 || end < begin || end > p.rows) {
        // n would count rows that are not there, and the tokens would land on those before them
        if ((tid & 31) == 0) atomicOr(&g_error_word, kErrLength);
      } else if (r >= begin && r < end) {
        const long long c = static_cast<long long>(load_i32(p.kv_len + s)) - (end - begin) + (r - begin);
        const long long pos = c + (p.pos_offset ? load_i32(p.pos_offset + s) : 0);
        if (c < 0 || c >= static_cast<long long>(p.max_pages) * p.P || pos < 0 ||
            pos >= static_cast<long long>(p.T) * p.Hg * p.Wg) {
          if ((tid & 31) == 0) atomicOr(&g_error_word, kErrPosition);
        } else {
          const int area = p.Hg * p.Wg;
          frame = static_cast<int>(pos / area);
          const int rest = static_cast<int>(pos - static_cast<long long>(frame) * area);
          row = rest / p.Wg;
          col = rest - row * p.Wg;
          at = pos;
        }
        if (kKind != 0 && at >= 0) {
          at = -1;
          const int pg = static_cast<int>(c / p.P), slot = static_cast<int>(c - static_cast<long long>(pg) * p.P);
          const int page = load_i32(p.table + s * p.table_stride + pg);
          if (page < 0 || page >= p.num_pages) {
            if ((tid & 31) == 0) atomicOr(&g_error_word, kErrPage);
          } else {
            at = kKind == 1 ? page * p.kc_page + slot * p.kc_token : page * p.vc_page + slot * p.vc_token;
          }
        }
      }
    }
    if ((tid & 31) == 0) {
      s_at[j] = at;
      s_axis[j][0] = frame;
      s_axis[j][1] = row;
      s_axis[j][2] = col;
    }
  }
  // Every sequence's range is looked at (a row's look-up sees only its own), 32 of them by a warp of each block:
  // many blocks for many sequences.
  if (kKind == 1 && blockIdx.y == 0 && tid >= kThreads - 32) {
    bool bad = false;
    for (long long s = blockIdx.x * 32ll + (tid & 31); s < p.S; s += gridDim.x * 32ll) {
      const int begin = load_i32(p.cu + s), end = load_i32(p.cu + s + 1);
      bad = bad || begin < 0 || end < begin || end > p.rows;
    }
    if (bad) atomicOr(&g_error_word, kErrLength);
  }
  __syncthreads();
  if (kKind < 2) {
    for (int i = tid; i < kTok * (D / 2); i += kThreads) {
      const int j = i / (D / 2), pr = i % (D / 2);
      const unsigned long long x = static_cast<unsigned>(s_axis[j][pr < p.half_t ? 0 : (pr < p.half_t + p.half_h ? 1 : 2)]);
      const int hi = static_cast<int>((x * p.turn[pr]) >> 32);        // turns in [-1/2, 1/2) * 2^32
      float sn, cn;
      sincospif(static_cast<float>(hi) * 0x1p-31f, &sn, &cn);
      cs[j][pr] = make_float2(cn, sn);
    }
    __syncthreads();
  }
  for (; rows.more(); rows.load()) rows.finish(p, cs, s_at, (kKind == 0 ? p.q_norm : p.k_norm) != nullptr);
}

template <typename T, int D, int kTok>
__global__ void __launch_bounds__(kThreads, kResident)
kv_append(const __grid_constant__ AppendParams p) {
  const int row0 = blockIdx.x * kTok;
  wait_for_earlier_work();
  // One tensor per block, q, k and v side by side (gridDim.z = 3): walked one after another they would
  // wait for memory three times over.  What a row reads depends on its number alone, so the first batch
  // is under way before the block has looked up its tokens' sequences and pages.
  if (blockIdx.z == 0)
    append_rows<T, D, kTok, 1>(p, row0);
  else if (blockIdx.z == 1)
    append_rows<T, D, kTok, 2>(p, row0);
  else
    append_rows<T, D, kTok, 0>(p, row0);
}

template <typename T, int D, int kTok>
cudaError_t launch_tok(const AppendParams& p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const int heads = p.Hq > p.Hkv ? p.Hq : p.Hkv;
  // Few tokens: split the heads over blocks too, until the device is covered (four blocks to a
  // multiprocessor) or a block's groups have one row each.  us with 2, 4 and 8 blocks to a multiprocessor: 256
  // tokens of 12 heads 3.9, 3.6, 3.4; 400 of 12 4.0, 3.9, 4.8; 256 of 40 7.3, 5.3, 5.7; 1100 of 4 4.6, 4.6, 6.7.
  const int blocks = (p.rows - 1) / kTok + 1, kinds = p.Hq > 0 ? 3 : 2;
  int ny = 1;
  const int most = (kTok * heads + kGroups - 1) / kGroups;
  while (ny < most && static_cast<long long>(blocks) * ny * kinds < 4ll * sms) ny *= 2;
  if (ny > most) ny = most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, ny, kinds);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append<T, D, kTok>, p);
}
template <typename T, int D>
cudaError_t launch(const AppendParams& p, int sms, cudaStream_t stream) {
  // Blocks of 2 tokens while the device holds all of them at once (912 tokens with q): each has half the work
  // in turn.  Past that 4 tokens share a block's look-ups.  us, 2 and 4 tokens to a block, d = 128:
  //   heads   256 tokens   700 tokens   900 tokens   1000 tokens   1560 tokens   3120 tokens
  //     4     2.8   3.7    3.3   4.7    3.7   4.3    4.7   4.3      5.8   5.2     9.6   8.6
  //    12     3.6   4.3    4.5   4.9    5.4   5.7    6.5   5.7      8.2   7.1    13.7  12.2
  //    40     5.3   5.6    8.7   9.3   10.3  11.8   12.7  11.9     19.7  17.1    43.6  36.4
  // (d = 64 the same up to 900; of 1100 to 2000 tokens, 4 and 40 heads are up to a tenth faster by twos).
  const long long pairs = ((p.rows - 1) / 2 + 1) * (p.Hq > 0 ? 3ll : 2ll);
  return pairs <= static_cast<long long>(kResident) * sms ? launch_tok<T, D, 2>(p, sms, stream) : launch_tok<T, D, 4>(p, sms, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int d, int dtype, int sms, cudaStream_t stream) {
  note_launch();
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, sms, stream) : launch<__nv_bfloat16, 64>(p, sms, stream);
  return d == 128 ? launch<__half, 128>(p, sms, stream) : launch<__half, 64>(p, sms, stream);
}

cudaError_t read_and_clear_error_word_append(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
