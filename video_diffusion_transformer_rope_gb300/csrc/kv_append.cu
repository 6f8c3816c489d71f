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

#include "kv8.cuh"
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

// 8 channels of a row, d/8 lanes together: the norm, if there is one, and the turn of their pairs by cs[0..3].
template <int D>
__device__ __forceinline__ void norm_rotate(float (&f)[8], bool norm, const float (&w)[8], float eps, const float2* cs) {
  if (norm) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float inv = rsqrtf(sq * (1.f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv * w[i];
  }
  const float4* c4 = reinterpret_cast<const float4*>(cs);
  const float4 c01 = c4[0], c23 = c4[1];
  const float cn[4] = {c01.x, c01.z, c23.x, c23.z}, sn[4] = {c01.y, c01.w, c23.y, c23.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u = f[2 * i], v = f[2 * i + 1];
    f[2 * i] = fmaf(u, cn[i], -v * sn[i]);
    f[2 * i + 1] = fmaf(u, sn[i], v * cn[i]);
  }
}

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
  // by, ny: which of how many blocks share the heads of these tokens
  __device__ __forceinline__ void init(const AppendParams& p, int row0, int by, int ny) {
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
    step = (kThreads / kLanes) * ny;
    j = 0;
    h = by * (kThreads / kLanes) + threadIdx.x / kLanes;
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
        norm_rotate<D>(f, norm, w, p.eps, &cs[t][lane * 4]);
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

// Every sequence's range is looked at (a row's look-up sees only its own), 32 of them by a warp of each of n blocks:
// many blocks for many sequences.
__device__ __forceinline__ void look_at_ranges(const AppendParams& p, int block, int n) {
  bool bad = false;
  for (long long s = block * 32ll + (threadIdx.x & 31); s < p.S; s += n * 32ll) {
    const int begin = load_i32(p.cu + s), end = load_i32(p.cu + s + 1);
    bad = bad || begin < 0 || end < begin || end > p.rows;
  }
  if (bad) atomicOr(&g_error_word, kErrLength);
}

// Cosine and sine of channel pair `pr` at position x of its axis.
__device__ __forceinline__ float2 cos_sin(const AppendParams& p, int pr, unsigned x) {
  const int hi = static_cast<int>((static_cast<unsigned long long>(x) * p.turn[pr]) >> 32);        // turns in [-1/2, 1/2) * 2^32
  float sn, cn;
  sincospif(static_cast<float>(hi) * 0x1p-31f, &sn, &cn);
  return make_float2(cn, sn);
}

template <typename T, int D, int kTok, int kKind>
__device__ __forceinline__ void append_rows(const AppendParams& p, int row0, int by, int ny) {
  __shared__ __align__(16) float2 cs[kTok][D / 2];
  __shared__ long long s_at[kTok];    // where each token goes: cache offset, or grid token for q; < 0: nowhere
  __shared__ int s_axis[kTok][3];     // its (t, h, w)
  const int tid = threadIdx.x;
  RowWalk<T, D, kTok, kKind> rows;
  rows.init(p, row0, by, ny);
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
  if (kKind == 1 && by == 0 && tid >= kThreads - 32) look_at_ranges(p, blockIdx.x, gridDim.x);
  __syncthreads();
  if (kKind < 2) {
    for (int i = tid; i < kTok * (D / 2); i += kThreads) {
      const int j = i / (D / 2), pr = i % (D / 2);
      cs[j][pr] = cos_sin(p, pr, static_cast<unsigned>(s_axis[j][pr < p.half_t ? 0 : (pr < p.half_t + p.half_h ? 1 : 2)]));
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
    append_rows<T, D, kTok, 1>(p, row0, blockIdx.y, gridDim.y);
  else if (blockIdx.z == 1)
    append_rows<T, D, kTok, 2>(p, row0, blockIdx.y, gridDim.y);
  else
    append_rows<T, D, kTok, 0>(p, row0, blockIdx.y, gridDim.y);
}

// ------------------------------------------------------------------------------------------ into an 8-bit cache
// The scale of a block of 16 tokens and a head comes from all of its new values, so a warp takes the whole block of
// a head: its rows are loaded, normed and turned into registers (d/8 lanes a row), their largest |x| is a shuffle
// maximum, and the codes leave, 8 bytes a lane.  Where older tokens of the block must be rounded again, the same warp
// does that too, so nothing is shared between warps.
//
// Bound: DRAM, and nearly the issue slots (the rows are worked out twice, kv_append's once): 21600 tokens of 3 x 40 heads,
// 1.11 GB, 227 us, 4.9 TB/s, 73 % of a plain copy's rate.
//
// A thread block takes the blocks ("segments") of the cache whose first new token is among its kRows (16 or fewer) rows,
// for keys or values; a segment may reach up to 15 rows further.  One warp looks up those rows, one to a lane.
constexpr int kResident8 = 7;

// The 8 channels of a lane as pairs of pairs: even channels (0, 2), (4, 6), odd channels (1, 3), (5, 7), so that the turn of
// two channel pairs is two packed instructions for each of their channels.
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& x, uint64_t (&even)[2], uint64_t (&odd)[2]) {
  const float2 a = unpack2<T>(x.x), b = unpack2<T>(x.y), c = unpack2<T>(x.z), d = unpack2<T>(x.w);
  even[0] = f32x2(a.x, b.x);
  even[1] = f32x2(c.x, d.x);
  odd[0] = f32x2(a.y, b.y);
  odd[1] = f32x2(c.y, d.y);
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float largest2(uint64_t a, float m) {
  float x, y;
  f32x2_split(a, x, y);
  return fmax3(m, fabsf(x), fabsf(y));
}
// Codes of 8 channels in order.
__device__ __forceinline__ uint2 encode_pairs(const uint64_t (&even)[2], const uint64_t (&odd)[2]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float a, b, c, d;
    f32x2_split(even[i], a, b);
    f32x2_split(odd[i], c, d);
    w[i] = encode4(a, c, b, d);
  }
  return make_uint2(w[0], w[1]);
}

struct Segment8 {
  int row, count;              // first row in the window, new tokens
  int older;                   // tokens of the block ahead of them
  int fits;                    // bit i: the i-th token has a place
  long long at, scale;         // cache offset of the block's first token, offset of its scales (head 0)
};

// The last s in [0, S) with cu[s] <= r, by one lane alone (find_sequence has the conditions).
__device__ __forceinline__ int find_sequence_lane(const int* cu, int S, int r) {
  int lo = 0, n = S;
  while (n > 1) {
    const int half = n / 2;
    if (load_i32(cu + lo + half) <= r) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return lo;
}

// cos_sin with the angle reduced to an eighth of a turn before it becomes a float: within 2^-28 turns, not 2^-26.  A code has 4
// bits, and a value that rounds to its neighbour is off by an eighth of itself, so here each bit of the angle halves
// the number of codes that differ from those of exact keys.
__device__ __forceinline__ float2 cos_sin8(const AppendParams& p, int pr, unsigned x) {
  const unsigned long long frac = static_cast<unsigned long long>(x) * p.turn[pr];       // turns * 2^64
  const unsigned quarter = static_cast<unsigned>((frac + (1ull << 61)) >> 62);
  const int rest = static_cast<int>(static_cast<long long>(frac - (static_cast<unsigned long long>(quarter) << 62)) >> 30);     // [-1/8, 1/8] turns * 2^34
  float sn, cn;
  sincospif(static_cast<float>(rest) * 0x1p-33f, &sn, &cn);
  const float a = quarter & 1 ? sn : cn, b = quarter & 1 ? cn : sn;
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

template <typename T, int D, bool kKeys, int kRows>
__device__ __forceinline__ void append_blocks(const AppendParams& p, int bx, int nx, int by, int ny) {
  constexpr int kLanes = D / 8;                  // of a row
  constexpr int kPer = 32 / kLanes;              // rows of a warp's step
  constexpr int kSteps = kBlock8 / kPer;
  constexpr int kWindow = kRows + kBlock8 - 1;
  static_assert(kWindow <= 32, "a lane looks up a row");
  __shared__ __align__(16) float s_cos[kKeys ? kWindow : 1][D / 2], s_sin[kKeys ? kWindow : 1][D / 2];
  __shared__ Segment8 segs[kRows];
  __shared__ int s_axis[kWindow][3];
  __shared__ int s_count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = bx * kRows;

  if (warp == 0) {
    const int r = row0 + lane;
    int seq = 0, begin = 0, end = 0, slot = 0, page = -1, axis[3] = {0, 0, 0};
    bool mine = false, fits = false, bad_page = false, bad_position = false;
    if (lane < kWindow && r < p.rows) {
      seq = find_sequence_lane(p.cu, p.S, r);
      begin = load_i32(p.cu + seq);
      end = load_i32(p.cu + seq + 1);
      mine = begin >= 0 && end >= begin && end <= p.rows && r >= begin && r < end;      // broken ranges: look_at_ranges
    }
    if (mine) {
      const long long c = static_cast<long long>(load_i32(p.kv_len + seq)) - (end - begin) + (r - begin);
      const long long pos = c + (p.pos_offset ? load_i32(p.pos_offset + seq) : 0);
      if (c < 0 || c >= static_cast<long long>(p.max_pages) * p.P) {
        mine = false;
        bad_position = true;
      } else {
        const int pg = static_cast<int>(c / p.P);
        slot = static_cast<int>(c - static_cast<long long>(pg) * p.P);
        page = load_i32(p.table + seq * p.table_stride + pg);
        bad_page = page < 0 || page >= p.num_pages;
        fits = pos >= 0 && pos < static_cast<long long>(p.T) * p.Hg * p.Wg;
        bad_position = !fits;
        if (fits) {
          const int area = p.Hg * p.Wg;
          axis[0] = static_cast<int>(pos / area);
          const int rest = static_cast<int>(pos - static_cast<long long>(axis[0]) * area);
          axis[1] = rest / p.Wg;
          axis[2] = rest - axis[1] * p.Wg;
        }
      }
    }
    if (lane < kRows && (bad_page || bad_position)) atomicOr(&g_error_word, (bad_page ? kErrPage : 0u) | (bad_position ? kErrPosition : 0u));
    if (lane < kWindow)
#pragma unroll
      for (int i = 0; i < 3; ++i) s_axis[lane][i] = axis[i];
    const unsigned placed = __ballot_sync(0xffffffffu, fits);
    // a segment starts with its sequence's first new row or a block's first token (so does index 0, whatever is before it)
    const bool leads = mine && lane < kRows && !bad_page && (slot % kBlock8 == 0 || r == begin);
    const unsigned all = __ballot_sync(0xffffffffu, leads);
    if (leads) {
      Segment8& g = segs[__popc(all & ((1u << lane) - 1))];
      g.row = lane;
      g.older = slot % kBlock8;
      g.count = min(min(kBlock8 - g.older, p.P - slot), end - r);
      g.fits = static_cast<int>((placed >> lane) & ((1u << g.count) - 1));
      const long long tok = slot - g.older;
      g.at = kKeys ? page * p.kc_page + tok * p.kc_token : page * p.vc_page + tok * p.vc_token;
      const Scales8& sc = p.scales;
      g.scale = kKeys ? page * sc.k_page + tok / kBlock8 * sc.k_block : page * sc.v_page + tok / kBlock8 * sc.v_block;
    }
    if (lane == 0) s_count = __popc(all);
  }
  if (kKeys && by == 0 && warp == 1) look_at_ranges(p, bx, nx);
  __syncthreads();
  const int count = s_count;
  if (count == 0) return;
  if (kKeys) {
    const int from = segs[0].row, to = segs[count - 1].row + segs[count - 1].count;
    for (int i = from * (D / 2) + tid; i < to * (D / 2); i += kThreads) {
      const int j = i / (D / 2), pr = i % (D / 2);
      const float2 t = cos_sin8(p, pr, static_cast<unsigned>(s_axis[j][pr < p.half_t ? 0 : (pr < p.half_t + p.half_h ? 1 : 2)]));
      s_cos[j][pr] = t.x;
      s_sin[j][pr] = t.y;
    }
    __syncthreads();
  }

  const T* src = static_cast<const T*>(kKeys ? p.k : p.v);
  const long long src_row = kKeys ? p.k_row : p.v_row, src_head = kKeys ? p.k_head : p.v_head;
  const long long dst_token = kKeys ? p.kc_token : p.vc_token, dst_head = kKeys ? p.kc_head : p.vc_head;
  uint8_t* cache = static_cast<uint8_t*>(kKeys ? p.k_cache : p.v_cache);
  uint8_t* scale = kKeys ? p.scales.k : p.scales.v;
  const long long scale_head = kKeys ? p.scales.k_head : p.scales.v_head;
  const int ch = lane % kLanes, sub = lane / kLanes;
  const bool norm = kKeys && p.k_norm;
  uint64_t w_even[2], w_odd[2];
  unpack_pairs<T>(norm ? load_b128(static_cast<const T*>(p.k_norm) + ch * 8) : make_uint4(0u, 0u, 0u, 0u), w_even, w_odd);
  bool past = false;
  for (int t = by * (kThreads / 32) + warp; t < count * p.Hkv; t += ny * (kThreads / 32)) {
    const int si = t / p.Hkv, h = t - si * p.Hkv;
    const Segment8 g = segs[si];
    const T* from = src + static_cast<long long>(row0 + g.row) * src_row + h * src_head + ch * 8;
    uint8_t* to = cache + g.at + h * dst_head + ch * 8;
    uint8_t* to_scale = scale + g.scale + h * scale_head;
    uint4 x[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int j = i * kPer + sub;
      x[i] = (g.fits >> j & 1) ? load_b128(from + j * src_row) : make_uint4(0u, 0u, 0u, 0u);      // 0 or NaN below: no maximum
    }
    const int e_old = g.older ? scale_exponent(*to_scale) : kMinExp8;
    // Twice over the rows, as they were read: their largest value, then their codes.  Held in between the fp32 values
    // would take twice the registers, and half as many warps would be loading.
    float inv_rms[kSteps];
    // a row times the norm's weights, turned; its rsqrt(mean square) is left to the caller
    auto turned = [&](int i, uint64_t (&even)[2], uint64_t (&odd)[2]) {
      if (norm) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          even[c] = fmul2(even[c], w_even[c]);
          odd[c] = fmul2(odd[c], w_odd[c]);
        }
      }
      const int j = min(g.row + i * kPer + sub, kWindow - 1);
      const float4 cn = *reinterpret_cast<const float4*>(&s_cos[j][ch * 4]), sn = *reinterpret_cast<const float4*>(&s_sin[j][ch * 4]);
      const uint64_t c2[2] = {f32x2(cn.x, cn.y), f32x2(cn.z, cn.w)}, s2[2] = {f32x2(sn.x, sn.y), f32x2(sn.z, sn.w)};
      const uint64_t n2[2] = {f32x2(-sn.x, -sn.y), f32x2(-sn.z, -sn.w)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint64_t u = even[c], v = odd[c];
        even[c] = ffma2(u, c2[c], fmul2(v, n2[c]));
        odd[c] = ffma2(u, s2[c], fmul2(v, c2[c]));
      }
    };
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i * kPer >= g.count) break;                   // a single token fills one row in 16
      uint64_t even[2], odd[2];
      unpack_pairs<T>(x[i], even, odd);
      float scale = 1.f;
      if (kKeys) {
        if (norm) {
          float a, b;
          f32x2_split(ffma2(odd[1], odd[1], ffma2(even[1], even[1], ffma2(odd[0], odd[0], fmul2(even[0], even[0])))), a, b);
          float sq = a + b;
#pragma unroll
          for (int o = D / 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
          scale = rsqrtf(sq * (1.f / D) + p.eps);
        }
        turned(i, even, odd);
      }
      inv_rms[i] = scale;
      const float m = largest2(odd[1], largest2(odd[0], largest2(even[1], largest2(even[0], 0.f))));
      top = fmaxf(top, m * scale);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    past |= top > 448.f * 128.f;
    const int e = max(e_old, block_exponent(top));
    const float inv = two_to(-e);
    if (g.older && e > e_old) {
      const float down = two_to(e_old - e);
      for (int j = sub; j < g.older; j += kPer) {
        uint2* q = reinterpret_cast<uint2*>(to + j * dst_token);
        float v[8];
        decode8(*q, v);
        *q = make_uint2(encode4(v[0] * down, v[1] * down, v[2] * down, v[3] * down),
                        encode4(v[4] * down, v[5] * down, v[6] * down, v[7] * down));
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i * kPer >= g.count) break;
      const int j = i * kPer + sub;
      asm volatile("" : "+r"(x[i].x), "+r"(x[i].y), "+r"(x[i].z), "+r"(x[i].w));      // worked out anew, not held
      uint64_t even[2], odd[2];
      unpack_pairs<T>(x[i], even, odd);
      if (kKeys) turned(i, even, odd);
      const float by = inv_rms[i] * inv;
      const uint64_t by2 = f32x2(by, by);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        even[c] = fmul2(even[c], by2);
        odd[c] = fmul2(odd[c], by2);
      }
      if (g.fits >> j & 1) *reinterpret_cast<uint2*>(to + (g.older + j) * dst_token) = encode_pairs(even, odd);
    }
    if (lane == 0 && g.fits) *to_scale = static_cast<uint8_t>(e + 127);
  }
  if (past) atomicOr(&g_error_word, kErrRange8);
}

// The blocks of keys, which take longest, first; then those of values and of queries.  (Side by side, so that issue slots
// and memory are wanted at the same time, 21600 tokens of 3 x 40 heads take 286 us, not 264.)
template <typename T, int D, int kTok, int kRows>
__global__ void __launch_bounds__(kThreads, kResident8)
kv_append8(const __grid_constant__ AppendParams p, const int nx, const int ny, const int qx) {
  wait_for_earlier_work();
  const int b = blockIdx.x, each = nx * ny;
  if (b < each)
    append_blocks<T, D, true, kRows>(p, b % nx, nx, b / nx, ny);
  else if (b < 2 * each)
    append_blocks<T, D, false, kRows>(p, (b - each) % nx, nx, (b - each) / nx, ny);
  else
    append_rows<T, D, kTok, 0>(p, (b - 2 * each) % qx * kTok, (b - 2 * each) / qx, (gridDim.x - 2 * each) / qx);
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

template <typename T, int D, int kTok, int kRows>
cudaError_t launch8_tok(const AppendParams& p, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8), kWarps = kThreads / 32;
  const int nx = (p.rows - 1) / kRows + 1, qx = p.Hq > 0 ? (p.rows - 1) / kTok + 1 : 0;
  // few rows: the heads over blocks too, as in launch_tok
  int ny = 1, qy = 1;
  const int most = (p.Hkv * kRows + kWarps - 1) / kWarps, q_most = (kTok * p.Hq + kGroups - 1) / kGroups;
  while (ny < most && static_cast<long long>(nx) * ny < sms) ny *= 2;
  while (qy < q_most && static_cast<long long>(qx) * qy < 2ll * sms) qy *= 2;
  ny = ny < most ? ny : most;
  qy = qy < q_most || qx == 0 ? qy : q_most;
  const long long blocks = 2ll * nx * ny + static_cast<long long>(qx) * qy;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append8<T, D, kTok, kRows>, p, nx, ny, qx);
}
template <typename T, int D>
cudaError_t launch8(const AppendParams& p, int sms, cudaStream_t stream) {
  // Few rows: blocks of 4 rows, which have fewer angles to work out one after the other; but of a chunk one in four of them has
  // a segment.  us with 4 and 16 rows to a block, single tokens of many sequences | one sequence's chunk, d = 128:
  //   kv heads   48 tokens                 256 tokens                 512 tokens
  //      8       4.9   6.2 | 7.3   8.7      7.1   9.4 |  9.3  10.0     9.9  12.5 | 10.0  10.4
  //     12       5.1   6.7 | 7.7   9.2      7.7  10.2 |  8.9   9.6    12.3  14.6 | 13.3  10.2
  //     40       7.2   8.5 | 8.0   9.4     17.2  20.0 | 17.0  13.4    31.1  33.5 | 27.1  17.0
  if (static_cast<long long>(p.rows) * p.Hkv <= 4096) return launch8_tok<T, D, 2, 4>(p, sms, stream);
  // queries by two tokens as in launch while there are few (21600 tokens by fours: 233, by twos 259 us)
  return p.rows <= 1024 ? launch8_tok<T, D, 2, 16>(p, sms, stream) : launch8_tok<T, D, 4, 16>(p, sms, stream);
}

}  // namespace

cudaError_t launch_append8(const AppendParams& p, int d, int dtype, int sms, cudaStream_t stream) {
  note_launch();
  if (dtype == 0) return d == 128 ? launch8<__nv_bfloat16, 128>(p, sms, stream) : launch8<__nv_bfloat16, 64>(p, sms, stream);
  return d == 128 ? launch8<__half, 128>(p, sms, stream) : launch8<__half, 64>(p, sms, stream);
}

cudaError_t launch_append(const AppendParams& p, int d, int dtype, int sms, cudaStream_t stream) {
  note_launch();
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, sms, stream) : launch<__nv_bfloat16, 64>(p, sms, stream);
  return d == 128 ? launch<__half, 128>(p, sms, stream) : launch<__half, 64>(p, sms, stream);
}

cudaError_t read_and_clear_error_word_append(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
