// The weight that each cached key gathers from the rows of a call (what eviction goes by):
//
//     w[c] = (c < len - n ? decay * w[c] : 0) + sum over rows r that see c of 2^(s_rc * scale*log2(e) - lse_r*log2(e))
//
// for a kv head's rows r, the (token, query head of its group) pairs; lse comes from the attention call.
//
// This file, few rows: bound by DRAM, which each key crosses once (its value is not needed), so K streams as in attn_rows.cu:
// a warp takes 32 keys at a time through a ring of its own, S^T = K Q^T by m16n8k16 products with the keys on the
// 16-wide side, and a key's sum over its rows ends as a shuffle over four lanes.  Nothing is shared between warps and
// each w is written by one lane: the same call gives the same bits (48 tokens over 8-33 thousand keys of 8 heads in 8
// bits, 1.14 GB: 178 us, 6.4 TB/s, 96 % of a plain copy's rate; with 16 keys a step 327 us, as many
// look-ups and shuffles served half the keys).  More than 32 rows: weigh_tiles_sm103.cu.
#include <cstdint>

#include "kv_mma.cuh"

namespace vdx {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;        // keys of one stage, a lane each
constexpr int kStages = 3;

template <typename T, int D, int kNT, bool k8>
__global__ void __launch_bounds__(kWarps * 32, 2)
weigh_rows(const __grid_constant__ WeighParams wp) {
  using M = std::conditional_t<k8, __half, T>;         // what the products take (attn_rows8.cu)
  constexpr int kElem = k8 ? 1 : 2;
  constexpr int kRowBytes = D * kElem;
  constexpr int kChunks = kRowBytes / 16;              // 16-byte chunks of a key
  constexpr int kTileBytes = kKeys * kRowBytes;
  constexpr int kPer = 32 / kChunks;                   // rows that the lanes copy at once
  const KvParams& p = wp.kv;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, c4 = lane & 3;
  wait_for_earlier_work();

  const int z = blockIdx.x % wp.nsplit;
  const int unit = blockIdx.x / wp.nsplit;
  const int hk = unit % p.Hkv, s = unit / p.Hkv;
  const SeqInfo sq = sequence_info(p, s, threadIdx.x == 0 && z == 0);
  const int rows = min(sq.n, p.max_q) * p.g;            // at most 8 * kNT
  if (rows == 0) return;                                // its entries stay as they are
  const long long lo64 = static_cast<long long>(z) * wp.split_keys;
  const int lo = static_cast<int>(min(lo64, static_cast<long long>(sq.len)));
  const int hi = static_cast<int>(min(lo64 + wp.split_keys, static_cast<long long>(sq.len)));

  constexpr int step = kKeys * kWarps;
  const uint32_t ring = smem_addr(smem) + warp * kStages * kTileBytes;
  const int k_first = lo + kKeys * warp;
  const int nblocks = k_first < hi ? (hi - k_first + step - 1) / step : 0;
  const int* table = p.table + static_cast<long long>(s) * p.table_stride;
  const int ch = lane % kChunks, r_in = lane / kChunks;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + hk * p.k_h * kElem + ch * 16;
  const uint8_t* kscale = p.scales.k + hk * p.scales.k_head;
  float* w = wp.w + s * wp.w_seq + hk * wp.w_head;
  const int old_to = sq.len - sq.n;                     // keys below were there before the call
  auto swizzle = [](int c, int r) { return kRowBytes == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); };

  // This lane's key of the block to be copied next: entry of the page table and token in the page; its page, when it has come.
  int pg = 0, off = 0, page = 0;
  if (nblocks > 0) {
    pg = (k_first + lane) / p.P;
    off = k_first + lane - pg * p.P;
    if (k_first + lane < hi) page = load_i32(table + pg);
  }
  // Scales and weights so far of the blocks being copied, oldest first: those of this lane's key
  int exps[kStages];
  float old[kStages];
  auto copy_block = [&](int i) {
    const int key = k_first + i * step + lane;
    const bool there = key < hi, ok = there && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
    if (there && !ok) atomicOr(&g_error_word, kErrPage);              // reads as zeros
    long long at = -1;
    exps[kStages - 1] = 127;
    if (ok) {
      at = (page * p.k_p + off * p.k_t) * kElem;
      if (k8) exps[kStages - 1] = kscale[page * p.scales.k_page + off / kBlock8 * p.scales.k_block];
    }
    old[kStages - 1] = there && key < old_to ? w[key] : 0.f;
    off += step;
    while (off >= p.P) {
      off -= p.P;
      ++pg;
    }
    if (key + step < hi) page = load_i32(table + pg);                 // of the next block
    const uint32_t dst = ring + (i % kStages) * kTileBytes;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int row = c * kPer + r_in;
      const long long from = __shfl_sync(0xffffffffu, at, row);
      cp_async16(dst + row * kRowBytes + (swizzle(ch, row) << 4), kbase + max(from, 0ll), from >= 0);
    }
  };
  auto shift = [&] {
#pragma unroll
    for (int j = 0; j + 1 < kStages; ++j) {
      exps[j] = exps[j + 1];
      old[j] = old[j + 1];
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    shift();
    if (i < nblocks) copy_block(i);
    cp_commit();
  }

  uint32_t qf[kNT][D / 16][2];
  float row_scale[kNT][2], lse2[kNT][2];
  int limit[kNT][2];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int r = nt * 8 + gq;
    const T* src = nullptr;
    if (r < rows) {
      const int tok = r / p.g, h = hk * p.g + (r - tok * p.g);
      src = static_cast<const T*>(p.q) + (static_cast<long long>(sq.row0) + tok) * p.q_t + h * p.q_h;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[nt][ks][0] = src ? load_b32(src + ks * 16 + (k8 ? 4 : 2) * c4) : 0u;
      qf[nt][ks][1] = src ? load_b32(src + ks * 16 + (k8 ? 4 * c4 + 2 : 8 + 2 * c4)) : 0u;
    }
    row_scale[nt][0] = row_scale[nt][1] = p.scale_log2;
    if constexpr (k8) query_to_half<T, D>(qf[nt], nt, c4, row_scale, p.scale_log2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = nt * 8 + 2 * c4 + e;
      limit[nt][e] = hi;
      lse2[nt][e] = INFINITY;                         // 2^(s - inf) = 0: a row that is none, or saw no key
      if (rr < rows) {
        const int tok = rr / p.g, h = hk * p.g + (rr - tok * p.g);
        limit[nt][e] = min(visible_limit(p, sq, tok), hi);
        const float l = wp.lse[lse_index(p, s, sq, h, tok)];
        if (l != -INFINITY) lse2[nt][e] = l * 1.4426950408889634f;
      }
    }
  }
  const int full_to = min(hi, visible_limit(p, sq, 0));     // below it every row sees everything

  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
  for (int i = 0; i < nblocks; ++i) {
    cp_wait<kStages - 2>();
    __syncwarp();                       // every lane's copies of block i are in; stage i-1 is free
    shift();
    if (i + kStages - 1 < nblocks) copy_block(i + kStages - 1);
    cp_commit();
    const uint32_t kt = ring + (i % kStages) * kTileBytes;
    const int key0 = k_first + i * step;
    const float key_scale = k8 ? two_to(scale_exponent(static_cast<uint8_t>(exps[0]))) : 1.f;
    float mine = 0.f;                   // this lane's key's sum
#pragma unroll
    for (int h = 0; h < 2; ++h) {       // 16 keys
      const int row = h * 16 + lrow;
      float st[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[nt][e] = 0.f;
      if constexpr (k8) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2) {
          uint32_t c[4];
          ldsm4(c, kt + row * kRowBytes + (swizzle(ks + lch, row) << 4));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a[4] = {decode2<false>(c[2 * x]), decode2<false>(c[2 * x + 1]), decode2<true>(c[2 * x]), decode2<true>(c[2 * x + 1])};
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma16816<M>(st[nt], a, qf[nt][ks + x][0], qf[nt][ks + x][1]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t a[4];
          ldsm4(a, kt + row * kRowBytes + (swizzle(2 * ks + lch, row) << 4));
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma16816<M>(st[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
        }
      }
      const float f[2] = {__shfl_sync(0xffffffffu, key_scale, h * 16 + gq), __shfl_sync(0xffffffffu, key_scale, h * 16 + gq + 8)};
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = fmaf(st[nt][e] * f[e >> 1], row_scale[nt][e & 1], -lse2[nt][e & 1]);
          if (key0 + kKeys > full_to && key0 + h * 16 + gq + (e >> 1) * 8 >= limit[nt][e & 1]) x = -INFINITY;
          sum[e >> 1] += ex2_approx(x);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        // key h * 16 + x * 8 + k is in lanes 4k to 4k + 3; its own lane is the one of its number
        const float y = __shfl_sync(0xffffffffu, sum[x], (lane & 7) * 4);
        if (lane >> 3 == 2 * h + x) mine = y;
      }
    }
    // one store of 32 neighbours
    if (key0 + lane < hi) w[key0 + lane] = old[0] * wp.decay + mine;
  }
  cp_wait<0>();
}

template <typename T, int D, int kNT, bool k8>
cudaError_t launch_nt(const WeighParams& p, cudaStream_t stream) {
  const int smem = kWarps * kStages * kKeys * D * (k8 ? 1 : 2);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(weigh_rows<T, D, kNT, k8>, smem, &done);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.kv.S) * p.kv.Hkv * p.nsplit;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_rows<T, D, kNT, k8>, p);
}
template <typename T, int D, bool k8>
cudaError_t launch_kind(const WeighParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.kv.max_q) * p.kv.g;
  if (rows <= 8) return launch_nt<T, D, 1, k8>(p, stream);
  if (rows <= 16) return launch_nt<T, D, 2, k8>(p, stream);
  return launch_nt<T, D, 4, k8>(p, stream);
}
template <typename T, int D>
cudaError_t launch(const WeighParams& p, cudaStream_t stream) {
  return p.kv.eight ? launch_kind<T, D, true>(p, stream) : launch_kind<T, D, false>(p, stream);
}

}  // namespace

cudaError_t launch_weigh_rows(WeighParams p, int d, int dtype, int sms, cudaStream_t stream) {
  note_launch();
  // Blocks of 64 to 2048 keys, eight to a multiprocessor where there are enough keys: ragged lengths even out (48 x 8 heads over
  // 8-33 thousand keys: at most 1024 keys a block 184 us, 2048 178, 4096 185).
  const long long units = static_cast<long long>(p.kv.S) * p.kv.Hkv;
  long long n = (8ll * sms + units - 1) / units;
  n = n < (p.kv.max_kv + 2047) / 2048 ? (p.kv.max_kv + 2047) / 2048 : n;
  long long keys = (p.kv.max_kv + n - 1) / n;
  keys = (keys + 63) / 64 * 64;
  p.split_keys = static_cast<int>(keys < 64 ? 64 : keys);
  p.nsplit = (p.kv.max_kv + p.split_keys - 1) / p.split_keys;
  if (p.nsplit < 1) p.nsplit = 1;
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, stream) : launch<__nv_bfloat16, 64>(p, stream);
  return d == 128 ? launch<__half, 128>(p, stream) : launch<__half, 64>(p, stream);
}

cudaError_t read_and_clear_error_word_weigh_rows(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
