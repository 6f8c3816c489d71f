// The weight that each cached key gathers from the rows of a call (what eviction goes by):
//
//     w[c] = (c < len - n ? decay * w[c] : 0) + sum over rows r that see c of 2^(s_rc * scale*log2(e) - lse_r*log2(e))
//
// for a kv head's rows r, the (token, query head of its group) pairs; lse comes from the attention call.
//
// This file, few rows: bound by DRAM, which each key crosses once (its value is not needed), so K streams as in attn_rows.cu:
// a warp takes 16 keys at a time through a ring of its own, S^T = K Q^T by m16n8k16 products with the keys on the
// 16-wide side, and a key's sum over its rows ends as a shuffle over four lanes.  Nothing is shared between warps and
// each w is written by one lane: the same call gives the same bits.  More than 32 rows: weigh_tiles_sm103.cu.
#include <cstdint>

#include "kv_mma.cuh"

namespace vdx {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;
constexpr int kStages = 4;

template <typename T, int D, int kNT, bool k8>
__global__ void __launch_bounds__(kWarps * 32, 2)
weigh_rows(const __grid_constant__ WeighParams wp) {
  using M = std::conditional_t<k8, __half, T>;
  constexpr int kElem = k8 ? 1 : 2;
  constexpr int kChunks = D * kElem / 16;
  constexpr int kRowBytes = D * kElem;
  constexpr int kTileBytes = kKeys * kRowBytes;
  constexpr int kCopies = kKeys * kChunks / 32;
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

  const uint32_t ring = smem_addr(smem) + warp * kStages * kTileBytes;
  const int step = kKeys * kWarps;
  const int k_first = lo + kKeys * warp;
  const int nblocks = k_first < hi ? (hi - k_first + step - 1) / step : 0;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + hk * p.k_h * kElem;
  const int* table = p.table + static_cast<long long>(s) * p.table_stride;
  float* w = wp.w + s * wp.w_seq + hk * wp.w_head;
  const int old_to = sq.len - sq.n;                     // keys below were there before the call
  auto swizzle = [](int c, int r) { return kRowBytes == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); };
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
  const int ch = lane % kChunks, r_in = lane / kChunks;

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

  int pg = nblocks > 0 ? k_first / p.P : 0;
  int off = nblocks > 0 ? k_first - pg * p.P : 0;
  int e0 = 0, e1 = 0;
  auto fetch_pages = [&](int key) {
    e0 = key < hi ? load_i32(table + pg) : 0;
    e1 = (off + kKeys > p.P && key + (p.P - off) < hi) ? load_i32(table + pg + 1) : 0;
    if (static_cast<unsigned>(e0) >= static_cast<unsigned>(p.num_pages) ||
        static_cast<unsigned>(e1) >= static_cast<unsigned>(p.num_pages)) {
      if (lane == 0) atomicOr(&g_error_word, kErrPage);
    }
  };
  fetch_pages(k_first);
  // scales and weights so far of the blocks being copied, oldest first: lane l has those of key l
  int exps[kStages - 1];
  float old[kStages - 1];
  auto copy_block = [&](int i) {
    const int key = k_first + i * step;
    const uint32_t dst = ring + (i % kStages) * kTileBytes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int row = r_in + c * (32 / kChunks);
      int o2 = off + row, page = e0;
      if (o2 >= p.P) {
        o2 -= p.P;
        page = e1;
      }
      const bool ok = key + row < hi && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
      cp_async16(dst + row * kRowBytes + (swizzle(ch, row) << 4),
                 ok ? kbase + (page * p.k_p + o2 * p.k_t) * kElem + ch * 16 : kbase, ok);
    }
    const int row = lane & 15, mine = key + row;
    if constexpr (k8) {
      int o2 = off + row, page = e0;
      if (o2 >= p.P) {
        o2 -= p.P;
        page = e1;
      }
      exps[kStages - 2] = mine < hi && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)
                              ? scale_exponent(p.scales.k[page * p.scales.k_page + o2 / kBlock8 * p.scales.k_block + hk * p.scales.k_head])
                              : 0;
    }
    old[kStages - 2] = mine < hi && mine < old_to ? w[mine] * wp.decay : 0.f;
    off += step;
    while (off >= p.P) {
      off -= p.P;
      ++pg;
    }
    if (i + 1 < nblocks) fetch_pages(key + step);
  };
  auto shift = [&] {
#pragma unroll
    for (int j = 0; j + 1 < kStages - 1; ++j) {
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
  for (int i = 0; i < nblocks; ++i) {
    cp_wait<kStages - 2>();
    __syncwarp();
    float key_scale[2] = {1.f, 1.f}, before[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if constexpr (k8) key_scale[x] = two_to(__shfl_sync(0xffffffffu, exps[0], gq + 8 * x));
      before[x] = __shfl_sync(0xffffffffu, old[0], gq + 8 * x);
    }
    shift();
    if (i + kStages - 1 < nblocks) copy_block(i + kStages - 1);
    cp_commit();
    const uint32_t kt = ring + (i % kStages) * kTileBytes;
    const int key0 = k_first + i * step;
    float sum[2] = {0.f, 0.f};
    float st[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[nt][e] = 0.f;
    if constexpr (k8) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ks += 2) {
        uint32_t c[4];
        ldsm4(c, kt + lrow * kRowBytes + (swizzle(ks + lch, lrow) << 4));
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
        ldsm4(a, kt + lrow * kRowBytes + (swizzle(2 * ks + lch, lrow) << 4));
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) mma16816<M>(st[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = fmaf(st[nt][e] * (k8 ? key_scale[e >> 1] : 1.f), row_scale[nt][e & 1], -lse2[nt][e & 1]);
        if (key0 + kKeys > full_to && key0 + gq + (e >> 1) * 8 >= limit[nt][e & 1]) x = -INFINITY;
        sum[e >> 1] += ex2_approx(x);
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
      const int key = key0 + gq + 8 * x;
      if (c4 == 0 && key < hi) w[key] = before[x] + sum[x];
    }
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
  // blocks of 64 to 1024 keys, several to a multiprocessor where there are enough
  const long long units = static_cast<long long>(p.kv.S) * p.kv.Hkv;
  long long n = (8ll * sms + units - 1) / units;
  n = n < (p.kv.max_kv + 1023) / 1024 ? (p.kv.max_kv + 1023) / 1024 : n;
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
