// Attention of few query rows per kv head over an 8-bit cache: attn_rows.cu's form with codes in place of keys and values.
//
// Bound: DRAM still, at half the bytes, so that instructions count: a warp takes 32 keys a step (a lane looks up a key's page,
// and the scales of its key and value, for all), and the products are of fp16 whatever the call's type, since
// codes become fp16 in one instruction (and bf16 in five).  Queries of bf16 are brought into fp16's range by a power
// of two of the row's own (query_to_half), which scores are multiplied back by, as they are by the key's scale; values are
// multiplied by their scale on the way, exactly; weights are taken times 2^7 (of at most 2^8), so that fp16 keeps
// those down to 2^-21 of a row's largest.  Codes are put in the fragments' order by what can be exchanged for free: the
// channels within a step of K Q^T, and those of the output.
//
// 48 tokens over 8-33 thousand keys of 8 heads, 2.16 GB: 346 us, 6.2 TB/s, 93 % of a plain copy's rate (16 keys a step in
// attn_rows.cu's own form 588 us; two stages and three CTAs to a multiprocessor 350, four CTAs 353).
#include <cstdint>

#include "kv_mma.cuh"
#include "rows_join.cuh"

namespace vdx {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;        // keys of one stage, a lane each
constexpr int kStages = 3;
constexpr float kLift = 7.f;     // log2 of what weights are multiplied by

// kNT tiles of 8 query rows.
template <typename T, int D, int kNT>
__global__ void __launch_bounds__(kWarps * 32, 2)
attn_rows8(const __grid_constant__ KvParams p) {
  constexpr int kChunks = D / 16;                      // 16-byte chunks of a key
  constexpr int kTileBytes = kKeys * D;                // K or V of one stage
  constexpr int kPer = 32 / kChunks;                   // rows that the lanes copy at once
  extern __shared__ __align__(128) uint8_t smem[];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, c4 = lane & 3;
  wait_for_earlier_work();

  const int z = blockIdx.x % p.nsplit;
  const int unit = blockIdx.x / p.nsplit;
  const int hk = unit % p.Hkv, s = unit / p.Hkv;        // all rows of a kv head are one block
  const SeqInfo sq = sequence_info(p, s, threadIdx.x == 0);
  const int live = min(sq.n, p.max_q) * p.g;            // max_q * g <= 8 * kNT
  if (live == 0) return;

  // Keys of this split, as in attn_rows.
  constexpr int step = kKeys * kWarps;
  const int len = visible_limit(p, sq, (live - 1) / p.g);
  const long long keys = p.cluster ? (len / step / p.nsplit + 1) * step : p.split_keys;
  const long long lo64 = z * keys;
  const int lo = static_cast<int>(min(lo64, static_cast<long long>(len)));
  const int hi = static_cast<int>(min(lo64 + keys, static_cast<long long>(len)));

  // ---- the warp's ring of key blocks lo + 32*(warp + 4*i)
  const uint32_t ring = smem_addr(smem) + warp * kStages * 2 * kTileBytes;
  const int k_first = lo + kKeys * warp;
  const int nblocks = k_first < hi ? (hi - k_first + step - 1) / step : 0;
  const int* table = p.table + static_cast<long long>(s) * p.table_stride;
  const int ch = lane % kChunks, r_in = lane / kChunks;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + hk * p.k_h + ch * 16;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + hk * p.v_h + ch * 16;
  const uint8_t* kscale = p.scales.k + hk * p.scales.k_head;
  const uint8_t* vscale = p.scales.v + hk * p.scales.v_head;
  // Chunk `c` of row r of a tile lies at chunk swizzle(c, r): 8 rows' chunks of one number fill all banks.
  auto swizzle = [](int c, int r) { return D == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); };
  // This lane's key of the block to be copied next: entry of the page table and token in the page; its page, when it has come.
  int pg = 0, off = 0, page = 0;
  if (nblocks > 0) {
    pg = (k_first + lane) / p.P;
    off = k_first + lane - pg * p.P;
    if (k_first + lane < hi) page = load_i32(table + pg);
  }
  // Scales of the blocks being copied, oldest first: the exponents of this lane's key and value
  int k_exp[kStages], v_exp[kStages];
  auto copy_block = [&](int i) {
    const int key = k_first + i * step + lane;
    const bool there = key < hi, ok = there && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
    if (there && !ok) atomicOr(&g_error_word, kErrPage);              // reads as zeros
    k_exp[kStages - 1] = v_exp[kStages - 1] = 127;
    long long at_k = -1, at_v = 0;
    if (ok) {
      const long long b = off / kBlock8;
      k_exp[kStages - 1] = kscale[page * p.scales.k_page + b * p.scales.k_block];
      v_exp[kStages - 1] = vscale[page * p.scales.v_page + b * p.scales.v_block];
      at_k = page * p.k_p + off * p.k_t;
      at_v = page * p.v_p + off * p.v_t;
    }
    off += step;
    while (off >= p.P) {
      off -= p.P;
      ++pg;
    }
    if (key + step < hi) page = load_i32(table + pg);                 // of the next block
    const uint32_t dst = ring + (i % kStages) * 2 * kTileBytes;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int row = c * kPer + r_in;
      const long long from_k = __shfl_sync(0xffffffffu, at_k, row), from_v = __shfl_sync(0xffffffffu, at_v, row);
      const uint32_t d = dst + row * D + (swizzle(ch, row) << 4);
      cp_async16(d, kbase + max(from_k, 0ll), from_k >= 0);
      cp_async16(d + kTileBytes, vbase + from_v, from_k >= 0);
    }
  };
  auto shift = [&] {
#pragma unroll
    for (int j = 0; j + 1 < kStages; ++j) {
      k_exp[j] = k_exp[j + 1];
      v_exp[j] = v_exp[j + 1];
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    shift();
    if (i < nblocks) copy_block(i);
    cp_commit();
  }

  // Query fragments (B operand: k = channel, n = row): row 8*nt + gq; channels 16*ks + 4*c4 and up, the order in which a
  // lane gets its codes.
  uint32_t qf[kNT][D / 16][2];
  float row_scale[kNT][2];               // scale_log2 and the query's power of two, for the two rows below
  int limit[kNT][2];                     // of the two rows whose scores this lane holds
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int r = nt * 8 + gq;
    const T* src = nullptr;
    if (r < live) {
      const int tok = r / p.g, h = hk * p.g + (r - tok * p.g);
      src = static_cast<const T*>(p.q) + (static_cast<long long>(sq.row0) + tok) * p.q_t + h * p.q_h;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[nt][ks][0] = src ? load_b32(src + ks * 16 + 4 * c4) : 0u;
      qf[nt][ks][1] = src ? load_b32(src + ks * 16 + 4 * c4 + 2) : 0u;
    }
    query_to_half<T, D>(qf[nt], nt, c4, row_scale, p.scale_log2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = nt * 8 + 2 * c4 + e;
      limit[nt][e] = rr < live ? min(visible_limit(p, sq, rr / p.g), hi) : hi;
    }
  }
  const int full_to = min(hi, visible_limit(p, sq, 0));      // below this key every row sees everything

  float o[kNT][D / 16][4];
  float m[kNT][2], l[kNT][2];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
  }

  const int lrow_k = (lane & 7) + ((lane >> 3) & 1) * 8, lch_k = lane >> 4;          // K: matrices (rows, rows+8) x 2 chunks
  const int lrow_v = (lane & 7) + ((lane >> 4) & 1) * 8, lch_v = (lane >> 3) & 1;    // V^T: 2 chunks x (keys, keys+8)
  for (int i = 0; i < nblocks; ++i) {
    cp_wait<kStages - 2>();
    __syncwarp();                       // every lane's copies of block i are in; stage i-1 is free
    shift();
    if (i + kStages - 1 < nblocks) copy_block(i + kStages - 1);
    cp_commit();
    const uint32_t kt = ring + (i % kStages) * 2 * kTileBytes;
    const uint32_t vt = kt + kTileBytes;
    const int key0 = k_first + i * step;

    float st[2][kNT][4];                // of keys gq and gq + 8 of each half
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[h][nt][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ks += 2)              // a chunk of 16 codes is a step of 16 channels
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = h * 16 + lrow_k;
        uint32_t c[4];
        ldsm4(c, kt + row * D + (swizzle(ks + lch_k, row) << 4));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a[4] = {decode2<false>(c[2 * x]), decode2<false>(c[2 * x + 1]), decode2<true>(c[2 * x]), decode2<true>(c[2 * x + 1])};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma16816<__half>(st[h][nt], a, qf[nt][ks + x][0], qf[nt][ks + x][1]);
        }
      }
    const float key_scale = two_to(scale_exponent(static_cast<uint8_t>(k_exp[0])));
    bool grow = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f[2] = {__shfl_sync(0xffffffffu, key_scale, h * 16 + gq), __shfl_sync(0xffffffffu, key_scale, h * 16 + gq + 8)};
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) st[h][nt][e] *= row_scale[nt][e & 1] * f[e >> 1];
        if (key0 + kKeys > full_to) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + h * 16 + gq + (e >> 1) * 8 >= limit[nt][e & 1]) st[h][nt][e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) grow |= st[h][nt][e] > m[nt][e & 1] + 8.f;
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(st[0][nt][e], st[0][nt][e + 2]), fmaxf(st[1][nt][e], st[1][nt][e + 2]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          if (mx > m[nt][e]) {
            const float alpha = ex2_approx(m[nt][e] - mx);
            m[nt][e] = mx;
            l[nt][e] *= alpha;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              o[nt][mt][e] *= alpha;
              o[nt][mt][e + 2] *= alpha;
            }
          }
        }
      }
    }
    // scales of the values of keys 2*c4 and 2*c4 + 1, and of those 8, 16 and 24 on, as pairs
    const uint32_t mine = half_two_to(scale_exponent(static_cast<uint8_t>(v_exp[0])));
    const uint32_t both = mine | (__shfl_xor_sync(0xffffffffu, mine, 1) << 16);       // right in even lanes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t vs[2] = {__shfl_sync(0xffffffffu, both, h * 16 + 2 * c4), __shfl_sync(0xffffffffu, both, h * 16 + 8 + 2 * c4)};
      uint32_t b[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        // a row that has seen no key yet: every score is -inf and weighs 2^-inf = 0
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kLift;
        const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kLift;
        const float p0 = ex2_approx(st[h][nt][0] - m0), p1 = ex2_approx(st[h][nt][1] - m1);
        const float p2 = ex2_approx(st[h][nt][2] - m0), p3 = ex2_approx(st[h][nt][3] - m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        b[nt][0] = transpose8x8(pack2<__half>(p0, p1));
        b[nt][1] = transpose8x8(pack2<__half>(p2, p3));
      }
      // Transposed as pairs of codes, a lane gets channels 2*gq and 2*gq + 1 of two keys: they are the product's
      // rows gq and gq + 8, once the four codes are put in order.
      const int row = h * 16 + lrow_v;
#pragma unroll
      for (int mt = 0; mt < D / 16; mt += 2) {
        uint32_t c[4];
        ldsm4_trans(c, vt + row * D + (swizzle(mt + lch_v, row) << 4));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t low = __byte_perm(c[x], 0u, 0x3120), up = __byte_perm(c[x + 2], 0u, 0x3120);
          const uint32_t a[4] = {half2_mul(decode2<false>(low), vs[0]), half2_mul(decode2<true>(low), vs[0]),
                                 half2_mul(decode2<false>(up), vs[1]), half2_mul(decode2<true>(up), vs[1])};
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma16816<__half>(o[nt][mt + x], a, b[nt][0], b[nt][1]);
        }
      }
    }
    __syncwarp();
  }
  cp_wait<0>();
  __syncthreads();                      // the rings become the warps' partial results
  join_warps<T, D, kNT, kWarps, true>(p, s, hk, unit, z, sq, live, smem, o, m, l, kLift);
}

template <typename T, int D, int kNT>
cudaError_t launch_nt(const KvParams& p, cudaStream_t stream) {
  constexpr int kRing = kWarps * kStages * 2 * kKeys * D, kJoin = join_bytes<D, kNT, kWarps>(), kSmem = kRing > kJoin ? kRing : kJoin;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(attn_rows8<T, D, kNT>, kSmem, &done);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSmem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster ? static_cast<unsigned>(p.nsplit) : 1u;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = launch_early();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, attn_rows8<T, D, kNT>, p);
}
template <typename T, int D>
cudaError_t launch(const KvParams& p, cudaStream_t stream) {
  if (p.block_rows == 8) return launch_nt<T, D, 1>(p, stream);
  if (p.block_rows == 16) return launch_nt<T, D, 2>(p, stream);
  return launch_nt<T, D, 4>(p, stream);
}

}  // namespace

cudaError_t launch_attn_rows8(const KvParams& p, int d, int dtype, cudaStream_t stream) {
  note_launch();
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, stream) : launch<__nv_bfloat16, 64>(p, stream);
  return d == 128 ? launch<__half, 128>(p, stream) : launch<__half, 64>(p, stream);
}

cudaError_t read_and_clear_error_word_rows8(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
