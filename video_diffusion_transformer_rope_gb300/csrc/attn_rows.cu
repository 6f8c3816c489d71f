// Attention of few query rows per kv head (single new tokens, short chunks, the rows of grouped
// heads) over a paged cache or dense keys, plus the kernel that joins key splits.
//
//     S^T = K Q^T (keys x rows),  P^T = 2^(S^T * scale*log2(e) - m),  O^T += V^T P^T
//
// Bound: DRAM, every key and value is read once and used for a handful of rows (2 flops per byte
// and row), so what counts is bytes in flight, not tensor rate: m16n8k16 MMAs with the KEYS (and
// the channels of V) on the 16-wide side and 8 query rows on the narrow side waste nothing on
// padding, and a warp needs no other warp: it streams its own 16-key blocks through its own
// ring of cp.async stages (any page size, stride or token order; rows past the end are filled
// with zeros, so what the cache holds there is never used), and keeps its own running maximum,
// sum and accumulator.  The warps of a CTA join through shared memory at the end.  Splits of the keys,
// up to 8 of them, are the CTAs of a cluster and join through one another's shared memory (no second
// launch, no scratch: 15.6 to 9.9 us for 4 sequences of up to 1000 keys); more, for a few heads over a
// long cache, join through the workspace and the kernel below.
//
// Weights are rounded to the call's type for the product with V (an fp32 operand would be two products);
// scores, sums and accumulators are fp32, and the sum is of the unrounded weights.  What that costs: 0.0023
// of the result against 64 bits in bf16 where the output's own rounding makes 0.0017, 0.00028 against 0.00021 in
// fp16 (root mean squares, 48 tokens over 8-33 thousand keys and 9 chunks).  fp16 weights below 2^-14 of the
// largest lose bits and below 2^-25 vanish.
//
// The running maximum moves only when a score exceeds it by more than 8 (log2 units): until then
// weights stay below 2^8, exact in the fp32 sums, and no lane has to talk to another.
#include <cstdint>

#include "kv_common.cuh"

namespace vdx {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;        // keys of one stage
constexpr int kStages = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr)
               : "memory");
  return v;
}

// kNT tiles of 8 query rows.
template <typename T, int D, int kNT>
__global__ void __launch_bounds__(kWarps * 32, 2)
attn_rows(const __grid_constant__ KvParams p) {
  constexpr int kRows = 8 * kNT;
  constexpr int kChunks = D / 8;                       // 16-byte chunks of a key
  constexpr int kRowBytes = D * 2;
  constexpr int kTileBytes = kKeys * kRowBytes;        // K or V of one stage
  constexpr int kCopies = kKeys * kChunks / 32;        // 16-byte copies per lane and tile
  constexpr int kPad = D + 4;
  extern __shared__ __align__(128) uint8_t smem[];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, c4 = lane & 3;
  wait_for_earlier_work();

  const int z = blockIdx.x % p.nsplit;
  const int unit = blockIdx.x / p.nsplit;
  const int hk = unit % p.Hkv, s = unit / p.Hkv;        // all rows of a kv head are one block
  const SeqInfo sq = sequence_info(p, s, threadIdx.x == 0);
  const int live = min(sq.n, p.max_q) * p.g;            // max_q * g <= kRows
  if (live == 0) return;

  // Keys of this split, up to the last row's limit: an equal part for each CTA of a cluster, which
  // wait for one another; fixed ranges otherwise (a CTA past a short sequence's end leaves).
  const int len = visible_limit(p, sq, (live - 1) / p.g);
  const long long keys = p.cluster ? (len / (kKeys * kWarps) / p.nsplit + 1) * (kKeys * kWarps) : p.split_keys;
  const long long lo64 = z * keys;
  const int lo = static_cast<int>(min(lo64, static_cast<long long>(len)));
  const int hi = static_cast<int>(min(lo64 + keys, static_cast<long long>(len)));

  // Query fragments (B operand: k = channel, n = row): row 8*nt + gq, channels 16*ks + 2*c4 (+8).
  uint32_t qf[kNT][D / 16][2];
  int limit[kNT][2];                     // of the two rows whose scores this lane holds
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int r = nt * 8 + gq;
    const T* src = nullptr;
    if (r < live) {
      const int tok = r / p.g, h = hk * p.g + (r - tok * p.g);
      src = static_cast<const T*>(p.q) + (p.cu ? 0 : s * p.q_b) + (static_cast<long long>(sq.row0) + tok) * p.q_t + h * p.q_h;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[nt][ks][0] = src ? load_b32(src + ks * 16 + 2 * c4) : 0u;
      qf[nt][ks][1] = src ? load_b32(src + ks * 16 + 8 + 2 * c4) : 0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = nt * 8 + 2 * c4 + e;
      limit[nt][e] = rr < live ? min(visible_limit(p, sq, rr / p.g), hi) : hi;
    }
  }
  // Below this key every row sees everything.
  const int full_to = p.causal_block > 0
                          ? min(hi, visible_limit(p, sq, 0))
                          : hi;

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

  // ---- the warp's ring of key blocks lo + 16*(warp + 4*i)
  const uint32_t ring = smem_addr(smem) + warp * kStages * 2 * kTileBytes;
  const int step = kKeys * kWarps;
  const int k_first = lo + kKeys * warp;
  const int nblocks = k_first < hi ? (hi - k_first + step - 1) / step : 0;
  const T* kbase = static_cast<const T*>(p.k) + hk * p.k_h;
  const T* vbase = static_cast<const T*>(p.v) + hk * p.v_h;
  const int* table = p.table ? p.table + static_cast<long long>(s) * p.table_stride : nullptr;
  // Page of the next block to copy and the one after it (a block crosses at most one page end:
  // paged sizes are >= 16, and a dense "page" holds every key).
  int pg = nblocks > 0 ? k_first / p.P : 0;
  int off = nblocks > 0 ? k_first - pg * p.P : 0;
  int e0 = s, e1 = s;
  auto fetch_pages = [&](int key) {
    if (table) {
      e0 = key < hi ? load_i32(table + pg) : 0;
      e1 = (off + kKeys > p.P && key + (p.P - off) < hi) ? load_i32(table + pg + 1) : 0;
      if (static_cast<unsigned>(e0) >= static_cast<unsigned>(p.num_pages) ||
          static_cast<unsigned>(e1) >= static_cast<unsigned>(p.num_pages)) {
        if (lane == 0) atomicOr(&g_error_word, kErrPage);
      }
    }
  };
  fetch_pages(k_first);
  const int ch = lane % kChunks, r_in = lane / kChunks;
  auto copy_block = [&](int i) {
    const int key = k_first + i * step;
    const uint32_t dst = ring + (i % kStages) * 2 * kTileBytes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int row = r_in + c * (32 / kChunks);
      int o2 = off + row, page = e0;
      if (o2 >= p.P) {
        o2 -= p.P;
        page = e1;
      }
      const bool ok = key + row < hi && static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
      const uint32_t d = dst + row * kRowBytes + ((ch ^ (row & 7)) << 4);
      const T* ks = kbase;
      const T* vs = vbase;
      if (ok) {
        ks += page * p.k_p + o2 * p.k_t + ch * 8;
        vs += page * p.v_p + o2 * p.v_t + ch * 8;
      }
      cp_async16(d, ks, ok);
      cp_async16(d + kTileBytes, vs, ok);
    }
    off += step;
    while (off >= p.P && table) {
      off -= p.P;
      ++pg;
    }
    if (i + 1 < nblocks) fetch_pages(key + step);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < nblocks) copy_block(i);
    cp_commit();
  }

  const int lrow_k = (lane & 7) + ((lane >> 3) & 1) * 8, lch_k = lane >> 4;          // K: matrices (rows, rows+8) x 2 chunks
  const int lrow_v = (lane & 7) + ((lane >> 4) & 1) * 8, lch_v = (lane >> 3) & 1;    // V^T: 2 chunks x (keys, keys+8)
  for (int i = 0; i < nblocks; ++i) {
    cp_wait<kStages - 2>();
    __syncwarp();                       // every lane's copies of block i are in; stage i-1 is free
    if (i + kStages - 1 < nblocks) copy_block(i + kStages - 1);
    cp_commit();
    const uint32_t kt = ring + (i % kStages) * 2 * kTileBytes;
    const uint32_t vt = kt + kTileBytes;
    const int key0 = k_first + i * step;

    float st[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[nt][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      ldsm4(a, kt + lrow_k * kRowBytes + (((2 * ks + lch_k) ^ (lrow_k & 7)) << 4));
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) mma16816<T>(st[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
    }
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) st[nt][e] *= p.scale_log2;
      if (key0 + kKeys > full_to) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + gq + (e >> 1) * 8 >= limit[nt][e & 1]) st[nt][e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) grow |= st[nt][e] > m[nt][e & 1] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(st[nt][e], st[nt][e + 2]);
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
    uint32_t b[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      // a row that has seen no key yet: every score is -inf and weighs 2^-inf = 0
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
      const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
      const float p0 = ex2_approx(st[nt][0] - m0), p1 = ex2_approx(st[nt][1] - m1);
      const float p2 = ex2_approx(st[nt][2] - m0), p3 = ex2_approx(st[nt][3] - m1);
      l[nt][0] += p0 + p2;
      l[nt][1] += p1 + p3;
      b[nt][0] = transpose8x8(pack2<T>(p0, p1));
      b[nt][1] = transpose8x8(pack2<T>(p2, p3));
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      uint32_t a[4];
      ldsm4_trans(a, vt + lrow_v * kRowBytes + (((2 * mt + lch_v) ^ (lrow_v & 7)) << 4));
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) mma16816<T>(o[nt][mt], a, b[nt][0], b[nt][1]);
    }
    __syncwarp();
  }
  cp_wait<0>();
  __syncthreads();                      // the rings become the warps' partial results

  float* so = reinterpret_cast<float*>(smem);                       // [kWarps][kRows][kPad]
  float* sm = so + kWarps * kRows * kPad;                           // [kWarps][kRows]
  float* sl = sm + kWarps * kRows;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[nt][e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
      const int r = nt * 8 + 2 * c4 + e;
      if (gq == 0) {
        sm[warp * kRows + r] = m[nt][e];
        sl[warp * kRows + r] = t;
      }
      float* dst = so + (warp * kRows + r) * kPad;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        dst[mt * 16 + gq] = o[nt][mt][e];
        dst[mt * 16 + gq + 8] = o[nt][mt][e + 2];
      }
    }
  }
  __syncthreads();
  // Four channels per thread.
  const long long slot = static_cast<long long>(unit) * p.nsplit + z;
  float* cm = sl + kWarps * kRows;                                  // [kRows]: this CTA's maximum and sum
  float* cl = cm + kRows;
  auto store = [&](int r, int dq, float mx, float lt, const float4& acc) {
    const int tok = r / p.g, h = hk * p.g + (r - tok * p.g);
    const bool none = mx == -INFINITY && lt == lt;                  // no key seen; a NaN sum is an answer
    const float inv = none ? 0.f : 1.f / lt;
    uint2 w2;
    w2.x = pack2<T>(acc.x * inv, acc.y * inv);
    w2.y = pack2<T>(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (out_row(p, s, sq, tok) * p.Hq + h) * D + dq) = w2;
    if (dq == 0 && p.lse)
      p.lse[lse_index(p, s, sq, h, tok)] = none ? -INFINITY : (mx + __log2f(lt)) * 0.69314718055994530942f;
  };
  for (int i = threadIdx.x; i < live * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), dq = (i % (D / 4)) * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w * kRows + r]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float lt = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wt = ex2_approx(sm[w * kRows + r] - base);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * kRows + r) * kPad + dq);
      lt += wt * sl[w * kRows + r];
      acc.x += wt * v.x; acc.y += wt * v.y; acc.z += wt * v.z; acc.w += wt * v.w;
    }
    if (p.cluster) {
      *reinterpret_cast<float4*>(so + r * kPad + dq) = acc;          // over warp 0's, which only this thread reads
      if (dq == 0) {
        cm[r] = mx;
        cl[r] = lt;
      }
    } else if (p.nsplit > 1) {
      *reinterpret_cast<float4*>(p.part_o + (slot * kRows + r) * D + dq) = acc;
      if (dq == 0) p.part_ml[slot * kRows + r] = make_float2(mx, lt);
    } else {
      store(r, dq, mx, lt, acc);
    }
  }
  if (!p.cluster) return;
  cluster_sync_all();                   // every CTA's part is in its shared memory
  for (int i = threadIdx.x + z * kWarps * 32; i < live * (D / 4); i += p.nsplit * kWarps * 32) {
    const int r = i / (D / 4), dq = (i % (D / 4)) * 4;
    const uint32_t am = smem_addr(cm + r), al = smem_addr(cl + r), ao = smem_addr(so + r * kPad + dq);
    float mx = -INFINITY;
    for (int w = 0; w < p.nsplit; ++w) mx = fmaxf(mx, ld_cluster_f32(mapa_shared(am, w)));
    const float base = mx == -INFINITY ? 0.f : mx;
    float lt = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < p.nsplit; ++w) {
      const float wt = ex2_approx(ld_cluster_f32(mapa_shared(am, w)) - base);
      const float4 v = ld_cluster_f32x4(mapa_shared(ao, w));
      lt += wt * ld_cluster_f32(mapa_shared(al, w));
      acc.x += wt * v.x; acc.y += wt * v.y; acc.z += wt * v.z; acc.w += wt * v.w;
    }
    store(r, dq, mx, lt, acc);
  }
  cluster_sync_all();                   // no CTA leaves while another reads its part
}

// Join the key splits of every row: out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z.  kPer warps per
// row (8 where there are few rows with many splits, 1 where there are many rows), each taking every
// kPer-th split: first the maxima, a split to a lane, then the rows of O, whose loads do not depend on one
// another (read one after another, 195 splits of one row took 60 us).  Bound by reading O (L2).
template <typename T, int D, int kPer>
__global__ void __launch_bounds__(256)
attn_join(const __grid_constant__ KvParams p) {
  constexpr int kVals = D / 32;
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kPer;
  wait_for_earlier_work();
  const unsigned unit = blockIdx.x, sh = unit / p.nblk;               // a block stays within one unit
  const int r = blockIdx.y * (8 / kPer) + warp / kPer;
  const int hk = static_cast<int>(sh % p.Hkv), s = static_cast<int>(sh / p.Hkv);
  const SeqInfo sq = sequence_info(p, s, false);
  const int R = static_cast<int>(unit - sh * p.nblk) * p.block_rows + r;      // rows of a kv head are < 2^31
  const bool live = r < p.block_rows && R < min(sq.n, p.max_q) * p.g;
  const int tok = R / p.g, h = hk * p.g + (R - tok * p.g);
  float m = -INFINITY, l = 0.f, acc[kVals];
#pragma unroll
  for (int e = 0; e < kVals; ++e) acc[e] = 0.f;
  if (live) {
    const long long base = static_cast<long long>(unit) * p.nsplit * p.block_rows + r;      // + z * block_rows
    for (int z = part + kPer * lane; z < p.nsplit; z += kPer * 32)
      m = fmaxf(m, p.part_ml[base + static_cast<long long>(z) * p.block_rows].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int z0 = part; z0 < p.nsplit; z0 += kPer * 32) {
      // weights of up to 32 splits, a lane each; a split without keys for this row has none, and no O
      const int z = z0 + kPer * lane;
      float w = 0.f;
      bool has = false;
      if (z < p.nsplit) {
        const float2 ml = p.part_ml[base + static_cast<long long>(z) * p.block_rows];
        has = ml.x > -INFINITY || ml.y != ml.y;           // a NaN sum is an answer
        w = ml.x > -INFINITY ? ex2_approx(ml.x - m) : 1.f;
        if (has) l += w * ml.y;
      }
      unsigned todo = __ballot_sync(0xffffffffu, has);
#pragma unroll 4
      while (todo) {
        const int i = __ffs(todo) - 1;
        todo &= todo - 1;
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* src = p.part_o + (base + static_cast<long long>(z0 + kPer * i) * p.block_rows) * D + lane * kVals;
        float v[kVals];
        if constexpr (kVals == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[0] = x.x; v[1] = x.y;
        }
#pragma unroll
        for (int e = 0; e < kVals; ++e) acc[e] += wi * v[e];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  }
  if (kPer > 1) {
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kVals; ++e) s_o[warp][lane * kVals + e] = acc[e];
    __syncthreads();
    if (part != 0) return;
    float top = m;
#pragma unroll
    for (int w = 1; w < kPer; ++w) top = fmaxf(top, s_m[warp + w]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kVals; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kPer; ++w) {
      const float f = s_m[warp + w] > -INFINITY ? ex2_approx(s_m[warp + w] - top) : 1.f;   // no keys: l and O are 0
      l += f * s_l[warp + w];
#pragma unroll
      for (int e = 0; e < kVals; ++e) acc[e] += f * s_o[warp + w][lane * kVals + e];
    }
    m = top;
  }
  if (!live) return;
  const bool empty = !(m > -INFINITY) && !(l != l);
  const float inv = empty ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + (out_row(p, s, sq, tok) * p.Hq + h) * D) + lane * (kVals / 2);
#pragma unroll
  for (int e = 0; e < kVals / 2; ++e) dst[e] = pack2<T>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0 && p.lse)
    p.lse[lse_index(p, s, sq, h, tok)] = empty ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
}

template <typename T, int D, int kNT>
cudaError_t launch_nt(const KvParams& p, cudaStream_t stream) {
  const int ring = kWarps * kStages * 2 * kKeys * D * 2;
  const int join = (kWarps * (D + 4 + 2) + 2) * 8 * kNT * 4;
  const int smem = ring > join ? ring : join;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(attn_rows<T, D, kNT>, smem, &done);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster ? static_cast<unsigned>(p.nsplit) : 1u;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = launch_early();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, attn_rows<T, D, kNT>, p);
}
template <typename T, int D>
cudaError_t launch(const KvParams& p, cudaStream_t stream) {
  if (p.block_rows == 8) return launch_nt<T, D, 1>(p, stream);
  if (p.block_rows == 16) return launch_nt<T, D, 2>(p, stream);
  return launch_nt<T, D, 4>(p, stream);
}
template <typename T, int D>
cudaError_t join(const KvParams& p, cudaStream_t stream) {
  const long long units = static_cast<long long>(p.S) * p.Hkv * p.nblk;
  if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units), p.rows_kernel ? p.block_rows : (p.block_rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.rows_kernel ? cudaLaunchKernelEx(&cfg, attn_join<T, D, 8>, p) : cudaLaunchKernelEx(&cfg, attn_join<T, D, 1>, p);
}

}  // namespace

cudaError_t launch_attn_rows(const KvParams& p, int d, int dtype, cudaStream_t stream) {
  note_launch();
  if (dtype == 0) return d == 128 ? launch<__nv_bfloat16, 128>(p, stream) : launch<__nv_bfloat16, 64>(p, stream);
  return d == 128 ? launch<__half, 128>(p, stream) : launch<__half, 64>(p, stream);
}
cudaError_t launch_attn_combine(const KvParams& p, int d, int dtype, cudaStream_t stream) {
  if (dtype == 0) return d == 128 ? join<__nv_bfloat16, 128>(p, stream) : join<__nv_bfloat16, 64>(p, stream);
  return d == 128 ? join<__half, 128>(p, stream) : join<__half, 64>(p, stream);
}

cudaError_t read_and_clear_error_word_rows(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
