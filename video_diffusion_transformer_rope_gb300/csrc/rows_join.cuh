// The end of the few-row attention kernels (attn_rows.cu, attn_rows8.cu): the warps of a block join through shared
// memory, the blocks of a cluster through one another's, more splits through the workspace.
#pragma once
#include "kv_common.cuh"

namespace vdx {

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

// o, m, l: this warp's accumulators of kNT tiles of 8 rows, their running maxima (log2 units) and its lanes' sums of weights,
// which are those against m - lift.  kPairs: rows gq and gq + 8 of a 16-channel step are channels 2*gq and 2*gq + 1.
// Every warp of the block has finished with `smem`.
template <typename T, int D, int kNT, int kWarps, bool kPairs>
__device__ __forceinline__ void join_warps(const KvParams& p, int s, int hk, int unit, int z, const SeqInfo& sq, int live, uint8_t* smem,
                                           const float (&o)[kNT][D / 16][4], const float (&m)[kNT][2], const float (&l)[kNT][2],
                                           float lift) {
  constexpr int kRows = 8 * kNT, kPad = D + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, c4 = lane & 3;
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
        sm[warp * kRows + r] = m[nt][e] - lift;
        sl[warp * kRows + r] = t;
      }
      float* dst = so + (warp * kRows + r) * kPad;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        dst[mt * 16 + (kPairs ? 2 * gq : gq)] = o[nt][mt][e];
        dst[mt * 16 + (kPairs ? 2 * gq + 1 : gq + 8)] = o[nt][mt][e + 2];
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

// Bytes of shared memory that it takes.
template <int D, int kNT, int kWarps>
constexpr int join_bytes() {
  return (kWarps * (D + 4 + 2) + 2) * 8 * kNT * 4;
}

}  // namespace vdx
