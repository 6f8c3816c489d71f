// Warp-level pieces shared by the few-row kernels (attn_rows.cu, kv_weigh.cu): asynchronous copies, fragments,
// m16n8k16 products, queries as fp16.
#pragma once
#include <type_traits>

#include "kv8.cuh"
#include "kv_common.cuh"

namespace vdx {

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

// The query fragments of one row (channels of four lanes) from T to fp16, and the two row factors this lane's scores need.
template <typename T, int D>
__device__ __forceinline__ void query_to_half(uint32_t (&q)[D / 16][2], int nt, int c4, float (*row_scale)[2], float scale_log2) {
  int e = 0;                             // the row is multiplied by 2^e
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float2 x = unpack2<T>(q[i / 2][i % 2]);
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // into [2^14, 2^15); what falls below fp16's steps is less than 2^-39 of the row's largest
    const int x = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = min(max(14 - x, -120), 120);
    const float up = two_to(e);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float2 v = unpack2<T>(q[i / 2][i % 2]);
      q[i / 2][i % 2] = pack2<__half>(v.x * up, v.y * up);
    }
  }
  const float down = scale_log2 * two_to(-e);           // of row 8*nt + gq, the same in its four lanes
#pragma unroll
  for (int i = 0; i < 2; ++i) row_scale[nt][i] = __shfl_sync(0xffffffffu, down, (2 * c4 + i) * 4);
}

}  // namespace vdx
