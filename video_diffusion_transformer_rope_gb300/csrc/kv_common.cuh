// Device helpers shared by the paged-cache and cross-attention kernels: element conversions,
// sequence lookup, visibility limits, and the translation unit's error word.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kv_internal.h"
#include "sm103_ptx.cuh"

namespace vdx {

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack2<T>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}

// Loads of what the work just ahead in the stream may have written (lengths, page tables, rows, weights): ordinary
// ones, which wait_for_earlier_work() holds back (it clobbers memory) and makes see those writes.  Neither
// holds for the read-only path (ld.global.nc): that is for memory that nobody writes while the kernel runs, and a
// kernel that starts early is running while the work before it still writes.  Cached in L1, where the
// look-ups of neighbouring blocks and pages hit (through L2 alone 48 tokens over 8-33 thousand keys take 882 us,
// not 662, and 3120 appended tokens 18.1, not 13.9).
__device__ __forceinline__ int load_i32(const int* p) { return *p; }
__device__ __forceinline__ uint32_t load_b32(const void* p) { return *static_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint4 load_b128(const void* p) { return *static_cast<const uint4*>(p); }

// The last s in [0, S) with cu[s] <= r (0 if none), found by the whole warp: each step its lanes
// probe 32 evenly spaced starts, so up to 32 sequences take one load.  With cu not decreasing it
// is the sequence that owns row r, if any does; the caller checks cu[s] <= r < cu[s + 1].
__device__ __forceinline__ int find_sequence(const int* cu, int S, int r) {
  int lo = 0, n = S;                      // the answer is in [lo, lo + n)
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const bool le = off < n && load_i32(cu + lo + off) <= r;
    // the highest probe at or below r; probes past a decreasing cu only make the result wrong,
    // not out of range
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int top = m ? 31 - __clz(m) : 0;
    lo += top * step;
    n = min(step, n - top * step);
  }
  return lo;
}

// Rows and keys of one sequence, clamped to what was passed by the host.
struct SeqInfo {
  int row0;   // first token in q / out
  int n;      // tokens
  int len;    // keys
  int shift;  // tokens of its block of causal_block that lie before key 0 (dropped ones)
};
__device__ __forceinline__ SeqInfo sequence_info(const KvParams& p, int s, bool report) {
  SeqInfo q;
  bool bad = false;
  if (p.cu) {
    int a = load_i32(p.cu + s), b = load_i32(p.cu + s + 1);
    bad = a < 0 || b < a || b > p.N;
    a = min(max(a, 0), p.N);
    b = min(max(b, a), p.N);
    q.row0 = a;
    q.n = b - a;
    bad = bad || q.n > p.max_q;
  } else {
    q.row0 = 0;
    q.n = p.N;
  }
  if (p.kv_len) {
    const int len = load_i32(p.kv_len + s);
    q.len = min(max(len, 0), p.max_kv);
    bad = bad || len != q.len;
  } else {
    q.len = p.max_kv;
  }
  q.shift = 0;
  if (p.pos_offset) {
    q.shift = load_i32(p.pos_offset + s) % p.causal_block;
    if (q.shift < 0) q.shift += p.causal_block;
  }
  if (bad && report) atomicOr(&g_error_word, kErrLength);
  return q;
}
// Keys that row i of the sequence sees: keys 0 .. limit-1.
__device__ __forceinline__ int visible_limit(const KvParams& p, const SeqInfo& q, int i) {
  if (p.causal_block <= 0) return q.len;
  const int pos = q.len - q.n + i;        // q.n may exceed q.len: negative positions see nothing
  if (pos < 0) return 0;
  // to the end of its block; pos < 2^30, shift and causal_block < 2^31
  const unsigned in_block = (static_cast<unsigned>(pos) + q.shift) % static_cast<unsigned>(p.causal_block);
  return static_cast<int>(min(static_cast<unsigned>(pos) + (p.causal_block - in_block), static_cast<unsigned>(q.len)));
}

// Offset of token `tok` of sequence s in q, and in out (elements, head 0).
__device__ __forceinline__ long long out_row(const KvParams& p, int s, const SeqInfo& q, int tok) {
  return p.cu ? static_cast<long long>(q.row0) + tok : static_cast<long long>(s) * p.N + tok;
}
__device__ __forceinline__ long long lse_index(const KvParams& p, int s, const SeqInfo& q, int h, int tok) {
  return p.cu ? static_cast<long long>(h) * p.N + q.row0 + tok
              : (static_cast<long long>(s) * p.Hq + h) * p.N + tok;
}

// Everything before this call in its stream has finished and is visible.  The kernels are launched so that
// they may start while the work before them drains (launch_early), and touch no memory of the caller's until
// here: 0.5 us less for each of a chain of calls (8 tokens appended 4.2 -> 3.7 us, 4 x 12 heads over 1000
// keys 9.3 -> 8.8).  None of them lets the next one start before its blocks have finished: that gained nothing.
__device__ __forceinline__ void wait_for_earlier_work() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Host: the launch attribute for it.
inline cudaLaunchAttribute launch_early() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// Host: whether this translation unit has launched a kernel (or captured one) in this process.  Until then its
// error word is 0, and reading it would load its kernels and cost every synchronising check a copy.
static std::atomic<bool> g_launched{false};
inline void note_launch() {
  if (!g_launched.load(std::memory_order_relaxed)) g_launched.store(true, std::memory_order_release);
}

// Host: read and reset this translation unit's error word.
static cudaError_t read_and_clear_word(unsigned int* word) {
  *word = 0;
  if (!g_launched.load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaMemcpyFromSymbol(word, g_error_word, sizeof(unsigned int));
  if (e != cudaSuccess || *word == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
}

}  // namespace vdx
