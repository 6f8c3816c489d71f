// Argument checks shared by the C-ABI front ends of the paged-cache calls (kv_capi.cu, kv_evict_capi.cu): messages,
// strided tensors, and what may lie over what.  Host code; nothing here touches the device.
#pragma once
#include <algorithm>
#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <numeric>

#include <nvtx3/nvToolsExt.h>

#include "kv_internal.h"
#include "vdx.h"

namespace vdx {
namespace checks {

inline vdx_status fail(vdx_status s, const char* fmt, ...) noexcept {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    vdx::set_last_error(buf);
  } catch (...) {               // no memory for the message: the status still says what happened
  }
  return s;
}
inline void clear_error() noexcept { fail(VDX_OK, "%s", ""); }

struct NvtxScope {
  explicit NvtxScope(const char* name) { nvtxRangePushA(name); }
  ~NvtxScope() { nvtxRangePop(); }
};

inline int multiprocessors() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    return 152;
  }
  return sms;
}

// A strided [n0, n1, n2, d] tensor of 2-byte (or `size`-byte) elements; extents of 0 make it empty.
struct Tensor {
  const void* ptr;
  long long n[3];
  long long stride[3];
  int d;
  int size = 2;
  bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0; }
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(ptr); }
  uintptr_t end() const {
    if (empty()) return begin();
    long long last = d;
    for (int i = 0; i < 3; ++i) last += (n[i] - 1) * stride[i];
    return begin() + static_cast<uintptr_t>(last) * size;
  }
};
inline bool overlap(const Tensor& a, const Tensor& b) {
  return !a.empty() && !b.empty() && a.begin() < b.end() && b.begin() < a.end();
}
inline bool overlap(const Tensor& a, const void* p, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  return p && bytes && !a.empty() && a.begin() < x + bytes && x < a.end();
}

// What a call reads beside its tensors: lengths, page tables, weights.
struct Span {
  const void* p;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
inline Span ints(const int* p, long long n) { return {p, n > 0 ? static_cast<size_t>(n) * 4 : 0}; }
inline Span table_span(const int* table, int seqs, long long stride, int max_pages) {
  return ints(table, seqs > 0 ? (seqs - 1) * stride + max_pages : 0);
}

// Whether no row of `a` shares an element with a row of `b`, also where their spans interleave (slices of one
// fused projection): true if, with some of the dimensions walked inside a window, the windows of both
// repeat by steps with a common divisor and lie apart within it.  Both have elements of the same size.
inline bool rows_apart(const Tensor& a, const Tensor& b) {
  if (!overlap(a, b)) return true;
  const long long delta = (static_cast<long long>(b.begin()) - static_cast<long long>(a.begin())) / a.size;
  for (int inside = 0; inside < 7; ++inside) {
    long long wa = a.d, wb = b.d, step = 0;
    for (int i = 0; i < 3; ++i)
      if (inside >> i & 1) {
        wa += (a.n[i] - 1) * a.stride[i];
        wb += (b.n[i] - 1) * b.stride[i];
      } else {
        if (a.n[i] > 1) step = std::gcd(step, a.stride[i]);
        if (b.n[i] > 1) step = std::gcd(step, b.stride[i]);
      }
    if (step == 0) continue;
    const long long at = (delta % step + step) % step;
    if (at >= wa && at + wb <= step) return true;
  }
  return false;
}
// Whether the rows of a tensor that is written lie apart from one another.
inline bool rows_distinct(const Tensor& t) {
  if (t.empty()) return true;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return t.stride[x] < t.stride[y]; });
  long long span = t.d;
  for (int i : order) {
    if (t.n[i] <= 1) continue;
    if (t.stride[i] < span) return false;
    span += (t.n[i] - 1) * t.stride[i];
  }
  return true;
}

constexpr long long kMaxStride = 1ll << 38;   // elements: a tensor map's strides stay below 2^40 bytes
constexpr long long kMaxSpan = 1ll << 46;     // elements of a whole tensor

// 16-byte alignment, strides in multiples of 16 bytes, no zero stride but the batch's.
inline vdx_status check_tensor(const char* name, const Tensor& t, bool batch_may_repeat) {
  if (t.empty()) return VDX_OK;
  if (!t.ptr) return fail(VDX_ERR_ARG, "%s must be non-NULL", name);
  if (t.begin() & 15) return fail(VDX_ERR_ALIGN, "%s is not 16-byte aligned", name);
  long long span = t.d;
  for (int i = 0; i < 3; ++i) {
    if (t.n[i] == 1) continue;
    const long long s = t.stride[i];
    if (s < 0 || s > kMaxStride || s % (16 / t.size))
      return fail(VDX_ERR_ARG, "%s: stride %lld must be a multiple of %d elements in [0, 2^38]", name, s, 16 / t.size);
    if (s < t.d && !(s == 0 && i == 0 && batch_may_repeat))
      return fail(VDX_ERR_ARG, "%s: stride %lld is smaller than a row of %d channels", name, s, t.d);
    if (s && t.n[i] - 1 > kMaxSpan / s) return fail(VDX_ERR_ARG, "%s is too large", name);
    span += (t.n[i] - 1) * s;
  }
  if (span > kMaxSpan) return fail(VDX_ERR_ARG, "%s is too large", name);
  return VDX_OK;
}

inline vdx_status check_i32(const char* name, const int32_t* p, bool optional) {
  if (!p) return optional ? VDX_OK : fail(VDX_ERR_ARG, "%s must be non-NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 3) return fail(VDX_ERR_ALIGN, "%s is not 4-byte aligned", name);
  return VDX_OK;
}

inline vdx_status check_heads(int Hq, int Hkv, int d, int dtype) {
  if (dtype != VDX_DTYPE_BF16 && dtype != VDX_DTYPE_FP16) return fail(VDX_ERR_ARG, "unknown dtype %d", dtype);
  if (d != 64 && d != 128) return fail(VDX_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", d);
  if (Hkv < 1 || Hq < 1) return fail(VDX_ERR_ARG, "head counts must be >= 1 (got %d and %d)", Hq, Hkv);
  if (Hq % Hkv) return fail(VDX_ERR_ARG, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  if (Hq / Hkv > 128) return fail(VDX_ERR_UNSUPPORTED, "more than 128 query heads per kv head (%d / %d)", Hq, Hkv);
  return VDX_OK;
}

inline Tensor cache_tensor(const vdx_paged_kv& c, bool v, bool eight = false) {
  Tensor t{v ? c.v : c.k, {c.num_pages, c.page_size, c.Hkv}, {0, 0, 0}, c.d, eight ? 1 : 2};
  t.stride[0] = v ? c.v_page : c.k_page;
  t.stride[1] = v ? c.v_token : c.k_token;
  t.stride[2] = v ? c.v_head : c.k_head;
  return t;
}

// The scales of an 8-bit cache as a tensor of rows of one byte.
inline Tensor scale_tensor(const vdx_paged_kv& c, const vdx_kv8_scales& s, bool v) {
  Tensor t{v ? s.v : s.k, {c.num_pages, (c.page_size - 1) / VDX_KV8_BLOCK + 1, c.Hkv}, {0, 0, 0}, 1, 1};
  t.stride[0] = v ? s.v_page : s.k_page;
  t.stride[1] = v ? s.v_block : s.k_block;
  t.stride[2] = v ? s.v_head : s.k_head;
  return t;
}
inline vdx_status check_scales(const vdx_paged_kv& c, const vdx_kv8_scales& s) {
  for (bool v : {false, true}) {
    const Tensor t = scale_tensor(c, s, v);
    const char* name = v ? "the value scales" : "the key scales";
    if (!t.ptr) return fail(VDX_ERR_ARG, "%s must be non-NULL", name);
    long long span = 1;
    for (int i = 0; i < 3; ++i) {
      if (t.n[i] == 1) continue;
      if (t.stride[i] < 1 || t.stride[i] > kMaxStride) return fail(VDX_ERR_ARG, "%s: stride %lld must lie in [1, 2^38]", name, t.stride[i]);
      if (t.n[i] - 1 > kMaxSpan / t.stride[i]) return fail(VDX_ERR_ARG, "%s are too large", name);
      span += (t.n[i] - 1) * t.stride[i];
    }
    if (span > kMaxSpan) return fail(VDX_ERR_ARG, "%s are too large", name);
  }
  return VDX_OK;
}
inline Scales8 device_scales(const vdx_kv8_scales& s) {
  return {s.k, s.v, s.k_page, s.k_block, s.k_head, s.v_page, s.v_block, s.v_head};
}

// `scales`: of an 8-bit cache, NULL for one of 16 bits.
inline vdx_status check_cache(const vdx_paged_kv* c, int Hq, const vdx_kv8_scales* scales = nullptr) {
  if (!c) return fail(VDX_ERR_ARG, "the cache must be non-NULL");
  if (vdx_status s = check_heads(Hq, c->Hkv, c->d, c->dtype)) return s;
  if (c->seqs < 0 || c->num_pages < 1 || c->max_pages < 1)
    return fail(VDX_ERR_ARG, "seqs must be >= 0, num_pages and max_pages >= 1 (got %d, %d, %d)", c->seqs, c->num_pages,
                c->max_pages);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size < 128)
    return fail(VDX_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or >= 128 (got %d)", c->page_size);
  if (static_cast<long long>(c->max_pages) * c->page_size > 0x3fffffffll)
    return fail(VDX_ERR_ARG, "max_pages * page_size = %lld is too large",
                static_cast<long long>(c->max_pages) * c->page_size);
  if (c->table_stride < c->max_pages && c->seqs > 1)
    return fail(VDX_ERR_ARG, "table_stride %lld is smaller than max_pages %d", c->table_stride, c->max_pages);
  if (c->table_stride > kMaxStride && c->seqs > 1) return fail(VDX_ERR_ARG, "table_stride %lld is too large", c->table_stride);
  if (c->seqs > 0)
    if (vdx_status s = check_i32("page_table", c->page_table, false)) return s;
  if (vdx_status s = check_tensor("the key cache", cache_tensor(*c, false, scales), false)) return s;
  if (vdx_status s = check_tensor("the value cache", cache_tensor(*c, true, scales), false)) return s;
  return scales ? check_scales(*c, *scales) : VDX_OK;
}

// A cache that is written: no token, key or value may lie over another, nor a scale over anything else of it.
inline vdx_status check_written_cache(const vdx_paged_kv& c, const vdx_kv8_scales* scales) {
  const Tensor kc = cache_tensor(c, false, scales), vc = cache_tensor(c, true, scales);
  if (!rows_distinct(kc)) return fail(VDX_ERR_ARG, "tokens of the key cache overlap one another");
  if (!rows_distinct(vc)) return fail(VDX_ERR_ARG, "tokens of the value cache overlap one another");
  if (c.k == c.v) return fail(VDX_ERR_ARG, "the key and value caches are the same memory");
  if (!rows_apart(kc, vc)) return fail(VDX_ERR_ARG, "the key and value caches overlap");
  if (!scales) return VDX_OK;
  const Tensor ks = scale_tensor(c, *scales, false), vs = scale_tensor(c, *scales, true);
  if (!rows_distinct(ks) || !rows_distinct(vs)) return fail(VDX_ERR_ARG, "scales overlap one another");
  if (!rows_apart(ks, vs)) return fail(VDX_ERR_ARG, "the key and value scales overlap");
  if (overlap(ks, kc) || overlap(ks, vc) || overlap(vs, kc) || overlap(vs, vc)) return fail(VDX_ERR_ARG, "the scales overlap the cache");
  return VDX_OK;
}

}  // namespace checks
}  // namespace vdx
