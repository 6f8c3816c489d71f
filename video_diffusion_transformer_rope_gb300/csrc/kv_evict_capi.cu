// C-ABI front end of the calls that keep a cache small: gathered attention weights and eviction.  Argument checks and
// dispatch; nothing here allocates, synchronises or keeps state between calls.
#include <cmath>

#include "kv_checks.h"

namespace {

using namespace vdx::checks;

// [seqs, Hkv, width] floats with strides: what they span, and whether the heads' rows lie apart.
struct Weights {
  const float* p;
  long long seq, head;
  int seqs, heads, width;
  Tensor tensor() const { return {p, {1, seqs, heads}, {0, seq, head}, width, 4}; }
};
vdx_status check_weights(const char* name, const Weights& w, bool written) {
  const Tensor t = w.tensor();
  if (t.empty() || w.width == 0) return VDX_OK;
  if (!w.p) return fail(VDX_ERR_ARG, "%s must be non-NULL", name);
  if (t.begin() & 3) return fail(VDX_ERR_ALIGN, "%s is not 4-byte aligned", name);
  for (int i = 1; i < 3; ++i)
    if (t.n[i] > 1 && (t.stride[i] < w.width || t.stride[i] > kMaxStride || t.n[i] - 1 > kMaxSpan / t.stride[i]))
      return fail(VDX_ERR_ARG, "%s: stride %lld must lie in [%d, 2^38]", name, t.stride[i], w.width);
  if (written && !rows_distinct(t)) return fail(VDX_ERR_ARG, "rows of %s overlap one another", name);
  return VDX_OK;
}

}  // namespace

extern "C" {

vdx_status vdx_paged_attn_weights(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_paged_weights_args* a, void* stream) {
  NvtxScope nvtx("vdx_paged_attn_weights");
  clear_error();
  if (!a) return fail(VDX_ERR_ARG, "the arguments must be non-NULL");
  if (vdx_status s = check_cache(c, a->Hq, scales)) return s;
  if (a->rows < 0 || a->max_q < 0 || a->max_kv < 0 || a->causal_block < 0 || a->width < 0)
    return fail(VDX_ERR_ARG, "rows, max_q, max_kv, causal_block and width must be >= 0 (got %d, %d, %d, %d, %d)", a->rows, a->max_q,
                a->max_kv, a->causal_block, a->width);
  if (!std::isfinite(a->decay)) return fail(VDX_ERR_ARG, "decay must be finite");
  if (!std::isfinite(a->scale)) return fail(VDX_ERR_ARG, "scale must be finite");
  vdx::WeighParams wp{};
  vdx::KvParams& p = wp.kv;
  p.scale_log2 = static_cast<float>((a->scale > 0.f ? a->scale : 1.0 / std::sqrt(static_cast<double>(c->d))) * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return fail(VDX_ERR_ARG, "scale = %g is too large", static_cast<double>(a->scale));
  p.q = a->q; p.k = c->k;
  p.q_t = a->q_row; p.q_h = a->q_head;
  p.k_p = c->k_page; p.k_t = c->k_token; p.k_h = c->k_head;
  p.cu = a->cu; p.kv_len = a->kv_len; p.pos_offset = a->causal_block ? a->pos_offset : nullptr; p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages; p.num_pages = c->num_pages; p.P = c->page_size;
  p.S = c->seqs; p.N = a->rows; p.Hq = a->Hq; p.Hkv = c->Hkv; p.g = a->Hq / c->Hkv;
  const int cap = std::min(c->max_pages * c->page_size, a->width);
  p.max_q = a->max_q > 0 ? std::min(a->max_q, a->rows) : a->rows;
  p.max_kv = a->max_kv > 0 ? std::min(a->max_kv, cap) : cap;
  p.causal_block = a->causal_block;
  p.eight = scales != nullptr;
  if (scales) p.scales = device_scales(*scales);
  wp.lse = a->lse; wp.w = a->w; wp.w_seq = a->w_seq; wp.w_head = a->w_head; wp.decay = a->decay;
  const Tensor q{a->q, {1, c->seqs > 0 ? a->rows : 0, a->Hq}, {0, a->q_row, a->q_head}, c->d};
  const Weights w{a->w, a->w_seq, a->w_head, c->seqs, c->Hkv, a->width};
  if (q.empty()) return VDX_OK;
  if (static_cast<long long>(p.max_q) * p.g > 0x7ffff000ll)
    return fail(VDX_ERR_ARG, "%d rows of %d heads per kv head are too many", p.max_q, p.g);
  // 256 keys take 1.1 us for every 128 rows (0.6 s at this many), and a warp of the tile kernel waits for all of them, a second at most
  if (static_cast<long long>(p.max_q) * p.g > vdx::kMaxWeighRows)
    return fail(VDX_ERR_UNSUPPORTED, "more than %d rows per kv head (%d of %d heads); where sequences have fewer, pass max_q", vdx::kMaxWeighRows,
                p.max_q, p.g);
  if (static_cast<long long>(p.S) * p.Hkv > 0x3fffffffll)
    return fail(VDX_ERR_ARG, "%d sequences of %d kv heads are too many", p.S, p.Hkv);
  if (vdx_status s = check_i32("cu", a->cu, false)) return s;
  if (vdx_status s = check_i32("kv_len", a->kv_len, false)) return s;
  if (vdx_status s = check_i32("pos_offset", a->pos_offset, true)) return s;
  if (vdx_status s = check_tensor("q", q, true)) return s;
  if (!a->lse) return fail(VDX_ERR_ARG, "lse must be non-NULL");
  if (reinterpret_cast<uintptr_t>(a->lse) & 3) return fail(VDX_ERR_ALIGN, "lse is not 4-byte aligned");
  if (vdx_status s = check_weights("the weights", w, true)) return s;
  const Tensor wt = w.tensor(), kc = cache_tensor(*c, false, scales);
  const Span reads[5] = {ints(a->cu, c->seqs + 1ll), ints(a->kv_len, c->seqs), ints(p.pos_offset, c->seqs),
                         table_span(c->page_table, c->seqs, c->table_stride, c->max_pages),
                         {a->lse, static_cast<size_t>(a->rows) * a->Hq * 4}};
  if (overlap(wt, q) || overlap(wt, kc) || (scales && overlap(wt, scale_tensor(*c, *scales, false))))
    return fail(VDX_ERR_ARG, "the weights overlap q or the cache");
  if (a->width > 0)
    for (const Span& r : reads)
      if (overlap(wt, r.p, r.bytes)) return fail(VDX_ERR_ARG, "the weights overlap cu, kv_len, pos_offset, page_table or lse");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const char* what = nullptr;
  // No place for any key (width 0): the kernel of few rows looks at lengths, which are reported; that of tiles has no units.
  if (static_cast<long long>(p.max_q) * p.g <= 32 || p.max_kv == 0) {
    e = vdx::launch_weigh_rows(wp, c->d, c->dtype, multiprocessors(), st);
  } else {
    vdx::EncodeTiledFn encode = nullptr;
    if (!vdx::encode_tiled_fn(&encode)) return VDX_ERR_CUDA;
    e = vdx::launch_weigh_tiles(wp, c->d, c->dtype, encode, multiprocessors(), st, &what);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(VDX_ERR_CUDA, "weights kernel launch: %s%s%s", what ? what : "", what ? ": " : "", cudaGetErrorString(e));
  }
  return VDX_OK;
}

vdx_status vdx_paged_evict(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_paged_kv* to, const vdx_kv8_scales* to_scales,
                           const vdx_paged_evict_args* a, void* stream) {
  NvtxScope nvtx("vdx_paged_evict");
  clear_error();
  if (!a) return fail(VDX_ERR_ARG, "the arguments must be non-NULL");
  if (vdx_status s = check_cache(c, c ? c->Hkv : 1, scales)) return s;
  if (vdx_status s = check_cache(to, to ? to->Hkv : 1, to_scales)) return s;
  if (!scales != !to_scales || c->Hkv != to->Hkv || c->d != to->d || c->dtype != to->dtype || c->seqs != to->seqs)
    return fail(VDX_ERR_ARG, "the two caches must be of one kind: heads, channels, type, bits and sequences");
  if (a->keep < 1 || a->recent < 0 || a->recent > a->keep || a->width < 0 || a->max_kv < 0)
    return fail(VDX_ERR_ARG, "keep must be >= 1, recent in [0, keep], width and max_kv >= 0 (got %d, %d, %d, %d)", a->keep, a->recent,
                a->width, a->max_kv);
  if (static_cast<long long>(a->keep) > 0x3fffffffll) return fail(VDX_ERR_ARG, "keep = %d is too large", a->keep);
  if (c->seqs == 0) return VDX_OK;
  if (static_cast<long long>(c->seqs) * c->Hkv > 0x3fffffffll)
    return fail(VDX_ERR_ARG, "%d sequences of %d kv heads are too many", c->seqs, c->Hkv);
  const bool same = a->w == a->w_out;
  if (same && (a->w_seq != a->w_out_seq || a->w_head != a->w_out_head)) return fail(VDX_ERR_ARG, "w_out is w with other strides");
  if (same && a->width < a->keep) return fail(VDX_ERR_ARG, "width %d of w, which is w_out too, is smaller than keep %d", a->width, a->keep);
  const Weights w{a->w, a->w_seq, a->w_head, c->seqs, c->Hkv, a->width};
  const Weights wo{a->w_out, a->w_out_seq, a->w_out_head, c->seqs, c->Hkv, a->keep};
  if (vdx_status s = check_weights("w", w, same)) return s;       // in place a head is written while others are read
  if (vdx_status s = check_weights("w_out", wo, true)) return s;
  if (vdx_status s = check_i32("kv_len", a->kv_len, false)) return s;
  if (vdx_status s = check_i32("pos_offset", a->pos_offset, true)) return s;
  if (vdx_status s = check_i32("kv_len_out", a->kv_len_out, false)) return s;
  if (vdx_status s = check_i32("pos_offset_out", a->pos_offset_out, true)) return s;
  if (vdx_status s = check_i32("index", a->index, false)) return s;
  if (vdx_status s = check_written_cache(*to, to_scales)) return s;

  // The pools may be the same tensors (by pages apart); the tables may not be.
  const Tensor kc = cache_tensor(*c, false, scales), vc = cache_tensor(*c, true, scales);
  const Tensor kt = cache_tensor(*to, false, scales), vt = cache_tensor(*to, true, scales);
  const bool one_pool = c->k == to->k && c->v == to->v;
  if (one_pool) {
    bool alike = c->num_pages == to->num_pages && c->page_size == to->page_size && c->k_page == to->k_page && c->k_token == to->k_token &&
                 c->k_head == to->k_head && c->v_page == to->v_page && c->v_token == to->v_token && c->v_head == to->v_head;
    if (scales)
      alike = alike && scales->k == to_scales->k && scales->v == to_scales->v && scales->k_page == to_scales->k_page &&
              scales->k_block == to_scales->k_block && scales->k_head == to_scales->k_head && scales->v_page == to_scales->v_page &&
              scales->v_block == to_scales->v_block && scales->v_head == to_scales->v_head;
    if (!alike) return fail(VDX_ERR_ARG, "two caches in the same pools must have the same strides, pages and scales");
    if (c->page_table == to->page_table) return fail(VDX_ERR_ARG, "the two caches have the same page table: what stays needs pages of its own");
  } else if (!rows_apart(kc, kt) || !rows_apart(kc, vt) || !rows_apart(vc, kt) || !rows_apart(vc, vt)) {
    return fail(VDX_ERR_ARG, "the two caches overlap without being the same pools");
  }
  const Span reads[4] = {ints(a->kv_len, c->seqs), ints(a->pos_offset, c->seqs),
                         table_span(c->page_table, c->seqs, c->table_stride, c->max_pages),
                         table_span(to->page_table, to->seqs, to->table_stride, to->max_pages)};
  const Span writes[3] = {ints(a->kv_len_out, c->seqs), ints(a->pos_offset_out, c->seqs),
                          ints(a->index, static_cast<long long>(c->seqs) * c->Hkv * a->keep)};
  const Tensor wt = w.tensor(), wot = wo.tensor();
  std::initializer_list<Tensor> caches = {kc, vc, kt, vt};
  for (int i = 0; i < 3; ++i) {
    for (const Span& r : reads)
      if (overlap(r, writes[i])) return fail(VDX_ERR_ARG, "kv_len_out, pos_offset_out or index overlaps kv_len, pos_offset or a page table");
    for (int j = 0; j < i; ++j)
      if (overlap(writes[i], writes[j])) return fail(VDX_ERR_ARG, "kv_len_out, pos_offset_out and index overlap one another");
    if (overlap(wot, writes[i].p, writes[i].bytes) || (a->width > 0 && overlap(wt, writes[i].p, writes[i].bytes)))
      return fail(VDX_ERR_ARG, "kv_len_out, pos_offset_out or index overlaps w or w_out");
    for (const Tensor& t : caches)
      if (overlap(t, writes[i].p, writes[i].bytes)) return fail(VDX_ERR_ARG, "kv_len_out, pos_offset_out or index overlaps a cache");
  }
  for (const Span& r : reads) {
    if (overlap(wot, r.p, r.bytes)) return fail(VDX_ERR_ARG, "w_out overlaps kv_len, pos_offset or a page table");
    if (overlap(kt, r.p, r.bytes) || overlap(vt, r.p, r.bytes)) return fail(VDX_ERR_ARG, "a cache overlaps kv_len, pos_offset or a page table");
  }
  if (!same && a->width > 0 && !rows_apart(wot, wt)) return fail(VDX_ERR_ARG, "w_out overlaps w");
  for (const Tensor& t : caches)
    if (overlap(wot, t)) return fail(VDX_ERR_ARG, "w_out overlaps a cache");
  if (a->width > 0 && (overlap(wt, kt) || overlap(wt, vt))) return fail(VDX_ERR_ARG, "w overlaps the cache that is written");
  if (scales) {
    for (bool v : {false, true}) {
      const Tensor st = scale_tensor(*to, *to_scales, v), sf = scale_tensor(*c, *scales, v), other = scale_tensor(*c, *scales, !v);
      if (!one_pool && (!rows_apart(st, sf) || !rows_apart(st, other))) return fail(VDX_ERR_ARG, "the scales of the two caches overlap");
      for (const Tensor& t : caches)
        if (overlap(st, t) || (!one_pool && overlap(sf, t) && (t.ptr == kt.ptr || t.ptr == vt.ptr)))
          return fail(VDX_ERR_ARG, "scales overlap a cache");
      if (overlap(st, wot) || overlap(sf, wot) || (a->width > 0 && overlap(st, wt))) return fail(VDX_ERR_ARG, "scales overlap w or w_out");
      for (const Span& x : reads)
        if (overlap(st, x.p, x.bytes)) return fail(VDX_ERR_ARG, "scales overlap kv_len, pos_offset or a page table");
      for (const Span& x : writes)
        if (overlap(st, x.p, x.bytes) || overlap(sf, x.p, x.bytes)) return fail(VDX_ERR_ARG, "scales overlap kv_len_out, pos_offset_out or index");
    }
  }

  vdx::EvictParams p{};
  const int size = scales ? 1 : 2;
  p.k = static_cast<const uint8_t*>(c->k); p.v = static_cast<const uint8_t*>(c->v);
  p.k_to = static_cast<uint8_t*>(to->k); p.v_to = static_cast<uint8_t*>(to->v);
  p.k_p = c->k_page * size; p.k_t = c->k_token * size; p.k_h = c->k_head * size;
  p.v_p = c->v_page * size; p.v_t = c->v_token * size; p.v_h = c->v_head * size;
  p.kt_p = to->k_page * size; p.kt_t = to->k_token * size; p.kt_h = to->k_head * size;
  p.vt_p = to->v_page * size; p.vt_t = to->v_token * size; p.vt_h = to->v_head * size;
  p.table = c->page_table; p.table_stride = c->table_stride;
  p.table_to = to->page_table; p.table_to_stride = to->table_stride;
  p.P = c->page_size; p.num_pages = c->num_pages;
  p.P_to = to->page_size; p.num_pages_to = to->num_pages; p.max_pages_to = to->max_pages;
  p.S = c->seqs; p.Hkv = c->Hkv; p.keep = a->keep; p.recent = a->recent;
  const int cap = std::min(c->max_pages * c->page_size, a->width);
  p.max_kv = a->max_kv > 0 ? std::min(a->max_kv, cap) : cap;
  if (p.max_kv > vdx::kMaxEvictKeys)
    return fail(VDX_ERR_UNSUPPORTED, "eviction from up to %d keys; max_kv, the page table and width allow %d", vdx::kMaxEvictKeys, p.max_kv);
  p.w = a->w; p.w_out = a->w_out; p.w_seq = a->w_seq; p.w_head = a->w_head; p.w_out_seq = a->w_out_seq; p.w_out_head = a->w_out_head;
  p.kv_len = a->kv_len; p.pos_offset = a->pos_offset; p.kv_len_out = a->kv_len_out; p.pos_offset_out = a->pos_offset_out;
  p.index = a->index;
  if (scales) {
    p.scales = device_scales(*scales);
    p.scales_to = device_scales(*to_scales);
  }
  const cudaError_t e = vdx::launch_evict(p, c->d, scales != nullptr, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(VDX_ERR_CUDA, "eviction kernel launch: %s", cudaGetErrorString(e));
  }
  return VDX_OK;
}

}  // extern "C"
