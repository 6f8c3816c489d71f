// C-ABI front end of the paged-cache and cross-attention calls: argument checks, the launch plan,
// dispatch.  Nothing here allocates, synchronises or keeps state between calls.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kv_checks.h"

namespace {

using namespace vdx::checks;

// ------------------------------------------------------------------------------------- attention
struct Problem {
  vdx::KvParams p{};
  int d = 0, dtype = 0;
  bool nothing = false;        // no rows: nothing to launch
  size_t workspace = 0;
};

vdx_status finish(Problem* pb, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& k_scale, const Tensor& v_scale,
                  long long out_elems, long long lse_elems, float scale, const void* workspace, size_t workspace_bytes, bool size_only) {
  vdx::KvParams& p = pb->p;
  if (!std::isfinite(scale)) return fail(VDX_ERR_ARG, "scale must be finite");
  p.scale_log2 = static_cast<float>((scale > 0.f ? scale : 1.0 / std::sqrt(static_cast<double>(pb->d))) * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return fail(VDX_ERR_ARG, "scale = %g is too large", static_cast<double>(scale));
  pb->nothing = q.empty();
  if (pb->nothing) return VDX_OK;
  if (static_cast<long long>(p.max_q) * p.g > 0x7ffff000ll)     // row numbers of padded blocks stay in an int
    return fail(VDX_ERR_ARG, "%d rows of %d heads per kv head are too many", p.max_q, p.g);
  if (static_cast<long long>(p.S) * p.Hkv > 0x3fffffffll)       // a launch has fewer blocks; products below stay in 64 bits
    return fail(VDX_ERR_ARG, "%d sequences of %d kv heads are too many", p.S, p.Hkv);
  if (vdx_status s = check_tensor("q", q, true)) return s;
  if (vdx_status s = check_tensor("k", k, true)) return s;
  if (vdx_status s = check_tensor("v", v, true)) return s;
  pb->workspace = vdx::plan_attention(&p, pb->d, multiprocessors());
  if (size_only) return VDX_OK;
  if (!p.out) return fail(VDX_ERR_ARG, "out must be non-NULL");
  if ((reinterpret_cast<uintptr_t>(p.out) & 15) || (reinterpret_cast<uintptr_t>(p.lse) & 3))
    return fail(VDX_ERR_ALIGN, "out is not 16-byte aligned or lse not 4-byte aligned");
  const size_t out_bytes = static_cast<size_t>(out_elems) * 2, lse_bytes = static_cast<size_t>(lse_elems) * 4;
  const Tensor* in[3] = {&q, &k, &v};
  const Tensor out{p.out, {1, 1, out_elems / pb->d}, {0, 0, pb->d}, pb->d};
  for (const Tensor* t : in) {
    if (overlap(*t, out)) return fail(VDX_ERR_ARG, "out overlaps q, k or v");
    if (overlap(*t, p.lse, lse_bytes)) return fail(VDX_ERR_ARG, "lse overlaps q, k or v");
  }
  if (overlap(out, p.lse, lse_bytes)) return fail(VDX_ERR_ARG, "lse overlaps out");
  if (pb->workspace) {
    if (!workspace || workspace_bytes < pb->workspace)
      return fail(VDX_ERR_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace ? workspace_bytes : 0,
                  pb->workspace);
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return fail(VDX_ERR_ALIGN, "workspace is not 16-byte aligned");
    const uintptr_t w = reinterpret_cast<uintptr_t>(workspace);
    const uintptr_t l = reinterpret_cast<uintptr_t>(p.lse);
    if (overlap(q, workspace, pb->workspace) || overlap(k, workspace, pb->workspace) || overlap(v, workspace, pb->workspace) ||
        overlap(out, workspace, pb->workspace) || (p.lse && w < l + lse_bytes && l < w + pb->workspace))
      return fail(VDX_ERR_ARG, "workspace overlaps q, k, v, out or lse");
    uint8_t* ws = const_cast<uint8_t*>(static_cast<const uint8_t*>(workspace));
    const long long rows = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit * p.block_rows;
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + static_cast<size_t>(rows) * pb->d * 4);
  }
  const Span reads[4] = {ints(p.cu, p.cu ? p.S + 1ll : 0), ints(p.kv_len, p.S), ints(p.pos_offset, p.S),
                         table_span(p.table, p.S, p.table_stride, p.max_pages)};
  const Span writes[3] = {{p.out, out_bytes}, {p.lse, lse_bytes}, {pb->workspace ? workspace : nullptr, pb->workspace}};
  for (const Span& w : writes)
    if (overlap(k_scale, w.p, w.bytes) || overlap(v_scale, w.p, w.bytes)) return fail(VDX_ERR_ARG, "out, lse or workspace overlaps the scales");
  for (const Span& r : reads)
    for (const Span& w : writes)
      if (overlap(r, w)) return fail(VDX_ERR_ARG, "out, lse or workspace overlaps cu, kv_len, pos_offset or page_table");
  return VDX_OK;
}

vdx_status paged_problem(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_paged_attn_args* a, const int32_t* pos_offset,
                         bool size_only, Problem* pb) {
  if (!a) return fail(VDX_ERR_ARG, "the arguments must be non-NULL");
  if (vdx_status s = check_cache(c, a->Hq, scales)) return s;
  if (a->rows < 0 || a->max_q < 0 || a->max_kv < 0 || a->causal_block < 0)
    return fail(VDX_ERR_ARG, "rows, max_q, max_kv and causal_block must be >= 0 (got %d, %d, %d, %d)", a->rows, a->max_q,
                a->max_kv, a->causal_block);
  vdx::KvParams& p = pb->p;
  pb->d = c->d;
  pb->dtype = c->dtype;
  p.q = a->q; p.k = c->k; p.v = c->v; p.out = a->out; p.lse = a->lse;
  p.q_b = 0; p.q_t = a->q_row; p.q_h = a->q_head;
  p.k_p = c->k_page; p.k_t = c->k_token; p.k_h = c->k_head;
  p.v_p = c->v_page; p.v_t = c->v_token; p.v_h = c->v_head;
  p.cu = a->cu; p.kv_len = a->kv_len; p.pos_offset = a->causal_block ? pos_offset : nullptr; p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages; p.num_pages = c->num_pages; p.P = c->page_size;
  p.S = c->seqs; p.N = a->rows; p.Hq = a->Hq; p.Hkv = c->Hkv; p.g = a->Hq / c->Hkv;
  const int cap = c->max_pages * c->page_size;
  p.max_q = a->max_q > 0 ? std::min(a->max_q, a->rows) : a->rows;
  p.max_kv = a->max_kv > 0 ? std::min(a->max_kv, cap) : cap;
  p.causal_block = a->causal_block;
  const Tensor q{a->q, {1, c->seqs > 0 ? a->rows : 0, a->Hq}, {0, a->q_row, a->q_head}, c->d};
  if (!q.empty()) {
    if (vdx_status s = check_i32("cu", a->cu, false)) return s;
    if (vdx_status s = check_i32("kv_len", a->kv_len, false)) return s;
    if (vdx_status s = check_i32("pos_offset", pos_offset, true)) return s;
  }
  p.eight = scales != nullptr;
  if (scales) p.scales = device_scales(*scales);
  const Tensor none{};
  return finish(pb, q, cache_tensor(*c, false, scales), cache_tensor(*c, true, scales),
                scales ? scale_tensor(*c, *scales, false) : none, scales ? scale_tensor(*c, *scales, true) : none,
                static_cast<long long>(a->rows) * a->Hq * c->d, a->lse ? static_cast<long long>(a->rows) * a->Hq : 0,
                a->scale, a->workspace, a->workspace_bytes, size_only);
}

vdx_status cross_problem(const vdx_cross_attn_args* a, bool size_only, Problem* pb) {
  if (!a) return fail(VDX_ERR_ARG, "the arguments must be non-NULL");
  if (vdx_status s = check_heads(a->Hq, a->Hkv, a->d, a->dtype)) return s;
  if (a->B < 0 || a->N < 0 || a->M < 0) return fail(VDX_ERR_ARG, "B, N and M must be >= 0 (got %d, %d, %d)", a->B, a->N, a->M);
  if (a->M > 0x3fffffff) return fail(VDX_ERR_ARG, "M = %d is too large", a->M);
  vdx::KvParams& p = pb->p;
  pb->d = a->d;
  pb->dtype = a->dtype;
  p.q = a->q; p.k = a->k; p.v = a->v; p.out = a->out; p.lse = a->lse;
  p.q_b = a->q_batch; p.q_t = a->q_row; p.q_h = a->q_head;
  p.k_p = a->k_batch; p.k_t = a->k_token; p.k_h = a->k_head;
  p.v_p = a->v_batch; p.v_t = a->v_token; p.v_h = a->v_head;
  p.kv_len = a->kv_len;
  p.num_pages = a->B; p.P = a->M;
  p.S = a->B; p.N = a->N; p.Hq = a->Hq; p.Hkv = a->Hkv; p.g = a->Hq / a->Hkv;
  p.max_q = a->N; p.max_kv = a->M;
  if (vdx_status s = check_i32("kv_len", a->kv_len, true)) return s;
  const Tensor q{a->q, {a->B, a->N, a->Hq}, {a->q_batch, a->q_row, a->q_head}, a->d};
  const Tensor k{a->k, {a->B, a->M, a->Hkv}, {a->k_batch, a->k_token, a->k_head}, a->d};
  const Tensor v{a->v, {a->B, a->M, a->Hkv}, {a->v_batch, a->v_token, a->v_head}, a->d};
  const long long rows = static_cast<long long>(a->B) * a->N * a->Hq;
  if (rows > kMaxSpan / a->d) return fail(VDX_ERR_ARG, "out is too large");
  return finish(pb, q, k, v, Tensor{}, Tensor{}, rows * a->d, a->lse ? rows : 0, a->scale, a->workspace, a->workspace_bytes, size_only);
}

vdx_status launch(const Problem& pb, void* stream) {
  if (pb.nothing) return VDX_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const char* what = nullptr;
  if (pb.p.rows_kernel) {
    e = (pb.p.eight ? vdx::launch_attn_rows8 : vdx::launch_attn_rows)(pb.p, pb.d, pb.dtype, st);
  } else {
    vdx::EncodeTiledFn encode = nullptr;
    if (!vdx::encode_tiled_fn(&encode)) return VDX_ERR_CUDA;
    e = vdx::launch_attn_tiles(pb.p, pb.d, pb.dtype, encode, multiprocessors(), st, &what);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();          // reported here; not left for the process's next CUDA call
    return fail(VDX_ERR_CUDA, "attention kernel launch: %s%s%s", what ? what : "", what ? ": " : "", cudaGetErrorString(e));
  }
  if (pb.p.nsplit > 1 && !pb.p.cluster) {
    e = vdx::launch_attn_combine(pb.p, pb.d, pb.dtype, st);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(VDX_ERR_CUDA, "join kernel launch: %s", cudaGetErrorString(e));
    }
  }
  return VDX_OK;
}

// ------------------------------------------------------------------------------------- append
vdx_status append(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_append_args* a, void* stream) {
  if (!a) return fail(VDX_ERR_ARG, "the arguments must be non-NULL");
  if (vdx_status s = check_cache(c, a->q ? a->Hq : (c ? c->Hkv : 1), scales)) return s;
  const int d = c->d;
  if (a->rows < 0) return fail(VDX_ERR_ARG, "rows must be >= 0 (got %d)", a->rows);
  if (!a->q != !a->q_out) return fail(VDX_ERR_ARG, "q and q_out go together");
  if (a->T < 1 || a->Hgrid < 1 || a->Wgrid < 1)
    return fail(VDX_ERR_ARG, "T, Hgrid and Wgrid must be >= 1 (got %d %d %d)", a->T, a->Hgrid, a->Wgrid);
  if (static_cast<long long>(a->Hgrid) * a->Wgrid > 0x7fffffffll)
    return fail(VDX_ERR_ARG, "a frame of %d x %d tokens is too large", a->Hgrid, a->Wgrid);
  int st = a->sec_t, sh = a->sec_h, sw = a->sec_w;
  if (st == 0 && sh == 0 && sw == 0) {
    sh = sw = 2 * (d / 6);
    st = d - sh - sw;
  }
  if (st < 0 || sh < 0 || sw < 0 || ((st | sh | sw) & 1) || static_cast<long long>(st) + sh + sw != d)
    return fail(VDX_ERR_ARG, "rotary sections %d/%d/%d must be even, non-negative and sum to d=%d", st, sh, sw, d);
  if (!(a->theta > 0.0) || !std::isfinite(a->theta)) return fail(VDX_ERR_ARG, "theta must be > 0");
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return fail(VDX_ERR_ARG, "eps must be finite and >= 0");
  if (!a->q && a->q_norm) return fail(VDX_ERR_ARG, "q_norm without q");
  if (a->rows == 0 || c->seqs == 0) return VDX_OK;
  const Tensor q{a->q, {1, a->q ? a->rows : 0, a->Hq}, {0, a->q_row, a->q_head}, d};
  const Tensor qo{a->q_out, {1, a->q ? a->rows : 0, a->Hq}, {0, a->q_out_row, a->q_out_head}, d};
  const Tensor k{a->k, {1, a->rows, c->Hkv}, {0, a->k_row, a->k_head}, d};
  const Tensor v{a->v, {1, a->rows, c->Hkv}, {0, a->v_row, a->v_head}, d};
  if (vdx_status s = check_tensor("q", q, false)) return s;
  if (vdx_status s = check_tensor("q_out", qo, false)) return s;
  if (vdx_status s = check_tensor("k", k, false)) return s;
  if (vdx_status s = check_tensor("v", v, false)) return s;
  if (vdx_status s = check_i32("cu", a->cu, false)) return s;
  if (vdx_status s = check_i32("kv_len", a->kv_len, false)) return s;
  if (vdx_status s = check_i32("pos_offset", a->pos_offset, true)) return s;
  if ((reinterpret_cast<uintptr_t>(a->q_norm) | reinterpret_cast<uintptr_t>(a->k_norm)) & 15)
    return fail(VDX_ERR_ALIGN, "q_norm or k_norm is not 16-byte aligned");
  const Tensor kc = cache_tensor(*c, false, scales), vc = cache_tensor(*c, true, scales);
  const bool in_place = a->q && a->q == a->q_out && a->q_row == a->q_out_row && a->q_head == a->q_out_head;
  if (a->q && ((!in_place && !rows_apart(qo, q)) || !rows_apart(qo, k) || !rows_apart(qo, v)))
    return fail(VDX_ERR_ARG, "q_out overlaps q, k or v");
  if (!rows_distinct(qo)) return fail(VDX_ERR_ARG, "rows of q_out overlap one another");
  if (vdx_status s = check_written_cache(*c, scales)) return s;
  for (const Tensor* t : {&kc, &vc})
    if (overlap(*t, q) || overlap(*t, k) || overlap(*t, v) || overlap(*t, qo))
      return fail(VDX_ERR_ARG, "the cache overlaps q, k, v or q_out");
  const Span reads[6] = {ints(a->cu, c->seqs + 1ll), ints(a->kv_len, c->seqs), ints(a->pos_offset, c->seqs),
                         table_span(c->page_table, c->seqs, c->table_stride, c->max_pages),
                         {a->q_norm, static_cast<size_t>(d) * 2}, {a->k_norm, static_cast<size_t>(d) * 2}};
  for (const Span& r : reads)
    for (const Tensor* t : {&kc, &vc, &qo})
      if (overlap(*t, r.p, r.bytes))
        return fail(VDX_ERR_ARG, "the cache or q_out overlaps cu, kv_len, pos_offset, page_table, q_norm or k_norm");
  if (scales) {
    for (bool value : {false, true}) {
      const Tensor t = scale_tensor(*c, *scales, value);
      if (overlap(t, q) || overlap(t, k) || overlap(t, v) || overlap(t, qo)) return fail(VDX_ERR_ARG, "the scales overlap q, k, v or q_out");
      for (const Span& r : reads)
        if (overlap(t, r.p, r.bytes))
          return fail(VDX_ERR_ARG, "the scales overlap cu, kv_len, pos_offset, page_table, q_norm or k_norm");
    }
  }

  vdx::AppendParams p{};
  p.q = a->q; p.k = a->k; p.v = a->v; p.q_out = a->q_out; p.k_cache = c->k; p.v_cache = c->v;
  p.q_row = a->q_row; p.q_head = a->q_head; p.k_row = a->k_row; p.k_head = a->k_head;
  p.v_row = a->v_row; p.v_head = a->v_head; p.q_out_row = a->q_out_row; p.q_out_head = a->q_out_head;
  p.kc_page = c->k_page; p.kc_token = c->k_token; p.kc_head = c->k_head;
  p.vc_page = c->v_page; p.vc_token = c->v_token; p.vc_head = c->v_head;
  p.cu = a->cu; p.kv_len = a->kv_len; p.pos_offset = a->pos_offset;
  p.table = c->page_table; p.table_stride = c->table_stride;
  p.q_norm = a->q_norm; p.k_norm = a->k_norm; p.eps = a->eps;
  p.rows = a->rows; p.S = c->seqs; p.Hq = a->q ? a->Hq : 0; p.Hkv = c->Hkv;
  p.P = c->page_size; p.num_pages = c->num_pages; p.max_pages = c->max_pages;
  p.T = a->T; p.Hg = a->Hgrid; p.Wg = a->Wgrid;
  p.half_t = st / 2; p.half_h = sh / 2;
  const int sec[3] = {st, sh, sw};
  int pair = 0;
  for (int x = 0; x < 3; ++x)
    for (int j = 0; j < sec[x] / 2; ++j) {
      const double turns = std::pow(a->theta, -2.0 * j / sec[x]) / 6.283185307179586476925286766559;
      if (!std::isfinite(turns)) return fail(VDX_ERR_ARG, "theta = %g is too small: its powers are not finite", a->theta);
      const double frac = turns - std::floor(turns);
      p.turn[pair++] = frac >= 1.0 ? 0ull : static_cast<uint64_t>(std::ldexp(frac, 64));
    }
  if (scales) p.scales = device_scales(*scales);
  const cudaError_t e = (scales ? vdx::launch_append8 : vdx::launch_append)(p, d, c->dtype, multiprocessors(), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(VDX_ERR_CUDA, "append kernel launch: %s", cudaGetErrorString(e));
  }
  return VDX_OK;
}

}  // namespace

namespace vdx {

size_t plan_attention(KvParams* p, int d, int sms) {
  const long long rows = static_cast<long long>(p->max_q) * p->g;
  p->rows_kernel = rows <= 32;
  if (p->rows_kernel) {
    p->block_rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : 32);
    p->nblk = 1;
    const long long units = static_cast<long long>(p->S) * p->Hkv;
    // Two CTAs to a multiprocessor, in one wave where the units leave room for splits: the most
    // splits that fit with a tenth to spare (clusters do not fill every group of processors), of at
    // least 192 keys.  16 x 8 heads over 8192 keys: 2 splits 84.7 us, 1 split 131, 4 (two waves) 93, 8
    // 105; 4 x 12 over 1000: 5 splits 10.9, 1 split 20.7, 6 (all slots, did not fit) 17.6.  Units
    // that fill the device by themselves are split only where they are long, to even out ragged
    // lengths: 48 x 8 over 8-33 thousand keys: 4 splits 662 us, 1 split 856; 64 x 12 over 1000 keys: 1
    // split 76.8, 2 splits 94.4.  Up to 8 splits are a cluster and join in it; a few heads over a long
    // cache take more, joined through the workspace (8 heads over 16000 keys: 31 of 512 keys 19.7 us,
    // 8 in a cluster 39.6).
    const long long slots = 2ll * sms, room = slots * 9 / 10 / units;
    long long n;
    if (room < 2)
      n = std::min<long long>(8, (p->max_kv + 8191) / 8192);
    else if (room <= 8 || p->max_kv <= 8 * 1024)
      n = std::min<long long>({room, 8, (p->max_kv + 191) / 192});
    else
      n = std::min<long long>(slots / units, p->max_kv / 512);
    long long keys = n > 0 ? ((p->max_kv + n - 1) / n + 63) / 64 * 64 : 0;
    p->cluster = n > 1 && n <= 8;
    p->nsplit = static_cast<int>(std::max<long long>(1, n));
    if (!p->cluster && n > 1) p->nsplit = static_cast<int>((p->max_kv + keys - 1) / keys);
    p->split_keys = static_cast<int>(p->nsplit > 1 ? keys : std::max(p->max_kv, 1));
    if (p->cluster) return 0;
  } else {
    const int per = 4 * (128 / p->g);                 // tokens of a block: two Q tiles of two CTAs
    p->block_rows = per * p->g;
    p->nblk = (p->max_q - 1) / per + 1;
    const long long units = static_cast<long long>(p->S) * p->Hkv * p->nblk;
    // Tiles cross page ends where a page is a multiple of 8 keys (a swizzle atom of the copies); the
    // largest power of two up to 64 that divides it is the box.  Dense keys are one page.
    p->box_rows = 0;
    if (p->table && p->P % 8 == 0) p->box_rows = std::min(64, p->P & -p->P);
    if (p->eight) p->box_rows = 8;                    // no boxes: a lane looks up each key, whatever the page size
    long long tiles = 1;
    if (p->max_kv > 0)
      tiles = p->box_rows ? (p->max_kv + 127) / 128
                    : static_cast<long long>(p->max_kv / p->P) * ((p->P + 127) / 128) + (p->max_kv % p->P + 127) / 128;
    // Splits: the sms / 2 CTA pairs take ceil(units * splits / pairs) units each; a unit costs its
    // tiles and about two tiles' time to start and finish, a split one up to two more for its partial
    // results, as its rows fill a block, and their join two to six in all (tile time: 1.4 us).  480p
    // frame of 96 units of 256 tiles: 3 splits 514 us, 1 split 706, 4 557; 40 units of 32 tiles: 512
    // rows each 1 split 54 us, 3 splits 60; 33 rows each 53 and 44.
    const long long fill = std::min<long long>(16, rows * 16 / p->block_rows);      // of a block, in sixteenths
    long long best = 0;
    p->nsplit = 1;
    for (int n = 1; n <= 32 && n <= tiles; ++n) {
      const long long per_split = (tiles + n - 1) / n;
      const long long rounds = (units * n + sms / 2 - 1) / (sms / 2);
      const long long cost = n == 1 ? rounds * 16 * (per_split + 2) : rounds * (16 * (per_split + 2) + 2 * fill) + 32 + 4 * fill;
      if (n == 1 || cost < best) {
        best = cost;
        p->nsplit = n;
      }
    }
    // a unit of 2^17 tiles takes about 0.2 s, well inside the limit of the kernel's waits for it
    p->nsplit = static_cast<int>(std::max<long long>(p->nsplit, (tiles + (1 << 17) - 1) >> 17));
    p->split_keys = static_cast<int>((tiles + p->nsplit - 1) / p->nsplit);
    p->nsplit = static_cast<int>((tiles + p->split_keys - 1) / p->split_keys);
  }
  if (p->nsplit == 1) return 0;
  const long long units = static_cast<long long>(p->S) * p->Hkv * p->nblk;
  return static_cast<size_t>(units) * p->nsplit * p->block_rows * (static_cast<size_t>(d) * 4 + 8);
}

}  // namespace vdx

extern "C" {

vdx_status vdx_rope3d_append(const vdx_paged_kv* c, const vdx_append_args* a, void* stream) {
  NvtxScope nvtx("vdx_rope3d_append");
  clear_error();
  return append(c, nullptr, a, stream);
}

vdx_status vdx_rope3d_append8(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_append_args* a, void* stream) {
  NvtxScope nvtx("vdx_rope3d_append8");
  clear_error();
  if (!scales) return fail(VDX_ERR_ARG, "the scales must be non-NULL");
  return append(c, scales, a, stream);
}

vdx_status vdx_paged_attn(const vdx_paged_kv* c, const vdx_paged_attn_args* a, void* stream) {
  NvtxScope nvtx("vdx_paged_attn");
  clear_error();
  Problem pb;
  if (vdx_status s = paged_problem(c, nullptr, a, nullptr, false, &pb)) return s;
  return launch(pb, stream);
}

vdx_status vdx_paged_attn_offset(const vdx_paged_kv* c, const vdx_paged_attn_args* a, const int32_t* pos_offset, void* stream) {
  NvtxScope nvtx("vdx_paged_attn_offset");
  clear_error();
  Problem pb;
  if (vdx_status s = paged_problem(c, nullptr, a, pos_offset, false, &pb)) return s;
  return launch(pb, stream);
}

size_t vdx_paged_attn_workspace_bytes(const vdx_paged_kv* c, const vdx_paged_attn_args* a) {
  clear_error();
  Problem pb;
  return paged_problem(c, nullptr, a, nullptr, true, &pb) == VDX_OK ? pb.workspace : 0;
}

vdx_status vdx_paged_attn8(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_paged_attn_args* a, const int32_t* pos_offset,
                           void* stream) {
  NvtxScope nvtx("vdx_paged_attn8");
  clear_error();
  if (!scales) return fail(VDX_ERR_ARG, "the scales must be non-NULL");
  Problem pb;
  if (vdx_status s = paged_problem(c, scales, a, pos_offset, false, &pb)) return s;
  return launch(pb, stream);
}

size_t vdx_paged_attn8_workspace_bytes(const vdx_paged_kv* c, const vdx_kv8_scales* scales, const vdx_paged_attn_args* a) {
  clear_error();
  Problem pb;
  if (!scales) {
    fail(VDX_ERR_ARG, "the scales must be non-NULL");
    return 0;
  }
  return paged_problem(c, scales, a, nullptr, true, &pb) == VDX_OK ? pb.workspace : 0;
}

vdx_status vdx_cross_attn(const vdx_cross_attn_args* a, void* stream) {
  NvtxScope nvtx("vdx_cross_attn");
  clear_error();
  Problem pb;
  if (vdx_status s = cross_problem(a, false, &pb)) return s;
  return launch(pb, stream);
}

size_t vdx_cross_attn_workspace_bytes(const vdx_cross_attn_args* a) {
  clear_error();
  Problem pb;
  return cross_problem(a, true, &pb) == VDX_OK ? pb.workspace : 0;
}

}  // extern "C"
