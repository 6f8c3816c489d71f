/* vdx — 3D-RoPE full spatiotemporal self-attention for video diffusion transformers, on one
 * GB300 (sm_103a).
 *
 * Operation (vidax: A Unified JAX Framework for Video Generative Models on Accelerator
 * Meshes, §2 "3D RoPE, 3D VAEs, and flash attention": rotary 3D position embedding on Q and
 * K, then attention that never materialises the N x N score matrix; §1 "Motivation and gap":
 * tens of thousands of latent-patch tokens).  For batch b, head h, query token n:
 *
 *     q'_n  = R(n) q_n,   k'_m = R(m) k_m
 *     lse_n = log sum_m exp(scale * <q'_n, k'_m>)           (natural log, all m: non-causal)
 *     out_n = sum_m exp(scale * <q'_n, k'_m> - lse_n) v_m
 *
 * R(n) rotates adjacent channel pairs (2i, 2i+1) like a complex number times exp(i*angle).
 * head_dim d is split into three rotary sections, in this order: sec_t dims turning with the
 * frame index t, sec_h with the grid row h, sec_w with the grid column w.  Within a section of
 * S dims, pair j turns at angle pos * theta^(-2j/S).  Token n = t*Hgrid*Wgrid + h*Wgrid + w.
 *
 * Layouts (row-major, contiguous):
 *   q, k, v, out : [B, N, H, d]   with N = T*Hgrid*Wgrid
 *   lse          : [B, H, N]      float32, may be NULL
 *
 * Ownership: every pointer is a device pointer owned by the caller.  The library owns only a
 * per-device cache of cos/sin tables (one per distinct grid/sections/theta; built on the
 * first call with that key, which allocates and uploads synchronously) and an error word;
 * vdx_shutdown() frees the tables.  Calls are asynchronous on `stream` (a cudaStream_t; NULL
 * means the legacy default stream).
 *
 * Errors: argument problems are reported before anything is launched and return a non-zero
 * vdx_status; vdx_last_error() gives a message (per host thread).  Device-side problems (a
 * pipeline wait that gave up after 1 s) are latched in a device error word read and cleared
 * by vdx_sync_check().
 */
#ifndef VDX_H_
#define VDX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VDX_OK = 0,
  VDX_ERR_ARG = 1,          /* bad size, section split, NULL pointer, aliasing        */
  VDX_ERR_ALIGN = 2,        /* a pointer is not 16-byte aligned                       */
  VDX_ERR_UNSUPPORTED = 3,  /* valid, but outside what this build implements          */
  VDX_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed                      */
  VDX_ERR_TIMEOUT = 5,      /* a kernel pipeline wait gave up (see vdx_sync_check)    */
  VDX_ERR_RANGE = 6         /* a rotated q/k value left the fp16 operand range         */
} vdx_status;

/* How K gets rotated on the bf16 path. */
#define VDX_K_ROPE_DEFAULT 0  /* = VDX_K_ROPE_PREPASS                                          */
#define VDX_K_ROPE_PREPASS 1  /* a prepass kernel rotates every key token once into an fp16
                                 workspace [B, N, H, d]; the attention kernel streams it      */
#define VDX_K_ROPE_FUSED 2    /* each CTA rotates every K tile in shared memory as it lands
                                 (no workspace; the rotation is repeated per query block)     */

/* Precision of the rotated Q/K operands of QK^T on the bf16 path. */
#define VDX_QK_FP16 0         /* one fp16 value per rotated element (default; fastest)          */
#define VDX_QK_SPLIT 1        /* fp16 hi + lo per element and three products (~22 significant
                                 bits): for activations whose logits reach the hundreds; about
                                 half the speed; needs the K prepass and twice its workspace  */

/* Which attention kernel runs a dense bf16 call. */
#define VDX_KERNEL_DEFAULT 0  /* VDX_KERNEL_PAIR for dense calls with VDX_K_ROPE_FUSED, with
                                 VDX_QK_SPLIT, or with VDX_QK_FP16 and N >= 65536; else
                                 VDX_KERNEL_SINGLE                                                */
#define VDX_KERNEL_SINGLE 1   /* one CTA per 256 query rows, each streaming whole K/V tiles          */
#define VDX_KERNEL_PAIR 2     /* clusters of two CTAs: each holds half of every K/V tile and the pair
                                 multiplies both CTAs' 512 query rows with CTA-pair MMAs; dense
                                 calls only (block-sparse and query-subset calls get
                                 VDX_ERR_UNSUPPORTED).  With VDX_K_ROPE_FUSED each CTA rotates
                                 its own Q tiles and its 64 keys of every K tile                */

typedef struct vdx_attn_options {
  int k_rope;               /* one of VDX_K_ROPE_*                                              */
  int qk_precision;         /* one of VDX_QK_*                                                  */
  void* workspace;          /* device scratch for the prepass, >= vdx_rope3d_workspace_bytes()
                               bytes, 16-byte aligned, not overlapping q/k/v/out/lse; NULL = a
                               library-owned per-device buffer (allocated or grown with
                               cudaMalloc on first need; shared by every call on that device, so
                               calls that may overlap on different streams should pass their own) */
  size_t workspace_bytes;   /* size of `workspace` in bytes                                      */
  int test_withhold_kv;     /* testing only, keep 0: the kernel's copy engine issues no K/V tile,
                               so every pipeline wait runs out (after about 1 s); the kernel then
                               stops cleanly and vdx_sync_check reports VDX_ERR_TIMEOUT (this is
                               how the failure path is exercised without faulting the GPU)    */
  int kernel;               /* one of VDX_KERNEL_*                                              */
} vdx_attn_options;

/* bf16 path, tcgen05 tensor cores.  q, k, v, out: __nv_bfloat16 [B, N, H, d]; d must be 128.
 * Arithmetic: rotation in fp32; rotated k, and rotated q multiplied by scale*log2(e), rounded
 * to fp16 for QK^T (so |k| and |q|*scale*log2(e) must stay below ~46000, else values are
 * clamped and vdx_sync_check reports VDX_ERR_RANGE); scores (in log2 units), softmax
 * statistics and the output accumulator in fp32; P and v enter PV as bf16.
 * sec_t/sec_h/sec_w: even, sum to d; all three 0 selects d - 4*(d/6), 2*(d/6), 2*(d/6)
 * (44/42/42 at d = 128).  scale <= 0 selects 1/sqrt(d).  theta > 0 (10000 for Wan).
 * out must not overlap q, k or v.  B, H, T, Hgrid, Wgrid >= 1. */
vdx_status vdx_rope3d_attn(const void* q, const void* k, const void* v, void* out, float* lse,
                           int B, int H, int T, int Hgrid, int Wgrid, int d,
                           int sec_t, int sec_h, int sec_w, double theta, float scale,
                           void* stream);

/* Same as vdx_rope3d_attn with explicit options (NULL = defaults: K prepass, fp16 QK operands,
 * library-owned workspace). */
vdx_status vdx_rope3d_attn_ex(const void* q, const void* k, const void* v, void* out, float* lse,
                              int B, int H, int T, int Hgrid, int Wgrid, int d,
                              int sec_t, int sec_h, int sec_w, double theta, float scale,
                              const vdx_attn_options* opt, void* stream);

/* Bytes of workspace the prepass needs for this problem: the rotated K and the rotated,
 * scale*log2(e)-multiplied Q as fp16 [B, N, H, d] each (2*B*N*H*d*2), twice that with
 * VDX_QK_SPLIT (hi + lo parts); 0 for invalid sizes.  A query-subset call rotates its gathered
 * rows itself and uses only the first half (the rotated K). */
size_t vdx_rope3d_workspace_bytes(int B, int H, int T, int Hgrid, int Wgrid, int d,
                                  int qk_precision);

/* ---- Block-sparse attention (the bit-wise block-sparse kernel of the ScalingAttention abstract
 * on the papers page 2606.17566; masks here are caller-defined).  Keys are
 * cut into tiles of VDX_SPARSE_KBLOCK tokens and queries into blocks of VDX_SPARSE_QBLOCK
 * tokens; query n attends only to the key tiles its block's mask selects (a query whose mask
 * row selects nothing gets out = 0 and lse = -inf).  Skipped tiles cost no work.
 *   block_mask: device uint32 words, row-major [M][n_qblocks][W] with
 *     W = vdx_rope3d_block_mask_words(T, Hgrid, Wgrid), n_qblocks = ceil(N / 256),
 *     M = B*H (mask_per_head = 1, one mask per (b, h)) or 1 (mask_per_head = 0, shared);
 *     bit (kb % 32) of word kb / 32 selects key tile kb; bits at or beyond ceil(N/128) ignored.
 *   Other arguments, rules and options as vdx_rope3d_attn_ex (K prepass only). */
#define VDX_SPARSE_QBLOCK 256
#define VDX_SPARSE_KBLOCK 128
vdx_status vdx_rope3d_attn_sparse(const void* q, const void* k, const void* v, void* out,
                                  float* lse, int B, int H, int T, int Hgrid, int Wgrid, int d,
                                  int sec_t, int sec_h, int sec_w, double theta, float scale,
                                  const uint32_t* block_mask, int mask_per_head,
                                  const vdx_attn_options* opt, void* stream);

/* ---- Active-query subset (after the KV-cache synchronization of the Heterogeneous Step
 * Allocation abstract on the papers page 2606.17566: only active query tokens are recomputed,
 * against the full K/V).
 * Query rows are the tokens q_index[i], i < Nq (device int32; one list shared by every batch
 * entry when index_per_batch = 0, else [B][Nq]); each is rotated at its own grid position,
 * attends to all N keys, and its result is written to out[b, q_index[i], h, :] and
 * lse[b, h, q_index[i]].  Rows of out / lse not listed are left untouched.  An index outside
 * [0, N) is skipped and reported by vdx_sync_check (VDX_ERR_ARG).  Duplicate indices write
 * the same values twice.  Other arguments, rules and options as vdx_rope3d_attn_ex. */
vdx_status vdx_rope3d_attn_subset(const void* q, const void* k, const void* v, void* out,
                                  float* lse, int B, int H, int T, int Hgrid, int Wgrid, int d,
                                  int sec_t, int sec_h, int sec_w, double theta, float scale,
                                  const int32_t* q_index, int Nq, int index_per_batch,
                                  const vdx_attn_options* opt, void* stream);

/* Words per query block of a block mask for this grid (ceil(ceil(N/128)/32)); 0 if invalid. */
int vdx_rope3d_block_mask_words(int T, int Hgrid, int Wgrid);

/* Host helper: fill `mask` (host memory, [n_qblocks][W] words) with the block mask of 3D
 * windowed attention (the windowed-attention primitive of the vidax page, §2 "3D RoPE, 3D
 * VAEs, and flash attention"), at block granularity: query block Qb selects key tile Kb when
 * some token of Qb and some token of Kb are within (wt, wh, ww) of each other on every grid
 * axis (|dt| <= wt, |dh| <= wh, |dw| <= ww).  Pass it with mask_per_head = 0. */
vdx_status vdx_window_block_mask(uint32_t* mask, int T, int Hgrid, int Wgrid, int wt, int wh,
                                 int ww);

/* fp32 path (CUDA cores, fp32 arithmetic throughout).  Same operation and rules; q, k, v,
 * out are float [B, N, H, d]; d must be 64 or 128. */
vdx_status vdx_rope3d_attn_f32(const float* q, const float* k, const float* v, float* out,
                               float* lse, int B, int H, int T, int Hgrid, int Wgrid, int d,
                               int sec_t, int sec_h, int sec_w, double theta, float scale,
                               void* stream);

/* ---- No-allocation variant.  The vidax page has no counterpart: this is a deployment aid
 * for callers that cannot allocate device memory at call time (a frozen memory pool, an
 * allocator-free embedding, a host that sizes every buffer up front).  Same operation,
 * arguments, layouts and K-prepass arithmetic as vdx_rope3d_attn, but the cos/sin table and
 * the rotated keys live in one fixed static device array of the library instead of memory
 * allocated on first use, and the call makes no cudaMalloc/cudaFree.
 *   Limit: B*N*H*d*2 <= VDX_NOALLOC_MAX_WORKSPACE_BYTES and T*sec_t/2 + Hgrid*sec_h/2 +
 *   Wgrid*sec_w/2 <= VDX_NOALLOC_MAX_TABLE_ENTRIES; larger problems return
 *   VDX_ERR_UNSUPPORTED.
 *   The array (about 64 MiB) is held on every GPU that loads the library until exit.
 *   Every call shares it and it keeps the last call's contents, so calls that may overlap on
 *   the GPU (unordered streams) race; order them or use vdx_rope3d_attn_ex with a workspace.
 *   The first call on each device looks up the array's device address (make it before any
 *   stream capture). */
#define VDX_NOALLOC_MAX_WORKSPACE_BYTES (64ull << 20)
#define VDX_NOALLOC_MAX_TABLE_ENTRIES 8192
vdx_status vdx_rope3d_attn_noalloc(const void* q, const void* k, const void* v, void* out,
                                   float* lse, int B, int H, int T, int Hgrid, int Wgrid, int d,
                                   int sec_t, int sec_h, int sec_w, double theta, float scale,
                                   void* stream);

/* ---- Streaming and conditioning: a paged key/value cache, attention of new tokens over it, and
 * cross attention.  A transformer block that generates video chunk by chunk (each new chunk of
 * latent tokens attends to every token before it) appends the chunk's rotated keys and its
 * values to a cache and attends over the cache; the same block attends to the text or image
 * encoder's states.
 *
 * Element types VDX_DTYPE_BF16 and VDX_DTYPE_FP16 (all tensors of a call share one), head
 * dimension 64 or 128, Hq a multiple of Hkv with Hq / Hkv <= 128 (query head h reads key/value
 * head h / (Hq / Hkv)).  Strides count elements.  The channels of one (token, head) are
 * contiguous; base pointers are 16-byte aligned and strides are multiples of 8, so slices of
 * one fused projection and caches in [page, token, head] or [page, head, token] order are taken
 * as they are.  Every pointer is a device pointer; these calls allocate nothing and keep nothing
 * between calls (scratch comes from the caller), so they may be captured into CUDA graphs and
 * run at once on several streams, each with its own workspace.
 *
 * Lengths live on the device and may change between replays of a captured call; what the host
 * passes are upper bounds.  Values that break a bound are never followed: the kernel clamps or
 * skips them and vdx_sync_check reports VDX_ERR_ARG. */
#define VDX_DTYPE_BF16 0
#define VDX_DTYPE_FP16 1

/* A cache of num_pages pages of page_size tokens each.  Key c of sequence s is token
 * c % page_size of page page_table[s * table_stride + c / page_size], for every head.
 * page_size: 16, 32, 64, or any size >= 128 (a page may hold one latent frame).  Entries of
 * page_table past a sequence's length are not read; a page index outside [0, num_pages) is
 * reported, nothing is written through it and its keys read as zeros.  Slots past a sequence's
 * length may hold anything, NaN included; within it the cache has to be finite. */
typedef struct vdx_paged_kv {
  void* k;                  /* [num_pages, page_size, Hkv, d] with the strides below              */
  void* v;
  long long k_page, k_token, k_head;   /* strides of k                                            */
  long long v_page, v_token, v_head;   /* strides of v                                            */
  const int32_t* page_table;           /* [seqs][table_stride], the first max_pages of a row used */
  long long table_stride;
  int num_pages, page_size, max_pages;
  int Hkv, d, dtype;
  int seqs;
} vdx_paged_kv;

/* New tokens of seqs sequences, packed: row r of q, k and v belongs to the sequence s with
 * cu[s] <= r < cu[s + 1] (cu: device int32 [seqs + 1], not decreasing, cu[seqs] <= rows; rows
 * outside every sequence are left alone).  kv_len[s] (device int32) counts the sequence's keys
 * with its new ones: with n = cu[s + 1] - cu[s], row i of the sequence has cache index
 * c = kv_len[s] - n + i. */

/* Append: for every row, write v and the rotated key into the cache at index c, and the rotated
 * query into q_out.  The rotation is that of vdx_rope3d_attn at grid token
 * pos_offset[s] + c (pos_offset NULL: c; larger than 0 when a sequence's oldest pages have been
 * dropped from its table).  With q_norm / k_norm (d values of the call's type, shared by the
 * heads) x * rsqrt(mean(x^2) + eps) * weight is applied to each head before the rotation.
 * fp32 arithmetic (angles reduced in 64-bit fixed point, within 2^-25 turns up to position 5e8), one
 * rounding to the call's type at the end, where vdx_rope3d_attn keeps its rotated q and k in fp16; v is
 * copied bit for bit.  A norm over all heads of a token is not this one: it goes before the call.
 * q may be NULL (keys and values only).  q_out may equal q with the same strides (in place),
 * also inside a fused projection; otherwise the outputs (q_out and the cache) must not overlap an
 * input (lengths, page table and weights too), nor each other.  A token outside the grid's T*Hgrid*Wgrid
 * positions, or with a cache index below 0 or past its page table, is skipped and reported; so are the
 * tokens of a sequence whose range in cu is no range of the call's rows.
 * Two rows of one call that land in the same cache slot (sequences whose tables share a page that both
 * write) race for it: what it holds then is a mixture of the two, each 16 bytes from either. */
typedef struct vdx_append_args {
  const void* q;            /* [rows, Hq, d] or NULL                                              */
  const void* k;            /* [rows, Hkv, d]                                                     */
  const void* v;
  void* q_out;              /* [rows, Hq, d]; NULL with q NULL                                    */
  long long q_row, q_head, k_row, k_head, v_row, v_head, q_out_row, q_out_head;   /* strides      */
  int rows, Hq;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* pos_offset;   /* [seqs] or NULL                                                  */
  int T, Hgrid, Wgrid, sec_t, sec_h, sec_w;   /* as in vdx_rope3d_attn                            */
  double theta;
  const void* q_norm;       /* [d] or NULL                                                        */
  const void* k_norm;       /* [d] or NULL                                                        */
  float eps;
} vdx_append_args;
vdx_status vdx_rope3d_append(const vdx_paged_kv* cache, const vdx_append_args* args, void* stream);

/* Attention of the new tokens over the cache (q already rotated, keys already appended):
 *     lse = log sum_c exp(scale * <q, k_c>),   out = sum_c exp(scale * <q, k_c> - lse) v_c
 * over the visible keys c of row i of its sequence, with p = kv_len - n + i and o = pos_offset[s]
 * (that of the append, given to vdx_paged_attn_offset; otherwise 0):
 *     c < kv_len,  and with causal_block = m > 0 also  c + o < (floor((p + o) / m) + 1) * m
 * (m = 1: each token sees the tokens up to itself; m = tokens of a latent frame: whole frames up
 * to its own, also where the oldest pages that were dropped end inside a frame; m = 0: every key).
 * A row that sees no key, or with m > 0 one whose p is negative, gets out = 0 and lse = -inf.
 * q, k and v enter the products as they are; scores, softmax statistics and accumulators are
 * fp32; the softmax weights are rounded to the call's type for the product with v (fp16: weights below
 * 2^-14 of a row's largest lose bits).  There is no counterpart of qk_precision.
 *   out: [rows, Hq, d] contiguous;  lse: float32 [Hq, rows] or NULL.
 *   max_q, max_kv: host bounds on n and on kv_len (they size the launch; 0 takes rows and
 *   max_pages * page_size).  Rows and keys past them are not computed, and reported.
 *   scale <= 0 selects 1/sqrt(d).  out, lse and workspace must not overlap an input, nor each other.
 *   workspace: >= vdx_paged_attn_workspace_bytes() bytes of the device, 16-byte aligned, used by
 *   this call alone until it has run; NULL where that is 0. */
typedef struct vdx_paged_attn_args {
  const void* q;            /* [rows, Hq, d]                                                      */
  void* out;
  float* lse;
  long long q_row, q_head;  /* strides of q                                                       */
  int rows, Hq;
  const int32_t* cu;
  const int32_t* kv_len;
  int max_q, max_kv;
  int causal_block;
  float scale;
  void* workspace;
  size_t workspace_bytes;
} vdx_paged_attn_args;
vdx_status vdx_paged_attn(const vdx_paged_kv* cache, const vdx_paged_attn_args* args, void* stream);
/* With pos_offset (device int32 [seqs], or NULL: as vdx_paged_attn), read where causal_block > 0. */
vdx_status vdx_paged_attn_offset(const vdx_paged_kv* cache, const vdx_paged_attn_args* args,
                                 const int32_t* pos_offset, void* stream);
/* 0 also where the call would be refused: vdx_last_error() is not empty then. */
size_t vdx_paged_attn_workspace_bytes(const vdx_paged_kv* cache, const vdx_paged_attn_args* args);

/* Cross attention: q [B, N, Hq, d] over k, v [B, M, Hkv, d] (an encoder's states; no positions).
 * kv_len (device int32 [B], or NULL: M) limits batch entry b to its first kv_len[b] keys; keys
 * past it may hold anything.  A batch stride of 0 shares one q, k or v over the batch.
 * Formulas, arithmetic, scale and workspace as vdx_paged_attn; M may be 0 and N may be 0.
 *   out: [B, N, Hq, d] contiguous;  lse: float32 [B, Hq, N] or NULL. */
typedef struct vdx_cross_attn_args {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  long long q_batch, q_row, q_head, k_batch, k_token, k_head, v_batch, v_token, v_head;
  int B, N, M, Hq, Hkv, d, dtype;
  const int32_t* kv_len;
  float scale;
  void* workspace;
  size_t workspace_bytes;
} vdx_cross_attn_args;
vdx_status vdx_cross_attn(const vdx_cross_attn_args* args, void* stream);
size_t vdx_cross_attn_workspace_bytes(const vdx_cross_attn_args* args);

/* ---- The same cache in 8 bits: half the memory, and half the bytes to read.
 * k and v of a vdx_paged_kv hold e4m3 bytes (strides in elements, that is bytes, multiples of 16), its dtype is that
 * of the call's other tensors.  A block is VDX_KV8_BLOCK consecutive tokens of a page (the last one of a page
 * may be short); for each block and head there is a scale 2^e, held as the byte e + 127 (e8m0), and a value is
 * its code times that scale.  e lies in [VDX_KV8_MIN_EXP, VDX_KV8_MAX_EXP], within which every value is exact in
 * bf16 and in fp16; bytes outside are read as the nearer end.  With scales that are powers of two a value
 * keeps its four significant bits whatever the scale, down to 2^-13 of the block's largest (where that is above 2^-7).
 * What is said above of page sizes, page tables, lengths, heads, streams and reports holds here too. */
#define VDX_KV8_BLOCK 16
#define VDX_KV8_MIN_EXP (-15)
#define VDX_KV8_MAX_EXP 7
typedef struct vdx_kv8_scales {
  uint8_t* k;               /* [num_pages, ceil(page_size / VDX_KV8_BLOCK), Hkv], strides in bytes   */
  uint8_t* v;
  long long k_page, k_block, k_head, v_page, v_block, v_head;
} vdx_kv8_scales;

/* vdx_rope3d_append into such a cache.  Keys (normed and rotated) and values go from fp32 to e4m3 with one
 * rounding, to nearest even, after the block's scale has been found: the least e with |x| <= 448 * 2^e for all new
 * values x of the block, and for a block whose first token is older than this call, not less than its e so far.
 * Where e grows the older codes are rounded again (exact, but for those that become e4m3's subnormals).  So a
 * sequence appended at once and one appended token by token may differ by that.  A block whose first token is new
 * starts afresh, whatever page and scale held.  Values past 448 * 2^7 are clamped to it and
 * vdx_sync_check reports VDX_ERR_RANGE; NaN stays NaN.
 * A block belongs to one sequence: two sequences that share a page (a common prefix) must not append into
 * a block of it.  q and q_out as in vdx_rope3d_append. */
vdx_status vdx_rope3d_append8(const vdx_paged_kv* cache, const vdx_kv8_scales* scales, const vdx_append_args* args, void* stream);

/* vdx_paged_attn_offset over such a cache.  Codes and scales enter the products as the values they stand for; the
 * softmax weights are rounded to fp16 after a multiplication by 2^7 (weights below 2^-21 of a row's largest lose
 * bits, below 2^-32 they vanish).  Queries of bf16 are taken as fp16 times a power of two of the row's own: what lies below
 * 2^-29 of a row's largest loses bits. */
vdx_status vdx_paged_attn8(const vdx_paged_kv* cache, const vdx_kv8_scales* scales, const vdx_paged_attn_args* args,
                           const int32_t* pos_offset, void* stream);
/* 0 also where the call would be refused: vdx_last_error() is not empty then. */
size_t vdx_paged_attn8_workspace_bytes(const vdx_paged_kv* cache, const vdx_kv8_scales* scales, const vdx_paged_attn_args* args);

/* ---- Which keys are worth their place: the weight that each cached key gathers, and eviction.
 *
 * After vdx_paged_attn (or vdx_paged_attn8), with its q, cu, kv_len, causal_block, scale and lse: for every sequence s
 * that has rows in the call, kv head h and key c < kv_len[s],
 *     w[s, h, c] = (c < kv_len[s] - n ? decay * w[s, h, c] : 0) + sum over rows i that see c and query heads a of
 *                  h's group of exp(scale * <q_(i,a), k_c> - lse[a, i])
 * so that a key starts at 0 with the call that brings it (the buffer needs no clearing), and the entries of a
 * sequence sum to the rows it has had times Hq / Hkv where decay is 1.  Other entries are left as they were.
 * fp32 arithmetic; each entry is summed by one thread block in an order that the call's shape fixes, so the same call
 * gives the same bits.  A row whose lse is -inf (it saw no key) adds nothing, one whose lse is NaN makes its keys'
 * entries NaN.
 *   scales: NULL for a 16-bit cache.  The cache's values are not read.
 *   w: float32 [seqs, Hkv, width], the entries of a head contiguous; kv_len past width or max_kv is clamped and
 *   reported.  pos_offset as in vdx_paged_attn_offset.  max_q (or rows) times Hq / Hkv: at most 2^26 (VDX_ERR_UNSUPPORTED). */
typedef struct vdx_paged_weights_args {
  const void* q;            /* [rows, Hq, d]                                                      */
  const float* lse;         /* [Hq, rows]                                                         */
  float* w;
  long long q_row, q_head, w_seq, w_head;   /* strides                                            */
  int width;
  int rows, Hq;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* pos_offset;   /* [seqs] or NULL                                                  */
  int max_q, max_kv;        /* host bounds, as in vdx_paged_attn                                  */
  int causal_block;
  float scale;
  float decay;              /* finite                                                             */
} vdx_paged_weights_args;
vdx_status vdx_paged_attn_weights(const vdx_paged_kv* cache, const vdx_kv8_scales* scales, const vdx_paged_weights_args* args,
                                  void* stream);

/* Eviction: of every sequence's L = kv_len[s] keys at most `keep` stay, for each kv head its own.  Where L > keep
 * these are the last `recent` and, of the others, the keep - recent with the largest w (of equals the one with
 * the lowest index; NaN counts as the largest); otherwise all.  Keys and values of a head that stay move, in their order,
 * to cache indices 0, 1, .. of the same sequence of `into`: the same kind of cache by another page table, no page twice, and
 * possibly in the same pools, whose pages the call must not read too (the old pages are free afterwards).  In 8 bits the
 * blocks of `into` get scales by the rule of vdx_rope3d_append8, as if the values were appended at once.
 * Written beside: kv_len_out[s] = min(L, keep); pos_offset_out[s] = pos_offset[s] + L - kv_len_out[s] (NULL: not
 * wanted), with which the next token appended stands where it would have stood; index[s, h, j], the old
 * cache index of the key that is now at j, and w_out[s, h, j], its weight (both for j < keep; -1 and 0 past the new length; a
 * weight of -0 comes out as 0, a NaN as a NaN).
 *   w_out may be w (same strides); otherwise outputs must not overlap inputs, nor each other.
 *   max_kv: host bound on L (0: what the page table and width hold), at most 393216 (VDX_ERR_UNSUPPORTED past it); L past
 *   it is clamped and reported.
 *   Slots of `into` that `into`'s table does not reach, or whose page is outside it, are skipped and reported. */
typedef struct vdx_paged_evict_args {
  const float* w;           /* [seqs, Hkv, width], the entries of a head contiguous               */
  float* w_out;             /* [seqs, Hkv, >= keep]                                               */
  long long w_seq, w_head, w_out_seq, w_out_head;   /* strides                                    */
  int width;
  const int32_t* kv_len;
  const int32_t* pos_offset;   /* [seqs] or NULL: 0                                               */
  int32_t* kv_len_out;
  int32_t* pos_offset_out;  /* [seqs] or NULL                                                     */
  int32_t* index;           /* [seqs, Hkv, keep] contiguous                                       */
  int keep, recent, max_kv; /* keep >= 1, 0 <= recent <= keep                                     */
} vdx_paged_evict_args;
vdx_status vdx_paged_evict(const vdx_paged_kv* cache, const vdx_kv8_scales* scales, const vdx_paged_kv* into,
                           const vdx_kv8_scales* into_scales, const vdx_paged_evict_args* args, void* stream);

/* Synchronise `stream`, then read and clear the device error word.  Returns VDX_OK,
 * VDX_ERR_TIMEOUT (a kernel gave up on a pipeline wait; the output of that call is
 * undefined), VDX_ERR_RANGE (a rotated q/k value was clamped to the fp16 range; the output
 * is inexact), VDX_ERR_ARG (a q_index entry was out of range; its row was skipped; or a page,
 * length or position that the paged-cache or cross-attention calls clamped or skipped) or
 * VDX_ERR_CUDA (an asynchronous CUDA error is pending). */
vdx_status vdx_sync_check(void* stream);

/* Message for the last non-OK status returned on this host thread ("" if none). */
const char* vdx_last_error(void);

/* Free every cached cos/sin table on every device.  Not to be called while work that uses
 * them is in flight. */
void vdx_shutdown(void);

/* Library version: major*10000 + minor*100 + patch. */
int vdx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* VDX_H_ */
