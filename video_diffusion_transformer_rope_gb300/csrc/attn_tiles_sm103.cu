// Attention of many query rows over a paged cache or over dense keys of another length (cross
// attention), on the 5th-generation tensor cores.
//
//     S = Q K^T,  p = 2^(S * scale*log2(e) - m),  l = sum p,  O = sum p v  (online over key tiles)
//
// Bound: the tensor cores and the exponentials together (at d = 128 a 128 x 128 tile costs 1024
// tensor cycles for its two products, reading shared memory at its full rate for the first), with
// Q and the output through DRAM when the keys are few (cross attention over 512 keys: 512 flops a
// byte).
//
// A unit of work is (sequence, kv head, block of 4 x 128 query rows, range of 128-key tiles); the
// rows of a block are (token, query head of the group) pairs, so grouped heads share every key
// they read.  The grid has a cluster of two CTAs per unit, of which one per two multiprocessors run: each
// takes its own unit and then claims those of clusters that have not started (launch control answers
// with their index), one ahead of its work, so units of uneven length even out.
// Each CTA holds two Q tiles of 128 rows (tile i of rank r: rows 256 i + 128 r and up of the block)
// and half of every key tile (64 keys of K, half the channels of V); rank 0 issues cta_group::2
// MMAs over both CTAs' rows and halves.  The halves leave room for the Q tiles of two units, so
// the next unit's rows load, and a finished unit's output leaves through its Q buffers, while the
// products of the current one run: with 4 key tiles to a unit that work is as long as the products.
//
//   warps 0-3, 4-7   softmax and epilogue of Q tile 0 / 1 (thread = row = TMEM lane)
//   warp 8           TMA producer of the K and V rings; a tile inside one page is one box, another
//                    several, a lane looking up and issuing each
//   warp 9           rank 0: issues the MMAs (one elected lane); rank 1: relays its landed halves
//                    to rank 0 with remote arrivals
//   warp 10          works out the units ahead of the others, into a ring of descriptors (lengths and
//                    ranges: divisions and dependent loads, ~2000 cycles), and loads their Q tiles
//   warp 11          stores finished output tiles: one TMA store, or the live rows of a tile that
//                    ends with its sequence
//
// TMEM (512 columns): S0, S1 at 0 and 128, O0, O1 at 256 and 384; P overwrites the first half of S
// as packed 16-bit pairs and is the A operand of the second product.  Issue order per key tile j:
//     S0(j) ; O1 += P1(j-1) V(j-1) ; S1(j) ; O0 += P0(j) V(j)
// and O1's last product of a unit follows S0 of the next unit's first tile, so the tensor cores do
// not drain between units.  A block whose rows all fit Q tile 0 leaves tile 1 out.  Exponentials
// are taken against the running maximum and kept while the row sum shows every p <= 256 (P is rounded to the
// call's type, as the tensor cores take it; its sum is fp32 and of the unrounded weights); the
// first tile of a unit, or a row whose scores rose, takes the tile's maximum first.
//
// Masks: a row sees keys below its limit; rows of V past the last key any row of the block sees
// are overwritten with zeros in shared memory before the product reads them (the cache may hold
// anything there), and scores of keys past the limit become -inf, whatever K holds.
#include <cstdint>

#include "kv_common.cuh"

namespace vdx {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kQBufs = 4;          // two Q tiles of two units
constexpr int kUnitSlots = 4;
constexpr int kMaxStages = 6;
constexpr uint32_t kRegsSoftmax = 192, kRegsCtl = 120;     // 2 x 192 + 120 = 3 x 168 at launch
static_assert(2 * kRegsSoftmax + kRegsCtl <= 3 * 168, "register split over budget");

// Shared memory of one CTA.  Q tiles and K halves are 64-channel parts of 128-byte swizzled rows; a V
// half is 128 rows of D/2 channels (one part of 128-byte rows, or of 64-byte rows at D = 64).
template <int D>
struct Layout {
  static constexpr int kQBytes = kBM * D * 2;
  static constexpr int kQPart = kBM * 128;
  static constexpr int kParts = D / 64;
  static constexpr int kStageBytes = kBN * D;             // half a tile of K or V
  static constexpr int kKPart = (kBN / 2) * 128;
  static constexpr int kVRow = D;                         // bytes of a V half's row
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kOffK = kQBufs * kQBytes;
  static constexpr int kOffV = kOffK + kStages * kStageBytes;
  static constexpr int kOffCtl = kOffV + kStages * kStageBytes;
};

enum : int {
  kSiteQFull = 32, kSiteQEmpty, kSiteKFull, kSiteKEmpty, kSiteVFull, kSiteVEmpty, kSiteSFull, kSitePReady,
  kSiteOFull, kSiteOEmpty, kSiteDrain, kSiteUnitFull, kSiteUnitEmpty, kSiteStaged, kSiteRelay, kSiteClaim
};

// One unit of work, as warp 10 hands it to the other roles.
struct Unit {
  int s, hk, unit, z;      // sequence, kv head, index among (sequence, head, block), split; s < 0: no unit is left
  int row0, n, keys, shift;    // the sequence's first row, rows, keys and blocks' shift (SeqInfo)
  int tok0, ntok;          // first token of the block and live tokens in it (<= 0: none)
  int len;                 // keys that its last row sees
  int t0, t1;              // key tiles of this split
  int tail;                // rows of V to keep in the split's last tile; kBN: all of them
};

struct Ctl {
  uint64_t q_full[kQBufs], q_empty[kQBufs];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[2], p_ready[2];
  uint64_t o_full[2], o_empty[2], staged[2];
  uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
  uint64_t claim_full, claim_ready;
  uint64_t done;
  alignas(16) uint32_t claim[4];     // answer to the claim of a further cluster's work
  Unit unit[kUnitSlots];
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ int ld_shared_flag(uint32_t addr) {
  int v;
  asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_flag(uint32_t addr) {
  asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(1) : "memory");
}

// Latch a wait that gave up, and the first site that did, beside whatever else has been reported.
__device__ __forceinline__ void report_timeout(int site) {
  if ((atomicOr(&g_error_word, 1u) & 1u) == 0) atomicOr(&g_error_word, static_cast<unsigned>(site & 0xff) << 8);
}

// mbar_try_wait that pairs with another CTA's cluster-scope release: what that CTA wrote by plain stores (or
// read) before it arrived lies before what follows here.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The rest of a warp's wait for a barrier phase whose first look (mbar_try_wait, which itself blocks for
// a while) failed.  Kept out of line: a dozen inlined copies would spread the roles' loops over so
// much code that they miss the instruction caches.  The warp gives up as one, when the CTA's abort
// flag is raised or after kWaitLimitNs, and then raises the flag and records the site.
template <bool kCluster>
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  const unsigned long long t0 = global_timer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, ld_shared_flag(abort_flag) != 0)) return false;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) {
      st_shared_flag(abort_flag);
      if ((threadIdx.x & 31) == 0) report_timeout(site);
      return false;
    }
  }
}
// kCluster: for what the other CTA did by plain accesses.  Waits for copies, products and tensor memory need
// CTA scope only (the copies' bytes, the commits and the tcgen05 fences order those).
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  if (__all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
  return wait_more<kCluster>(bar, parity, abort_flag, site);
}
// The softmax warps' form: their registers are past what a function call leaves room for.
__device__ __forceinline__ bool warp_wait_inline(uint32_t bar, uint32_t parity, uint32_t abort_flag, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, ld_shared_flag(abort_flag) != 0 || global_timer_ns() - t0 > kWaitLimitNs)) {
      st_shared_flag(abort_flag);
      if ((threadIdx.x & 31) == 0) report_timeout(site);
      return false;
    }
  }
  return true;
}

// Shared-memory offsets within Ctl: every barrier address is one 32-bit base plus a constant.
constexpr uint32_t kBarQFull = offsetof(Ctl, q_full), kBarQEmpty = offsetof(Ctl, q_empty), kBarKFull = offsetof(Ctl, k_full),
                   kBarKEmpty = offsetof(Ctl, k_empty), kBarVFull = offsetof(Ctl, v_full), kBarVEmpty = offsetof(Ctl, v_empty),
                   kBarSFull = offsetof(Ctl, s_full), kBarPReady = offsetof(Ctl, p_ready), kBarOFull = offsetof(Ctl, o_full),
                   kBarOEmpty = offsetof(Ctl, o_empty), kBarStaged = offsetof(Ctl, staged),
                   kBarUnitFull = offsetof(Ctl, unit_full), kBarUnitEmpty = offsetof(Ctl, unit_empty),
                   kBarClaimFull = offsetof(Ctl, claim_full), kBarClaimReady = offsetof(Ctl, claim_ready),
                   kOffClaim = offsetof(Ctl, claim), kBarDone = offsetof(Ctl, done), kOffUnit = offsetof(Ctl, unit), kOffAbort = offsetof(Ctl, abort_flag);

// Bounded wait on the way out, whatever the abort flag says: copies and MMAs in flight finish
// before shared or tensor memory is released.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      report_timeout(kSiteDrain);
      return;
    }
  }
}

// How keys are cut into tiles.  Tiles of 128 consecutive keys whatever the page size, where pages are
// a multiple of box_rows >= 8 keys (whole swizzle atoms): a tile inside one page is one box of 128
// rows, another is 128 / box_rows boxes, a lane looking up the page of each.  Other page sizes
// (p.box_rows = 0): a tile ends with its page.
// Dense keys (kPaged = false) are one page.
template <bool kPaged>
struct TileGeom {
  int tiles_per_page;      // of the second kind
  __device__ __forceinline__ explicit TileGeom(const KvParams& p) { tiles_per_page = (p.P + kBN - 1) / kBN; }
  __device__ __forceinline__ int tiles(const KvParams& p, int len) const {
    if (len <= 0) return 0;
    if (!kPaged || p.box_rows) return (len + kBN - 1) / kBN;
    const int full = len / p.P;
    return full * tiles_per_page + (len - full * p.P + kBN - 1) / kBN;
  }
};
template <bool kPaged>
struct TileCursor {
  int page, off;           // entry of the page table and token in the page of the first key
  int key0, keys;          // first key, keys the tile can hold
  __device__ __forceinline__ void seek(const KvParams& p, const TileGeom<kPaged>& g, int t) {
    if (!kPaged) {
      page = 0;
      off = key0 = t * kBN;
      keys = min(kBN, p.P - off);
    } else if (p.box_rows) {
      key0 = t * kBN;
      page = key0 / p.P;
      off = key0 - page * p.P;
      keys = kBN;
    } else {
      page = t / g.tiles_per_page;
      off = (t - page * g.tiles_per_page) * kBN;
      key0 = page * p.P + off;
      keys = min(kBN, p.P - off);
    }
  }
  __device__ __forceinline__ void next(const KvParams& p) {
    key0 += keys;
    off += keys;
    if (!kPaged) {
      keys = min(kBN, p.P - off);
    } else if (p.box_rows) {
      while (off >= p.P) {
        off -= p.P;
        ++page;
      }
    } else {
      if (off == p.P) {
        off = 0;
        ++page;
      }
      keys = min(kBN, p.P - off);
    }
  }
};

template <bool kPaged>
__device__ __forceinline__ Unit make_unit(const KvParams& p, const TileGeom<kPaged>& g, int it, bool report) {
  Unit u;
  const int blk = it % p.nblk;
  int r = it / p.nblk;
  u.z = r % p.nsplit;
  r /= p.nsplit;
  u.hk = r % p.Hkv;
  u.s = r / p.Hkv;
  u.unit = r * p.nblk + blk;
  const SeqInfo sq = sequence_info(p, u.s, report);
  u.row0 = sq.row0;
  u.n = sq.n;
  u.keys = sq.len;
  u.shift = sq.shift;
  const int per = p.block_rows / p.g;
  u.tok0 = blk * per;                                    // nblk * per stays near max_q < 2^31
  u.ntok = min(per, min(sq.n, p.max_q) - u.tok0);
  u.len = u.ntok > 0 ? visible_limit(p, sq, u.tok0 + u.ntok - 1) : 0;
  const int nt = g.tiles(p, u.len);
  const long long a = static_cast<long long>(u.z) * p.split_keys;
  u.t0 = static_cast<int>(min(a, static_cast<long long>(nt)));
  u.t1 = static_cast<int>(min(a + p.split_keys, static_cast<long long>(nt)));
  u.tail = kBN;
  if (u.t0 < u.t1 && u.t1 == nt) {
    TileCursor<kPaged> c;
    c.seek(p, g, nt - 1);
    if (c.key0 + c.keys > u.len) u.tail = u.len - c.key0;
  }
  return u;
}

// A role's walk along the ring of units: wait() for the following one, read the fields it needs (broadcast
// from one lane, so that what follows from them, such as loop counts, stages and MMA descriptors, is
// warp-uniform to the compiler too), and release() its slot, which is free when every role has.
struct UnitReader {
  uint32_t ctl;
  int k = 0;
  __device__ __forceinline__ bool wait() const {
    return warp_wait(ctl + kBarUnitFull + 8 * (k % kUnitSlots), (k / kUnitSlots) & 1, ctl + kOffAbort, kSiteUnitFull);
  }
  __device__ __forceinline__ int get(uint32_t offset) const {
    return __shfl_sync(0xffffffffu, ld_shared_flag(ctl + kOffUnit + (k % kUnitSlots) * static_cast<uint32_t>(sizeof(Unit)) + offset), 0);
  }
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(ctl + kBarUnitEmpty + 8 * (k % kUnitSlots));
    ++k;
  }
};
#define VDX_UNIT(reader, field) (reader).get(offsetof(Unit, field))
constexpr int kUnitReaders = 8 + 3;     // softmax warps, producer, MMA / relay, store

// S = Q K^T over the pair (M = 256, N = 128): A = each CTA's Q tile, B = 64 keys from each CTA.
// The whole MMA warp calls, one elected lane issues.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem, uint32_t idesc) {
  const uint64_t a = smem_desc_sw128(q_smem, 16, 1024), b = smem_desc_sw128(k_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)       // addresses count 16 bytes; a K step is 32 bytes further on
    mma_ss_pair_warp(d_tmem, a + (kk >> 2) * (Layout<D>::kQPart >> 4) + (kk & 3) * 2,
                     b + (kk >> 2) * (Layout<D>::kKPart >> 4) + (kk & 3) * 2, idesc, kk > 0 ? 1u : 0u);
}
// O (+)= P V over the pair (M = 256, N = D): A = P from each CTA's TMEM, B = V, D/2 channels from each
// CTA, channel-contiguous (MN-major); 16 keys a step, 8-key groups 8 rows apart.  D = 64: 64-byte
// swizzled rows (layout 4 in bits 61-63 of the descriptor instead of 2).
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t idesc, bool accumulate) {
  uint64_t desc = smem_desc_sw128(v_smem, Layout<D>::kStageBytes, 8 * Layout<D>::kVRow);
  if (D == 64) desc = (desc & ~(7ull << 61)) | (4ull << 61);
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk)
    mma_ts_pair_warp(d_tmem, p_tmem + kk * 8, desc + kk * Layout<D>::kVRow, idesc, (accumulate || kk > 0) ? 1u : 0u);
}
// Arrival on the other CTA's barrier that orders this CTA's plain shared-memory writes before it
// for the whole cluster.
__device__ __forceinline__ void mbar_arrive_remote_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ float row_max128(const uint32_t (&s)[128]) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fmax3(__uint_as_float(s[i]), __uint_as_float(s[i + 8]), __uint_as_float(s[i + 16]));
#pragma unroll
  for (int j = 24; j < 120; j += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmax3(m[i], __uint_as_float(s[i + j]), __uint_as_float(s[i + j + 8]));
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], __uint_as_float(s[i + 120]));
  return fmaxf(fmax3(fmax3(m[0], m[1], m[2]), m[3], m[4]), fmax3(m[5], m[6], m[7]));
}

// p = 2^(s * c - base) of a 128-column row, packed to pairs of T; returns the fp32 row sum.
template <typename T>
__device__ __forceinline__ float exp_row128(const uint32_t (&s)[128], float c, float base, uint32_t (&pk)[64]) {
  const uint64_t c2 = f32x2(c, c), nb2 = f32x2(-base, -base);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 64; ++e) {
    const uint64_t a = ffma2(f32x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, nb2);
    float a0, a1;
    f32x2_split(a, a0, a1);
    const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
    acc[e & 3] = fadd2(acc[e & 3], f32x2(p0, p1));
    pk[e] = pack2<T>(p0, p1);
  }
  float l0, l1;
  f32x2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), l0, l1);
  return l0 + l1;
}

// Scores of a row (this thread's TMEM lane) at column `valid` and beyond become -inf, in place: a
// loop over 32 columns at a time, since ragged tiles are few and unrolled code in the row's path
// costs the others instruction-cache misses.
__device__ __forceinline__ void mask_row(uint32_t s_tmem, int valid) {
#pragma unroll 1
  for (int ch = 0; ch < kBN; ch += 32) {
    if (__all_sync(0xffffffffu, valid >= ch + 32)) continue;
    uint32_t r[32];
    tmem_ld32(s_tmem + ch, r);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (ch + e >= valid) r[e] = 0xff800000u;
    tmem_st32(s_tmem + ch, r);
  }
  tmem_wait_st();
}

// 32 bytes to global memory: one full sector per thread where the row is 32-byte aligned.
__device__ __forceinline__ void store32(void* dst, const uint32_t* r, bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
  } else {
    uint4* d = static_cast<uint4*>(dst);
    d[0] = make_uint4(r[0], r[1], r[2], r[3]);
    d[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// Ask for a cluster of the grid that has not been launched: the 16-byte answer goes to this offset of every CTA
// of this cluster, counted on its barrier.  Not to be asked again once an answer was "none".
__device__ __forceinline__ void claim_cluster(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];"
      ::"r"(answer), "r"(bar) : "memory");
}
// The unit of the claimed cluster (its index in the grid), or `none`.
__device__ __forceinline__ int claimed_cluster(uint32_t answer, int none) {
  const uint4 a = ld_shared_v4(answer);
  const uint64_t lo = a.x | (static_cast<uint64_t>(a.y) << 32), hi = a.z | (static_cast<uint64_t>(a.w) << 32);
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tmov.b128 r, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x) : "l"(lo), "l"(hi) : "memory");
  fence_proxy_async_smem();          // the next answer is written by the async proxy, after this read
  return got && static_cast<int>(x >> 1) < none ? static_cast<int>(x >> 1) : none;
}

// Rows of V past the last visible key become zeros (this CTA's half of the tile; whole warp).
template <int D>
__device__ __noinline__ void zero_v_rows(uint32_t v_smem, int from, int lane) {
  for (int i = from * (Layout<D>::kVRow / 16) + lane; i < kBN * (Layout<D>::kVRow / 16); i += 32)
    st_shared_v4(v_smem + i * 16, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async_smem();
  __syncwarp();
}

// One instance per kind of keys and of results, so that none carries the others' code: in this
// kernel, whose roles' code does not fit the instruction caches, that is time.
template <typename T, int D, bool kPaged, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
attn_tiles(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kbox,
           const __grid_constant__ CUtensorMap tm_vbox, const __grid_constant__ CUtensorMap tm_out,
           const __grid_constant__ KvParams p, const int units, const int claim) {
  using Lo = Layout<D>;
  constexpr int kS = Lo::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Lo::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = smem_addr(smem), sK = smem_addr(smem + Lo::kOffK), sV = smem_addr(smem + Lo::kOffV);
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (tid == 0) {
    // rank 0's full barriers also count one relayed arrival from rank 1, its P-ready and O-empty
    // barriers one arrival from each of rank 1's softmax warps
    const uint32_t full = leader ? 2 : 1, rows = leader ? 128 + 4 : 128;
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(smem_addr(&ctl->q_full[i]), full);
      mbar_init(smem_addr(&ctl->q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ctl->s_full[i]), 1);
      mbar_init(smem_addr(&ctl->p_ready[i]), rows);
      mbar_init(smem_addr(&ctl->o_full[i]), 1);
      mbar_init(smem_addr(&ctl->o_empty[i]), rows);
      mbar_init(smem_addr(&ctl->staged[i]), 128);
    }
    for (int i = 0; i < kS; ++i) {
      mbar_init(smem_addr(&ctl->k_full[i]), full);
      mbar_init(smem_addr(&ctl->k_empty[i]), 1);
      mbar_init(smem_addr(&ctl->v_full[i]), full);
      mbar_init(smem_addr(&ctl->v_empty[i]), 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(smem_addr(&ctl->unit_full[i]), 1);
      mbar_init(smem_addr(&ctl->unit_empty[i]), kUnitReaders);
    }
    mbar_init(smem_addr(&ctl->claim_full), 1);
    mbar_init(smem_addr(&ctl->claim_ready), 2);          // both CTAs' (used on rank 0)
    mbar_init(smem_addr(&ctl->done), 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc_pair(smem_addr(&ctl->tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();                 // both CTAs' barriers exist before any remote arrival
  tc_fence_after_sync();
  wait_for_earlier_work();
  const uint32_t tmem = ctl->tmem_base;
  const uint32_t sCtl = smem_addr(ctl);
  const TileGeom<kPaged> geom(p);
  const int per_tile = kBM / p.g;     // tokens of one Q tile
  auto wait = [&](uint32_t bar, int parity, int site) {      // the whole warp, which gives up as one
    return warp_wait(bar, parity & 1, sCtl + kOffAbort, site);
  };

  if (warp >= 8) {
    regs_decrease<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------------------------------------------ TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      int kv = 0, k_issued = 0;                         // key tiles so far; tiles of K (an abort may fall between)
      bool ok = true;
      UnitReader in{sCtl};
      while (ok) {
        if (!(ok = in.wait())) break;
        if (VDX_UNIT(in, s) < 0) {
          in.release();
          break;
        }
        const int t0 = VDX_UNIT(in, t0), t1 = VDX_UNIT(in, t1), s = VDX_UNIT(in, s), hk = VDX_UNIT(in, hk);
        const int len = kPaged ? VDX_UNIT(in, len) : 0;
        in.release();
        if (t0 >= t1) continue;
        const int* table = kPaged ? p.table + static_cast<long long>(s) * p.table_stride : nullptr;
        TileCursor<kPaged> c;
        c.seek(p, geom, t0);
        // K: this CTA's 64 keys; V: all 128 of its channels.  A tile is one box of each where it lies inside
        // one page (always, for dense keys and for tiles that end with their page), else box_rows-key
        // boxes, one to a lane, of the keys that some row sees.
        const int box = kPaged ? p.box_rows : 0;
        bool whole;
        int seen, page, tok;                            // of the tile: keys in boxes; of this lane's box
        auto look_up = [&](const TileCursor<kPaged>& c) {
          whole = !kPaged || !box || c.off + kBN <= p.P;
          seen = whole ? kBN : min(kBN, len - c.key0);
          page = !kPaged ? s : 0;
          tok = c.off + lane * box;
          if (kPaged && (lane == 0 || (!whole && lane * box < seen))) {
            int e = c.page;
            if (!whole)
              while (tok >= p.P) {
                tok -= p.P;
                ++e;
              }
            page = load_i32(table + e);
          }
        };
        look_up(c);
        for (int t = t0; ok && t < t1; ++t) {
          const bool one = whole;
          const int keys = seen, tok0 = kPaged ? tok : c.key0;
          int pg = page;
          if (kPaged && static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) {
            atomicOr(&g_error_word, kErrPage);
            pg = -1;                                    // out of the map's range: filled with zeros
          }
          c.next(p);
          if (kPaged && t + 1 < t1) look_up(c);         // the next tile's pages, while this one waits for its stages
          const int st = kv % kS;
          const int k_box0 = one ? 0 : static_cast<int>(rank) * (kBN / 2 / max(box, 1));   // first box of this CTA's keys
          const int k_rows = one ? kBN / 2 : max(0, min(kBN / 2, keys - static_cast<int>(rank) * (kBN / 2)));
#pragma unroll 1
          for (int which = 0; which < 2; ++which) {
            // boxes [b0, b0 + n) of the tile, in rows of this stage from 0
            const int b0 = which == 0 ? k_box0 : 0;
            const int n = one ? 1 : ((which == 0 ? k_rows : keys) + box - 1) / box;
            const uint32_t bytes = one ? Lo::kStageBytes : static_cast<uint32_t>(n * box) * (which == 0 ? D * 2 : D);
            const uint32_t empty = (which == 0 ? sCtl + kBarKEmpty : sCtl + kBarVEmpty) + 8 * st;
            if (kv >= kS && !(ok = wait(empty, kv / kS - 1, which == 0 ? kSiteKEmpty : kSiteVEmpty))) break;
            const uint32_t bar = (which == 0 ? sCtl + kBarKFull : sCtl + kBarVFull) + 8 * st;
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            if (which == 0) ++k_issued;
            __syncwarp();
            if (lane >= b0 && lane < b0 + n) {
              const uint32_t row = one ? 0u : static_cast<uint32_t>((lane - b0) * box);
              if (which == 0) {
                const int kp = !kPaged && p.k_p == 0 ? 0 : pg;       // one set of keys for the whole batch
#pragma unroll
                for (int h = 0; h < Lo::kParts; ++h)
                  tma_load_4d(sK + st * Lo::kStageBytes + h * Lo::kKPart + row * 128, one ? &tm_k : &tm_kbox, bar, h * 64,
                              tok0 + (one ? static_cast<int>(rank) * (kBN / 2) : 0), hk, kp);
              } else {
                tma_load_4d(sV + st * Lo::kStageBytes + row * Lo::kVRow, one ? &tm_v : &tm_vbox, bar,
                            static_cast<int>(rank) * (D / 2), tok0, hk, !kPaged && p.v_p == 0 ? 0 : pg);
              }
            }
            __syncwarp();
          }
          if (ok) ++kv;
        }
      }
      // every copy lands before the CTA can retire (rank 0's barriers also need rank 1's relay, which
      // an abort may have stopped: its own copies are waited for by the bounded drain)
      if (lane == 0) {
        for (int st = 0; st < kS; ++st) {
          if (k_issued > st) drain_wait(sCtl + kBarKFull + 8 * st, ((k_issued - 1 - st) / kS) & 1);
          if (kv > st) drain_wait(sCtl + kBarVFull + 8 * st, ((kv - 1 - st) / kS) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 9 && leader) {
      // ------------------------------------------------------------------ MMA issuer
      constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t kIdQK = idesc_f16kind_f32acc(2 * kBM, kBN, kType, 0);
      constexpr uint32_t kIdPV = idesc_f16kind_f32acc(2 * kBM, D, kType, 1);
      // This warp shares its scheduler with two softmax warps, and every instruction between two
      // products delays the next one: stages, phases and descriptors are carried, not computed.
      int st = 0, ph = 0;                                // K / V stage and its phase
      int pr0 = 0, pr1 = 0;                              // phases of p_ready
      int n = 0, n1 = 0;                                 // units, units with a second Q tile
      bool ok = true;
      // the second Q tile's product with V that is still to be issued
      bool have = false, first = false, last = false;
      int st1 = 0;
      auto finish_second = [&]() {                        // O1 += P1 V of the key tile before
        ok = wait(sCtl + kBarPReady + 8, pr1, kSitePReady);
        pr1 ^= 1;
        if (first && n1 > 1 && ok) ok = wait(sCtl + kBarOEmpty + 8, n1, kSiteOEmpty);
        if (!ok) return;
        tc_fence_after_sync();
        issue_pv<D>(tmem + 384, tmem + 128, sV + st1 * Lo::kStageBytes, kIdPV, !first);
        mma_commit_pair_warp(sCtl + kBarVEmpty + 8 * st1);
        if (last) mma_commit_pair_warp(sCtl + kBarOFull + 8);
        have = false;
      };
      UnitReader in{sCtl};
      while (ok) {
        if (!(ok = in.wait())) break;
        if (VDX_UNIT(in, s) < 0) {
          in.release();
          break;
        }
        int left = VDX_UNIT(in, t1) - VDX_UNIT(in, t0);
        const int tail = VDX_UNIT(in, tail);
        const bool two = VDX_UNIT(in, ntok) > 2 * per_tile;
        in.release();
        if (left <= 0) {
          // The pending product must not wait for a unit with tiles: until it is issued the softmax and
          // store warps do not get to the units after theirs, and with every slot of the ring taken by
          // such units none would follow.
          if (have) finish_second();
          continue;
        }
        const int q0 = sQ + 2 * (n & 1) * Lo::kQBytes, qph = n >> 1;
        const uint32_t q_full = sCtl + kBarQFull + 8 * (2 * (n & 1));
        if (!(ok = wait(q_full, qph, kSiteQFull) && wait(sCtl + kBarKFull + 8 * st, ph, kSiteKFull))) break;
        bool fresh = true;
        while (true) {
          const uint32_t kt = sK + st * Lo::kStageBytes, vt = sV + st * Lo::kStageBytes;
          const bool end = left == 1;
          tc_fence_after_sync();
          issue_qk<D>(tmem, q0, kt, kIdQK);
          mma_commit_pair_warp(sCtl + kBarSFull + 0);
          if (!two) mma_commit_pair_warp(sCtl + kBarKEmpty + 8 * st);
          if (have) {
            finish_second();
            if (!ok) break;
          }
          if (two) {
            if (fresh) {
              if (!(ok = wait(q_full + 8, qph, kSiteQFull))) break;
              tc_fence_after_sync();
            }
            issue_qk<D>(tmem + 128, q0 + Lo::kQBytes, kt, kIdQK);
            mma_commit_pair_warp(sCtl + kBarSFull + 8);
            mma_commit_pair_warp(sCtl + kBarKEmpty + 8 * st);
          }
          ok = wait(sCtl + kBarVFull + 8 * st, ph, kSiteVFull);
          if (end && tail < kBN) {
            // rank 1 zeroed rows of its half before it arrived: seen at cluster scope (the phase is complete,
            // so this returns at once)
            if (ok) ok = warp_wait<true>(sCtl + kBarVFull + 8 * st, ph, sCtl + kOffAbort, kSiteVFull);
            zero_v_rows<D>(vt, tail, lane);
          }
          // the next tile's keys are waited for here, so that its product follows this one's without a
          // wait in between
          const int st_was = st;
          if (++st == kS) {
            st = 0;
            ph ^= 1;
          }
          if (!end && ok) ok = wait(sCtl + kBarKFull + 8 * st, ph, kSiteKFull);
          if (ok) ok = wait(sCtl + kBarPReady, pr0, kSitePReady);
          pr0 ^= 1;
          if (fresh && n > 0 && ok) ok = wait(sCtl + kBarOEmpty, n + 1, kSiteOEmpty);
          if (!ok) break;
          tc_fence_after_sync();
          issue_pv<D>(tmem + 256, tmem, vt, kIdPV, !fresh);
          if (end) mma_commit_pair_warp(sCtl + kBarOFull + 0);
          if (two) {
            if (fresh) ++n1;
            have = true;
            first = fresh;
            last = end;
            st1 = st_was;
          } else {
            mma_commit_pair_warp(sCtl + kBarVEmpty + 8 * st_was);
          }
          fresh = false;
          if (--left == 0) break;
        }
        ++n;
      }
      if (ok && have) finish_second();
      mma_commit_pair_warp(sCtl + kBarDone);
      drain_wait(sCtl + kBarDone, 0);
    } else if (warp == 9) {
      // ------------------------------------------------------------------ relay (rank 1): tells rank 0
      // that this CTA's Q tiles and halves of K and V have landed
      int st = 0, ph = 0, n = 0;
      bool ok = true;
      UnitReader in{sCtl};
      while (ok) {
        if (!(ok = in.wait())) break;
        if (VDX_UNIT(in, s) < 0) {
          in.release();
          break;
        }
        int left = VDX_UNIT(in, t1) - VDX_UNIT(in, t0);
        const int tail = VDX_UNIT(in, tail);
        in.release();
        if (left <= 0) continue;
        for (int i = 0; ok && i < 2; ++i) {
          const int b = 2 * (n & 1) + i;
          ok = wait(sCtl + kBarQFull + 8 * b, n >> 1, kSiteRelay);
          if (ok && lane == 0) mbar_arrive_remote(mapa_shared(sCtl + kBarQFull + 8 * b, 0));
        }
        for (; ok && left > 0; --left) {
          if (!(ok = wait(sCtl + kBarKFull + 8 * st, ph, kSiteRelay))) break;
          if (lane == 0) mbar_arrive_remote(mapa_shared(sCtl + kBarKFull + 8 * st, 0));
          if (!(ok = wait(sCtl + kBarVFull + 8 * st, ph, kSiteRelay))) break;
          if (left == 1 && tail < kBN) {
            zero_v_rows<D>(sV + st * Lo::kStageBytes, tail, lane);
            if (lane == 0) mbar_arrive_remote_cluster(mapa_shared(sCtl + kBarVFull + 8 * st, 0));
          } else if (lane == 0) {
            mbar_arrive_remote(mapa_shared(sCtl + kBarVFull + 8 * st, 0));
          }
          if (++st == kS) {
            st = 0;
            ph ^= 1;
          }
        }
        ++n;
      }
      __syncwarp();
      // rank 0's last commit also arrives here; see it land before this CTA can retire
      drain_wait(sCtl + kBarDone, 0);
    } else if (warp == 10) {
      // ------------------------------------------------------------------ units ahead of the other roles,
      // and their Q tiles once the unit before the last has left its buffers
      if (lane == 0) tma_prefetch_desc(&tm_q);
      const uint32_t q_bytes = static_cast<uint32_t>(per_tile * p.g) * D * 2;
      bool ok = true;
      int n = 0, q_issued = 0;                          // units with key tiles, Q tiles
      int it = static_cast<int>(blockIdx.x >> 1), claims = 0;
      int busy = -1;                                    // the last unit with key tiles
      const uint32_t remote = mapa_shared(sCtl, 0);
      for (int k = 0;; ++k) {
        const int slot = k % kUnitSlots;
        if (k >= kUnitSlots && !(ok = wait(sCtl + kBarUnitEmpty + 8 * slot, k / kUnitSlots - 1, kSiteUnitEmpty))) break;
        Unit u;
        u.s = -1;
        u.t0 = u.t1 = u.ntok = 0;
        const bool more = it < units;
        if (more) u = make_unit<kPaged>(p, geom, it, leader && lane == 0);
        if (lane == 0) {
          ctl->unit[slot] = u;
          mbar_arrive(sCtl + kBarUnitFull + 8 * slot);
        }
        __syncwarp();
        if (!more) break;
        if (u.t0 < u.t1) {
          for (int i = 0; i < 2; ++i) {
            const int b = 2 * (n & 1) + i;
            if (n >= 2 && !(ok = wait(sCtl + kBarQEmpty + 8 * b, (n >> 1) - 1, kSiteQEmpty))) break;
            if (lane == 0) {
              const uint32_t bar = sCtl + kBarQFull + 8 * b;
              mbar_arrive_expect_tx(bar, q_bytes);
#pragma unroll
              for (int h = 0; h < Lo::kParts; ++h)
                tma_load_4d(sQ + b * Lo::kQBytes + h * Lo::kQPart, &tm_q, bar, h * 64, u.hk * p.g,
                            u.row0 + u.tok0 + (2 * i + static_cast<int>(rank)) * per_tile, kPaged || p.q_b == 0 ? 0 : u.s);
            }
            ++q_issued;
            __syncwarp();
          }
          if (!ok) break;
          ++n;
          // When the unit with tiles before this one is done, claim a further one.  Claimed any earlier, the units
          // of a short call would be dealt out before their lengths tell.  (Its slot, taken again, says so.)
          if (claim && busy >= 0 && k - busy < kUnitSlots &&
              !(ok = wait(sCtl + kBarUnitEmpty + 8 * (busy % kUnitSlots), busy / kUnitSlots, kSiteUnitEmpty)))
            break;
          busy = k;
        }
        it = units;
        if (!claim) continue;                           // every cluster of the grid runs at once
        // Claim the work of a cluster that has not started yet: rank 0 asks once both CTAs expect the answer
        // and have read the one before; it comes to both.
        if (lane == 0) {
          mbar_arrive_expect_tx(sCtl + kBarClaimFull, 16);
          mbar_arrive_remote_cluster(remote + kBarClaimReady);
        }
        __syncwarp();
        if (leader) {
          // the other CTA's read of the last answer lies before the next one is asked for
          if (!(ok = warp_wait<true>(sCtl + kBarClaimReady, claims & 1, sCtl + kOffAbort, kSiteClaim))) break;
          if (lane == 0) claim_cluster(sCtl + kOffClaim, sCtl + kBarClaimFull);
          __syncwarp();
        }
        ++claims;
        if (!(ok = wait(sCtl + kBarClaimFull, claims - 1, kSiteClaim))) break;
        it = claimed_cluster(sCtl + kOffClaim, units);
        __syncwarp();
      }
      if (lane == 0 && claims > 0) drain_wait(sCtl + kBarClaimFull, (claims - 1) & 1);
      if (lane == 0)
        for (int b = 0; b < kQBufs; ++b)
          if (q_issued > b) drain_wait(sCtl + kBarQFull + 8 * b, ((q_issued - 1 - b) / kQBufs) & 1);
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ output tiles
      bool ok = true;
      int n = 0, n1 = 0;
      UnitReader in{sCtl};
      while (ok) {
        if (!(ok = in.wait())) break;
        if (VDX_UNIT(in, s) < 0) {
          in.release();
          break;
        }
        const bool tiles = VDX_UNIT(in, t0) < VDX_UNIT(in, t1);
        const int ntok = VDX_UNIT(in, ntok), s = VDX_UNIT(in, s), hk = VDX_UNIT(in, hk);
        const int tok0 = VDX_UNIT(in, tok0) + (kPaged ? VDX_UNIT(in, row0) : 0);
        in.release();
        if (!tiles) continue;
        const bool two = ntok > 2 * per_tile;
        for (int i = 0; ok && i < 2; ++i) {
          const int b = 2 * (n & 1) + i;
          const int tok = (2 * i + static_cast<int>(rank)) * per_tile;      // within the block
          const int live = min(per_tile, ntok - tok);
          if (i == 0 || two) {
            ok = wait(sCtl + kBarStaged + 8 * i, i == 0 ? n : n1, kSiteStaged);
            if (!ok) break;
            const uint32_t src = sQ + b * Lo::kQBytes;
            if (kSplit || live <= 0) {
              // partial results leave from the registers; a tile without rows has none
            } else if (!kPaged || live == per_tile) {
              if (lane == 0) {
#pragma unroll
                for (int h = 0; h < Lo::kParts; ++h)
                  tma_store_4d(&tm_out, src + h * Lo::kQPart, h * 64, hk * p.g, tok0 + tok, kPaged ? 0 : s);
                bulk_commit_group();
                bulk_wait_group_read0();
              }
            } else {
              // the sequence ends inside the tile: its rows alone, 16 bytes a lane
              constexpr int kChunks = D / 8;
              for (int j = lane; j < live * p.g * kChunks; j += 32) {
                const int row = j / kChunks, ch = j % kChunks;
                const uint4 x = ld_shared_v4(src + (ch >> 3) * Lo::kQPart + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                const int tk = row / p.g, hd = row - tk * p.g;
                T* dst = static_cast<T*>(p.out) +
                         ((static_cast<long long>(tok0) + tok + tk) * p.Hq + hk * p.g + hd) * D + ch * 8;
                *reinterpret_cast<uint4*>(dst) = x;
              }
            }
          } else {
            ok = wait(sCtl + kBarQFull + 8 * b, n >> 1, kSiteQFull);   // the unused tile's copy has landed
            if (!ok) break;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sCtl + kBarQEmpty + 8 * b);
        }
        ++n;
        if (two) ++n1;
      }
      __syncwarp();
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------------- softmax + epilogue
    regs_increase<kRegsSoftmax>();
    const int qi = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_bits + 128 * qi;
    const uint32_t tO = tmem + lane_bits + 256 + 128 * qi;
    const int my_tok = row / p.g, my_head = row - my_tok * p.g;
    const bool in_tile = my_tok < per_tile;
    const int tok = (2 * qi + static_cast<int>(rank)) * per_tile + my_tok;   // within a block
    const uint32_t remote = mapa_shared(sCtl, 0);
    const float c = p.scale_log2;
    int g = 0, n = 0, nq = 0;                    // this Q tile's key tiles and units; units with key tiles
    bool ok = true;
    // one arrival per thread on rank 0, one per warp from rank 1, whose TMEM accesses are complete
    auto arrive = [&](uint32_t bar) {
      tc_fence_before_sync();
      if (leader) {
        mbar_arrive(sCtl + bar);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(remote + bar);
      }
    };
    for (int k = 0; ok; ++k) {
      // The unit's fields are read from its slot where they are needed (the score row leaves no
      // registers to keep them in); the slot is free when the unit is done.
      const int slot = k % kUnitSlots;
      const Unit& u = ctl->unit[slot];
      if (!(ok = warp_wait_inline(sCtl + kBarUnitFull + 8 * slot, (k / kUnitSlots) & 1, sCtl + kOffAbort, kSiteUnitFull))) break;
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(sCtl + kBarUnitEmpty + 8 * slot);
      };
      if (u.s < 0) {
        release();
        break;
      }
      int t = u.t0;
      const int t1 = u.t1;
      if (t < t1) ++nq;
      if (qi == 1 && u.ntok <= 2 * per_tile) {
        release();
        continue;
      }
      const bool live = in_tile && tok < u.ntok;
      const int limit = !live ? 0 : (kPaged ? visible_limit(p, SeqInfo{u.row0, u.n, u.keys, u.shift}, u.tok0 + tok) : u.len);
      const bool any_live = __any_sync(0xffffffffu, live);
      // tiles below this one are whole for every live row of the warp
      const int whole_to = !kPaged ? u.len / kBN
                           : !p.box_rows ? 0 : __reduce_min_sync(0xffffffffu, live ? limit : 0x7fffffff) / kBN;
      float m = -INFINITY, l = 0.f;
      bool fresh = true;                       // no tile of this unit has been weighed yet
      bool scaled = false;                     // O holds earlier tiles' sums (not before the second one)
      for (; t < t1; ++t) {
        if (!(ok = warp_wait_inline(sCtl + kBarSFull + 8 * qi, g, sCtl + kOffAbort, kSiteSFull))) break;
        g ^= 1;
        tc_fence_after_sync();
        int valid = kBN;
        bool seen = any_live;
        if (t >= whole_to) {
          TileCursor<kPaged> cur;
          cur.seek(p, geom, t);
          valid = min(limit - cur.key0, cur.keys);
          seen = __any_sync(0xffffffffu, live && valid > 0);
        }
        if (seen) {
          if (t >= whole_to) mask_row(tS, valid);
          uint32_t pk[64];
          float lt, alpha = 1.f;
          // Weigh the row against the running maximum; if that does not do (a sum above 256, or a row
          // that has seen no key yet, whose maximum is -inf), look at the tile's own maximum first and
          // weigh it again.  The first tile is looked at right away.  One copy of the code: a second
          // one costs more in instruction-cache misses than the branches do.
          bool look = fresh;
          while (true) {
            uint32_t s[128];
            tmem_ld128(tS, s);
            if (look) {
              const float mt = row_max128(s) * c;
              if (mt > m) {
                alpha = ex2_approx(m - mt);
                l *= alpha;
                m = mt;
              }
            }
            // a row without keys so far: its scores are -inf and weigh nothing
            lt = exp_row128<T>(s, c, look && !(m > -INFINITY) ? 0.f : m, pk);
            if (look || !__any_sync(0xffffffffu, live && !(lt <= 256.f))) break;
            look = true;
          }
          fresh = false;
          // S of this tile is complete, and with it every product issued before it: O holds the sum up
          // to the tile before and may be scaled
          if (look && scaled && __any_sync(0xffffffffu, live && alpha != 1.f)) {
            uint32_t r[32];
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tmem_ld32(tO + ch * 32, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st32(tO + ch * 32, r);
            }
          }
          uint32_t (&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[0]);
          uint32_t (&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[32]);
          tmem_st32(tS, lo);
          tmem_st32(tS + 32, hi);
          l += lt;
          tmem_wait_st();
        } else if (any_live) {
          // no row of this warp sees the tile: its weights are zeros
          uint32_t z[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) z[e] = 0u;
          tmem_st32(tS, z);
          tmem_st32(tS + 32, z);
          tmem_wait_st();
        }
        scaled = true;
        arrive(kBarPReady + 8 * qi);
      }
      if (!ok) break;
      const bool empty = !(m > -INFINITY) && !(l != l);  // saw no key (a NaN sum is an answer)
      const int h = u.hk * p.g + my_head;
      const long long prow = (static_cast<long long>(u.unit) * p.nsplit + u.z) * p.block_rows + tok * p.g + my_head;
      if (live) {
        const SeqInfo sq{u.row0, u.n, u.keys, u.shift};
        if (kSplit)
          p.part_ml[prow] = make_float2(empty ? -INFINITY : m, l);
        else if (p.lse)
          p.lse[lse_index(p, u.s, sq, h, u.tok0 + tok)] = empty ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
        if (!scaled && !kSplit) {
          // the block sees no key at all (a split without keys is not read)
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (out_row(p, u.s, sq, u.tok0 + tok) * p.Hq + h) * D);
#pragma unroll
          for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      release();
      if (!scaled) continue;
      if (!(ok = warp_wait_inline(sCtl + kBarOFull + 8 * qi, n & 1, sCtl + kOffAbort, kSiteOFull))) break;
      tc_fence_after_sync();
      if (any_live) {
        const float inv = empty ? 0.f : 1.f / l;
        const uint32_t tile = sQ + (2 * (~nq & 1) + qi) * Lo::kQBytes + row * 128;   // this row of the unit's Q tile
        float* dst = p.part_o + prow * D;
        const bool al = (reinterpret_cast<uintptr_t>(p.part_o) & 31) == 0;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t r[32];
          tmem_ld32(tO + ch * 32, r);
          if (empty) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (kSplit) {
            if (live && !empty) {                          // the join does not read an empty row
#pragma unroll
              for (int e = 0; e < 32; e += 8) store32(dst + ch * 32 + e, r + e, al);
            }
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = pack2<T>(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = ch * 4 + e;                     // 16-byte chunk of the row
              st_shared_v4(tile + (x >> 3) * Lo::kQPart + (((x & 7) ^ (row & 7)) << 4),
                           make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]));
            }
          }
        }
      }
      arrive(kBarOEmpty + 8 * qi);
      fence_proxy_async_smem();
      mbar_arrive(sCtl + kBarStaged + 8 * qi);
      ++n;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();                 // neither CTA leaves while the pair's MMAs may use it
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// A [n3][n2][n1] grid of rows of D channels (element strides s1, s2, s3) as a map with boxes of
// b1 x b2 rows of `channels` channels (64: 128-byte swizzle, 32: 64-byte).
template <typename T>
bool encode_rows(EncodeTiledFn encode, CUtensorMap* map, const void* base, int D, long long n1, long long s1, long long n2,
                 long long s2, long long n3, long long s3, int channels, int b1, int b2) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2),
                              static_cast<cuuint64_t>(n3)};
  auto bytes = [&](long long n, long long s) { return static_cast<cuuint64_t>(n > 1 ? s : D) * 2; };   // unused where n = 1
  const cuuint64_t strides[3] = {bytes(n1, s1), bytes(n2, s2), bytes(n3, s3)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(channels), static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                channels == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const KvParams& p, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  CUtensorMap mq, mk, mv, mkb{}, mvb{}, mo;            // no boxes: their maps are never used
  const bool one_q = p.cu != nullptr || p.q_b == 0;
  const bool has_keys = p.P > 0;
  // dimensions: q and out (d, head, token, batch), k and v (d, token, head, page)
  const long long kpages = !p.table && p.k_p == 0 ? 1 : p.num_pages, vpages = !p.table && p.v_p == 0 ? 1 : p.num_pages;
  const void* k = has_keys ? p.k : p.q;                  // no keys: the maps are never used
  const void* v = has_keys ? p.v : p.q;
  const int P = has_keys ? p.P : 1;
  const long long ob = static_cast<long long>(p.N) * p.Hq * D;
  if (!encode_rows<T>(encode, &mq, p.q, D, p.Hq, p.q_h, p.N, p.q_t, one_q ? 1 : p.S, p.q_b, 64, p.g, kBM / p.g) ||
      !encode_rows<T>(encode, &mk, k, D, P, p.k_t, p.Hkv, p.k_h, kpages, p.k_p, 64, kBN / 2, 1) ||
      !encode_rows<T>(encode, &mv, v, D, P, p.v_t, p.Hkv, p.v_h, vpages, p.v_p, D / 2, kBN, 1) ||
      (p.box_rows && (!encode_rows<T>(encode, &mkb, k, D, P, p.k_t, p.Hkv, p.k_h, kpages, p.k_p, 64, p.box_rows, 1) ||
                      !encode_rows<T>(encode, &mvb, v, D, P, p.v_t, p.Hkv, p.v_h, vpages, p.v_p, D / 2, p.box_rows, 1))) ||
      !encode_rows<T>(encode, &mo, p.out, D, p.Hq, D, p.N, static_cast<long long>(p.Hq) * D, p.cu ? 1 : p.S, ob, 64, p.g,
                      kBM / p.g)) {
    *what = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  const int smem = Layout<D>::kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
  static std::atomic<uint64_t> done[4] = {};
  auto* kernel = p.table ? (p.nsplit > 1 ? attn_tiles<T, D, true, true> : attn_tiles<T, D, true, false>)
                         : (p.nsplit > 1 ? attn_tiles<T, D, false, true> : attn_tiles<T, D, false, false>);
  const cudaError_t e = allow_shared(kernel, smem, &done[(p.table ? 2 : 0) + (p.nsplit > 1 ? 1 : 0)]);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit;
  if (units > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1] = launch_early();
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, mkb, mvb, mo, p, static_cast<int>(units), units > sms / 2 ? 1 : 0);
}

}  // namespace

cudaError_t launch_attn_tiles(const KvParams& p, int d, int dtype, EncodeTiledFn encode, int sms, cudaStream_t stream,
                              const char** what) {
  *what = nullptr;
  note_launch();
  if (dtype == 0)
    return d == 128 ? launch<__nv_bfloat16, 128>(p, encode, sms, stream, what)
                    : launch<__nv_bfloat16, 64>(p, encode, sms, stream, what);
  return d == 128 ? launch<__half, 128>(p, encode, sms, stream, what) : launch<__half, 64>(p, encode, sms, stream, what);
}

cudaError_t read_and_clear_error_word_tiles(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
