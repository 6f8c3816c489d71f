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
//   warps 12-15      8-bit caches only, in warp 8's place: load codes and write them to the K and V rings
//                    as the values they stand for (in fp16, as are Q, which they convert, and P times 2^7);
//                    rank 1's relay passes their arrivals on with a release of cluster scope
//
// A 720p frame of 3600 tokens of 40 heads over 75600 keys in 8 bits takes 4.28 ms, 1300 TFLOP/s: the converters keep up
// (waits for K and V are no more than in 16 bits), but leave the softmax 144 registers, so that a row comes in two halves and
// its maximum and its weights read S twice; P is ready ~500 cycles later.  Whole rows with 184 or 192 registers spill
// elsewhere: 4.47 and 4.63 ms; halves with 176: 4.53; 152 and 104: 4.43.  (Those with rank 1's converters telling rank 0
// themselves at CTA scope, which took 4.24 ms but orders nothing between two CTAs.  A second relay, for K alone: 4.45.)
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

#include "kv8.cuh"
#include "kv_common.cuh"
#include "kv_maps.h"
#include "sm103_wait.cuh"

namespace vdx {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kThreads = 384;
constexpr int kThreads8 = 512;     // with the converters of an 8-bit cache
constexpr int kTmemCols = 512;
constexpr int kQBufs = 4;          // two Q tiles of two units
constexpr int kUnitSlots = 4;
constexpr int kMaxStages = 6;
constexpr uint32_t kRegsSoftmax = 192, kRegsCtl = 120;     // 2 x 192 + 120 = 3 x 168 at launch
static_assert(2 * kRegsSoftmax + kRegsCtl <= 3 * 168, "register split over budget");
constexpr uint32_t kRegsSoftmax8 = 144, kRegsCtl8 = 112, kRegsConvert = 112;
static_assert(2 * kRegsSoftmax8 + kRegsCtl8 + kRegsConvert <= 4 * 128, "register split over budget");

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
  kSiteOFull, kSiteOEmpty, kSiteUnitFull = kSiteDrain + 1, kSiteUnitEmpty, kSiteStaged, kSiteRelay, kSiteClaim
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
  uint64_t q_ready[kQBufs], q_scaled[kQBufs];      // 8 bits: Q tiles are fp16, in both CTAs (rank 0) and in this one
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
  int8_t q_exp[kQBufs][kBM];         // 8 bits: what their rows were multiplied by
};

static_assert(Layout<128>::kOffCtl + sizeof(Ctl) + 1024 <= 232448, "shared memory of a block");

// Shared-memory offsets within Ctl: every barrier address is one 32-bit base plus a constant.
constexpr uint32_t kBarQReady = offsetof(Ctl, q_ready), kBarQScaled = offsetof(Ctl, q_scaled);
constexpr uint32_t kBarQFull = offsetof(Ctl, q_full), kBarQEmpty = offsetof(Ctl, q_empty), kBarKFull = offsetof(Ctl, k_full),
                   kBarKEmpty = offsetof(Ctl, k_empty), kBarVFull = offsetof(Ctl, v_full), kBarVEmpty = offsetof(Ctl, v_empty),
                   kBarSFull = offsetof(Ctl, s_full), kBarPReady = offsetof(Ctl, p_ready), kBarOFull = offsetof(Ctl, o_full),
                   kBarOEmpty = offsetof(Ctl, o_empty), kBarStaged = offsetof(Ctl, staged),
                   kBarUnitFull = offsetof(Ctl, unit_full), kBarUnitEmpty = offsetof(Ctl, unit_empty),
                   kBarClaimFull = offsetof(Ctl, claim_full), kBarClaimReady = offsetof(Ctl, claim_ready),
                   kOffClaim = offsetof(Ctl, claim), kBarDone = offsetof(Ctl, done), kOffUnit = offsetof(Ctl, unit), kOffAbort = offsetof(Ctl, abort_flag);

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
constexpr int kUnitReaders8 = 8 + 4 + 2;      // converters in the producer's place

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

// The same in two halves of 64 columns, straight from tensor memory, for the instances whose converters need the
// registers: `s` is not held, and the tile's maximum takes a walk of its own.
__device__ __forceinline__ float row_max_halves(uint32_t s_tmem) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t s[64];
    tmem_ld64(s_tmem + 64 * h, s);
#pragma unroll
    for (int i = 0; i < 64; i += 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = fmax3(m[j], __uint_as_float(s[i + j]), __uint_as_float(s[i + j + 4]));
  }
  return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}
template <typename T>
__device__ __forceinline__ float exp_row_halves(uint32_t s_tmem, float c, float base, uint32_t (&pk)[64]) {
  const uint64_t c2 = f32x2(c, c), nb2 = f32x2(-base, -base);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t s[64];
    tmem_ld64(s_tmem + 64 * h, s);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint64_t a = ffma2(f32x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, nb2);
      float a0, a1;
      f32x2_split(a, a0, a1);
      const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
      acc[e & 3] = fadd2(acc[e & 3], f32x2(p0, p1));
      pk[32 * h + e] = pack2<T>(p0, p1);
    }
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

// 16 bytes to shared memory without waiting for them; zeros unless `live`.
__device__ __forceinline__ void copy_code16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// 16 codes of row r, channels 16 c and up of a 64-channel part of 128-byte swizzled rows (64-byte ones: kRow 64), as
// fp16 times `scale` (a pair of equal powers of two).
template <int kRow>
__device__ __forceinline__ void expand_chunk(uint32_t part, int r, int c, const uint4& x, uint32_t scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = half2_mul(decode2<false>(w[i]), scale);
    y[2 * i + 1] = half2_mul(decode2<true>(w[i]), scale);
  }
  const int turn = kRow == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    st_shared_v4(part + r * kRow + (((2 * c + i) ^ turn) << 4), make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
}
// A row of a Q tile (64-channel parts kPart bytes apart, 128-byte swizzled) from bf16 to fp16, in place, times the power of
// two that brings its largest channel into [2^14, 2^15); what falls below fp16's steps is less than 2^-39 of
// that.  Returns the power's exponent.
template <int D, int kPart>
__device__ __forceinline__ int query_row_to_half(uint32_t tile, int r) {
  __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = ld_shared_v4(tile + (c >> 3) * kPart + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));      // NaN: the other
  }
  const float m = fmaxf(__low2float(top), __high2float(top));
  const int e = min(max(14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127), -120), 120);
  const float up = two_to(e);
#pragma unroll 2
  for (int c = 0; c < D / 8; ++c) {
    const uint32_t at = tile + (c >> 3) * kPart + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    const uint4 x = ld_shared_v4(at);
    float f[8];
    unpack8<__nv_bfloat16>(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= up;
    st_shared_v4(at, pack8<__half>(f));
  }
  return e;
}

// One instance per kind of keys and of results, so that none carries the others' code: in this
// kernel, whose roles' code does not fit the instruction caches, that is time.
//
// k8: the cache holds 8-bit codes with scales.  Four more warps copy this CTA's halves of a tile's codes into the stages
// they belong to, a tile ahead, 16 bytes a lane (a lane looks up the page and the scales of a key and of a
// value for the others of its warp); then they spread each row in place to fp16 times its scale, which is exact.  A row's
// codes and its values are the same lanes', so that a warp needs no other.  The products are of fp16 whatever
// T is, since codes become fp16 in one instruction and bf16 in five: queries of bf16 are brought into fp16's
// range by a power of two for each row, exactly, by the same warps at the start of a unit, and weights are taken
// times 2^7 (of at most 2^8), so that fp16 keeps those down to 2^-21 of a row's largest.
template <typename T, int D, bool kPaged, bool kSplit, bool k8>
__global__ void __launch_bounds__(k8 ? kThreads8 : kThreads, 1)
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
    const uint32_t landed = k8 ? full + 3 : full;       // K and V: four converter warps instead of the producer, and the relay
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(smem_addr(&ctl->q_full[i]), k8 ? 1 : full);
      mbar_init(smem_addr(&ctl->q_ready[i]), landed);
      mbar_init(smem_addr(&ctl->q_scaled[i]), 4);
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
      mbar_init(smem_addr(&ctl->k_full[i]), landed);
      mbar_init(smem_addr(&ctl->k_empty[i]), 1);
      mbar_init(smem_addr(&ctl->v_full[i]), landed);
      mbar_init(smem_addr(&ctl->v_empty[i]), 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(smem_addr(&ctl->unit_full[i]), 1);
      mbar_init(smem_addr(&ctl->unit_empty[i]), k8 ? kUnitReaders8 : kUnitReaders);
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

  if (k8 && warp >= 12) {
    // -------------------------------------------------------------------- converters of 8-bit keys and values
    regs_decrease<kRegsConvert>();
    constexpr int kKLanes = D / 16, kKStep = 32 / kKLanes, kKLoads = 16 / kKStep;        // K: 16 keys a warp
    constexpr int kVLanes = D / 32, kVStep = 32 / kVLanes, kVLoads = 32 / kVStep;        // V: 32 keys, this CTA's channels
    const int cw = warp - 12;
    // Converters arrive in their own CTA, each lane's writes fenced against the async proxy.  The products that rank 0 issues
    // read rank 1's shared memory too, so rank 1's relay passes its arrivals on with a release of cluster scope.  (From
    // here that would wait for every load in flight: 7.5 ms, not 6.2, for a 720p frame when this was the one change.)
    const int kc = lane % kKLanes, kr = lane / kKLanes, vc = lane % kVLanes, vr = lane / kVLanes;
    // Where this lane's codes of row r wait in a stage (in 128-byte rows of 64 channels: the upper part's row, where there
    // is one, else half of the row): within what the row's own lanes will write.
    auto raw_k = [&](int r) { return D == 128 ? Lo::kKPart + r * 128 + kc * 16 : r * 128 + (r & 1) * 64 + kc * 16; };
    auto raw_v = [&](int r) { return r * Lo::kVRow + (r & 1) * (Lo::kVRow / 2) + vc * 16; };
    int kv = 0, n = 0;                                  // tiles, units with tiles
    bool ok = true;
    UnitReader in{sCtl};
    while (ok) {
      if (!(ok = in.wait())) break;
      if (VDX_UNIT(in, s) < 0) {
        in.release();
        break;
      }
      const int t0 = VDX_UNIT(in, t0), t1 = VDX_UNIT(in, t1), s = VDX_UNIT(in, s), hk = VDX_UNIT(in, hk), len = VDX_UNIT(in, len);
      const bool two = VDX_UNIT(in, ntok) > 2 * per_tile;
      in.release();
      if (t0 >= t1) continue;
      const int* table = p.table + static_cast<long long>(s) * p.table_stride;
      const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + hk * p.k_h + kc * 16;
      const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + hk * p.v_h + static_cast<int>(rank) * (D / 2) + vc * 16;
      const uint8_t* kscale = p.scales.k + hk * p.scales.k_head;
      const uint8_t* vscale = p.scales.v + hk * p.scales.v_head;
      TileCursor<kPaged> c;                             // of the tile whose pages are looked up next
      c.seek(p, geom, t0);
      int ek, ev, ek_next = 0, ev_next = 0;             // scale bytes of this lane's key and value
      int k_page, k_slot, v_page, v_slot;               // of the tile to be copied next
      // The row of the tile at c that this lane looks up: its page and slot (negative: a key that is not there).
      auto look_up = [&](int row, int& page, int& slot) {
        slot = c.off + row;
        int e = c.page;
        while (slot >= p.P) {
          slot -= p.P;
          ++e;
        }
        page = 0;
        if (c.key0 + row < len)
          page = load_i32(table + e);
        else
          slot = -1;
      };
      auto look_up_key = [&] { look_up(static_cast<int>(rank) * (kBN / 2) + cw * 16 + (lane & 15), k_page, k_slot); };
      auto look_up_value = [&] {
        look_up(cw * 32 + lane, v_page, v_slot);
        c.next(p);
      };
      auto place = [&](int page, int slot, long long per_page, long long per_slot) {
        if (slot < 0) return -1ll;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) return page * per_page + slot * per_slot;
        atomicOr(&g_error_word, kErrPage);
        return -1ll;
      };
      // Codes of tile number n to the rows of its stage that they will fill, once that is free: 16 bytes a lane, which
      // the same lane reads again.
      auto copy_keys = [&](int n) {
        if (n >= kS && !(ok = wait(sCtl + kBarKEmpty + 8 * (n % kS), n / kS - 1, kSiteKEmpty))) return;
        const long long at = place(k_page, k_slot, p.k_p, p.k_t);
        ek_next = at < 0 ? 127 : kscale[k_page * p.scales.k_page + k_slot / kBlock8 * p.scales.k_block];
#pragma unroll
        for (int i = 0; i < kKLoads; ++i) {
          const long long from = __shfl_sync(0xffffffffu, at, i * kKStep + kr);
          copy_code16(sK + n % kS * Lo::kStageBytes + raw_k(cw * 16 + i * kKStep + kr), kbase + max(from, 0ll), from >= 0);
        }
      };
      auto copy_values = [&](int n) {
        if (n >= kS && !(ok = wait(sCtl + kBarVEmpty + 8 * (n % kS), n / kS - 1, kSiteVEmpty))) return;
        const long long at = place(v_page, v_slot, p.v_p, p.v_t);
        ev_next = at < 0 ? 127 : vscale[v_page * p.scales.v_page + v_slot / kBlock8 * p.scales.v_block];
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
          const long long from = __shfl_sync(0xffffffffu, at, i * kVStep + vr);
          copy_code16(sV + n % kS * Lo::kStageBytes + raw_v(cw * 32 + i * kVStep + vr), vbase + max(from, 0ll), from >= 0);
        }
      };
      look_up_key();
      look_up_value();
      copy_keys(kv);
      copies_commit();
      if (!ok) break;
      copy_values(kv);
      copies_commit();
      if (!ok) break;
      if (t0 + 1 < t1) {
        look_up_key();
        look_up_value();
      }
      // This unit's Q tiles to fp16, a row to a lane.  (An unused second one's buffer is already the next but one unit's.)
      for (int i = 0; ok && i < 2; ++i) {
        const int b = 2 * (n & 1) + i;
        if (!(ok = wait(sCtl + kBarQFull + 8 * b, n >> 1, kSiteQFull))) break;
        if (std::is_same<T, __nv_bfloat16>::value && (i == 0 || two)) {
          ctl->q_exp[b][cw * 32 + lane] = static_cast<int8_t>(query_row_to_half<D, Lo::kQPart>(sQ + b * Lo::kQBytes, cw * 32 + lane));
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sCtl + kBarQScaled + 8 * b);
          mbar_arrive(sCtl + kBarQReady + 8 * b);
        }
      }
      if (!ok) break;
      ++n;
      // Codes are copied a tile ahead: any further, and the stage they need would be that of a tile whose products wait
      // for what is written here.
      for (int t = t0; t < t1; ++t) {
        const int st = kv % kS;
        ek = ek_next;
        ev = ev_next;
        if (t + 1 < t1) copy_keys(kv + 1);
        copies_commit();
        if (!ok) break;
        if (t + 2 < t1) look_up_key();
        copies_wait<2>();                               // two parts are younger than this tile's keys
        uint4 x[kKLoads > kVLoads ? kKLoads : kVLoads];
        const uint32_t kt = sK + st * Lo::kStageBytes, vt = sV + st * Lo::kStageBytes;
#pragma unroll
        for (int i = 0; i < kKLoads; ++i) x[i] = ld_shared_v4(kt + raw_k(cw * 16 + i * kKStep + kr));
        __syncwarp();                                   // a row's codes are read before it is written
        const uint32_t sk = half_two_to(scale_exponent(static_cast<uint8_t>(ek))) * 0x10001u;
#pragma unroll
        for (int i = 0; i < kKLoads; ++i)
          expand_chunk<128>(kt + kc / 4 * Lo::kKPart, cw * 16 + i * kKStep + kr, kc % 4, x[i], __shfl_sync(0xffffffffu, sk, i * kKStep + kr));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sCtl + kBarKFull + 8 * st);
        if (t + 1 < t1) copy_values(kv + 1);
        copies_commit();
        if (!ok) break;
        if (t + 2 < t1) look_up_value();
        copies_wait<2>();
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) x[i] = ld_shared_v4(vt + raw_v(cw * 32 + i * kVStep + vr));
        __syncwarp();
        const uint32_t sv = half_two_to(scale_exponent(static_cast<uint8_t>(ev))) * 0x10001u;
#pragma unroll
        for (int i = 0; i < kVLoads; ++i)
          expand_chunk<Lo::kVRow>(vt, cw * 32 + i * kVStep + vr, vc, x[i], __shfl_sync(0xffffffffu, sv, i * kVStep + vr));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sCtl + kBarVFull + 8 * st);
        ++kv;
      }
      if (!ok) break;
    }
    copies_wait<0>();
    __syncwarp();
  } else if (warp >= 8) {
    regs_decrease<k8 ? kRegsCtl8 : kRegsCtl>();
    if (k8 && warp == 8) {
      // the converters do its work
    } else if (warp == 8) {
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
      constexpr uint32_t kType = !k8 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
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
      // K, V and (8 bits) Q: rank 1's converters wrote their halves by plain stores, so the wait acquires at cluster scope
      auto wait_tile = [&](uint32_t bar, int parity, int site) { return warp_wait<k8>(bar, parity & 1, sCtl + kOffAbort, site); };
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
        const uint32_t q_full = sCtl + (k8 ? kBarQReady : kBarQFull) + 8 * (2 * (n & 1));
        if (!(ok = wait_tile(q_full, qph, kSiteQFull) && wait_tile(sCtl + kBarKFull + 8 * st, ph, kSiteKFull))) break;
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
              if (!(ok = wait_tile(q_full + 8, qph, kSiteQFull))) break;
              tc_fence_after_sync();
            }
            issue_qk<D>(tmem + 128, q0 + Lo::kQBytes, kt, kIdQK);
            mma_commit_pair_warp(sCtl + kBarSFull + 8);
            mma_commit_pair_warp(sCtl + kBarKEmpty + 8 * st);
          }
          ok = wait_tile(sCtl + kBarVFull + 8 * st, ph, kSiteVFull);
          if (!k8 && end && tail < kBN) {
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
          if (!end && ok) ok = wait_tile(sCtl + kBarKFull + 8 * st, ph, kSiteKFull);
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
        constexpr uint32_t kBarQ = k8 ? kBarQReady : kBarQFull;
        auto pass_on = [&](uint32_t bar) {                  // copies have landed; what warps wrote must be seen as well
          if (lane != 0) return;
          if (k8)
            mbar_arrive_remote_cluster(mapa_shared(bar, 0));
          else
            mbar_arrive_remote(mapa_shared(bar, 0));
        };
        for (int i = 0; ok && i < 2; ++i) {
          const uint32_t bar = sCtl + kBarQ + 8 * (2 * (n & 1) + i);
          ok = wait(bar, n >> 1, kSiteRelay);
          if (ok) pass_on(bar);
        }
        for (; ok && left > 0; --left) {
          if (!(ok = wait(sCtl + kBarKFull + 8 * st, ph, kSiteRelay))) break;
          pass_on(sCtl + kBarKFull + 8 * st);
          if (!(ok = wait(sCtl + kBarVFull + 8 * st, ph, kSiteRelay))) break;
          if (!k8 && left == 1 && tail < kBN) {
            zero_v_rows<D>(sV + st * Lo::kStageBytes, tail, lane);
            if (lane == 0) mbar_arrive_remote_cluster(mapa_shared(sCtl + kBarVFull + 8 * st, 0));
          } else {
            pass_on(sCtl + kBarVFull + 8 * st);
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
    regs_increase<k8 ? kRegsSoftmax8 : kRegsSoftmax>();
    const int qi = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_bits + 128 * qi;
    const uint32_t tO = tmem + lane_bits + 256 + 128 * qi;
    const int my_tok = row / p.g, my_head = row - my_tok * p.g;
    const bool in_tile = my_tok < per_tile;
    const int tok = (2 * qi + static_cast<int>(rank)) * per_tile + my_tok;   // within a block
    const uint32_t remote = mapa_shared(sCtl, 0);
    using M = std::conditional_t<k8, __half, T>;     // what the products take
    constexpr float kLift = k8 ? 7.f : 0.f;          // log2 of what weights are multiplied by
    float c = p.scale_log2;
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
      if (k8 && std::is_same<T, __nv_bfloat16>::value && t < t1) {
        // the power of two that this row of Q was multiplied by
        const int b = 2 * (~nq & 1) + qi;
        if (!(ok = warp_wait_inline(sCtl + kBarQScaled + 8 * b, ((nq - 1) >> 1) & 1, sCtl + kOffAbort, kSiteQFull))) break;
        c = p.scale_log2 * two_to(-static_cast<int>(ctl->q_exp[b][row]));
      }
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
            uint32_t s[k8 ? 1 : 128];
            if constexpr (!k8) tmem_ld128(tS, s);
            if (look) {
              float mt;
              if constexpr (k8)
                mt = row_max_halves(tS) * c;
              else
                mt = row_max128(s) * c;
              if (mt > m) {
                alpha = ex2_approx(m - mt);
                l *= alpha;
                m = mt;
              }
            }
            // a row without keys so far: its scores are -inf and weigh nothing
            const float base = look && !(m > -INFINITY) ? 0.f : m - kLift;
            if constexpr (k8)
              lt = exp_row_halves<M>(tS, c, base, pk);
            else
              lt = exp_row128<M>(s, c, base, pk);
            if (look || !__any_sync(0xffffffffu, live && !(lt <= (k8 ? 32768.f : 256.f)))) break;
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
          p.part_ml[prow] = make_float2(empty ? -INFINITY : m - kLift, l);
        else if (p.lse)
          p.lse[lse_index(p, u.s, sq, h, u.tok0 + tok)] = empty ? -INFINITY : (m - kLift + __log2f(l)) * 0.69314718055994530942f;
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

template <typename T, int D>
cudaError_t launch(const KvParams& p, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  CUtensorMap mq, mk{}, mv{}, mkb{}, mvb{}, mo;        // no boxes, 8 bits: their maps are never used
  const bool one_q = p.cu != nullptr || p.q_b == 0;
  const bool has_keys = p.P > 0;
  // dimensions: q and out (d, head, token, batch), k and v (d, token, head, page)
  const long long kpages = !p.table && p.k_p == 0 ? 1 : p.num_pages, vpages = !p.table && p.v_p == 0 ? 1 : p.num_pages;
  const void* k = has_keys ? p.k : p.q;                  // no keys: the maps are never used
  const void* v = has_keys ? p.v : p.q;
  const int P = has_keys ? p.P : 1;
  const long long ob = static_cast<long long>(p.N) * p.Hq * D;
  if (!encode_rows<T>(encode, &mq, p.q, D, p.Hq, p.q_h, p.N, p.q_t, one_q ? 1 : p.S, p.q_b, 64, p.g, kBM / p.g) ||
      (!p.eight && (!encode_rows<T>(encode, &mk, k, D, P, p.k_t, p.Hkv, p.k_h, kpages, p.k_p, 64, kBN / 2, 1) ||
                    !encode_rows<T>(encode, &mv, v, D, P, p.v_t, p.Hkv, p.v_h, vpages, p.v_p, D / 2, kBN, 1))) ||
      (!p.eight && p.box_rows && (!encode_rows<T>(encode, &mkb, k, D, P, p.k_t, p.Hkv, p.k_h, kpages, p.k_p, 64, p.box_rows, 1) ||
                      !encode_rows<T>(encode, &mvb, v, D, P, p.v_t, p.Hkv, p.v_h, vpages, p.v_p, D / 2, p.box_rows, 1))) ||
      !encode_rows<T>(encode, &mo, p.out, D, p.Hq, D, p.N, static_cast<long long>(p.Hq) * D, p.cu ? 1 : p.S, ob, 64, p.g,
                      kBM / p.g)) {
    *what = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  const int smem = Layout<D>::kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
  static std::atomic<uint64_t> done[6] = {};
  auto* kernel = p.eight   ? (p.nsplit > 1 ? attn_tiles<T, D, true, true, true> : attn_tiles<T, D, true, false, true>)
                 : p.table ? (p.nsplit > 1 ? attn_tiles<T, D, true, true, false> : attn_tiles<T, D, true, false, false>)
                           : (p.nsplit > 1 ? attn_tiles<T, D, false, true, false> : attn_tiles<T, D, false, false, false>);
  const cudaError_t e = allow_shared(kernel, smem, &done[(p.eight ? 4 : p.table ? 2 : 0) + (p.nsplit > 1 ? 1 : 0)]);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit;
  if (units > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * units));
  cfg.blockDim = dim3(p.eight ? kThreads8 : kThreads);
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
