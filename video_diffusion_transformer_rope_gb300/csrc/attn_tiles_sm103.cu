// Attention of many query rows over a paged cache or over dense keys of another length (cross
// attention), on the 5th-generation tensor cores.
//
//     S = Q K^T,  p = 2^(S * scale*log2(e) - m),  l = sum p,  O = sum p v  (online over key tiles)
//
// Bound: the tensor cores and the exponentials together (at d = 128 a 128 x 128 tile costs 1024
// tensor cycles for its two products and as many exponentials per multiprocessor), with Q and the
// output through DRAM when the keys are few (cross attention over 512 keys: 512 flops a byte).
//
// A unit of work is (sequence, kv head, block of 2 x 128 query rows, range of 128-key tiles); the
// rows of a block are (token, query head of the group) pairs, so grouped heads share every key
// they read.  One persistent CTA per multiprocessor walks units blockIdx.x, + gridDim.x, ...; its
// roles run ahead of one another across units, so one unit's loads and epilogue hide behind the
// next one's products (with 4 key tiles to a unit they are as long as the products).
//
//   warps 0-3, 4-7   softmax and epilogue of the block's first / second 128 rows (thread = row =
//                    TMEM lane)
//   warp 8           TMA producer: Q tiles, then K and V tiles through rings; a tile is one box of
//                    a page of >= 128 tokens, or 128 / page_size boxes, each lane issuing one page
//   warp 9           issues the tcgen05 MMAs (one elected lane) and owns TMEM
//
// TMEM (512 columns): S0, S1 at 0 and 128, O0, O1 at 256 and 384; P overwrites the first half of S
// as packed 16-bit pairs and is the A operand of the second product.  Issue order per key tile j:
//     S0(j) ; O1 += P1(j-1) V(j-1) ; S1(j) ; O0 += P0(j) V(j)
// and O1's last product of a unit follows S0 of the next unit's first tile, so the tensor cores do
// not drain between units.  Exponentials are taken against the running maximum and kept while
// the row sum shows every p <= 256; the first tile of a unit, or a row whose scores rose, takes
// the tile's maximum first.
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
constexpr int kMaxStages = 6;
constexpr uint32_t kRegsSoftmax = 208, kRegsCtl = 88;      // 2 x 208 + 88 = 3 x 168 at launch
static_assert(2 * kRegsSoftmax + kRegsCtl <= 3 * 168, "register split over budget");

template <int D>
struct Layout {
  static constexpr int kTileBytes = kBN * D * 2;
  static constexpr int kHalfBytes = kBN * 128;            // 128 rows of 64 channels
  static constexpr int kHalves = D / 64;
  static constexpr int kKStages = D == 128 ? 3 : 5;
  static constexpr int kVStages = D == 128 ? 2 : 5;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kTileBytes;
  static constexpr int kOffCtl = kOffV + kVStages * kTileBytes;
};

enum : int {
  kSiteQFull = 32, kSiteQEmpty, kSiteKFull, kSiteKEmpty, kSiteVFull, kSiteVEmpty, kSiteSFull, kSitePReady,
  kSiteOFull, kSiteOEmpty, kSiteDrain
};

struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[2], p_ready[2];
  uint64_t o_full[2], o_empty[2];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};

// Bounded wait on the way out, whatever the abort flag says: copies and MMAs in flight finish
// before shared or tensor memory is released.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicCAS(&g_error_word, 0u, 1u | (static_cast<unsigned>(kSiteDrain) << 8));
      return;
    }
  }
}

// Plan values that every role derives from KvParams.
struct TileGeom {
  bool small_pages;        // several pages per tile
  int pages_per_tile;      // of small pages
  int tiles_per_page;      // of large ones
  __device__ __forceinline__ explicit TileGeom(const KvParams& p) {
    small_pages = p.table != nullptr && p.P < kBN;
    pages_per_tile = small_pages ? kBN / p.P : 1;
    tiles_per_page = (p.P + kBN - 1) / kBN;
  }
  __device__ __forceinline__ int tiles(const KvParams& p, int len) const {
    if (len <= 0) return 0;
    if (small_pages) return (len + kBN - 1) / kBN;
    const int full = len / p.P;
    return full * tiles_per_page + (len - full * p.P + kBN - 1) / kBN;
  }
};

// Key tile of a page of >= 128 tokens: tiles do not cross a page's end.  Small pages: tile t covers
// keys 128 t and up.
struct TileCursor {
  int page, sub;           // entry of the page table, tile within the page
  int key0, keys;          // first key, keys it can hold
  __device__ __forceinline__ void seek(const KvParams& p, const TileGeom& g, int t) {
    if (g.small_pages) {
      page = t * g.pages_per_tile;
      sub = 0;
      key0 = t * kBN;
      keys = kBN;
    } else {
      page = t / g.tiles_per_page;
      sub = t - page * g.tiles_per_page;
      key0 = page * p.P + sub * kBN;
      keys = min(kBN, p.P - sub * kBN);
    }
  }
  __device__ __forceinline__ void next(const KvParams& p, const TileGeom& g) {
    if (g.small_pages) {
      page += g.pages_per_tile;
      key0 += kBN;
    } else {
      key0 += keys;
      if (++sub == g.tiles_per_page) {
        sub = 0;
        ++page;
      }
      keys = min(kBN, p.P - sub * kBN);
    }
  }
};

// One unit of work, the same for every role.
struct Unit {
  int s, hk, blk, z;
  SeqInfo sq;
  int tok0, ntok;          // first token of the block and live tokens in it (0: none)
  int len;                 // keys that its last row sees
  int t0, t1;              // key tiles of this split
  __device__ __forceinline__ Unit(const KvParams& p, const TileGeom& g, int it, bool report) {
    blk = it % p.nblk;
    int r = it / p.nblk;
    z = r % p.nsplit;
    r /= p.nsplit;
    hk = r % p.Hkv;
    s = r / p.Hkv;
    sq = sequence_info(p, s, report);
    const int per = p.block_rows / p.g;
    tok0 = blk * per;                                    // nblk * per stays near max_q < 2^31
    ntok = min(per, min(sq.n, p.max_q) - tok0);
    len = ntok > 0 ? visible_limit(p, sq, tok0 + ntok - 1) : 0;
    const int nt = g.tiles(p, len);
    const long long a = static_cast<long long>(z) * p.split_keys;
    t0 = static_cast<int>(min(a, static_cast<long long>(nt)));
    t1 = static_cast<int>(min(a + p.split_keys, static_cast<long long>(nt)));
  }
};

// S(tmem) = A(128 x D, K-major) * B(128 x D, K-major)^T; operands in 64-channel halves of 128-byte
// swizzled rows.  The whole MMA warp calls, one elected lane issues.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * Layout<D>::kHalfBytes + (kk & 3) * 32;
    mma_ss_warp(d_tmem, smem_desc_sw128(a_smem + off, 16, 1024), smem_desc_sw128(b_smem + off, 16, 1024), idesc,
                kk > 0 ? 1u : 0u);
  }
}
// O(tmem) (+)= P(tmem, 128 x 128) * V(128 keys x D, channel-contiguous = MN-major).
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t idesc, bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk)
    mma_ts_warp(d_tmem, p_tmem + kk * 8, smem_desc_sw128(v_smem + kk * 2048, Layout<D>::kHalfBytes, 1024), idesc,
                (accumulate || kk > 0) ? 1u : 0u);
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

__device__ __forceinline__ void mask_row(uint32_t (&s)[128], int valid) {
#pragma unroll
  for (int e = 0; e < 128; ++e)
    if (e >= valid) s[e] = 0xff800000u;
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tiles(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ KvParams p, const int units) {
  using Lo = Layout<D>;
  constexpr int kKS = Lo::kKStages, kVS = Lo::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Lo::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = smem_addr(smem + Lo::kOffQ), sK = smem_addr(smem + Lo::kOffK), sV = smem_addr(smem + Lo::kOffV);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ctl->q_full[i]), 1);
      mbar_init(smem_addr(&ctl->q_empty[i]), 1);
      mbar_init(smem_addr(&ctl->s_full[i]), 1);
      mbar_init(smem_addr(&ctl->p_ready[i]), 128);
      mbar_init(smem_addr(&ctl->o_full[i]), 1);
      mbar_init(smem_addr(&ctl->o_empty[i]), 128);
    }
    for (int i = 0; i < kKS; ++i) {
      mbar_init(smem_addr(&ctl->k_full[i]), 1);
      mbar_init(smem_addr(&ctl->k_empty[i]), 1);
    }
    for (int i = 0; i < kVS; ++i) {
      mbar_init(smem_addr(&ctl->v_full[i]), 1);
      mbar_init(smem_addr(&ctl->v_empty[i]), 1);
    }
    mbar_init(smem_addr(&ctl->done), 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_addr(&ctl->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  volatile int* abort_flag = &ctl->abort_flag;
  const TileGeom geom(p);

  if (warp >= 8) {
    regs_decrease<kRegsCtl>();
    if (warp == 8) {
      // ------------------------------------------------------------------ TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      const int per_tile = kBM / p.g;                   // tokens of one Q tile
      const uint32_t q_bytes = static_cast<uint32_t>(per_tile * p.g) * D * 2;
      int kc = 0, vc = 0, n = 0;                        // K tiles, V tiles, units so far
      bool ok = true;
      for (int it = blockIdx.x; ok && it < units; it += gridDim.x) {
        const Unit u(p, geom, it, false);
        if (u.t0 >= u.t1) continue;
        const int* table = p.table ? p.table + static_cast<long long>(u.s) * p.table_stride : nullptr;
        TileCursor c;
        c.seek(p, geom, u.t0);
        for (int t = u.t0; ok && t < u.t1; ++t, c.next(p, geom)) {
          // this lane's page of the tile (small pages: one per lane)
          const int boxes = geom.small_pages ? (min(kBN, u.len - c.key0) + p.P - 1) / p.P : 1;
          int page = 0;
          if (lane < boxes) {
            if (table) {
              page = __ldg(table + c.page + lane);
              if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
                atomicOr(&g_error_word, kErrPage);
                page = -1;                              // out of the map's range: filled with zeros
              }
            } else {
              page = u.s;
            }
          }
          const int kpage = p.k_p == 0 && !table ? 0 : page, vpage = p.v_p == 0 && !table ? 0 : page;
          const uint32_t bytes = geom.small_pages ? static_cast<uint32_t>(boxes * p.P) * D * 2 : Lo::kTileBytes;
          const uint32_t box_off = static_cast<uint32_t>(lane * p.P) * 128;      // lane 0: 0
          const int tok = c.sub * kBN;
          {
            const int st = kc % kKS;
            if (kc >= kKS)
              ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->k_empty[st]), (kc / kKS - 1) & 1, abort_flag, kSiteKEmpty));
            if (!ok) break;
            const uint32_t bar = smem_addr(&ctl->k_full[st]);
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (lane < boxes)
#pragma unroll
              for (int h = 0; h < Lo::kHalves; ++h)
                tma_load_4d(sK + st * Lo::kTileBytes + h * Lo::kHalfBytes + box_off, &tm_k, bar, h * 64, tok, u.hk, kpage);
            ++kc;
          }
          if (t == u.t0) {
            for (int i = 0; ok && i < 2; ++i) {
              if (n > 0)
                ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->q_empty[i]), (n - 1) & 1, abort_flag, kSiteQEmpty));
              if (!ok) break;
              const uint32_t bar = smem_addr(&ctl->q_full[i]);
              if (lane == 0) {
                mbar_arrive_expect_tx(bar, q_bytes);
#pragma unroll
                for (int h = 0; h < Lo::kHalves; ++h)
                  tma_load_4d(sQ + i * Lo::kTileBytes + h * Lo::kHalfBytes, &tm_q, bar, h * 64, u.hk * p.g,
                              u.sq.row0 + u.tok0 + i * per_tile, p.cu || p.q_b == 0 ? 0 : u.s);
              }
              __syncwarp();
            }
            if (!ok) break;
            ++n;
          }
          {
            const int st = vc % kVS;
            if (vc >= kVS)
              ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->v_empty[st]), (vc / kVS - 1) & 1, abort_flag, kSiteVEmpty));
            if (!ok) break;
            const uint32_t bar = smem_addr(&ctl->v_full[st]);
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (lane < boxes)
#pragma unroll
              for (int h = 0; h < Lo::kHalves; ++h)
                tma_load_4d(sV + st * Lo::kTileBytes + h * Lo::kHalfBytes + box_off, &tm_v, bar, h * 64, tok, u.hk, vpage);
            ++vc;
          }
        }
      }
      // every copy lands before the CTA can retire (after an abort one of the two Q copies of the
      // last unit may not have been issued: its barrier then still shows the phase before)
      if (lane == 0) {
        for (int s = 0; s < kKS; ++s)
          if (kc > s) drain_wait(smem_addr(&ctl->k_full[s]), ((kc - 1 - s) / kKS) & 1);
        for (int s = 0; s < kVS; ++s)
          if (vc > s) drain_wait(smem_addr(&ctl->v_full[s]), ((vc - 1 - s) / kVS) & 1);
        for (int i = 0; i < 2; ++i)
          if (n > 0) drain_wait(smem_addr(&ctl->q_full[i]), (n - 1) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA issuer
      constexpr uint32_t kType = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t kIdQK = idesc_f16kind_f32acc(kBM, kBN, kType, 0);
      constexpr uint32_t kIdPV = idesc_f16kind_f32acc(kBM, D, kType, 1);
      const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 384};
      int g = 0, n = 0;                                  // key tiles and units so far
      bool ok = true;
      // the second Q tile's product with V that is still to be issued
      bool have = false, first = false, last = false;
      int pend_n = 0;
      auto wait = [&](uint64_t* bar, int parity, int site) {
        return __all_sync(0xffffffffu, mbar_wait(smem_addr(bar), parity & 1, abort_flag, site));
      };
      auto finish_second = [&]() {                        // O1 += P1(g-1) V(g-1)
        ok = wait(&ctl->p_ready[1], g - 1, kSitePReady);
        if (ok && first && pend_n > 0) ok = wait(&ctl->o_empty[1], pend_n - 1, kSiteOEmpty);
        if (!ok) return;
        tc_fence_after_sync();
        const int vs = (g - 1) % kVS;
        issue_pv<D>(tO[1], tS[1], sV + vs * Lo::kTileBytes, kIdPV, !first);
        mma_commit_warp(smem_addr(&ctl->v_empty[vs]));
        if (last) mma_commit_warp(smem_addr(&ctl->o_full[1]));
        have = false;
      };
      for (int it = blockIdx.x; ok && it < units; it += gridDim.x) {
        const Unit u(p, geom, it, false);
        if (u.t0 >= u.t1) continue;
        TileCursor c;
        c.seek(p, geom, u.t0);
        for (int t = u.t0; t < u.t1; ++t, c.next(p, geom)) {
          const int ks = g % kKS, vs = g % kVS;
          const uint32_t kt = sK + ks * Lo::kTileBytes, vt = sV + vs * Lo::kTileBytes;
          if (t == u.t0 && !(ok = wait(&ctl->q_full[0], n, kSiteQFull))) break;
          if (!(ok = wait(&ctl->k_full[ks], g / kKS, kSiteKFull))) break;
          tc_fence_after_sync();
          issue_qk<D>(tS[0], sQ, kt, kIdQK);
          mma_commit_warp(smem_addr(&ctl->s_full[0]));
          if (t == u.t1 - 1) mma_commit_warp(smem_addr(&ctl->q_empty[0]));
          if (have) {
            finish_second();
            if (!ok) break;
          }
          if (t == u.t0) {
            if (!(ok = wait(&ctl->q_full[1], n, kSiteQFull))) break;
            tc_fence_after_sync();
          }
          issue_qk<D>(tS[1], sQ + Lo::kTileBytes, kt, kIdQK);
          mma_commit_warp(smem_addr(&ctl->s_full[1]));
          mma_commit_warp(smem_addr(&ctl->k_empty[ks]));
          if (t == u.t1 - 1) mma_commit_warp(smem_addr(&ctl->q_empty[1]));
          if (!(ok = wait(&ctl->v_full[vs], g / kVS, kSiteVFull))) break;
          if (c.key0 + c.keys > u.len) {
            // rows of V past the last visible key become zeros
            const int from = u.len - c.key0;
            for (int i = from * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
              for (int h = 0; h < Lo::kHalves; ++h) st_shared_v4(vt + h * Lo::kHalfBytes + i * 16, make_uint4(0u, 0u, 0u, 0u));
            fence_proxy_async_smem();
            __syncwarp();
          }
          ok = wait(&ctl->p_ready[0], g, kSitePReady);
          if (ok && t == u.t0 && n > 0) ok = wait(&ctl->o_empty[0], n - 1, kSiteOEmpty);
          if (!ok) break;
          tc_fence_after_sync();
          issue_pv<D>(tO[0], tS[0], vt, kIdPV, t > u.t0);
          if (t == u.t1 - 1) mma_commit_warp(smem_addr(&ctl->o_full[0]));
          have = true;
          first = t == u.t0;
          last = t == u.t1 - 1;
          pend_n = n;
          ++g;
        }
        ++n;
      }
      if (ok && have) finish_second();
      mma_commit_warp(smem_addr(&ctl->done));
      drain_wait(smem_addr(&ctl->done), 0);
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
    const int per_tile = kBM / p.g;
    const int my_tok = row / p.g, my_head = row - my_tok * p.g;
    const bool in_tile = my_tok < per_tile;
    const float c = p.scale_log2;
    int g = 0, n = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < units; it += gridDim.x) {
      const Unit u(p, geom, it, tid == 0);
      const int tok = qi * per_tile + my_tok;            // within the block
      const bool live = in_tile && tok < u.ntok;
      const int limit = live ? visible_limit(p, u.sq, u.tok0 + tok) : 0;
      float m = -INFINITY, l = 0.f;
      const bool any_live = __any_sync(0xffffffffu, live);
      TileCursor cur;
      if (u.t0 < u.t1) cur.seek(p, geom, u.t0);
      for (int t = u.t0; t < u.t1; ++t, cur.next(p, geom)) {
        // a warp gives up as one: its lanes meet again in the votes and TMEM accesses below
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->s_full[qi]), g & 1, abort_flag, kSiteSFull)))) break;
        ++g;
        tc_fence_after_sync();
        if (any_live) {
          uint32_t s[128], pk[64];
          tmem_ld128(tS, s);
          const int valid = min(limit - cur.key0, cur.keys);
          const bool ragged = __any_sync(0xffffffffu, live && valid < kBN);
          if (ragged) mask_row(s, valid);
          bool redo = t == u.t0;
          float lt = 0.f;
          if (!redo) {
            lt = exp_row128<T>(s, c, m, pk);
            redo = __any_sync(0xffffffffu, live && !(lt <= 256.f));
            if (redo) {
              tmem_ld128(tS, s);
              if (ragged) mask_row(s, valid);
            }
          }
          float alpha = 1.f;
          if (redo) {
            const float mt = row_max128(s) * c;
            if (mt > m) {
              alpha = ex2_approx(m - mt);
              l *= alpha;
              m = mt;
            }
            // a row that has seen no key yet: its scores are -inf and weigh nothing
            lt = exp_row128<T>(s, c, m == -INFINITY ? 0.f : m, pk);
          }
          uint32_t (&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[0]);
          uint32_t (&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[32]);
          tmem_st32(tS, lo);
          tmem_st32(tS + 32, hi);
          l += lt;
          // S of this tile is complete, and with it every product issued before it: O holds the
          // sum up to the tile before and may be scaled
          if (t > u.t0 && redo && __any_sync(0xffffffffu, live && alpha != 1.f)) {
            uint32_t r[32];
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tmem_ld32(tO + ch * 32, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st32(tO + ch * 32, r);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&ctl->p_ready[qi]));
      }
      if (!ok) break;
      if (u.t0 < u.t1) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->o_full[qi]), n & 1, abort_flag, kSiteOFull)))) break;
        ++n;
        tc_fence_after_sync();
      }
      if (any_live) {
        const bool empty = !(m > -INFINITY) && !(l != l);  // saw no key (a NaN sum is an answer)
        const float inv = empty ? 0.f : 1.f / l;
        const int unit = (u.s * p.Hkv + u.hk) * p.nblk + u.blk;
        const long long slot = (static_cast<long long>(unit) * p.nsplit + u.z) * p.block_rows + qi * per_tile * p.g + row;
        const int h = u.hk * p.g + my_head;
        const bool split = p.nsplit > 1;
        T* orow = live && !split ? static_cast<T*>(p.out) + (out_row(p, u.s, u.sq, u.tok0 + tok) * p.Hq + h) * D : nullptr;
        float* prow = live && split ? p.part_o + slot * D : nullptr;
        const bool al = ((split ? reinterpret_cast<uintptr_t>(p.part_o) : reinterpret_cast<uintptr_t>(p.out)) & 31) == 0;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t r[32];
          if (u.t0 < u.t1) {
            tmem_ld32(tO + ch * 32, r);
          }
          if (u.t0 >= u.t1 || empty) {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0u;
          }
          if (!live) continue;
          if (split) {
            if (empty) continue;                          // the join does not read it
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(prow + ch * 32 + e, r + e, al);
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = pack2<T>(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
            store32(orow + ch * 32, pk, al);
            store32(orow + ch * 32 + 16, pk + 8, al);
          }
        }
        if (live) {
          if (split)
            p.part_ml[slot] = make_float2(empty ? -INFINITY : m, l);
          else if (p.lse)
            p.lse[lse_index(p, u.s, u.sq, h, u.tok0 + tok)] =
                empty ? -INFINITY : (m + __log2f(l)) * 0.69314718055994530942f;
        }
      }
      if (u.t0 < u.t1) {
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&ctl->o_empty[qi]));
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// A [n3][n2][n1] grid of rows of D channels (element strides s1, s2, s3) as a map with 64-channel
// boxes of b1 x b2 rows.
template <typename T>
bool encode_rows(EncodeTiledFn encode, CUtensorMap* map, const void* base, int D, long long n1, long long s1, long long n2,
                 long long s2, long long n3, long long s3, int b1, int b2) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2),
                              static_cast<cuuint64_t>(n3)};
  auto bytes = [&](long long n, long long s) { return static_cast<cuuint64_t>(n > 1 ? s : D) * 2; };   // unused where n = 1
  const cuuint64_t strides[3] = {bytes(n1, s1), bytes(n2, s2), bytes(n3, s3)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const KvParams& p, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  CUtensorMap mq, mk, mv;
  const bool one_q = p.cu != nullptr || p.q_b == 0;
  const bool small = p.table != nullptr && p.P < kBN;
  const bool has_keys = p.P > 0;
  // dimensions: q (d, head, token, batch), k and v (d, token, head, page)
  const long long kpages = !p.table && p.k_p == 0 ? 1 : p.num_pages, vpages = !p.table && p.v_p == 0 ? 1 : p.num_pages;
  const void* k = has_keys ? p.k : p.q;                  // no keys: the maps are never used
  const void* v = has_keys ? p.v : p.q;
  const int P = has_keys ? p.P : 1;
  if (!encode_rows<T>(encode, &mq, p.q, D, p.Hq, p.q_h, p.N, p.q_t, one_q ? 1 : p.S, p.q_b, p.g, kBM / p.g) ||
      !encode_rows<T>(encode, &mk, k, D, P, p.k_t, p.Hkv, p.k_h, kpages, p.k_p, small ? p.P : kBN, 1) ||
      !encode_rows<T>(encode, &mv, v, D, P, p.v_t, p.Hkv, p.v_h, vpages, p.v_p, small ? p.P : kBN, 1)) {
    *what = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  const int smem = Layout<D>::kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(attn_tiles<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.S) * p.Hkv * p.nblk * p.nsplit;
  if (units > 0x7fffffffLL - sms) return cudaErrorInvalidConfiguration;
  attn_tiles<T, D><<<static_cast<unsigned>(units < sms ? units : sms), kThreads, smem, stream>>>(mq, mk, mv, p,
                                                                                                 static_cast<int>(units));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tiles(const KvParams& p, int d, int dtype, EncodeTiledFn encode, int sms, cudaStream_t stream,
                              const char** what) {
  *what = nullptr;
  if (dtype == 0)
    return d == 128 ? launch<__nv_bfloat16, 128>(p, encode, sms, stream, what)
                    : launch<__nv_bfloat16, 64>(p, encode, sms, stream, what);
  return d == 128 ? launch<__half, 128>(p, encode, sms, stream, what) : launch<__half, 64>(p, encode, sms, stream, what);
}

cudaError_t read_and_clear_error_word_tiles(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
