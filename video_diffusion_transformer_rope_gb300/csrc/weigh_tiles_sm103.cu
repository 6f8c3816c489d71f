// The weight that each cached key gathers (kv_weigh.cu has the formula) where a kv head has many rows, on the
// 5th-generation tensor cores.
//
//     S^T = K Q^T  (128 keys x 128 rows),   w[key] += sum over the tile's rows of 2^(S^T * scale*log2(e) - lse*log2(e))
//
// With the keys as the M side a key is a thread's TMEM lane and its sum stays in that thread's registers: no sum
// goes through memory, and the same call gives the same bits.  The keys are the A operand in tensor memory (64
// columns for 128 channels): only Q streams through shared memory, by TMA, each tile used for two key tiles.  Read as
// an operand of both and written once that is three quarters of shared memory's rate; with the keys there too it
// would be past it.  A warp copies the next unit's keys to shared memory meanwhile (any page size), from where the
// threads that own them put them into tensor memory, 8-bit codes as T, exactly.
//
// Bound: the tensor cores and the exponentials together (a 128 x 128 tile at d = 128 is 512 cycles of either).  1560
// tokens of 2 x 12 heads over 32760 keys, a causal block each: 287 us, 1090 TFLOP/s, the exponential units 46 % busy; what it
// waits for is the way from a product to its weighers and back over three S tiles.  While masked and whole tiles shared a loop
// it was 304 us; from there eight weighing warps of whole rows took 335 to 349 us, loads of 64 columns 376, the odd tiles'
// warps writing keys 312 to 318, a register split of 104 and 64 363, a unit's Q tiles over clusters of two 429.
//
// A unit is (sequence, kv head, 256 keys); a block per multiprocessor takes every gridDim-th of them.
//   warps 0-15       exponentials and sums (thread = key = TMEM lane): four warps to a key tile and every other Q tile,
//                    the pairs of them added at the end; the first eight also put the keys into tensor memory
//   warp 16          TMA producer of the Q ring; copies half of the keys of units of few Q tiles
//   warp 17          issues the products                 warp 18  -lse*log2(e) of a Q tile's rows
//   warp 19          copies keys
// TMEM (512 columns): the keys of both tiles at 0 and 64, three S tiles at 128, 256 and 384, used in turn; a tile is
// free as soon as its scores are in registers.
#include <cstdint>

#include "kv8.cuh"
#include "kv_common.cuh"
#include "kv_maps.h"
#include "sm103_wait.cuh"

namespace vdx {
namespace {

constexpr int kKeys = 128;             // of a tile; a unit has two
constexpr int kRowTile = 128;
constexpr int kThreads = 640;
constexpr int kSBufs = 3;
constexpr int kLseSlots = 4;
constexpr int kMaxStages = 8;

template <int D>
struct Layout {
  static constexpr int kStageBytes = kRowTile * D * 2;      // 64-channel parts of 128-byte swizzled rows
  static constexpr int kPart = kRowTile * 128;
  static constexpr int kParts = D / 64;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffKeys = kStages * kStageBytes;
  static constexpr int kOffCtl = kOffKeys + 2 * kKeys * D * 2;
};

enum : int {
  kSiteQFull = 64, kSiteQEmpty, kSiteKeys, kSiteSFull, kSiteSEmpty, kSiteLseFull, kSiteLseEmpty, kSiteLoaded, kSiteTaken, kSiteKeysFree,
  kSitePart
};

struct Ctl {
  uint64_t q_full[kMaxStages], q_empty[kMaxStages];
  uint64_t keys[2], keys_free[2];      // in tensor memory
  uint64_t loaded, taken;              // in shared memory
  uint64_t part_full[2], part_empty[2];
  // S tiles for each of the four groups of warps that weigh, by its own count: a group does not see every use of an S buffer,
  // and it may have as many tiles waiting as there are buffers.
  uint64_t s_full[4][kSBufs], s_empty[kSBufs];
  // Rows' lse for the warps of the even and of the odd Q tiles apart, by their own counts: in units of one Q tile the odd
  // ones wait for nothing, so of barriers that they shared they could miss more than one phase.
  uint64_t l_full[2][kLseSlots], l_empty[2][kLseSlots];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float nl[2][kLseSlots][kRowTile];
  float part[2][kKeys];
  int8_t exponent[2 * kKeys];
};

struct Unit {
  int it;                  // its number; `units`: none is left
  int s, hk, key0, keys;   // keys of its two tiles
  SeqInfo sq;
  int rows, t0, t1;        // rows of the kv head; Q tiles that some key of the unit is seen by
  __device__ __forceinline__ bool has(int tile) const { return keys > tile * kKeys; }
};

// The first row token of the sequence that sees key c (visible_limit the other way round).
__device__ __forceinline__ int first_token(const KvParams& p, const SeqInfo& q, int c) {
  if (p.causal_block <= 0) return 0;
  const int pos = static_cast<int>(c - (static_cast<unsigned>(c) + q.shift) % static_cast<unsigned>(p.causal_block));
  return max(max(pos, 0) - (q.len - q.n), 0);
}

// The next unit from number `it` on that has work.
__device__ __forceinline__ Unit next_unit(const KvParams& p, int it, int units, int blocks, int row_tile, bool report) {
  Unit u;
  for (; it < units; it += gridDim.x) {
    const int kb = it % blocks, r = it / blocks;
    u.hk = r % p.Hkv;
    u.s = r / p.Hkv;
    u.sq = sequence_info(p, u.s, report && kb == 0 && u.hk == 0);
    u.rows = min(u.sq.n, p.max_q) * p.g;
    u.key0 = kb * 2 * kKeys;
    u.keys = min(2 * kKeys, u.sq.len - u.key0);
    if (u.rows > 0 && u.keys > 0) {
      u.t1 = (u.rows + row_tile - 1) / row_tile;
      u.t0 = static_cast<int>(min(static_cast<long long>(first_token(p, u.sq, u.key0)) * p.g / row_tile, static_cast<long long>(u.t1)));
      break;
    }
  }
  u.it = min(it, units);
  return u;
}

// sum over 32 columns of 2^(s * c + nl), those below lo or from hi on left out where kMask.
template <bool kMask>
__device__ __forceinline__ void weigh32(const uint32_t (&s)[32], uint32_t nl, float c, int lo, int hi, uint64_t (&acc)[4]) {
  const uint64_t c2 = f32x2(c, c);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const uint4 l = ld_shared_v4(nl + e * 4);
    const uint64_t a = ffma2(f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, f32x2(__uint_as_float(l.x), __uint_as_float(l.y)));
    const uint64_t b = ffma2(f32x2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, f32x2(__uint_as_float(l.z), __uint_as_float(l.w)));
    float x[4];
    f32x2_split(a, x[0], x[1]);
    f32x2_split(b, x[2], x[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kMask && (e + i < lo || e + i >= hi)) x[i] = -INFINITY;
      x[i] = ex2_approx(x[i]);
    }
    acc[(e >> 1) & 3] = fadd2(acc[(e >> 1) & 3], f32x2(x[0], x[1]));
    acc[((e >> 1) + 1) & 3] = fadd2(acc[((e >> 1) + 1) & 3], f32x2(x[2], x[3]));
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <typename T, int D, bool k8>
__global__ void __launch_bounds__(kThreads, 1)
weigh_tiles(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ WeighParams wp, const int units, const int blocks) {
  using Lo = Layout<D>;
  constexpr int kS = Lo::kStages;
  const KvParams& p = wp.kv;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Lo::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sQ = smem_addr(smem), sK = smem_addr(smem + Lo::kOffKeys);
  const int row_tile = kRowTile / p.g * p.g;           // whole tokens
  constexpr int kElem = k8 ? 1 : 2, kLanes = D * kElem / 16;      // 16-byte chunks of a key
  // Where chunk ch of key r of the unit lies: eight keys' chunks of one number are in different banks.
  auto key_chunk = [&](int r, int ch) {
    return sK + r * (kLanes * 16) + (kLanes == 4 ? ch ^ ((r >> 1) & 3) : (ch & ~7) | ((ch ^ r) & 7)) * 16;
  };

  if (tid == 0) {
    for (int i = 0; i < kS; ++i) {
      mbar_init(smem_addr(&ctl->q_full[i]), 1);
      mbar_init(smem_addr(&ctl->q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ctl->keys[i]), kKeys);
      mbar_init(smem_addr(&ctl->keys_free[i]), 1);
      mbar_init(smem_addr(&ctl->part_full[i]), kKeys);
      mbar_init(smem_addr(&ctl->part_empty[i]), kKeys);
    }
    mbar_init(smem_addr(&ctl->loaded), 2);
    mbar_init(smem_addr(&ctl->taken), 8);
    for (int i = 0; i < 4 * kSBufs; ++i) mbar_init(smem_addr(&ctl->s_full[0][i]), 1);
    for (int i = 0; i < kSBufs; ++i) mbar_init(smem_addr(&ctl->s_empty[i]), 4);
    for (int i = 0; i < 2 * kLseSlots; ++i) {
      mbar_init(smem_addr(&ctl->l_full[0][i]), 1);
      mbar_init(smem_addr(&ctl->l_empty[0][i]), 8);
    }
    mbar_init(smem_addr(&ctl->done), 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  // rows of a stage behind the last whole token are never copied: they weigh nothing, so they must not be NaN
  for (int i = tid; i < kS * Lo::kParts * (kRowTile - row_tile) * 8; i += kThreads) {
    const int ch = i & 7, r = i >> 3, part = r / (kRowTile - row_tile);
    st_shared_v4(sQ + part * Lo::kPart + (row_tile + r - part * (kRowTile - row_tile)) * 128 + ch * 16, make_uint4(0u, 0u, 0u, 0u));
  }
  fence_proxy_async_smem();
  if (warp == 17) {
    tmem_alloc(smem_addr(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  wait_for_earlier_work();
  const uint32_t tmem = ctl->tmem_base;
  const uint32_t flag = smem_addr(&ctl->abort_flag);
  auto wait = [&](const uint64_t* bar, int phase, int site) { return warp_wait(smem_addr(bar), phase & 1, flag, site); };
  auto first = [&](int it, bool report = false) { return next_unit(p, it, units, blocks, row_tile, report); };
  const int stride = gridDim.x;

  // Keys `from` .. of every `step`, 32 each, of a unit to shared memory, by one warp.
  auto copy_keys = [&](const Unit& u, int from, int step) {
    const int* table = p.table + u.s * p.table_stride;
    const uint8_t* base = static_cast<const uint8_t*>(p.k) + u.hk * p.k_h * kElem;
#pragma unroll 1
    for (int r0 = from; r0 < u.keys; r0 += step) {
      // a lane looks up a key; kLanes lanes copy its row
      const int c = u.key0 + r0 + lane, pg = c / p.P, slot = c - pg * p.P;
      long long at = -1;                               // zeros
      int e = 0;
      if (c < u.sq.len) {
        const int page = load_i32(table + pg);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
          at = (page * p.k_p + slot * p.k_t) * kElem;
          if (k8) e = scale_exponent(p.scales.k[page * p.scales.k_page + slot / kBlock8 * p.scales.k_block + u.hk * p.scales.k_head]);
        } else {
          atomicOr(&g_error_word, kErrPage);
        }
      }
      if (k8) ctl->exponent[r0 + lane] = static_cast<int8_t>(e);
      const int ch = lane % kLanes;
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        const int r = i * (32 / kLanes) + lane / kLanes;
        const long long row = __shfl_sync(0xffffffffu, at, r);
        copy16(key_chunk(r0 + r, ch), base + max(row, 0ll) + ch * 16, row >= 0);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&ctl->loaded));
  };
  auto short_unit = [&](const Unit& u) { return u.t1 - u.t0 <= kS; };

  if (warp == 16) {
    // -------------------------------------------------------------------- Q tiles
    if (lane == 0) tma_prefetch_desc(&tm_q);
    int n = 0, loads = 0;
    bool ok = true;
    for (Unit u = first(blockIdx.x, lane == 0); ok && u.it < units; u = first(u.it + stride, lane == 0)) {
      if (u.t0 == u.t1) continue;
      // A warp's copies are ~3 bytes a clock.  The keys of a unit whose Q tiles are all under way at once would be waited for: this
      // warp copies half of them (12 heads of 30 tokens over 35 thousand keys of 3 sequences 70 -> 53 us; of all units' keys, a
      // 480p frame takes 293 us, not 287).  Of others it says that it has none to copy: who waits for `taken` sees every phase.
      if (loads > 0 && !(ok = wait(&ctl->taken, loads - 1, kSiteTaken))) break;
      ++loads;
      copy_keys(u, short_unit(u) ? 32 : u.keys, 64);
      for (int t = u.t0; t < u.t1; ++t, ++n) {
        const int st = n % kS;
        if (n >= kS && !(ok = wait(&ctl->q_empty[st], n / kS - 1, kSiteQEmpty))) break;
        if (lane == 0) {
          const uint32_t bar = smem_addr(&ctl->q_full[st]);
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(row_tile) * D * 2);
#pragma unroll
          for (int h = 0; h < Lo::kParts; ++h)
            tma_load_4d(sQ + st * Lo::kStageBytes + h * Lo::kPart, &tm_q, bar, h * 64, u.hk * p.g, u.sq.row0 + t * (row_tile / p.g), 0);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int st = 0; st < kS; ++st)
        if (n > st) drain_wait(smem_addr(&ctl->q_full[st]), ((n - 1 - st) / kS) & 1);
    __syncwarp();
  } else if (warp == 17) {
    // -------------------------------------------------------------------- products
    constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    int n = 0, seq = 0, filled[2] = {0, 0};
    int given = 0;                                       // a byte for each group: tiles given to it, mod kSBufs
    bool ok = true;
    for (Unit u = first(blockIdx.x); ok && u.it < units; u = first(u.it + stride)) {
      if (u.t0 == u.t1) continue;
      const int tiles = u.has(1) ? 2 : 1;
      for (int x = 0; ok && x < tiles; ++x) ok = wait(&ctl->keys[x], filled[x]++, kSiteKeys);
      for (int t = u.t0; ok && t < u.t1; ++t, ++n) {
        const int st = n % kS;
        if (!(ok = wait(&ctl->q_full[st], n / kS, kSiteQFull))) break;
        const int cols = min(row_tile, u.rows - t * row_tile);
        // whole tiles take the zero rows too; the last tile only what it has, in sixteens
        const uint32_t id = idesc_f16kind_f32acc(kKeys, cols == row_tile ? kRowTile : (cols + 15) & ~15, kType, 0);
        const uint64_t b = smem_desc_sw128(sQ + st * Lo::kStageBytes, 16, 1024);
        for (int x = 0; x < tiles; ++x, ++seq) {
          const int buf = seq % kSBufs;
          if (seq >= kSBufs && !(ok = wait(&ctl->s_empty[buf], seq / kSBufs - 1, kSiteSEmpty))) break;
          tc_fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_warp(tmem + 128 + buf * 128, tmem + x * 64 + kk * 8, b + (kk >> 2) * (Lo::kPart >> 4) + (kk & 3) * 2, id, kk > 0 ? 1u : 0u);
          const int group = x + 2 * ((t - u.t0) & 1), at = given >> (8 * group) & 255;
          mma_commit_warp(smem_addr(&ctl->s_full[group][at]));
          given += at == kSBufs - 1 ? -(at << (8 * group)) : 1 << (8 * group);
        }
        if (!ok) break;
        mma_commit_warp(smem_addr(&ctl->q_empty[st]));
      }
      for (int x = 0; ok && x < tiles; ++x) mma_commit_warp(smem_addr(&ctl->keys_free[x]));
    }
    mma_commit_warp(smem_addr(&ctl->done));
    drain_wait(smem_addr(&ctl->done), 0);
  } else if (warp == 18) {
    // -------------------------------------------------------------------- lse of the rows
    constexpr int kPer = kRowTile / 32;
    int evens = 0, odds = 0;                             // Q tiles so far
    bool ok = true;
    long long at[kPer];                                  // where this lane's rows of a head's first tile lie
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = i * 32 + lane;
      at[i] = x < row_tile ? static_cast<long long>(x % p.g) * p.N + x / p.g : -1;
    }
    for (Unit u = first(blockIdx.x); ok && u.it < units; u = first(u.it + stride)) {
      const float* lse = wp.lse + static_cast<long long>(u.hk) * p.g * p.N + u.sq.row0;
      float v[kPer], ahead[kPer];                        // of this tile and the next
      auto load = [&](int t, float (&to)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          to[i] = -INFINITY;                             // no row
          if (at[i] >= 0 && t * row_tile + i * 32 + lane < u.rows) to[i] = lse[at[i] + t * (row_tile / p.g)];
        }
      };
      load(u.t0, ahead);
      for (int t = u.t0; t < u.t1; ++t) {
        const int odd = (t - u.t0) & 1, n = odd ? odds++ : evens++, slot = n % kLseSlots;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = ahead[i];
        if (t + 1 < u.t1) load(t + 1, ahead);
        if (n >= kLseSlots && !(ok = wait(&ctl->l_empty[odd][slot], n / kLseSlots - 1, kSiteLseEmpty))) break;
        // a row that saw no key weighs 2^-inf = 0
#pragma unroll
        for (int i = 0; i < kPer; ++i) ctl->nl[odd][slot][i * 32 + lane] = v[i] == -INFINITY ? -INFINITY : v[i] * -1.4426950408889634f;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl->l_full[odd][slot]));
      }
    }
    __syncwarp();
  } else if (warp == 19) {
    // -------------------------------------------------------------------- keys to shared memory, a unit ahead
    int n = 0;
    bool ok = true;
    for (Unit u = first(blockIdx.x); ok && u.it < units; u = first(u.it + stride)) {
      if (u.t0 == u.t1) continue;
      if (n > 0 && !(ok = wait(&ctl->taken, n - 1, kSiteTaken))) break;
      copy_keys(u, 0, short_unit(u) ? 64 : 32);
      ++n;
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------------- exponentials, sums; keys to tensor memory
    const int x = (warp >> 2) & 1, half = warp >> 3;     // key tile; every other Q tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int n = 0, seq = 0, weighed = 0, parts = 0;          // n: this half's Q tiles
    int loads = 0, writes = 0;                           // units, units whose keys this tile has
    bool ok = true;
    // 32 columns are 64 channels
    auto write_keys = [&](const Unit& u) {
      if (u.it >= units || u.t0 == u.t1) return;
      if (u.has(x) && writes > 0 && !(ok = warp_wait_inline(smem_addr(&ctl->keys_free[x]), (writes - 1) & 1, flag, kSiteKeysFree))) return;
      if (!(ok = warp_wait_inline(smem_addr(&ctl->loaded), loads & 1, flag, kSiteLoaded))) return;
      ++loads;
      if (u.has(x)) {
        ++writes;
        tc_fence_after_sync();
        const int r = x * kKeys + row;
        const uint32_t scale = k8 ? pair_two_to<T>(ctl->exponent[r]) : 0u;
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t y[32];
#pragma unroll
          for (int i = 0; i < 4 * kElem; ++i) {
            const uint4 v = ld_shared_v4(key_chunk(r, h * 4 * kElem + i));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (k8)
                decode4<T>(w[e], scale, y[i * 8 + 2 * e], y[i * 8 + 2 * e + 1], top);
              else
                y[i * 4 + e] = w[e];
            }
          }
          // a NaN channel makes every score of the key NaN: the last one stands for all
          if (k8 && h == D / 64 - 1 && any_nan(top)) y[31] = 0x7fff7fffu;
          tmem_st32(tmem + lanes + x * 64 + h * 32, y);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&ctl->keys[x]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl->taken));
    };
    Unit u = first(blockIdx.x);
    if (half == 0) write_keys(u);
    while (ok && u.it < units) {
      const int c = u.key0 + x * kKeys + row;
      const bool live = c < u.sq.len;
      float* w = wp.w + u.s * wp.w_seq + u.hk * wp.w_head + c;
      const float old = half == 0 && live && c < u.sq.len - u.sq.n ? *w : 0.f;
      // rows below this one do not see the key; the whole warp's keys are seen from `clear` on
      const long long r0 = live ? static_cast<long long>(first_token(p, u.sq, c)) * p.g : 0;
      const int from = static_cast<int>(min(r0, static_cast<long long>(u.rows)));
      const int clear = __reduce_max_sync(0xffffffffu, from);
      const int tiles = u.has(1) ? 2 : 1;
      float total = 0.f;
      for (int t = u.t0; t < u.t1; ++t, seq += tiles) {
        if (((t - u.t0) & 1) != half) continue;
        const int slot = n % kLseSlots;
        if (!(ok = warp_wait_inline(smem_addr(&ctl->l_full[half][slot]), (n / kLseSlots) & 1, flag, kSiteLseFull))) break;
        if (u.has(x)) {
          const int buf = (seq + x) % kSBufs;
          if (!(ok = warp_wait_inline(smem_addr(&ctl->s_full[x + 2 * half][weighed % kSBufs]), (weighed / kSBufs) & 1, flag, kSiteSFull))) break;
          tc_fence_after_sync();
          ++weighed;
          const int cols = min(row_tile, u.rows - t * row_tile), lo = from - t * row_tile;
          const uint32_t ts = tmem + lanes + 128 + buf * 128, nl = smem_addr(&ctl->nl[half][slot][0]);
          const bool whole = cols == row_tile && clear <= t * row_tile;
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
          auto free_s = [&] {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl->s_empty[buf]));
          };
          if (whole) {
#pragma unroll 1
            for (int ch = 0; ch < row_tile; ch += 32) {
              uint32_t s[32];
              tmem_ld32(ts + ch, s);
              if (ch + 32 >= row_tile) free_s();
              weigh32<false>(s, nl + ch * 4, p.scale_log2, 0, 32, acc);
            }
          } else {
#pragma unroll 1
            for (int ch = 0; ch < cols; ch += 32) {
              uint32_t s[32];
              tmem_ld32(ts + ch, s);
              if (ch + 32 >= cols) free_s();
              weigh32<true>(s, nl + ch * 4, p.scale_log2, lo - ch, cols - ch, acc);
            }
          }
          float a, b;
          f32x2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), a, b);
          total += a + b;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl->l_empty[half][slot]));
        ++n;
      }
      if (!ok) break;
      const Unit next = first(u.it + stride);
      if (half == 0) write_keys(next);
      if (!ok) break;
      // the sums of the odd Q tiles to those of the even ones
      if (u.has(x)) {
        if (u.t1 - u.t0 > 1) {
          const uint32_t bar = smem_addr(half ? &ctl->part_empty[x] : &ctl->part_full[x]);
          if (half) {
            if (parts > 0 && !(ok = warp_wait_inline(bar, (parts - 1) & 1, flag, kSitePart))) break;
            ctl->part[x][row] = total;
            mbar_arrive(smem_addr(&ctl->part_full[x]));
          } else {
            if (!(ok = warp_wait_inline(bar, parts & 1, flag, kSitePart))) break;
            total += ctl->part[x][row];
            mbar_arrive(smem_addr(&ctl->part_empty[x]));
          }
          ++parts;
        }
        if (half == 0 && live) *w = old * wp.decay + total;
      }
      u = next;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool k8>
cudaError_t launch_kind(const WeighParams& p, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  CUtensorMap mq;
  if (!encode_rows<T>(encode, &mq, p.kv.q, D, p.kv.Hq, p.kv.q_h, p.kv.N, p.kv.q_t, 1, 0, 64, p.kv.g, kRowTile / p.kv.g)) {
    *what = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  constexpr int kSmem = Layout<D>::kOffCtl + static_cast<int>(sizeof(Ctl)) + 1024;
  static_assert(kSmem <= 232448, "shared memory of a block");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(weigh_tiles<T, D, k8>, kSmem, &done);
  if (e != cudaSuccess) return e;
  const int blocks = (p.kv.max_kv + 2 * kKeys - 1) / (2 * kKeys);
  const long long units = static_cast<long long>(p.kv.S) * p.kv.Hkv * blocks;
  if (units > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  if (units == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSmem);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_tiles<T, D, k8>, mq, p, static_cast<int>(units), blocks);
}
template <typename T, int D>
cudaError_t launch(const WeighParams& p, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  return p.kv.eight ? launch_kind<T, D, true>(p, encode, sms, stream, what) : launch_kind<T, D, false>(p, encode, sms, stream, what);
}

}  // namespace

cudaError_t launch_weigh_tiles(const WeighParams& p, int d, int dtype, EncodeTiledFn encode, int sms, cudaStream_t stream, const char** what) {
  *what = nullptr;
  note_launch();
  if (dtype == 0)
    return d == 128 ? launch<__nv_bfloat16, 128>(p, encode, sms, stream, what) : launch<__nv_bfloat16, 64>(p, encode, sms, stream, what);
  return d == 128 ? launch<__half, 128>(p, encode, sms, stream, what) : launch<__half, 64>(p, encode, sms, stream, what);
}

cudaError_t read_and_clear_error_word_weigh_tiles(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
