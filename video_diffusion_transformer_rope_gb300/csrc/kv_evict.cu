// Eviction from a paged cache by the weight that each key has gathered: which keys of a (sequence, kv head) stay, and
// the move of what stays into the pages of another table.
//
// evict_select, a cluster of up to 8 blocks per (sequence, head), a run of the weights in each one's shared memory: of the
// first L - recent weights the `need` largest, of equals the lowest indices.  The border is found digit by digit (8 bits
// of the weights as ordered integers, from the top: a histogram of those that share the digits so far, summed over the
// blocks, then the digit that holds the need-th largest; no further one where all that share the digits so far stay), then
// one walk in order writes index and weights of what stays; a key's place is the number of keys above the border before it
// and of those equal to it, up to the last that fits.
// Bound by latency: passes and barriers (75600 weights of 40 heads: one block a head 76 us, clusters of 8 37 us).
//
// evict_move, a warp per (16 slots of a page, head): rows of 16 keys and values, found through the index and the old
// page table, 16 bytes a lane; in 8 bits their largest value gives the new scale first.  Bound by DRAM: what stays is read
// and written once (28800 of 75600 keys of 40 heads of 128 channels in 16 bits, 1.18 GB: 171 us, the rate of a plain copy;
// in 8 bits 166 for half of that, rows of 128 bytes gathered by head).
#include <cstdint>

#include "kv8.cuh"
#include "kv_common.cuh"

namespace vdx {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;               // weights of a thread in one step of a walk
constexpr int kMaxRun = kMaxEvictKeys / 8;      // weights that a block's shared memory holds

// Larger weights are larger numbers; NaN is the largest, -0 is 0.
__device__ __forceinline__ uint32_t ordered(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return b >> 31 ? ~b : b | 0x80000000u;
}

// The weight that it was (-0 comes back as 0, a NaN as some NaN).
__device__ __forceinline__ float weight_of(uint32_t u) { return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u); }

__device__ __forceinline__ int evict_length(const EvictParams& p, int s, bool report) {
  const int len = load_i32(p.kv_len + s), used = min(max(len, 0), p.max_kv);
  if (report && used != len) atomicOr(&g_error_word, kErrLength);
  return used;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_addr(p), rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads)
evict_select(const __grid_constant__ EvictParams p, const int cluster) {
  extern __shared__ __align__(16) uint32_t run[];          // this block's weights, as ordered integers
  __shared__ uint32_t hist[kWarps][256 + 1];
  __shared__ uint32_t s_total[2][256], s_all[256], s_count[2];
  __shared__ uint32_t s_prefix, s_need, s_whole;
  __shared__ uint2 s_sum[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / cluster, hk = unit % p.Hkv, s = unit / p.Hkv;
  auto sync_all = [&] {
    if (cluster > 1)
      cluster_sync_all();
    else
      __syncthreads();
  };
  wait_for_earlier_work();
  const int len = evict_length(p, s, tid == 0 && rank == 0 && hk == 0), left = min(len, p.keep);
  if (tid == 0 && rank == 0 && hk == 0) {
    p.kv_len_out[s] = left;
    if (p.pos_offset_out) p.pos_offset_out[s] = (p.pos_offset ? load_i32(p.pos_offset + s) : 0) + (len - left);
  }
  const float* w = p.w + s * p.w_seq + hk * p.w_head;
  float* w_out = p.w_out + s * p.w_out_seq + hk * p.w_out_head;
  int* index = p.index + (static_cast<long long>(s) * p.Hkv + hk) * p.keep;

  const int per = ((len + cluster - 1) / cluster + kPer - 1) / kPer * kPer;
  const int begin = min(rank * per, len), count = min(per, len - begin);
  for (int base = tid; base < count; base += 8 * kThreads) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (base + e * kThreads < count) x[e] = w[begin + base + e * kThreads];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (base + e * kThreads < count) run[base + e * kThreads] = ordered(x[e]);
  }
  const int older = len > p.keep ? len - p.recent : 0;      // the candidates; the rest stays
  const int mine = min(max(older - begin, 0), count);       // of them in this run
  uint32_t border = 0, need = len > p.keep ? p.keep - p.recent : 0;
  if (need > 0) {
    uint32_t prefix = 0;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < kWarps * 257; i += kThreads) (&hist[0][0])[i] = 0;
      __syncthreads();
      for (int i = tid; i < mine; i += kThreads) {
        const uint32_t u = run[i];
        // a histogram per warp: weights crowd into few digits
        if (pass == 0 || (u >> (shift + 8)) == prefix) atomicAdd(&hist[warp][(u >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid < 256) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) n += hist[i][tid];
        s_total[pass & 1][tid] = n;
      }
      sync_all();
      if (tid < 256) {
        uint32_t n = s_total[pass & 1][tid];
        if (cluster > 1) {
          n = 0;
#pragma unroll
          for (int r = 0; r < 8; ++r) n += ld_cluster_u32(&s_total[pass & 1][tid], min(r, cluster - 1)) * (r < cluster ? 1u : 0u);
        }
        s_all[tid] = n;
      }
      __syncthreads();
      if (warp == 0) {
        // from the top digit down, 8 digits to a lane: where the need-th largest lies
        uint32_t n[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += n[i] = s_all[255 - (lane * 8 + i)];
        uint32_t before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && need <= before + n[i]) {
            s_prefix = (prefix << 8) | static_cast<uint32_t>(255 - (lane * 8 + i));
            s_need = need - before;
            s_whole = need - before == n[i];
          }
          before += n[i];
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;                                        // of the weights that share these digits
      border = prefix << shift;
      if (s_whole) break;                                   // all of them stay: no digit further down matters
    }
  }
  auto above_border = [&](int i, uint32_t u) { return i >= mine || (need > 0 && u > border); };
  auto at_border = [&](int i, uint32_t u) { return i < mine && need > 0 && u == border; };
  // What lies before this run: counted by its blocks.
  uint32_t above = 0, equal = 0;
  if (cluster > 1) {
    if (tid < 2) s_count[tid] = 0;
    __syncthreads();
    uint32_t g = 0, q = 0;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t u = run[i];
      g += above_border(i, u);
      q += at_border(i, u);
    }
    g = __reduce_add_sync(0xffffffffu, g);
    q = __reduce_add_sync(0xffffffffu, q);
    if (lane == 0) {
      atomicAdd(&s_count[0], g);
      atomicAdd(&s_count[1], q);
    }
    cluster_sync_all();
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      above += ld_cluster_u32(&s_count[0], min(r, rank)) * (r < rank ? 1u : 0u);
      equal += ld_cluster_u32(&s_count[1], min(r, rank)) * (r < rank ? 1u : 0u);
    }
  } else {
    __syncthreads();
  }
  // In order: above the border stays, of those at it the first `need`.  Every weight of the head is in shared memory by
  // now, so w_out may be w.
  for (int base = 0, step = 0; base < count; base += kThreads * kPer, ++step) {
    uint32_t x[kPer];
    uint32_t gt = 0, eq = 0;                                // bits
#pragma unroll
    for (int e = 0; e < kPer; e += 4) {
      const int i = base + tid * kPer + e;                  // runs are padded to kPer
      const uint4 v = i < count ? *reinterpret_cast<const uint4*>(run + i) : make_uint4(0u, 0u, 0u, 0u);
      x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + tid * kPer + e;
      if (i < count) {
        if (above_border(i, x[e])) gt |= 1u << e;
        if (at_border(i, x[e])) eq |= 1u << e;
      }
    }
    uint2 sum = make_uint2(__popc(gt), __popc(eq));
    const uint2 own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, sum.x, o), b = __shfl_up_sync(0xffffffffu, sum.y, o);
      if (lane >= o) sum = make_uint2(sum.x + a, sum.y + b);
    }
    if (lane == 31) s_sum[step & 1][warp] = sum;
    __syncthreads();
    const uint2 of_warp = lane < kWarps ? s_sum[step & 1][lane] : make_uint2(0u, 0u);
    uint2 all = of_warp;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, all.x, o), b = __shfl_up_sync(0xffffffffu, all.y, o);
      if (lane >= o) all = make_uint2(all.x + a, all.y + b);
    }
    uint32_t g = above + sum.x - own.x + __shfl_sync(0xffffffffu, all.x - of_warp.x, warp);
    uint32_t q = equal + sum.y - own.y + __shfl_sync(0xffffffffu, all.y - of_warp.y, warp);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const bool is_gt = gt >> e & 1, is_eq = eq >> e & 1;
      if (is_gt || (is_eq && q < need)) {
        const uint32_t at = g + min(q, need);
        index[at] = begin + base + tid * kPer + e;
        w_out[at] = weight_of(x[e]);
      }
      g += is_gt;
      q += is_eq;
    }
    above += __shfl_sync(0xffffffffu, all.x, kWarps - 1);
    equal += __shfl_sync(0xffffffffu, all.y, kWarps - 1);
  }
  for (int j = left + rank * kThreads + tid; j < p.keep; j += cluster * kThreads) {
    index[j] = -1;
    w_out[j] = 0.f;
  }
  if (cluster > 1) cluster_sync_all();                      // no block leaves while another reads its counts
}

constexpr int kMoveWarps = 4;

// Rows of D * (k8 ? 1 : 2) bytes.
template <int D, bool k8>
__global__ void __launch_bounds__(kMoveWarps * 32)
evict_move(const __grid_constant__ EvictParams p, const int blocks, const int blocks_page) {
  constexpr int kRowBytes = D * (k8 ? 1 : 2), kLanes = kRowBytes / 16, kRowsStep = 32 / kLanes, kSteps = kBlock8 / kRowsStep;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, ch = lane % kLanes;
  wait_for_earlier_work();
  const long long task = static_cast<long long>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  // heads of a block of slots are neighbours: their rows lie side by side in a token-major cache
  const int hk = static_cast<int>(task % p.Hkv);
  const long long rest = task / p.Hkv;
  const int b = static_cast<int>(rest % blocks), s = static_cast<int>(rest / blocks);
  if (s >= p.S) return;
  const int left = min(evict_length(p, s, false), p.keep);
  const int pg = b / blocks_page, slot0 = (b - pg * blocks_page) * kBlock8;
  const long long j0 = static_cast<long long>(pg) * p.P_to + slot0;
  const int count = static_cast<int>(min(static_cast<long long>(min(kBlock8, p.P_to - slot0)), left - j0));
  if (count <= 0) return;
  const int page_to = pg < p.max_pages_to ? load_i32(p.table_to + s * p.table_to_stride + pg) : -1;
  if (page_to < 0 || page_to >= p.num_pages_to) {
    if (lane == 0) atomicOr(&g_error_word, pg < p.max_pages_to ? kErrPage : kErrInto);
    return;
  }
  // lane l (and 16 + l): where the l-th key comes from
  int page = -1, slot = 0;
  if ((lane & 15) < count) {
    const int c = load_i32(p.index + (static_cast<long long>(s) * p.Hkv + hk) * p.keep + j0 + (lane & 15));
    page = load_i32(p.table + s * p.table_stride + c / p.P);
    slot = c % p.P;
    if (page < 0 || page >= p.num_pages) {
      page = -1;                                            // its key and value are zeros
      if (lane < 16) atomicOr(&g_error_word, kErrPage);
    }
  }
  int exps = kMinExp8;                                      // lane l: exponent of key l, 16 + l: of value l
  if (k8 && page >= 0) {
    const Scales8& sc = p.scales;
    exps = scale_exponent(*(lane < 16 ? sc.k + page * sc.k_page + slot / kBlock8 * sc.k_block + hk * sc.k_head
                                      : sc.v + page * sc.v_page + slot / kBlock8 * sc.v_block + hk * sc.v_head));
  }
  uint4 x[2][kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = i * kRowsStep + sub;
    const long long from = __shfl_sync(0xffffffffu, page, r);
    const int sl = __shfl_sync(0xffffffffu, slot, r);
    x[0][i] = x[1][i] = make_uint4(0u, 0u, 0u, 0u);
    if (from >= 0) {
      x[0][i] = load_b128(p.k + from * p.k_p + sl * p.k_t + hk * p.k_h + ch * 16);
      x[1][i] = load_b128(p.v + from * p.v_p + sl * p.v_t + hk * p.v_h + ch * 16);
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    uint8_t* to = kind ? p.v_to + page_to * p.vt_p + slot0 * p.vt_t + hk * p.vt_h : p.k_to + page_to * p.kt_p + slot0 * p.kt_t + hk * p.kt_h;
    const long long token = kind ? p.vt_t : p.kt_t;
    float lift[kSteps];
    if (k8) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        lift[i] = two_to(__shfl_sync(0xffffffffu, exps, kind * 16 + i * kRowsStep + sub));
        float f[16];
        decode8(make_uint2(x[kind][i].x, x[kind][i].y), reinterpret_cast<float (&)[8]>(f[0]));
        decode8(make_uint2(x[kind][i].z, x[kind][i].w), reinterpret_cast<float (&)[8]>(f[8]));
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) m = fmaxf(m, fabsf(f[c]));
        top = fmaxf(top, m * lift[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = block_exponent(top);
      const float inv = two_to(-e);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const float by = lift[i] * inv;
        uint32_t* word = reinterpret_cast<uint32_t*>(&x[kind][i]);
        float f[16];
        decode8(make_uint2(word[0], word[1]), reinterpret_cast<float (&)[8]>(f[0]));
        decode8(make_uint2(word[2], word[3]), reinterpret_cast<float (&)[8]>(f[8]));
#pragma unroll
        for (int c = 0; c < 4; ++c) word[c] = encode4(f[4 * c] * by, f[4 * c + 1] * by, f[4 * c + 2] * by, f[4 * c + 3] * by);
      }
      const Scales8& sc = p.scales_to;
      if (lane == 0)
        *(kind ? sc.v + page_to * sc.v_page + slot0 / kBlock8 * sc.v_block + hk * sc.v_head
               : sc.k + page_to * sc.k_page + slot0 / kBlock8 * sc.k_block + hk * sc.k_head) = static_cast<uint8_t>(e + 127);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = i * kRowsStep + sub;
      if (r < count) *reinterpret_cast<uint4*>(to + r * token + ch * 16) = x[kind][i];
    }
  }
}

template <int D, bool k8>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  const int most = p.keep < p.max_kv ? p.keep : p.max_kv;
  const int blocks_page = (p.P_to - 1) / kBlock8 + 1;
  const long long blocks = static_cast<long long>(most / p.P_to) * blocks_page + (most % p.P_to + kBlock8 - 1) / kBlock8;
  if (blocks == 0) return cudaSuccess;
  const long long grid = (blocks * p.Hkv * p.S + kMoveWarps - 1) / kMoveWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kMoveWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr = launch_early();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move<D, k8>, p, static_cast<int>(blocks), blocks_page);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int d, bool eight, cudaStream_t stream) {
  note_launch();
  // runs of about 4096 weights; one block reads them fast enough, and barriers of a cluster cost more than they save
  int cluster = 1;
  while (cluster < 8 && p.max_kv > cluster * 4096) cluster *= 2;
  const int run = ((p.max_kv + cluster - 1) / cluster + kPer - 1) / kPer * kPer;
  const int smem = run * 4;
  const long long blocks = static_cast<long long>(p.S) * p.Hkv * cluster;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_shared(evict_select, kMaxRun * 4, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = launch_early();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select, p, cluster);
  if (e != cudaSuccess) return e;
  if (eight) return d == 128 ? launch_move<128, true>(p, stream) : launch_move<64, true>(p, stream);
  return d == 128 ? launch_move<128, false>(p, stream) : launch_move<64, false>(p, stream);
}

cudaError_t read_and_clear_error_word_evict(unsigned int* word) { return read_and_clear_word(word); }

}  // namespace vdx
