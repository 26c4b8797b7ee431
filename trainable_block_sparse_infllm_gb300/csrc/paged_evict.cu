// Eviction from a paged cache by accumulated attention weight.
//
// Of a (sequence, KV head) with n > budget slots the `budget` best stay: first
// the slots whose position is below n_init or among the sequence's newest
// n_local positions, then by weight, descending; equal ones by slot,
// ascending.  Attention does not depend on the order of a cache's slots, so
// nothing is compacted: the i-th kept slot at or past `budget` moves into the
// i-th evicted slot below it (both ascending), which moves the fewest rows and
// never overwrites a row that is still to be read.  A decode loop that evicts
// one token per step moves one row per step, not the cache.
//
// evict_select_kernel, one cluster of C CTAs per (sequence, KV head): every
// thread holds kKeys consecutive slots' keys (weight order-mapped to 32 bits)
// in registers.  The key that divides kept from evicted is found by 256-bin
// histograms in shared memory (for C > 1 summed through distributed shared
// memory): the first spans the keys from the smallest to the largest, each
// further one the bin that holds the boundary, until a bin holds just the keys
// that are still wanted.  (Digits of fixed bits would put most softmax sums
// into the two or three bins of their exponents.)  Ordered scans then number
// the holes and the movers, whose lists go out through shared memory, in whole
// lines.  evict_move_kernel moves the rows over the whole GPU; where the capacity
// past the budget allows few moves (kFewMoves) the selecting CTAs do it themselves
// and save the launch.
//
// Measured (GB300): 32 sequences of 2K to 16K, 8 KV heads, pages of 16, to 4096:
// selection 33 us (barriers and shared-memory counts; 2 CTAs per unit, 1.7
// waves), moves 89 us (454 MB of rows and 50 MB of their weights' and positions'
// sectors: 5.7 TB/s, 85% of the copy rate, in rows of 256 bytes).  One of 128K to
// 32K, 2 KV heads: 17 and 12 us.  One slot of each of 16 sequences of 4097, 2 KV
// heads: 8.7 us, one launch.
#include "paged.cuh"
#include "kernels.h"

namespace infllmv2 {

namespace {

constexpr int kSelThreads = 512;
constexpr int kShortThreads = 128;   // of a CTA for a short cache among many
constexpr int kMoveThreads = 256;
constexpr int kMaxCluster = 16;

struct EvictArgs {
  PagedShape s;
  int budget, n_init, n_local;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* count;    // [B Hkv] rows to move; -1: a page was bad, the sequence stays
  // [B Hkv][most] evicted slots below the budget, kept slots at or past it, as
  // page * page size + row (the pool's slots are fewer than 2^31).
  int32_t* hole;
  int32_t* mover;
  int most;          // cap / 2: min(budget, n - budget) at most
};

// Larger key: kept first.  NaN (a weight that no softmax produced) goes first
// of all, and -0 equals 0.
__device__ __forceinline__ uint32_t evict_key(float w) { return w != w ? 0u : float_to_ordered(w + 0.f); }

// Moves warp, warp + warps, ... (in batches of kBatch) of a unit's `count`.  A
// row of D 16-bit values takes D / 8 lanes of 16 bytes; all loads of a batch
// are issued before its first store, and the next batch's places are fetched
// meanwhile.
template <int kDim, int kBatch>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int unit, int h, int count, int warp, int warps) {
  constexpr int kLanes = kDim / 8, kRowsAtOnce = 32 / kLanes;
  constexpr int kSteps = 2 * kBatch / kRowsAtOnce;
  const PagedShape& s = a.s;
  const int lane = threadIdx.x & 31;
  const long long list = static_cast<long long>(unit) * a.most;
  const int step = warps * kBatch;
  int first = warp * kBatch;
  int to_next = 0, from_next = 0;
  auto fetch = [&](int at) {
    if (lane < kBatch && at + lane < count) {
      to_next = a.hole[list + at + lane];
      from_next = a.mover[list + at + lane];
    }
  };
  fetch(first);
  for (; first < count; first += step) {
    const int have = min(kBatch, count - first);
    const int to_page = to_next / s.ps, to_row = to_next % s.ps;
    const int from_page = from_next / s.ps, from_row = from_next % s.ps;
    fetch(first + step);
    float w = 0.f;
    int p = 0;
    if (lane < have) {
      const long long f = paged_meta(from_page, h, from_row, s.Hkv, s.ps);
      w = s.weights[f];
      p = s.positions[f];
    }
    uint4 x[kSteps];
    uint16_t* dst[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = i * kRowsAtOnce + lane / kLanes;     // row of the batch: move r / 2, K then V
      const int move = r >> 1;
      const long long* st = (r & 1) ? s.vst : s.kst;
      uint16_t* base = static_cast<uint16_t*>((r & 1) ? s.v : s.k) + h * st[1] + (lane % kLanes) * 8;
      const int fp = __shfl_sync(0xffffffffu, from_page, move), fr = __shfl_sync(0xffffffffu, from_row, move);
      const int tp = __shfl_sync(0xffffffffu, to_page, move), tr = __shfl_sync(0xffffffffu, to_row, move);
      dst[i] = move < have ? base + tp * st[0] + tr * st[2] : nullptr;
      if (move < have) x[i] = *reinterpret_cast<const uint4*>(base + fp * st[0] + fr * st[2]);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
    if (lane < have) {
      const long long d = paged_meta(to_page, h, to_row, s.Hkv, s.ps);
      s.weights[d] = w;
      s.positions[d] = p;
    }
  }
}

__device__ __forceinline__ void count_if(bool in, uint32_t* bin) {   // no branch around the increment
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(smem_u32(bin)),
               "r"(static_cast<uint32_t>(in))
               : "memory");
}

constexpr uint32_t kAlways = 0xffffffffu;   // above every weight's key

// What warps and CTAs tell each other about their keys, (a page is bad; the
// smallest and largest key of a weight; slots that always stay), over the warp's
// lanes that have one.
__device__ __forceinline__ uint4 reduce_range(uint4 v, bool has) {
  return make_uint4(__any_sync(0xffffffffu, has && v.x != 0), __reduce_min_sync(0xffffffffu, has ? v.y : kAlways),
                    __reduce_max_sync(0xffffffffu, has ? v.z : 0u), __reduce_add_sync(0xffffffffu, has ? v.w : 0u));
}

// kDim = 0: the moves are left to evict_move_kernel.
template <int kThreads, int kKeys, int kDim>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a, int C) {
  constexpr int kSelWarps = kThreads / 32;
  extern __shared__ int32_t stage[];                       // [kKeys kThreads]: holes up, movers down
  __shared__ __align__(16) uint32_t hist[2][256];
  __shared__ __align__(16) uint32_t total[256];            // of the cluster
  __shared__ uint4 range_warp[kSelWarps];
  __shared__ uint4 range[kMaxCluster];
  __shared__ int4 boundary;                                // a round's (keys above the bin, keys in it, bin)
  __shared__ unsigned long long warp_tot[2][kSelWarps];
  __shared__ unsigned long long cta_tot[2][kMaxCluster];
  const PagedShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C, b = unit / s.Hkv, h = unit % s.Hkv;
  if (C > 1) cluster_arrive_relaxed();
  for (int i = tid; i < 256; i += kThreads) hist[0][i] = hist[1][i] = 0;   // visible by the barrier after the loads
  pdl_wait();
  pdl_trigger();
  if (C > 1) cluster_wait();   // every CTA runs: its shared memory may be written
  const int n = paged_len(s.kv_lens, b, s.cap, s.status);
  const bool writes_len = kDim > 0 && rank == 0 && h == 0 && tid == 0;
  if (n <= a.budget) {   // the same for the whole cluster
    if (kDim == 0 && rank == 0 && tid == 0) a.count[unit] = 0;
    if (writes_len) a.new_lens[b] = n;
    return;
  }
  const int seen = a.seq_lens ? a.seq_lens[b] : n;
  const int slot0 = (rank * kThreads + tid) * kKeys;
  // Slots at or past n get key 0.  They never stay: of equal keys the lower
  // slots do, and more than `budget` of those exist.
  uint32_t key[kKeys];
  uint32_t low = kAlways, high = 0, always = 0;
  bool bad = false;
  constexpr int kPart = kKeys < 16 ? kKeys : 16;   // 16 slots at a multiple of 16 are in one page
  int place[kKeys / kPart];                        // page * page size + row of a part's first slot
  {
    const int32_t* table = s.table + static_cast<long long>(b) * s.maxp;
    const int local = seen - a.n_local;
#pragma unroll
    for (int c = 0; c < kKeys / kPart; ++c) {
      const int first = slot0 + c * kPart;
      long long at = -1;
      place[c] = 0;
      if (first < n) {
        const int page = table[first / s.ps], row = first % s.ps;
        if (page < 0 || page >= s.P) {
          bad = true;
        } else {
          at = paged_meta(page, h, row, s.Hkv, s.ps);
          place[c] = page * s.ps + row;
        }
      }
#pragma unroll
      for (int v = 0; v < kPart / 4; ++v) {
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        int4 p = make_int4(0, 0, 0, 0);
        if (at >= 0) {
          w = *reinterpret_cast<const float4*>(s.weights + at + v * 4);
          p = *reinterpret_cast<const int4*>(s.positions + at + v * 4);
        }
        const float ws[4] = {w.x, w.y, w.z, w.w};
        const int ps[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool held = first + v * 4 + e < n, stays = ps[e] < a.n_init || ps[e] >= local;
          const uint32_t k = evict_key(ws[e]);
          if (held && !stays) {
            low = min(low, k);
            high = max(high, k);
          }
          always += held && stays ? 1u : 0u;
          key[c * kPart + v * 4 + e] = held ? (stays ? kAlways : k) : 0u;
        }
      }
    }
  }
  if (bad) atomicOr(s.status, kStatusBadPage);
  {
    const uint4 mine = reduce_range(make_uint4(bad, low, high, always), true);
    if (lane == 0) range_warp[warp] = mine;
  }
  __syncthreads();
  if (warp == 0) {   // the CTA's, to every CTA
    const uint4 v = range_warp[lane % kSelWarps];
    const uint4 sum = reduce_range(v, lane < kSelWarps);
    if (C == 1) {
      if (lane == 0) range[0] = sum;
    } else if (lane < C) {
      const uint32_t to = dsmem_addr(&range[rank], lane);
      st_dsmem_u32(to, sum.x);
      st_dsmem_u32(to + 4, sum.y);
      st_dsmem_u32(to + 8, sum.z);
      st_dsmem_u32(to + 12, sum.w);
    }
  }
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  const uint4 all_range = reduce_range(range[lane < C ? lane : 0], lane < C);
  if (all_range.x) {
    if (kDim == 0 && rank == 0 && tid == 0) a.count[unit] = -1;
    if (writes_len) a.new_lens[b] = n;
    return;
  }

  // ---- where the boundary is ---------------------------------------------------
  // Keys above `at + last` stay, keys below `at` go; `match` keys are between,
  // of which the `want` largest (of equal ones the lowest slots) stay.
  uint32_t at = kAlways, last = 0;
  int want = a.budget, match = static_cast<int>(all_range.w);
  if (match < want) {
    want -= match;
    at = all_range.y;
    last = all_range.z - all_range.y;
    match = n - static_cast<int>(all_range.w);
  }
#pragma unroll 1
  for (int round = 0; match != want && last != 0; ++round) {
    const int buf = round & 1;
    const int shift = max(0, 24 - __clz(last));   // 256 bins of 2^shift keys
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const uint32_t off = key[i] - at;
      count_if(off <= last, &hist[buf][(off >> shift) & 255u]);
    }
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
    // The next round's (last read before the barrier above).
    for (int i = tid; i < 256; i += kThreads) hist[buf ^ 1][i] = 0;
    if (C > 1) {
      // Bin tid over the cluster: each CTA sums all of it by itself.  (Clusters
      // have at least 256 threads per CTA.)
      if (tid < 256) {
        uint32_t sum = 0;
        for (int r0 = 0; r0 < C; r0 += 8) {   // 8 remote loads in flight
          uint32_t v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = r0 + r < C ? ld_dsmem_u32(dsmem_addr(&hist[buf][tid], r0 + r)) : 0u;
#pragma unroll
          for (int r = 0; r < 8; ++r) sum += v[r];
        }
        total[tid] = sum;
      }
      __syncthreads();
    }
    if (warp == 0) {   // lane l holds bins 255 - 8 l - (0..7), largest first
      const uint32_t* hs = C > 1 ? total : hist[buf];
      const uint4 hi = *reinterpret_cast<const uint4*>(hs + 252 - 8 * lane);
      const uint4 lo = *reinterpret_cast<const uint4*>(hs + 248 - 8 * lane);
      const int c[8] = {static_cast<int>(hi.w), static_cast<int>(hi.z), static_cast<int>(hi.y), static_cast<int>(hi.x),
                        static_cast<int>(lo.w), static_cast<int>(lo.z), static_cast<int>(lo.y), static_cast<int>(lo.x)};
      int sum[8];
      sum[0] = c[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) sum[j] = sum[j - 1] + c[j];
      const int incl = warp_inclusive_scan(sum[7]), above = incl - sum[7];   // above: keys in larger bins
      if (above < want && incl >= want) {
        int j = 0;   // bins of the lane that lie above the boundary's
#pragma unroll
        for (int e = 0; e < 7; ++e) j += above + sum[e] < want ? 1 : 0;
        int before = above, in_bin = c[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
          if (e == j) {
            before = above + sum[e - 1];
            in_bin = c[e];
          }
        boundary = make_int4(before, in_bin, 255 - 8 * lane - j, 0);
      }
    }
    __syncthreads();   // the boundary is found; hist[buf ^ 1] is zero
    const int4 found = boundary;
    want -= found.x;
    match = found.y;
    const uint32_t skip = static_cast<uint32_t>(found.z) << shift;
    at += skip;
    last = min(last - skip, (1u << shift) - 1);
  }

  // ---- which slots stay, and their numbers ------------------------------------
  // Exclusive sum over the unit's threads, in slot order, of two counts packed
  // into 16 bits each; `cta0`: before this CTA, `cta`: this CTA's, `all`: the
  // unit's, 32 bits each.
  unsigned long long cta0 = 0, cta = 0, all = 0;
  auto scan = [&](uint32_t v, int buf) {
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    auto wide = [](uint32_t x) { return (static_cast<unsigned long long>(x >> 16) << 32) | (x & 0xffffu); };
    if (lane == 31) warp_tot[buf][warp] = wide(inc);
    __syncthreads();
    unsigned long long before = 0;
    cta = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      if (w == warp) before = cta;
      cta += warp_tot[buf][w];
    }
    cta0 = 0;
    all = cta;
    if (C > 1) {
      if (tid < C) st_dsmem_u64(dsmem_addr(&cta_tot[buf][rank], tid), cta);
      cluster_sync();
      all = 0;
      for (int r = 0; r < C; ++r) {
        if (r == rank) cta0 = all;
        all += cta_tot[buf][r];
      }
    }
    return before + wide(inc) - wide(v);   // within the CTA
  };
  int rank_eq = 0;
  const bool ties = match > want;   // of equal keys (last = 0): the lowest slots stay
  if (ties) {
    uint32_t equal = 0;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) equal += key[i] == at ? 1u : 0u;
    rank_eq = static_cast<int>(scan(equal, 0));
    rank_eq += static_cast<int>(cta0);
  }
  unsigned long long stay = 0;   // kKeys bits
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const bool eq = ties && key[i] == at;
    if (key[i] >= at && (!eq || rank_eq < want)) stay |= 1ull << i;
    rank_eq += eq ? 1 : 0;
  }
  const int below = min(kKeys, a.budget - slot0);   // slots below the budget
  const unsigned long long below_mask = below <= 0 ? 0ull : (below >= 64 ? ~0ull : (1ull << below) - 1);
  const unsigned long long holes = ~stay & below_mask, movers = stay & ~below_mask;
  const unsigned long long mine =
      scan((static_cast<uint32_t>(__popcll(holes)) << 16) | static_cast<uint32_t>(__popcll(movers)), 1);
  const int count = static_cast<int>(all & 0xffffffffu);   // as many holes as movers
  constexpr int kSlots = kKeys * kThreads;
  {
    int32_t* up = stage + static_cast<int>(mine >> 32);
    int32_t* down = stage + kSlots - 1 - static_cast<int>(mine & 0xffffffffu);
#pragma unroll
    for (int c = 0; c < kKeys / kPart; ++c) {
      const uint32_t mask = (1u << kPart) - 1;
      for (uint32_t x = static_cast<uint32_t>(holes >> (c * kPart)) & mask; x; x &= x - 1)
        *up++ = place[c] + __ffs(x) - 1;
      for (uint32_t x = static_cast<uint32_t>(movers >> (c * kPart)) & mask; x; x &= x - 1)
        *down-- = place[c] + __ffs(x) - 1;
    }
  }
  __syncthreads();
  {
    const int n_holes = static_cast<int>(cta >> 32), n_movers = static_cast<int>(cta & 0xffffffffu);
    int32_t* to = a.hole + static_cast<long long>(unit) * a.most + static_cast<int>(cta0 >> 32);
    int32_t* from = a.mover + static_cast<long long>(unit) * a.most + static_cast<int>(cta0 & 0xffffffffu);
    for (int i = tid; i < n_holes; i += kThreads) to[i] = stage[i];
    for (int i = tid; i < n_movers; i += kThreads) from[i] = stage[kSlots - 1 - i];
  }
  if constexpr (kDim == 0) {
    if (rank == 0 && tid == 0) a.count[unit] = count;
  } else {
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
    if (writes_len) a.new_lens[b] = a.budget;
    move_rows<kDim, 4>(a, unit, h, count, rank * kSelWarps + warp, C * kSelWarps);
  }
}

// The moves over the whole GPU: CTA (x, unit).  Also writes
// new_lens; its writer is the only reader of kv_lens in this launch, so the two
// may be one array.
template <int kDim>
__global__ void __launch_bounds__(kMoveThreads, 3) evict_move_kernel(const EvictArgs a) {
  const PagedShape& s = a.s;
  const int unit = blockIdx.y, b = unit / s.Hkv, h = unit % s.Hkv;
  pdl_wait();
  pdl_trigger();
  const int count = a.count[unit];
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int n = paged_len(s.kv_lens, b, s.cap, s.status);
    a.new_lens[b] = count < 0 ? n : min(n, a.budget);
  }
  constexpr int kWarps = kMoveThreads / 32;
  move_rows<kDim, 8>(a, unit, h, count, blockIdx.x * kWarps + threadIdx.x / 32, gridDim.x * kWarps);
}

struct EvictPlan {
  int threads, keys, cluster;
};

// Moves of a unit up to which the selecting CTAs make them.  d 128, pages of 16,
// every slot past the budget to be moved, in a graph, one against two launches:
// 128 moves: 11.5 and 10.7 us (2 units of 4096), 12.0 and 12.9 (32 of 4096), 17.2
// and 20.4 (256 of 4096), 14.3 and 19.9 (32 of 16384), 178 and 168 (800 of 16384);
// 256 moves: 14.9 and 10.7, 15.6 and 13.8, 23.8 and 24.5, 14.4 and 20.6, 197 and
// 191; 512 moves: 19.5 and 11.6, 21.0 and 17.4, 33.2 and 33.6, 18.0 and 23.1, 240
// and 229.  With one of them to be moved: 7.1 and 8.5, 8.0 and 10.2, 10.3 and 14.9,
// 11.6 and 16.1, 141 and 134.
constexpr int kFewMoves = 128;

// Threads per CTA, slots per thread and CTAs per unit.  A cache of up to 8192
// slots takes one CTA of 512 threads with 4, 8 or 16 slots each.  With more
// units than the SMs hold such CTAs at once, caches of up to 4096 slots take
// CTAs of 128 threads with up to 32, more of which share an SM (468 units of
// 844 slots: 29.2 us with 512 threads, 16.8 us with 128; 800 units of 4000: 113
// and 109 us; but 800 of 6000: 165 and 179 us).  Longer caches take clusters of
// up to 16 CTAs, and past 131072 slots more slots per thread.
EvictPlan evict_plan(int cap, long long units) {
  if (cap <= 4096 && units > 2 * device_sm_count())
    return {kShortThreads, cap <= 512 ? 4 : (cap <= 1024 ? 8 : (cap <= 2048 ? 16 : 32)), 1};
  if (cap <= 2048) return {kSelThreads, 4, 1};
  if (cap <= 4096) return {kSelThreads, 8, 1};
  int c = 1;
  while (c < kMaxCluster && cap > kSelThreads * 16 * c) c *= 2;
  int keys = 16;
  while (keys < 64 && cap > kSelThreads * keys * c) keys *= 2;
  return {kSelThreads, keys, c};
}

template <int kThreads, int kKeys, int kDim>
cudaError_t launch_select(const EvictArgs& a, int C, cudaStream_t st) {
  auto kernel = evict_select_kernel<kThreads, kKeys, kDim>;
  constexpr int kSmem = kKeys * kThreads * 4;
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (kSmem > 32768) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.B * a.s.Hkv * C), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, C);
}

template <int kDim>
cudaError_t launch_select_any(const EvictArgs& a, EvictPlan plan, cudaStream_t st) {
  if (plan.threads == kShortThreads) {
    if (plan.keys == 4) return launch_select<kShortThreads, 4, kDim>(a, 1, st);
    if (plan.keys == 8) return launch_select<kShortThreads, 8, kDim>(a, 1, st);
    if (plan.keys == 16) return launch_select<kShortThreads, 16, kDim>(a, 1, st);
    return launch_select<kShortThreads, 32, kDim>(a, 1, st);
  }
  switch (plan.keys) {
    case 4: return launch_select<kSelThreads, 4, kDim>(a, plan.cluster, st);
    case 8: return launch_select<kSelThreads, 8, kDim>(a, plan.cluster, st);
    case 16: return launch_select<kSelThreads, 16, kDim>(a, plan.cluster, st);
    case 32: return launch_select<kSelThreads, 32, kDim>(a, plan.cluster, st);
    default: return launch_select<kSelThreads, 64, kDim>(a, plan.cluster, st);
  }
}

template <int kDim>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t st) {
  // About 16 CTAs per SM over all units, no more than a unit's moves can use.
  const long long units = static_cast<long long>(a.s.B) * a.s.Hkv;
  const long long per_cta = kMoveThreads / 32 * 8;
  const long long most = a.most < a.budget ? a.most : a.budget;
  long long x = (16LL * device_sm_count() + units - 1) / units;
  const long long use = (most + per_cta - 1) / per_cta;
  if (x > use) x = use;
  if (x < 1) x = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(units), 1);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<kDim>, a);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int most_moves(const PagedShape& s) { return s.cap / 2; }

}  // namespace

bool paged_evict_supported(const PagedShape& s) { return s.cap <= kSelThreads * 64 * kMaxCluster; }

size_t paged_evict_workspace_bytes(const PagedShape& s) {
  const size_t units = static_cast<size_t>(s.B) * s.Hkv;
  return up256(units * 4) + 2 * up256(units * most_moves(s) * 4);
}

cudaError_t launch_paged_evict(const PagedShape& s, int budget, int n_init, int n_local, const int32_t* seq_lens,
                               int32_t* new_lens, void* ws, cudaStream_t st) {
  const size_t units = static_cast<size_t>(s.B) * s.Hkv;
  EvictArgs a;
  a.s = s;
  a.budget = budget;
  a.n_init = n_init;
  a.n_local = n_local;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.most = most_moves(s);
  a.count = static_cast<int32_t*>(ws);
  a.hole = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + up256(units * 4));
  a.mover = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(a.hole) + up256(units * a.most * 4));
  const EvictPlan plan = evict_plan(s.cap, static_cast<long long>(units));
  // The selecting CTAs move the rows themselves, without a second launch, where
  // the page table has room for at most kFewMoves slots past the budget (the host
  // does not know the lengths, so this bounds a unit's moves).  new_lens over
  // kv_lens would be read by the other KV heads' CTAs: that goes by the second
  // launch.
  if (new_lens != s.kv_lens && s.cap - budget <= kFewMoves)
    return s.D == 128 ? launch_select_any<128>(a, plan, st) : launch_select_any<64>(a, plan, st);
  cudaError_t e = launch_select_any<0>(a, plan, st);
  if (e != cudaSuccess) return e;
  return s.D == 128 ? launch_move<128>(a, st) : launch_move<64>(a, st);
}

}  // namespace infllmv2
