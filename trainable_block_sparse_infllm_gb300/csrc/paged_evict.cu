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
// Two launches:
//  * evict_select_kernel, one cluster of C CTAs per (sequence, KV head): every
//    thread holds kKeys consecutive slots' keys (weight order-mapped to 32
//    bits) in registers, and the budget-th largest key is found 8 bits at a
//    time by 256-bin histograms in shared memory, for C > 1 summed through
//    distributed shared memory.  Ordered scans then number the holes and the
//    movers.
//  * evict_move_kernel: the numbered moves, over the whole GPU whatever the
//    number of (sequence, KV head) pairs; this is where the bytes are.
#include "paged.cuh"
#include "kernels.h"

namespace infllmv2 {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMaxCluster = 16;

struct EvictArgs {
  PagedShape s;
  int budget, n_init, n_local;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* count;    // [B Hkv] rows to move; -1: a page was bad, the sequence stays
  int2* hole;        // [B Hkv][most] (page, row) of the evicted slots below the budget
  int2* mover;       // [B Hkv][most] of the kept slots at or past it
  int most;          // cap / 2: min(budget, n - budget) at most
};

// Larger key: kept first.  NaN (a weight that no softmax produced) goes first
// of all, and -0 equals 0.
__device__ __forceinline__ uint32_t evict_key(float w) { return w != w ? 0u : float_to_ordered(w + 0.f); }

template <int kKeys>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int C) {
  __shared__ __align__(16) uint32_t hist[2][256];
  __shared__ __align__(16) uint32_t total[256];            // of the cluster
  __shared__ unsigned long long warp_tot[kSelWarps];
  __shared__ unsigned long long cta_tot[2][kMaxCluster];
  __shared__ uint32_t bad_by_rank[kMaxCluster];
  const PagedShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C, b = unit / s.Hkv, h = unit % s.Hkv;
  if (C > 1) cluster_arrive_relaxed();
  if (tid < 256) hist[0][tid] = hist[1][tid] = 0;   // visible by the barrier after the loads
  pdl_wait();
  pdl_trigger();
  if (C > 1) cluster_wait();   // every CTA runs: its shared memory may be written
  const int n = paged_len(s.kv_lens, b, s.cap, s.status);
  if (n <= a.budget) {   // the same for the whole cluster
    if (rank == 0 && tid == 0) a.count[unit] = 0;
    return;
  }
  const int seen = a.seq_lens ? __ldg(a.seq_lens + b) : n;
  const int slot0 = (rank * kSelThreads + tid) * kKeys;
  const int mine = max(0, min(kKeys, n - slot0));
  uint32_t key[kKeys];
  bool bad = false;
  {
    const int32_t* table = s.table + static_cast<long long>(b) * s.maxp;
    constexpr int kPart = kKeys < 16 ? kKeys : 16;   // 16 slots at a multiple of 16 are in one page
#pragma unroll
    for (int c = 0; c < kKeys / kPart; ++c) {
      const int first = slot0 + c * kPart;
      long long at = -1;
      if (first < n) {
        const int page = __ldg(table + first / s.ps);
        if (page < 0 || page >= s.P)
          bad = true;
        else
          at = paged_meta(page, h, first % s.ps, s.Hkv, s.ps);
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
          const bool always = ps[e] < a.n_init || ps[e] >= seen - a.n_local;
          key[c * kPart + v * 4 + e] = always ? 0xffffffffu : evict_key(ws[e]);
        }
      }
    }
  }
  if (bad) atomicOr(s.status, kStatusBadPage);
  bad = __syncthreads_or(bad);
  if (C > 1) {
    if (tid < C) st_dsmem_u32(dsmem_addr(&bad_by_rank[rank], tid), bad ? 1u : 0u);
    cluster_sync();
    for (int r = 0; r < C; ++r) bad |= bad_by_rank[r] != 0;
  }
  if (bad) {
    if (rank == 0 && tid == 0) a.count[unit] = -1;
    return;
  }

  // ---- the budget-th largest key, 8 bits per round from the top -------------
  // `want`: how many of the keys that match the prefix stay.  The counts are
  // shared-memory increments; those of a warp that meet in one bin are one.
  uint32_t prefix = 0;
  int want = a.budget;
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round, buf = round & 1;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const uint32_t k = key[i];
      if (i < mine && (round == 0 || (k >> (shift + 8)) == prefix)) atomicAdd(&hist[buf][(k >> shift) & 255u], 1u);
    }
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
    if (tid < 256) hist[buf ^ 1][tid] = 0;   // the next round's (last read before the barrier above)
    if (C > 1) {
      // Bin tid over the cluster: each CTA sums all of it by itself.
      if (tid < 256) {
        uint32_t sum = 0;
        for (int r = 0; r < C; ++r) sum += ld_dsmem_u32(dsmem_addr(&hist[buf][tid], r));
        total[tid] = sum;
      }
      __syncthreads();
    }
    // Every warp finds the bin for itself: lane l holds bins 255 - 8 l - (0..7), largest first.
    const uint32_t* h = C > 1 ? total : hist[buf];
    const uint4 hi = *reinterpret_cast<const uint4*>(h + 252 - 8 * lane);
    const uint4 lo = *reinterpret_cast<const uint4*>(h + 248 - 8 * lane);
    const int c[8] = {static_cast<int>(hi.w), static_cast<int>(hi.z), static_cast<int>(hi.y), static_cast<int>(hi.x),
                      static_cast<int>(lo.w), static_cast<int>(lo.z), static_cast<int>(lo.y), static_cast<int>(lo.x)};
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += c[j];
    const int incl = warp_inclusive_scan(sum);
    int above = incl - sum;   // keys in larger bins
    int bin = 0;
    const bool here = above < want && incl >= want;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (above + c[j] >= want) {
        bin = 255 - 8 * lane - j;
        break;
      }
      above += c[j];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    want -= __shfl_sync(0xffffffffu, above, src);
    prefix = (prefix << 8) | static_cast<uint32_t>(__shfl_sync(0xffffffffu, bin, src));
    __syncthreads();   // hist[buf ^ 1] is zero
  }

  // ---- which slots stay: larger keys, and the first `want` equal ones --------
  // Two ordered scans over all threads: the equal keys, then holes and movers.
  auto scan = [&](unsigned long long v, int buf) {   // exclusive, over the unit's threads
    unsigned long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (buf) __syncthreads();   // the first scan's totals have been read
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    unsigned long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      if (w == warp) before = all;
      all += warp_tot[w];
    }
    if (C > 1) {
      if (tid < C) st_dsmem_u64(dsmem_addr(&cta_tot[buf][rank], tid), all);
      cluster_sync();
      for (int r = 0; r < rank; ++r) before += cta_tot[buf][r];
    }
    return before + inc - v;
  };
  int equal = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) equal += (i < mine && key[i] == prefix) ? 1 : 0;
  int rank_eq = static_cast<int>(scan(equal, 0));
  unsigned long long stay = 0;   // kKeys bits
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const bool eq = key[i] == prefix;
    if (i < mine && (key[i] > prefix || (eq && rank_eq < want))) stay |= 1ull << i;
    rank_eq += (i < mine && eq) ? 1 : 0;
  }
  const int below = max(0, min(mine, a.budget - slot0));   // slots below the budget
  const unsigned long long below_mask = below >= 64 ? ~0ull : (1ull << below) - 1;
  unsigned long long holes = ~stay & below_mask, movers = stay & ~below_mask;
  const unsigned long long at =
      scan((static_cast<unsigned long long>(__popcll(holes)) << 32) | static_cast<unsigned long long>(__popcll(movers)), 1);
  const long long list = static_cast<long long>(unit) * a.most;
  auto place = [&](unsigned long long bits) {
    const int slot = slot0 + __ffsll(bits) - 1;
    return make_int2(__ldg(s.table + static_cast<long long>(b) * s.maxp + slot / s.ps), slot % s.ps);
  };
  for (int i = static_cast<int>(at >> 32); holes; holes &= holes - 1, ++i) a.hole[list + i] = place(holes);
  int last = static_cast<int>(at & 0xffffffffu);
  for (; movers; movers &= movers - 1, ++last) a.mover[list + last] = place(movers);
  // The unit's last thread has every mover before it.
  if (rank == C - 1 && tid == kSelThreads - 1) a.count[unit] = last;
}

// CTA (x, unit): moves x, x + gridDim.x, ... of the unit in batches of kBatch
// per warp.  A row of D 16-bit values takes D / 8 lanes of 16 bytes; all loads
// of a batch are issued before its first store.
template <int kDim>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  constexpr int kLanes = kDim / 8, kRowsAtOnce = 32 / kLanes;
  constexpr int kBatch = 8;                              // moves: 2 kBatch rows
  constexpr int kSteps = 2 * kBatch / kRowsAtOnce;
  const PagedShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.y, b = unit / s.Hkv, h = unit % s.Hkv;
  pdl_wait();
  pdl_trigger();
  const int count = a.count[unit];
  if (blockIdx.x == 0 && h == 0 && tid == 0) {
    // The only reader of kv_lens in this launch is new_lens' writer, so the two may be one array.
    const int n = paged_len(s.kv_lens, b, s.cap, s.status);
    a.new_lens[b] = count < 0 ? n : min(n, a.budget);
  }
  const long long list = static_cast<long long>(unit) * a.most;
  const int step = gridDim.x * (kMoveThreads / 32) * kBatch;
  int first = (blockIdx.x * (kMoveThreads / 32) + warp) * kBatch;
  int2 to_next = make_int2(0, 0), from_next = make_int2(0, 0);
  auto fetch = [&](int at) {   // one batch ahead
    if (lane < kBatch && at + lane < count) {
      to_next = a.hole[list + at + lane];
      from_next = a.mover[list + at + lane];
    }
  };
  fetch(first);
  for (; first < count; first += step) {
    const int have = min(kBatch, count - first);
    const int to_page = to_next.x, to_row = to_next.y, from_page = from_next.x, from_row = from_next.y;
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

struct EvictPlan {
  int keys, cluster;
};

// Slots per thread and CTAs per unit.  One CTA holds 512 x 4, 8 or 16 slots;
// longer caches take clusters of up to 16 CTAs, and past 131072 slots more
// keys per thread.
EvictPlan evict_plan(int cap) {
  if (cap <= kSelThreads * 4) return {4, 1};
  if (cap <= kSelThreads * 8) return {8, 1};
  int c = 1;
  while (c < kMaxCluster && cap > kSelThreads * 16 * c) c *= 2;
  int keys = 16;
  while (keys < 64 && cap > kSelThreads * keys * c) keys *= 2;
  return {keys, c};
}

template <int kKeys>
cudaError_t launch_select(const EvictArgs& a, int C, cudaStream_t st) {
  auto kernel = evict_select_kernel<kKeys>;
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.B * a.s.Hkv * C), 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
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
  return up256(units * 4) + 2 * up256(units * most_moves(s) * sizeof(int2));
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
  a.hole = reinterpret_cast<int2*>(static_cast<char*>(ws) + up256(units * 4));
  a.mover = reinterpret_cast<int2*>(reinterpret_cast<char*>(a.hole) + up256(units * a.most * sizeof(int2)));
  const EvictPlan plan = evict_plan(s.cap);
  cudaError_t e;
  switch (plan.keys) {
    case 4: e = launch_select<4>(a, plan.cluster, st); break;
    case 8: e = launch_select<8>(a, plan.cluster, st); break;
    case 16: e = launch_select<16>(a, plan.cluster, st); break;
    case 32: e = launch_select<32>(a, plan.cluster, st); break;
    default: e = launch_select<64>(a, plan.cluster, st); break;
  }
  if (e != cudaSuccess) return e;
  return s.D == 128 ? launch_move<128>(a, st) : launch_move<64>(a, st);
}

}  // namespace infllmv2
