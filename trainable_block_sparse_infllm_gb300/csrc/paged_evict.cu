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
//    bits) in registers, and the budget-th largest key is found 4 bits at a
//    time: 16 counts per round, packed in registers, summed by redux, shared
//    memory and, for C > 1, distributed shared memory.  Unlike a shared-memory
//    histogram its time does not depend on how the weights are spread (sums of
//    softmax weights crowd into a few exponents).  Ordered scans then number
//    the holes and the movers.
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
  int32_t* hole;     // [B Hkv][most] evicted slots below the budget
  int32_t* mover;    // [B Hkv][most] kept slots at or past it
  int most;          // cap / 2: min(budget, n - budget) at most
};

// Larger key: kept first.  NaN (a weight that no softmax produced) goes first
// of all, and -0 equals 0.
__device__ __forceinline__ uint32_t evict_key(float w) { return w != w ? 0u : float_to_ordered(w + 0.f); }

template <int kKeys>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int C) {
  __shared__ uint32_t warp_hist[2][kSelWarps][8];          // 16 counts of 16 bits per warp
  __shared__ uint32_t cta_hist[2][kMaxCluster][16];        // by rank, written by every rank
  __shared__ unsigned long long warp_tot[kSelWarps];
  __shared__ unsigned long long cta_tot[2][kMaxCluster];
  __shared__ uint32_t bad_by_rank[kMaxCluster];
  const PagedShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C, b = unit / s.Hkv, h = unit % s.Hkv;
  if (C > 1) cluster_arrive_relaxed();
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

  // ---- the budget-th largest key, 4 bits per round from the top -------------
  uint32_t prefix = 0;
  int want = a.budget;   // how many of the keys that match the prefix stay
#pragma unroll 1
  for (int round = 0; round < 8; ++round) {
    const int shift = 28 - 4 * round, buf = round & 1;
    // Counts of this thread's digits, 8 bits each, digits 0-3, 4-7, 8-11, 12-15.
    uint32_t c8[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const uint32_t k = key[i];
      const bool in = i < mine && (round == 0 || (k >> (shift + 4)) == prefix);
      const uint32_t d = (k >> shift) & 15u;
      const uint32_t one = in ? 1u << ((d & 3) * 8) : 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) c8[q] += (d >> 2) == static_cast<uint32_t>(q) ? one : 0u;
    }
    uint32_t sum[8];   // digits 2 j and 2 j + 1, 16 bits each
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      sum[2 * q] = __reduce_add_sync(0xffffffffu, __byte_perm(c8[q], 0, 0x4140));
      sum[2 * q + 1] = __reduce_add_sync(0xffffffffu, __byte_perm(c8[q], 0, 0x4342));
    }
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) warp_hist[buf][warp][j] = sum[j];
    }
    __syncthreads();
    int have = 0;   // lane d < 16: keys with digit d
    if (C == 1 || warp == 0) {
      if (lane < 16) {
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) have += (warp_hist[buf][w][lane >> 1] >> ((lane & 1) * 16)) & 0xffffu;
      }
    }
    if (C > 1) {
      if (warp == 0) {
        for (int r = lane >> 4; r < C; r += 2) {
          const int v = __shfl_sync(0xffffffffu, have, lane & 15);
          st_dsmem_u32(dsmem_addr(&cta_hist[buf][rank][lane & 15], r), v);
        }
      }
      cluster_sync();
      have = 0;
      if (lane < 16)
        for (int r = 0; r < C; ++r) have += cta_hist[buf][r][lane];
    }
    // Keys with a larger digit than lane's (lanes 16.. hold 0).
    const int incl = warp_inclusive_scan(have);
    const int total = __shfl_sync(0xffffffffu, incl, 15);
    const int above = total - incl;
    const bool here = lane < 16 && above < want && above + have >= want;
    const int d = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    want -= __shfl_sync(0xffffffffu, above, d);
    prefix = (prefix << 4) | static_cast<uint32_t>(d);
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
  for (int i = static_cast<int>(at >> 32); holes; holes &= holes - 1, ++i) a.hole[list + i] = slot0 + __ffsll(holes) - 1;
  int last = static_cast<int>(at & 0xffffffffu);
  for (; movers; movers &= movers - 1, ++last) a.mover[list + last] = slot0 + __ffsll(movers) - 1;
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
  const int32_t* table = s.table + static_cast<long long>(b) * s.maxp;
  const long long list = static_cast<long long>(unit) * a.most;
  const int step = gridDim.x * (kMoveThreads / 32) * kBatch;
  for (int first = (blockIdx.x * (kMoveThreads / 32) + warp) * kBatch; first < count; first += step) {
    const int have = min(kBatch, count - first);
    int to_page = 0, to_row = 0, from_page = 0, from_row = 0;
    if (lane < have) {
      const int to = a.hole[list + first + lane], from = a.mover[list + first + lane];
      to_page = __ldg(table + to / s.ps);
      to_row = to % s.ps;
      from_page = __ldg(table + from / s.ps);
      from_row = from % s.ps;
      const long long d = paged_meta(to_page, h, to_row, s.Hkv, s.ps);
      const long long f = paged_meta(from_page, h, from_row, s.Hkv, s.ps);
      const float w = s.weights[f];
      const int p = s.positions[f];
      s.weights[d] = w;
      s.positions[d] = p;
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
  a.mover = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + up256(units * 4) + up256(units * a.most * 4));
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
