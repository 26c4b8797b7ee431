// Page tables and slot maps of one step, from the lengths of its requests.
//
// Sequence b goes from kv_lens[b] to kv_lens[b] + n_new[b] tokens, which need
// need_b = ceil(that / page size) pages; it owns the first held[b] entries of its
// row of the table.  Rows that shrink give back entries [need, held), rows that
// grow take entries [held, need): take j of all (in order of sequence and entry)
// is the stack's j-th page from the top, and past the stack's end page j - n of
// those that this call gives back.  What is left of those goes onto the stack.
// Then token t of sequence b has its slot, page * page size + row, and position.
// Three sums over the batch (pages taken, pages given, tokens) say where each
// sequence's share starts.  A call that lacks pages or finds a bad length changes
// no table and maps no token.
//
// Bound by latency: of the launches, and of the few loads that depend on each other
// (lengths, then an entry of the stack or table, then the slot).  One cluster, for
// small steps one CTA, makes the sums for itself in shared memory.  Takes only write
// rows that grow, and read the stack and rows that shrink; after the cluster's barrier
// come the writes to the stack and to the lengths, which every CTA has read by then.
// The slots are found beside the takes, a new page's through the stack in place of the
// table.  Measured (GB300, with the copy that resets its tables): 64 sequences of one
// token 4.8 us in a graph, 48 with 70,000 tokens 10.5 us.  (A second launch over the
// whole device for the slots of a large step cost more than it saved: 21.4 us a pass
// from Python instead of 17.6.)
#include "paged.cuh"
#include "packed.h"

namespace infllmv2 {

namespace {

constexpr int kMost = 1024;          // threads of a CTA
constexpr int kMaxWarps = kMost / 32;
constexpr int kMaxCluster = 16;
constexpr int kTokensPerCta = 4096;  // before another CTA joins

struct Sums {
  long long take, give, tokens;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.take + b.take, a.give + b.give, a.tokens + b.tokens};
}

__device__ __forceinline__ Sums shfl_up(const Sums& s, int o) {
  return {__shfl_up_sync(0xffffffffu, s.take, o), __shfl_up_sync(0xffffffffu, s.give, o),
          __shfl_up_sync(0xffffffffu, s.tokens, o)};
}

// The sequence whose share [start[b], start[b + 1]) holds i; start[n] > i >= start[0].
__device__ __forceinline__ int owner(const int* start, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Row `row` of a page; none for a page that is not of the pool (a foreign entry on the stack).
__device__ __forceinline__ int slot_of(int page, int row, const ReserveArgs& a) {
  if (page >= 0 && page < a.pages) return page * a.ps + row;
  atomicOr(a.status, kStatusBadPage);
  return -1;
}

__global__ void __launch_bounds__(kMost) paged_reserve_kernel(const ReserveArgs a, int ctas) {
  extern __shared__ int shared[];
  __shared__ Sums warp_sum[kMaxWarps];
  __shared__ int bad_any;
  const int n1 = a.batch + 1;
  int* take0 = shared;            // first take, give and token of each sequence
  int* give0 = take0 + n1;
  int* token0 = give0 + n1;
  int* held = token0 + n1;        // the entries it owns and needs
  int* need = held + n1;
  int* kv = need + n1;
  const int threads = blockDim.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  pdl_wait();
  if (tid == 0) bad_any = 0;
  const int n_free = *a.n_free;
  __syncthreads();

  // Each thread: the sums of its run of sequences.
  const int per = (a.batch + threads - 1) / threads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  const long long cap = static_cast<long long>(a.maxp) * a.ps;
  Sums mine = {0, 0, 0};
  bool bad = n_free < 0 || n_free > a.pages;
  for (int b = b0; b < b1; ++b) {
    const int L = a.kv_lens[b], m = a.n_new[b], h = a.held[b];
    const long long after = static_cast<long long>(L) + m;
    bad |= L < 0 || m < 0 || after > cap || h < 0 || h > a.maxp;
    const int pages = bad ? 0 : static_cast<int>((after + a.ps - 1) / a.ps);
    held[b] = h;
    need[b] = pages;
    kv[b] = L;
    if (!bad) mine = mine + Sums{max(pages - h, 0), max(h - pages, 0), m};
  }
  Sums incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up = shfl_up(incl, o);
    if (lane >= o) incl = incl + up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (bad) bad_any = 1;
  __syncthreads();
  Sums total = {0, 0, 0}, at = {0, 0, 0};
  for (int w = 0; w < (a.batch + 32 * per - 1) / (32 * per); ++w) {   // the warps that have sequences
    if (w == warp) at = total;
    total = total + warp_sum[w];
  }
  const long long on_stack = total.take < n_free ? total.take : n_free;   // takes from the stack
  const long long kept = n_free - on_stack;
  const long long reused = total.take - on_stack;                         // takes of what is given back
  const long long lacking = reused - total.give;
  const long long most = a.slots || a.positions ? a.max_tokens : 0x7fffffffll;
  const bool refuse = bad_any || n_free + total.give > a.pages || total.tokens > most;
  const bool go = !refuse && lacking <= 0;
  at = {at.take + incl.take - mine.take, at.give + incl.give - mine.give, at.tokens + incl.tokens - mine.tokens};
  if (go) {
    for (int b = b0; b < b1; ++b) {
      take0[b] = static_cast<int>(at.take);
      give0[b] = static_cast<int>(at.give);
      token0[b] = static_cast<int>(at.tokens);
      at.take += max(need[b] - held[b], 0);
      at.give += max(held[b] - need[b], 0);
      at.tokens += a.n_new[b];
    }
    if (tid == 0) {
      take0[a.batch] = static_cast<int>(total.take);
      give0[a.batch] = static_cast<int>(total.give);
      token0[a.batch] = static_cast<int>(total.tokens);
    }
  }
  __syncthreads();

  const int stride = ctas * threads, first = rank * threads + tid;
  // Page i of those given back, in order.
  auto given = [&](int i) {
    const int b = owner(give0, a.batch, i);
    return a.table[static_cast<long long>(b) * a.maxp + need[b] + (i - give0[b])];
  };
  auto taken = [&](int j) { return j < n_free ? a.free_pages[n_free - 1 - j] : given(j - n_free); };
  if (go) {
    for (int j = first; j < total.take; j += stride) {
      const int b = owner(take0, a.batch, j);
      a.table[static_cast<long long>(b) * a.maxp + held[b] + (j - take0[b])] = taken(j);
    }
  }
  const int tokens = go ? static_cast<int>(total.tokens) : 0;
  if (a.slots || a.positions) {
    for (int t = first; t < a.max_tokens; t += stride) {
      int slot = -1, position = 0;
      if (t < tokens) {
        const int b = owner(token0, a.batch, t), i = t - token0[b];
        const int s = kv[b] + i, c = s / a.ps;
        if (a.slots) {
          const int page = c < held[b] ? a.table[static_cast<long long>(b) * a.maxp + c]
                                       : taken(take0[b] + c - held[b]);
          slot = slot_of(page, s - c * a.ps, a);
        }
        position = (a.seq_lens ? a.seq_lens[b] : kv[b]) + i;
      }
      if (a.slots) a.slots[t] = slot;
      if (a.positions) a.positions[t] = position;
    }
  }
  if (ctas > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  pdl_trigger();
  if (go) {
    for (int i = first + static_cast<int>(reused); i < total.give; i += stride)
      a.free_pages[kept + (i - reused)] = given(i);
  }
  if (rank == 0) {
    for (int b = b0; b < b1; ++b) {
      a.starts[b] = go ? token0[b] : 0;
      a.new_lens[b] = go ? kv[b] + (token0[b + 1] - token0[b]) : kv[b];
      if (go) a.held[b] = need[b];
    }
    if (tid == 0) {
      a.starts[a.batch] = tokens;
      if (go) *a.n_free = static_cast<int>(kept + total.give - reused);
      *a.missing = refuse ? -1 : static_cast<int>(min(max(lacking, 0ll), 0x7fffffffll));
      if (refuse) atomicOr(a.status, kStatusBadKvLen);
    }
  }
}

}  // namespace

cudaError_t launch_paged_reserve(const ReserveArgs& a, cudaStream_t st) {
  const size_t bytes = 6 * sizeof(int) * (static_cast<size_t>(a.batch) + 1);
  // Small steps in 256 threads, whose barriers and sums cost less (in a graph, 256 or 1024 threads: 64 sequences
  // of one token 2.9 or 3.7 us, 256 of one 3.5 or 4.4; 2048 tokens 7.3 or 4.8; between, at 1024 tokens of 16
  // to 64 sequences, 256 already cost 0.6 to 0.9 us more).
  const int threads = a.batch <= 256 && a.max_tokens <= 1024 ? 256 : kMost;
  int ctas = 1;
  while (ctas < kMaxCluster && a.max_tokens > ctas * kTokensPerCta) ctas *= 2;
  cudaError_t e = cudaSuccess;
  if (bytes > 40 * 1024)
    e = cudaFuncSetAttribute(paged_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(6 * sizeof(int) * (kPagedMaxBatch + 1)));
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(paged_reserve_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = ctas;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, paged_reserve_kernel, a, ctas);
}

}  // namespace infllmv2
