// Append to a paged cache: token t of sequence b's n_new[b] newest tokens goes
// to slot kv_lens[b] - n_new[b] + t, which is row slot % page_size of page
// table[b, slot / page_size]; its weight starts at 0 and its position is
// seq_lens[b] - n_new[b] + t.
//
// A copy: bound by latency for one token per sequence and by memory for a
// prompt.  A row (a key or a value of one head) takes D / 8 lanes of 16 bytes;
// a group of lanes carries kRows consecutive tokens of one (b, h), all loads
// before the first store, so that a long prompt keeps enough bytes in flight.
// The page table is read once per token.
//
// Measured (GB300): 8 prompts of up to 8192 tokens, 4 KV heads, 37,700 tokens in
// all, 25.9 us, 93% of the copy rate; one token of each of 64 sequences, 8 KV
// heads, 2.4 us in a graph, 7.0 us a call from Python.
#include "paged.cuh"

namespace infllmv2 {

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  PagedShape s;
  PagedRows r;
  int nq;
  const int32_t* n_new;
  const int32_t* seq_lens;
};

template <int kLanes, int kRows>   // kLanes = D / 8
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
  const PagedShape& s = a.s;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % kLanes;
  const int b = blockIdx.z;
  const int which = blockIdx.y & 1;   // 0: keys, 1: values
  const int h = blockIdx.y >> 1;
  const int t0 = (blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes) * kRows;
  const int n_new = a.n_new ? __ldg(a.n_new + b) : a.nq;
  const int L = __ldg(s.kv_lens + b);
  if (n_new < 0 || n_new > a.nq || L < n_new || L > s.cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(s.status, kStatusBadKvLen);
    return;
  }
  if (t0 >= n_new) return;
  const long long* sst = which ? a.r.vst : a.r.kst;
  const long long* dst = which ? s.vst : s.kst;
  const uint16_t* src = static_cast<const uint16_t*>(which ? a.r.v : a.r.k) + b * sst[0] + h * sst[1] + lane * 8;
  uint16_t* to = static_cast<uint16_t*>(which ? s.v : s.k) + h * dst[1] + lane * 8;
  uint4 x[kRows];
  int page[kRows], row[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    page[i] = -1;
    if (t0 + i < n_new) {
      const int slot = L - n_new + t0 + i;
      page[i] = __ldg(s.table + static_cast<long long>(b) * s.maxp + slot / s.ps);
      row[i] = slot % s.ps;
      x[i] = *reinterpret_cast<const uint4*>(src + (t0 + i) * sst[2]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t0 + i >= n_new) break;
    if (page[i] < 0 || page[i] >= s.P) {   // no such page: the token is not written
      atomicOr(s.status, kStatusBadPage);
      continue;
    }
    *reinterpret_cast<uint4*>(to + page[i] * dst[0] + row[i] * dst[2]) = x[i];
    if (lane == 0) {
      const long long m = paged_meta(page[i], h, row[i], s.Hkv, s.ps);
      if (which == 0 && s.weights) s.weights[m] = 0.f;
      if (which == 1 && s.positions)
        s.positions[m] = (a.seq_lens ? __ldg(a.seq_lens + b) : L) - n_new + t0 + i;
    }
  }
}

template <int kLanes, int kRows>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
  const int per_block = kThreads / kLanes * kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.nq + per_block - 1) / per_block), 2 * a.s.Hkv, a.s.B);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<kLanes, kRows>, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedShape& s, int nq, const PagedRows& rows, const int32_t* n_new,
                                const int32_t* seq_lens, cudaStream_t st) {
  const AppendArgs a{s, rows, nq, n_new, seq_lens};
  return s.D == 128 ? launch<16, 4>(a, st) : launch<8, 4>(a, st);
}

}  // namespace infllmv2
