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
// The packed form takes rows [token, head, d] of several sequences, and each
// token's slot in place of a table: slots[t] = page * page size + row, below 0
// for a token that is not written.
//
// Measured (GB300): 8 prompts of up to 8192 tokens, 4 KV heads, 37,700 tokens in
// all, 25.9 us, 93% of the copy rate; one token of each of 64 sequences, 8 KV
// heads, 2.4 us in a graph, 7.0 us a call from Python.  Packed: 40,000 tokens, 4 KV
// heads, into token-major pages, 26.1 us in a graph, 93%; 64 tokens, 8 KV heads, 2.0 us in a graph,
// 5.3 us a call from Python.
#include "packed.h"
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
  const int n_new = a.n_new ? a.n_new[b] : a.nq;
  const int L = s.kv_lens[b];
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
      page[i] = s.table[static_cast<long long>(b) * s.maxp + slot / s.ps];
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
        s.positions[m] = (a.seq_lens ? a.seq_lens[b] : L) - n_new + t0 + i;
    }
  }
}

template <int kLanes, int kRows>   // kLanes = D / 8
__global__ void __launch_bounds__(kThreads) packed_append_kernel(const PagedShape s, const PackedAppend a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % kLanes;
  const int which = blockIdx.y & 1;   // 0: keys, 1: values
  const int h = blockIdx.y >> 1;
  const int t0 = (blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes) * kRows;
  const long long* dst = which ? s.vst : s.kst;
  const long long step = which ? a.v_token : a.k_token;
  const uint16_t* src = static_cast<const uint16_t*>(which ? a.v : a.k) + h * (which ? a.v_head : a.k_head) + lane * 8;
  uint16_t* to = static_cast<uint16_t*>(which ? s.v : s.k) + h * dst[1] + lane * 8;
  uint4 x[kRows];
  int slot[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    slot[i] = -1;
    if (t0 + i < a.tokens) {
      slot[i] = a.slots[t0 + i];
      x[i] = *reinterpret_cast<const uint4*>(src + (t0 + i) * step);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slot[i] < 0) continue;
    const int page = slot[i] / s.ps, row = slot[i] - page * s.ps;
    if (page >= s.P) {   // no such page: the token is not written
      atomicOr(s.status, kStatusBadPage);
      continue;
    }
    *reinterpret_cast<uint4*>(to + page * dst[0] + row * dst[2]) = x[i];
    if (lane == 0) {
      const long long m = paged_meta(page, h, row, s.Hkv, s.ps);
      if (which == 0 && s.weights) s.weights[m] = 0.f;
      if (which == 1 && s.positions) s.positions[m] = a.positions[t0 + i];
    }
  }
}

cudaLaunchConfig_t launch_config(dim3 grid, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int kLanes, int kRows>
cudaError_t launch_packed(const PagedShape& s, const PackedAppend& a, cudaStream_t st) {
  const int per_block = kThreads / kLanes * kRows;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      launch_config(dim3(static_cast<unsigned>((a.tokens + per_block - 1) / per_block), 2 * s.Hkv, 1), st, &attr);
  return cudaLaunchKernelEx(&cfg, packed_append_kernel<kLanes, kRows>, s, a);
}

template <int kLanes, int kRows>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
  const int per_block = kThreads / kLanes * kRows;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = launch_config(
      dim3(static_cast<unsigned>((a.nq + per_block - 1) / per_block), 2 * a.s.Hkv, a.s.B), st, &attr);
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<kLanes, kRows>, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedShape& s, int nq, const PagedRows& rows, const int32_t* n_new,
                                const int32_t* seq_lens, cudaStream_t st) {
  const AppendArgs a{s, rows, nq, n_new, seq_lens};
  return s.D == 128 ? launch<16, 4>(a, st) : launch<8, 4>(a, st);
}

cudaError_t launch_paged_append_packed(const PagedShape& s, const PackedAppend& a, cudaStream_t st) {
  return s.D == 128 ? launch_packed<16, 4>(s, a, st) : launch_packed<8, 4>(s, a, st);
}

}  // namespace infllmv2
