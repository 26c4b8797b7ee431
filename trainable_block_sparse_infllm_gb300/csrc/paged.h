// Internal launch interface of the paged-cache kernels (paged_append.cu,
// paged_attn.cu, paged_evict.cu).  Host-side only; every pointer is a device
// pointer unless its comment says otherwise.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace infllmv2 {

// A paged cache as the kernels see it.  Strides are in elements.
struct PagedShape {
  int B, Hkv, D, ps, P, maxp;   // batch, KV heads, head dim, page size, pages of the pool, page-table width
  int cap;                      // maxp * ps: slots a sequence can hold
  bool fp16;
  long long kst[3], vst[3];     // page, head, token
  void* k;
  void* v;
  float* weights;               // [P, Hkv, ps] or null
  int32_t* positions;           // [P, Hkv, ps] or null
  const int32_t* table;         // [B, maxp]
  const int32_t* kv_lens;       // [B]
  uint32_t* status;
};

// Source of an append: rows [batch, head, token, d] with their strides (elements).
struct PagedRows {
  const void* k;
  const void* v;
  long long kst[3], vst[3];   // batch, head, token
};

cudaError_t launch_paged_append(const PagedShape& s, int nq, const PagedRows& rows, const int32_t* n_new,
                                const int32_t* seq_lens, cudaStream_t st);

// Tensor-map order of the pool's dimensions: which of map dimensions 1..3
// (0 is d) holds the token, head and page coordinate.
struct PagedMapOrder {
  int token, head, page;
};

size_t paged_attn_workspace_bytes(const PagedShape& s, int G);
cudaError_t launch_paged_attn(const PagedShape& s, int G, const CUtensorMap& k_map, PagedMapOrder k_order,
                              const CUtensorMap& v_map, PagedMapOrder v_order, int box_rows, const void* q,
                              float scale2, bool accumulate, void* out, float* lse, void* ws, cudaStream_t st);

constexpr int kPagedMaxGroup = 32;
constexpr int kPagedMaxBatch = 4096;

size_t paged_evict_workspace_bytes(const PagedShape& s);
bool paged_evict_supported(const PagedShape& s);
cudaError_t launch_paged_evict(const PagedShape& s, int budget, int n_init, int n_local, const int32_t* seq_lens,
                               int32_t* new_lens, void* ws, cudaStream_t st);

}  // namespace infllmv2
