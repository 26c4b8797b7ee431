// Internal launch interface of the packed-step kernels (rotary.cu,
// paged_reserve.cu, paged_append.cu's packed form).  Host-side only; every
// pointer is a device pointer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"

namespace infllmv2 {

// Tokens of a rotary or append call (their rounding up to whole CTAs stays within 32 bits).
constexpr int kPackedMaxTokens = 1 << 30;

// One packed tensor [tokens, heads, d]; strides in elements.
struct PackedRows {
  void* x;
  long long token, head;
};

// ------------------------------------------------------------- rotary ----

struct RotaryArgs {
  PackedRows q_in, q_out, k_in, k_out;
  const int32_t* positions;
  const uint64_t* turns;   // [part / 2]: 2^64 times the turns per position
  float scale;
  int tokens, q_heads, k_heads, dim, part;
  bool interleaved, transpose, in_place;
};

enum class RotaryType { kBf16, kFp16, kFp32 };
cudaError_t launch_rotary(const RotaryArgs& a, RotaryType type, cudaStream_t st);

// ------------------------------------------------------ pages and slots ----

struct ReserveArgs {
  int batch, maxp, ps, pages, max_tokens;
  int32_t* table;        // [batch, maxp]
  int32_t* held;         // [batch]
  int32_t* free_pages;   // [pages]
  int32_t* n_free;       // [1]
  const int32_t* kv_lens;
  const int32_t* n_new;
  const int32_t* seq_lens;   // or null: kv_lens
  int32_t* new_lens;
  int32_t* starts;       // [batch + 1]
  int32_t* slots;        // [max_tokens] or null
  int32_t* positions;    // [max_tokens] or null
  int32_t* missing;      // [1]
  uint32_t* status;
};

cudaError_t launch_paged_reserve(const ReserveArgs& a, cudaStream_t st);

// ------------------------------------------------------- packed append ----

struct PackedAppend {
  const void* k;
  const void* v;
  long long k_token, k_head, v_token, v_head;
  int tokens;
  const int32_t* slots;
  const int32_t* positions;   // or null
};

cudaError_t launch_paged_append_packed(const PagedShape& s, const PackedAppend& a, cudaStream_t st);

}  // namespace infllmv2
