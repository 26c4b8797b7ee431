// Internal launch interface of the packed attention kernels (packed_attn.cu,
// packed_attn_bwd.cu).  Host-side only; every pointer is a device pointer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace infllmv2 {

constexpr int kPackedMaxBatch = 4096;
constexpr int kPackedMaxGroup = 32;

// Strides in elements between tokens and heads.
struct PackedStride {
  long long token, head;
};

struct PackedAttnShape {
  int B, Hkv, G, Tq, Tk;
  float scale, scale2;        // of the scores; scale2 = scale log2(e)
  const int32_t* q_starts;    // [B + 1]
  const int32_t* k_starts;    // [B + 1]
  uint32_t* status;
};

// Tensor maps.  q, out (the forward pass's only where by_tile), dout: [d, group, KV
// head, token], one box of 64 columns = the
// rows (token, head of the group) of packed_tile_tokens(G) tokens; k, v: [d,
// token, KV head], one box of 64 columns x 128 tokens.  128-byte swizzle.
struct PackedAttnMaps {
  CUtensorMap q, k, v, out, dout;
};

// Tokens whose rows, one per head of the group, fill a tile of 128.
__host__ __device__ constexpr int packed_tile_tokens(int G) { return 128 / G; }

struct PackedAttnOut {
  void* out;
  PackedStride st;
  float* lse;   // [Tq, Hkv * G] or null
  bool by_tile;   // whole tiles through maps.out
};

// Whether the forward pass writes whole tiles by TMA.
bool packed_attn_by_tile(const PackedAttnShape& s);

// The inputs behind the maps, for single rows.
struct PackedAttnIn {
  const void *q, *k, *v;
  PackedStride q_st, k_st, v_st;
};

cudaError_t launch_packed_attn(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                               const PackedAttnIn& in, const PackedAttnOut& o, cudaStream_t st);

struct PackedAttnGrads {
  const float* lse;
  void *dq, *dk, *dv;
  PackedStride dq_st, dk_st, dv_st;
  // Workspace [Tq, Hkv * G]: of each row D and, before it, lse log2(e), or in fp16 two exponents of dS (its own, and
  // in the first row of a tile that of the tile's rows).
  float2* rows;
};

cudaError_t launch_packed_attn_bwd(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                                   const PackedAttnGrads& g, cudaStream_t st);

}  // namespace infllmv2
