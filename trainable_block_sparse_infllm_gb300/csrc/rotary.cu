// Rotary positions: the first `part` values of every head form part / 2 pairs
// (x, y), and pair i of a token at position p becomes
//     scale (x cos a - y sin a,  x sin a + y cos a),   a = p * frequency_i,
// or, transposed (the gradient), the same with -a.
//
// An angle matters modulo one turn, and p * frequency loses all of it in 32
// bits for far positions (p = 10^6 leaves an error of 0.06 rad).  Frequencies
// are therefore 64-bit fixed-point turns per position: the 64-bit product
// p * turns wraps around exactly at whole turns, and its upper 32 bits are the
// angle to 2^-32 turn.  The nearest quarter turn comes off those bits before
// they become a float, so the conversion costs 2^-24 of an eighth turn at most.
// No table of angles is read: a token's part / 2 sines and cosines are computed
// once in its CTA and shared by all its heads.
//
// Bound by memory.  An item is two 16-byte vectors of one head that turn into
// each other (half layout: x's and y's; interleaved: two neighbours, four or
// eight pairs), or two of the part that stays.  A thread loads its first kAhead
// items before the angles are computed.
#include <cuda_fp16.h>

#include "common.cuh"
#include "packed.h"

namespace infllmv2 {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;        // items in flight per thread (8 vectors of 16 bytes)
constexpr int kMaxTokens = 8;    // tokens of one CTA
constexpr int kMaxPairs = 256;   // head_dim 512

template <typename T>
struct Vec;   // 16 bytes of T as floats

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void get(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};

template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  __device__ static void get(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  __device__ static uint4 put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ static void get(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// (cos, sin) of position * turns, times scale.
__device__ __forceinline__ float2 turned(int32_t position, uint64_t turns, float scale, bool transpose) {
  const uint64_t whole = static_cast<uint64_t>(static_cast<int64_t>(position)) * turns + (1ull << 31);
  const uint32_t angle = static_cast<uint32_t>(whole >> 32);
  const uint32_t quarter = (angle + (1u << 29)) >> 30;                        // the nearest quarter turn, 0..3
  const int32_t rest = static_cast<int32_t>(angle - (quarter << 30));         // in [-2^29, 2^29) of 2^32
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  float cs = (quarter & 1) ? -s : c, sn = (quarter & 1) ? c : s;
  if (quarter & 2) {
    cs = -cs;
    sn = -sn;
  }
  return make_float2(cs * scale, transpose ? -sn * scale : sn * scale);
}

// Where item `i` of a CTA's tokens lies: vectors at x and x + second (elements).
struct Item {
  const void* in;
  void* out;
  int second;   // elements between the item's vectors
  int pairs;    // index of its first (cos, sin), or -1: copied
};

template <typename T>
__device__ __forceinline__ Item locate(const RotaryArgs& a, int i, int token0, int per_row, int per_token) {
  constexpr int kN = Vec<T>::kN;
  const int t = i / per_token, j = i - t * per_token;
  const int h = j / per_row, c = j - h * per_row;
  const bool is_q = h < a.q_heads;
  const PackedRows& in = is_q ? a.q_in : a.k_in;
  const PackedRows& out = is_q ? a.q_out : a.k_out;
  const int head = is_q ? h : h - a.q_heads;
  const bool turns = c < a.part / (2 * kN);
  const int at = turns && !a.interleaved ? c * kN : 2 * c * kN;
  Item r;
  r.second = turns && !a.interleaved ? a.part / 2 : kN;
  r.pairs = turns ? t * (a.part / 2) + c * kN : -1;
  const long long token = token0 + t;
  r.in = static_cast<const T*>(in.x) + token * in.token + head * in.head + at;
  r.out = static_cast<T*>(out.x) + token * out.token + head * out.head + at;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int per_cta) {
  constexpr int kN = Vec<T>::kN;
  __shared__ float2 angles[kMaxTokens * kMaxPairs];
  pdl_wait();
  pdl_trigger();
  const int token0 = blockIdx.x * per_cta;
  const int tokens = min(per_cta, a.tokens - token0);
  // Items of a row: in place, what stays need not be copied.
  const int per_row = (a.in_place ? a.part : a.dim) / (2 * kN);
  const int per_token = per_row * (a.q_heads + a.k_heads);
  const int items = tokens * per_token;
  uint4 u[kAhead][2];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < items) {
      const Item it = locate<T>(a, i, token0, per_row, per_token);
      u[k][0] = *static_cast<const uint4*>(it.in);
      u[k][1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(it.in) + it.second);
    }
  }
  const int half = a.part / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = i / half;
    angles[i] = turned(__ldg(a.positions + token0 + t), __ldg(a.turns + (i - t * half)), a.scale, a.transpose);
  }
  __syncthreads();
  for (int base = 0; base < items; base += kAhead * kThreads) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + threadIdx.x + k * kThreads;
      if (i >= items) break;
      const Item it = locate<T>(a, i, token0, per_row, per_token);
      uint4 r0 = u[k][0], r1 = u[k][1];
      if (it.pairs >= 0) {
        float x[kN], y[kN];
        Vec<T>::get(r0, x);
        Vec<T>::get(r1, y);
        if (a.interleaved) {
          // Pairs (x0, x1), (x2, x3), ... then those of y.
#pragma unroll
          for (int e = 0; e < kN; e += 2) {
            const float2 f = angles[it.pairs + e / 2], g = angles[it.pairs + kN / 2 + e / 2];
            const float p = x[e], q = x[e + 1], r = y[e], s = y[e + 1];
            x[e] = p * f.x - q * f.y;
            x[e + 1] = p * f.y + q * f.x;
            y[e] = r * g.x - s * g.y;
            y[e + 1] = r * g.y + s * g.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const float2 f = angles[it.pairs + e];
            const float p = x[e], q = y[e];
            x[e] = p * f.x - q * f.y;
            y[e] = p * f.y + q * f.x;
          }
        }
        r0 = Vec<T>::put(x);
        r1 = Vec<T>::put(y);
      }
      *static_cast<uint4*>(it.out) = r0;
      *reinterpret_cast<uint4*>(static_cast<T*>(it.out) + it.second) = r1;
      // The item kAhead rounds on takes its place.
      const int next = i + kAhead * kThreads;
      if (next < items) {
        const Item n = locate<T>(a, next, token0, per_row, per_token);
        u[k][0] = *static_cast<const uint4*>(n.in);
        u[k][1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(n.in) + n.second);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RotaryArgs& a, cudaStream_t st) {
  // Tokens of a CTA: as many as give each thread kAhead items, while every SM
  // keeps several CTAs.
  const int per_token = (a.in_place ? a.part : a.dim) / (2 * Vec<T>::kN) * (a.q_heads + a.k_heads);
  int per_cta = 1;
  while (per_cta < kMaxTokens && 2 * per_cta * per_token <= kAhead * kThreads && a.tokens / (2 * per_cta) >= 608)
    per_cta *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.tokens + per_cta - 1) / per_cta), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T>, a, per_cta);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, RotaryType type, cudaStream_t st) {
  switch (type) {
    case RotaryType::kBf16: return launch<__nv_bfloat16>(a, st);
    case RotaryType::kFp16: return launch<__half>(a, st);
    default: return launch<float>(a, st);
  }
}

}  // namespace infllmv2
