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
// Bound by memory.  A thread has one item of one head, two 16-byte vectors, for
// kTokens tokens: half of the turned part apart (half of the rest, which is copied), so
// that neighbouring threads read neighbouring vectors, whole sectors at a time.  In the
// half layout the two turn into each other, interleaved each holds pairs of its own.
// All its loads go out before the CTA computes its tokens' angles.
//
// Measured (GB300): 16,384 tokens of 40 heads of 128, 50 us with a quarter of each head
// turned, 99% of the copy rate (fp32: 97 us, 102%); 64 tokens of 34 heads 1.9 us in a graph, 5.7 us a call
// from Python.  With two vectors side by side for a thread the first took 64 us.
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "packed.h"

namespace infllmv2 {

namespace {

constexpr int kThreads = 512;      // of a CTA at most
constexpr int kMaxTokens = 16;     // of a CTA

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

// What a thread does with every row: its two vectors and their (cos, sin).
struct Item {
  int at, second;           // elements from the head's first to the first vector, and on to the second
  int pairs, second_pairs;  // which vector's (cos, sin) (half layout: one of both); -1: copied
};

template <typename T>
__device__ __forceinline__ Item item_of(const RotaryArgs& a, int c) {
  constexpr int kN = Vec<T>::kN;
  const int turned = a.part / (2 * kN);
  Item r;
  if (c < turned) {
    r.at = c * kN;
    r.second = turned * kN;
    r.pairs = c;
    r.second_pairs = turned + c;
  } else {
    r.at = a.part + (c - turned) * kN;
    r.second = (a.dim - a.part) / 2;
    r.pairs = r.second_pairs = -1;
  }
  return r;
}

// blockDim: items of a head, heads, groups of kTokens tokens.
template <typename T, int kTokens>
__global__ void __launch_bounds__(kThreads, 2) rotary_kernel(const RotaryArgs a) {
  constexpr int kN = Vec<T>::kN;
  // [tokens of the CTA][pair of a vector][vector]: neighbouring threads' angles are neighbours.
  extern __shared__ float2 angles[];
  pdl_wait();
  pdl_trigger();
  const Item it = item_of<T>(a, threadIdx.x);
  const int group = a.interleaved ? kN / 2 : kN;   // pairs of a vector
  const int half = a.part / 2, vectors = half / group, per_cta = kTokens * blockDim.z;
  const int cta0 = blockIdx.x * per_cta, token0 = cta0 + threadIdx.z * kTokens;
  const int tokens = min(kTokens, a.tokens - token0);   // (of this thread)
  for (int h0 = 0; h0 < a.q_heads + a.k_heads; h0 += blockDim.y) {
    const int h = h0 + threadIdx.y;
    const bool is_q = h < a.q_heads, is_head = h < a.q_heads + a.k_heads;
    const PackedRows& in = is_q ? a.q_in : a.k_in;
    const PackedRows& out = is_q ? a.q_out : a.k_out;
    const int head = is_q ? h : h - a.q_heads;
    const T* x = static_cast<const T*>(in.x) + token0 * in.token + head * in.head + it.at;
    uint4 u[kTokens][2];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      if (is_head && k < tokens) {
        u[k][0] = *reinterpret_cast<const uint4*>(x + k * in.token);
        u[k][1] = *reinterpret_cast<const uint4*>(x + k * in.token + it.second);
      }
    }
    if (h0 == 0) {
      const int me = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x;
      const int n = min(per_cta, a.tokens - cta0) * half;
      for (int i = me; i < n; i += blockDim.x * blockDim.y * blockDim.z) {
        const int t = i / half, pair = i - t * half;
        angles[t * half + (pair % group) * vectors + pair / group] =
            turned(a.positions[cta0 + t], a.turns[pair], a.scale, a.transpose);
      }
      __syncthreads();
    }
    if (!is_head) continue;
    T* y = static_cast<T*>(out.x) + token0 * out.token + head * out.head + it.at;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      if (k >= tokens) break;
      if (it.pairs >= 0) {
        const float2* angle = angles + (threadIdx.z * kTokens + k) * half;
        float v[kN], w[kN];
        Vec<T>::get(u[k][0], v);
        Vec<T>::get(u[k][1], w);
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < kN; e += 2) {
            const float2 f = angle[e / 2 * vectors + it.pairs], g = angle[e / 2 * vectors + it.second_pairs];
            const float p = v[e], q = v[e + 1], r = w[e], s = w[e + 1];
            v[e] = p * f.x - q * f.y;
            v[e + 1] = p * f.y + q * f.x;
            w[e] = r * g.x - s * g.y;
            w[e + 1] = r * g.y + s * g.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const float2 f = angle[e * vectors + it.pairs];
            const float p = v[e], q = w[e];
            v[e] = p * f.x - q * f.y;
            w[e] = p * f.y + q * f.x;
          }
        }
        u[k][0] = Vec<T>::put(v);
        u[k][1] = Vec<T>::put(w);
      }
      *reinterpret_cast<uint4*>(y + k * out.token) = u[k][0];
      *reinterpret_cast<uint4*>(y + k * out.token + it.second) = u[k][1];
    }
  }
}

template <typename T, int kTokens>
cudaError_t launch_tokens(const RotaryArgs& a, int items, int heads, cudaStream_t st) {
  const int hy = std::min(heads, kThreads / items);
  // Groups of tokens: about 256 threads, within the angles' room.
  const int tz = std::max(1, std::min(256 / (items * hy), kMaxTokens / kTokens));
  const int per_cta = kTokens * tz;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.tokens + per_cta - 1) / per_cta), 1, 1);
  cfg.blockDim = dim3(items, hy, tz);
  cfg.dynamicSmemBytes = per_cta * (a.part / 2) * sizeof(float2);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T, kTokens>, a);
}

template <typename T>
cudaError_t launch(const RotaryArgs& a, cudaStream_t st) {
  // Items of a head: in place, what stays need not be copied.
  const int items = (a.in_place ? a.part : a.dim) / (2 * Vec<T>::kN);
  const int heads = a.q_heads + a.k_heads;
  // One token for a thread while the grid is small, where latency counts: 34 heads of 128, bf16, in place, in a
  // graph, one or four tokens: 1.9 or 3.0 us for 64 tokens, 4.1 or 4.6 for 963 (the border), 5.7 or 4.6 for 1500,
  // 61.7 or 43.6 for 16,384.
  return static_cast<long long>(a.tokens) * items * heads < 1 << 18 ? launch_tokens<T, 1>(a, items, heads, st)
                                                                    : launch_tokens<T, 4>(a, items, heads, st);
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
