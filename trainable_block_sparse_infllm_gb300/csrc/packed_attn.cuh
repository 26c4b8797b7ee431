// What the packed attention kernels share: which sequence and tile a CTA works
// on, 3D and 4D TMA loads, and packing of probabilities.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "packed_attn.h"
#include "tc.cuh"

namespace infllmv2 {
namespace packed {

// Asks once per device for the dynamic shared memory that a kernel needs.
class SharedMemory {
 public:
  template <typename Kernel>
  cudaError_t allow(Kernel kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && known) done_[dev].store(true, std::memory_order_relaxed);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> done_[kDevices] = {};
};

// A sequence's rows.  One whose starts are out of range or descend is empty.
struct Sequence {
  int q0, n_q, k0, n_k;
};

__device__ __forceinline__ Sequence sequence(const PackedAttnShape& s, int b, bool* bad) {
  Sequence r;
  r.q0 = s.q_starts[b];
  r.k0 = s.k_starts[b];
  const int q1 = s.q_starts[b + 1], k1 = s.k_starts[b + 1];
  if (r.q0 < 0 || q1 < r.q0 || q1 > s.Tq || r.k0 < 0 || k1 < r.k0 || k1 > s.Tk) {
    *bad = true;
    return {0, 0, 0, 0};
  }
  r.n_q = q1 - r.q0;
  r.n_k = k1 - r.k0;
  return r;
}

// Tiles of `step` tokens cut from the sequences' queries (of_keys: keys).  A
// tile's level is its index among the queries' tiles, or that of the keys' tiles
// counted from the last: either way causal work grows with it.
__device__ __forceinline__ int tile_count(const PackedAttnShape& s, int b, int step, bool of_keys, bool* bad) {
  const Sequence q = sequence(s, b, bad);
  return ((of_keys ? q.n_k : q.n_q) + step - 1) / step;
}

// The order of all tiles, for one warp that asks for one after another (i rising).  Up
// to 32 sequences: down the levels, sequence by sequence within one, so that what
// starts last has the least to do; the counts stay in registers.  More: the
// sequences in turn, each from its last tile down, walked once (there is nothing to
// balance among so many, and a search by level would read them all each time).
struct Walker {
  int count;     // of sequence base + lane
  int base;      // more than 32: the 32 sequences at hand, and the tiles before them
  int before;

  __device__ __forceinline__ void load(const PackedAttnShape& s, int step, bool of_keys, bool* bad) {
    const int b = base + static_cast<int>(threadIdx.x & 31);
    count = b < s.B ? tile_count(s, b, step, of_keys, bad) : 0;
  }

  __device__ __forceinline__ void start(const PackedAttnShape& s, int step, bool of_keys, bool* bad) {
    base = before = 0;
    load(s, step, of_keys, bad);
  }

  // All lanes: the sequence and level of tile i; false past the last one.
  __device__ __forceinline__ bool find(const PackedAttnShape& s, int i, int step, bool of_keys, int* b, int* level,
                                       bool* bad) {
    const int lane = threadIdx.x & 31;
    if (s.B > 32) {
      for (;;) {
        const int incl = warp_inclusive_scan(count), all = __shfl_sync(0xffffffffu, incl, 31);
        if (i < before + all) {
          const unsigned mask = __ballot_sync(0xffffffffu, i < before + incl);
          const int at = __ffs(mask) - 1;
          *b = base + at;
          *level = __shfl_sync(0xffffffffu, incl, at) - 1 - (i - before);   // from its last tile down
          return true;
        }
        before += all;
        base += 32;
        if (base >= s.B) return false;
        load(s, step, of_keys, bad);
      }
    }
    auto at_least = [&](int t) {   // tiles of level t and up
      return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(max(count - t, 0))));
    };
    if (at_least(0) <= i) return false;
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, count);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at_least(mid) > i) lo = mid; else hi = mid;
    }
    // Among the sequences that have a tile of this level, number `rank`.
    const int rank = i - at_least(lo + 1);
    const unsigned mask = __ballot_sync(0xffffffffu, count > lo);
    const unsigned here = __ballot_sync(0xffffffffu, ((mask >> lane) & 1) && __popc(mask & ((1u << lane) - 1)) == rank);
    *b = __ffs(here) - 1;
    *level = lo;
    return true;
  }
};

// Tile `i` of the same order, once, for a whole CTA; false past the last one.  (More
// than 32 sequences: every thread sums a run of them.)  `scratch`: 40 ints of shared
// memory.  The CTA that has tile 0 flags bad starts.
__device__ __forceinline__ bool find_tile(const PackedAttnShape& s, int i, int step, bool of_keys, int* scratch, int* b,
                                          int* level) {
  const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x / 32;
  bool bad = false;
  int* found = scratch + 32;   // whether, sequence, level
  if (tid == 0) found[0] = 0;
  if (s.B <= 32) {
    __syncthreads();
    if (tid < 32) {
      Walker w;
      w.start(s, step, of_keys, &bad);
      int at = 0, its = 0;
      const bool ok = w.find(s, i, step, of_keys, &at, &its, &bad);
      if (lane == 0) {
        found[0] = ok;
        found[1] = at;
        found[2] = its;
      }
    }
  } else {
    const int per = (s.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int b0 = min(tid * per, s.B), b1 = min(b0 + per, s.B);
    int mine = 0;
    for (int x = b0; x < b1; ++x) mine += tile_count(s, x, step, of_keys, &bad);
    const int incl = warp_inclusive_scan(mine);
    if (lane == 31) scratch[tid >> 5] = incl;
    __syncthreads();
    int first = incl - mine;   // the tiles before this thread's
    for (int w = 0; w < warps; ++w) first += w < (tid >> 5) ? scratch[w] : 0;
    if (i >= first && i < first + mine) {
      for (int x = b0; x < b1; ++x) {
        const int n = tile_count(s, x, step, of_keys, &bad);
        if (i < first + n) {
          found[0] = 1;
          found[1] = x;
          found[2] = n - 1 - (i - first);
          break;
        }
        first += n;
      }
    }
  }
  if (bad && i == 0) atomicOr(s.status, kStatusBadKvLen);
  __syncthreads();
  *b = found[1];
  *level = found[2];
  return found[0] != 0;
}

// Whether all `threads` that meet at barrier `bar` say so (all of the first eight warps).
// They go on to the next unit together or not at all: a warp whose wait gave up would
// leave the others at a barrier.
__device__ __forceinline__ bool all_agree(bool mine, int bar = 1, int threads = 256) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(mine ? 1u : 0u), "r"(bar), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// The thread's stores have read shared memory; have been done.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (kFp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kFp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 32 consecutive 16-bit values (16 words) to global memory: in whole 32-byte sectors
// where `wide` (every row starts on one), which halves the store instructions.
__device__ __forceinline__ void store_row(uint16_t* to, const uint32_t (&w)[16], bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 16 * i), "r"(w[8 * i]),
                   "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                   "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(to + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// Whether every row of a tensor starts on 32 bytes.
__device__ __forceinline__ bool wide_rows(const void* x, const PackedStride& st) {
  return reinterpret_cast<uint64_t>(x) % 32 == 0 && st.token % 16 == 0 && st.head % 16 == 0;
}

template <bool kFp16>
constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
  return kFp16 ? tc::idesc_fp16(M, N, a_mn, b_mn) : tc::idesc_bf16(M, N, a_mn, b_mn);
}

// One lane of a converged warp, in a form from which the compiler knows that the
// rest of the warp's work stays uniform.  Products are issued so: the whole warp
// runs the issuer's loop, which keeps descriptors and addresses in uniform
// registers, where tcgen05.mma takes them from; in a branch of lane 0 each product
// moved them there first.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// The warp's index, uniform for the compiler too.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

// A converged warp that issued products: waits until all of them are done.
__device__ __forceinline__ void products_end(uint64_t* bar, bool issuer, uint32_t* status) {
  if (issuer) tc::commit(bar);
  __syncwarp();
  mbar_wait(bar, 0, status);
}

// One product of a 128-row A by D-step K extent: both operands K-major tiles of
// [rows][kD] in boxes of 64 columns x 128 rows.
template <int kD>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id) {
#pragma unroll
  for (int k = 0; k < kD / 16; ++k) {
    const uint64_t off = static_cast<uint64_t>(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
    tc::mma_ss(d_tmem, a + off, b + off, id, k > 0 ? 1u : 0u);
  }
}

// The same with A in tensor memory, two values to a 32-bit column.
template <int kD>
__device__ __forceinline__ void mma_rows_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id) {
#pragma unroll
  for (int k = 0; k < kD / 16; ++k) {
    const uint64_t off = static_cast<uint64_t>(((k >> 2) * 16384 + (k & 3) * 32) >> 4);
    tc::mma_ts(d_tmem, a_tmem + 8 * k, b + off, id, k > 0 ? 1u : 0u);
  }
}

__device__ __forceinline__ void st_words(uint32_t addr, const uint32_t (&w)[32]) { tc::st32(addr, w); }
__device__ __forceinline__ void st_words(uint32_t addr, const uint32_t (&w)[16]) { tc::st16(addr, w); }

// D += A B over 128 rows of B: A [128 x 128] two to a 32-bit column of tensor
// memory, the columns of its second half kHalf behind the first's, B the
// [128][kD] tile read along its rows (MN-major).
template <int kHalf = 32>
__device__ __forceinline__ void mma_cols(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, bool accumulate) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    tc::mma_ts(d_tmem, a_tmem + kHalf * (k >> 2) + 8 * (k & 3), b + static_cast<uint64_t>((k * 2048) >> 4), id,
               accumulate || k > 0 ? 1u : 0u);
}

__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr) { return tc::sdesc_sw128(saddr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_cols(uint32_t saddr) { return tc::sdesc_sw128(saddr, 16384, 1024); }

// One warp: clears rows [from, 128) of a [128][kD] tile, so that a zero
// probability never multiplies what lies behind a sequence's end.
template <int kD>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from) {
  const int lane = threadIdx.x & 31;
  for (int e = lane; e < (128 - from) * (kD / 8); e += 32) {
    const int row = from + e / (kD / 8), c = e % (kD / 8);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * 16384 + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Two warps (half 0 and 1): looks through the 64 rows [64 half, 64 half + 64) of a
// [128][kD] tile.  Rows from `valid` on are cleared; so are the ones with an
// infinity or NaN, and their bits set in flags[0 .. 3].
template <int kD, bool kFp16>
__device__ __forceinline__ void check_rows(uint8_t* tile, int half, int valid, uint32_t* flags) {
  constexpr uint32_t kExponent = kFp16 ? 0x7c007c00u : 0x7f807f80u;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int row = 64 * half + 32 * k + lane;
    uint8_t* at = tile + row * 128;
    uint32_t most = 0u;   // the largest exponent of each 16-bit lane
#pragma unroll
    for (int c = 0; c < kD / 8; ++c) {   // (in an order without bank conflicts)
      const uint4 u = *reinterpret_cast<const uint4*>(at + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
      most = __vmaxu2(__vmaxu2(most, __vmaxu2(u.x & kExponent, u.y & kExponent)),
                      __vmaxu2(u.z & kExponent, u.w & kExponent));
    }
    const bool odd = ((most ^ kExponent) & 0xffffu) == 0u || ((most ^ kExponent) >> 16) == 0u;
    const uint32_t mask = __ballot_sync(0xffffffffu, odd && row < valid);
    if (lane == 0) flags[2 * half + k] = mask;
    if (odd || row >= valid) {
#pragma unroll
      for (int c = 0; c < kD / 8; ++c)
        *reinterpret_cast<uint4*>(at + (c >> 3) * 16384 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Where float4 c4 of row `row` lies in a table of fp32 rows of kD in shared
// memory: a warp's 32 rows meet different banks.
template <int kD>
__device__ __forceinline__ int swizzled(int row, int c4) {
  return row * (kD / 4) + (c4 ^ (row & (kD / 4 - 1)));
}

__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

}  // namespace packed
}  // namespace infllmv2
