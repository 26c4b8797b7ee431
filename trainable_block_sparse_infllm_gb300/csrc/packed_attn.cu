// Causal attention over packed sequences: out = softmax(scale q k^T) v.
//
// The group's heads share their keys, so the rows of a tile are (token, head of
// the group) pairs, token by token: 128 / G tokens of G heads fill a 128-row
// product whatever the group, and a short prompt wastes few rows.  Online softmax
// in base 2: with m >= the row's scores (up to 2^8, see below), x = sum 2^(z - m) v
// and l = sum 2^(z - m) are kept per row, and out = x / l.  One pass over the keys.
//
// A CTA takes two adjacent tiles (256 rows) of one sequence and KV head, and walks
// the keys in tiles of 128 up to the last one that a row attends:
//   warps 0-3, 4-7  softmax of the first and second tile; a thread is a row.  S
//              comes from tensor memory, P (16 bits) goes back over it, which makes
//              it the A operand of P V.  The running maximum moves only when it
//              grows by more than 2^8, which is rare, so x is rarely rescaled.
//   warp 8     issues the products of both tiles in turn: while one tile's softmax
//              runs, the other's P V and next Q K^T keep the tensor cores busy.
//              P V of key tile j before S of j + 1 in issue order: S overwrites P.
//   warp 9     TMA: both Q tiles, then K_0, V_0, K_1, V_1, ... through a ring.
//   warps 10, 11  look through the V tiles that some row attends in part (at most
//              three): a zero probability must meet no infinity or NaN.  Rows behind
//              the sequence's end are cleared; a row of the sequence that holds one is
//              cleared too, and the rows that attend it add it at the end, one by one.
// Few queries against many keys (drafted tokens, a short chunk after a long past)
// leave most SMs without a unit: its key tiles are then divided over a cluster,
// whose CTAs join their (m, l, x) through distributed shared memory.
// Tensor memory: two S / P buffers of 128 columns and two accumulators of D.
#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "packed_attn.cuh"

namespace infllmv2 {

namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kCheckWarp = 10;
constexpr int kMaxPartial = 3;   // V tiles that rows attend in part: 256 queries' own keys lie in three tiles at most
constexpr int kRing = 163840;   // bytes of the K / V ring
constexpr float kLazy = 8.0f;   // log2 of how far scores may pass the running maximum
// log2 of P at the running maximum.  fp16 loses what is below 2^-25, which many
// small probabilities could add up to; its largest value leaves room for 2^(6 + 8).
template <bool kFp16>
constexpr float kTop = kFp16 ? 6.0f : 0.0f;
constexpr uint32_t kColO = 256;

template <int kD>
struct Layout {
  static constexpr int kTile = kD / 64 * 16384;   // 128 rows of kD
  static constexpr int kStages = kRing / kTile;
  static constexpr int kBars = 2 * kTile + kRing;
  // Barriers: Q of each tile, ring full and empty, V tiles attended in part, before and after they were
  // looked through, then S, P and O of each tile.
  static constexpr int kQFull = 0, kFull = 2, kEmpty = kFull + kStages, kPartial = kEmpty + kStages,
                       kChecked = kPartial + kMaxPartial, kSFull = kChecked + kMaxPartial, kPFull = kSFull + 2,
                       kODone = kPFull + 2, kNumBars = kODone + 2;
  static constexpr int kScratch = kBars + 8 * kNumBars;
  static constexpr int kFlags = kScratch + 32;   // [kMaxPartial][4]: rows of those tiles that were cleared
  static constexpr int kBytes = kFlags + kMaxPartial * 16 + 1024;   // and slack to align the tiles
};

template <int kD, bool kFp16>
__device__ __forceinline__ float dot(const uint16_t* q, const uint16_t* k) {
  float z = 0.f;
#pragma unroll 1
  for (int i = 0; i < kD / 2; ++i) {
    const float2 a = packed::unpack2<kFp16>(reinterpret_cast<const uint32_t*>(q)[i]);
    const float2 b = packed::unpack2<kFp16>(reinterpret_cast<const uint32_t*>(k)[i]);
    z = fmaf(a.x, b.x, fmaf(a.y, b.y, z));
  }
  return z;
}

// kSplit: a unit's key tiles are divided over a cluster of `ctas` CTAs.
template <int kD, bool kFp16, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnIn in,
                       const PackedAttnOut o, const int ctas) {
  using L = Layout<kD>;
  constexpr int kTile = L::kTile, kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int* scratch = reinterpret_cast<int*>(smem + L::kScratch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 4);
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + L::kFlags);
  uint8_t* ring = smem + 2 * kTile;
  // kSplit, at the end, over the ring: x of this CTA's 256 rows, their (m, l), and the weights of the share it joins.
  float4* parts = reinterpret_cast<float4*>(ring);
  float2* sums = reinterpret_cast<float2*>(ring + 256 * kD * 4);
  float* weights = reinterpret_cast<float*>(sums + 256);   // [256 / ctas][16]
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;

  pdl_wait();
  pdl_trigger();
  const int tile_tokens = packed_tile_tokens(s.G);
  const int rank = kSplit ? static_cast<int>(blockIdx.x) % ctas : 0;
  const int index = kSplit ? static_cast<int>(blockIdx.x) / ctas : static_cast<int>(blockIdx.x);
  const int h = index % s.Hkv;
  int b, unit;
  if (!packed::find_tile(s, index / s.Hkv, 2 * tile_tokens, false, scratch, &b, &unit)) return;   // the whole cluster
  bool bad = false;
  const packed::Sequence seq = packed::sequence(s, b, &bad);
  const int t0 = unit * 2 * tile_tokens;   // the CTA's first query
  const int before = seq.n_k - seq.n_q;    // query t attends keys 0 .. before + t
  // Key tiles of each half: up to its last query's own key.
  int n_tiles[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = t0 + x * tile_tokens, last = min(first + tile_tokens, seq.n_q) - 1;
    n_tiles[x] = last < first ? 0 : (max(before + last + 1, 0) + 127) / 128;
  }
  int j0 = 0;   // this CTA's first key tile; all tile indexes below count from it
  if (kSplit) {
    const int all = max(n_tiles[0], n_tiles[1]);
    j0 = rank * all / ctas;
    const int j1 = (rank + 1) * all / ctas;
    n_tiles[0] = max(min(n_tiles[0], j1) - j0, 0);
    n_tiles[1] = max(min(n_tiles[1], j1) - j0, 0);
  }
  const int n = max(n_tiles[0], n_tiles[1]);
  const int partial = max(before + t0 + 1, 0) / 128 - j0;   // the first key tile that some row attends in part
  const int looked = max(partial, 0);                        // the first of this CTA's that is looked through

  if (tid == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool by_warps = i == L::kPFull || i == L::kPFull + 1;
      mbar_init(&bars[i], by_warps ? 4 : i >= L::kChecked && i < L::kChecked + kMaxPartial ? 2 : 1);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    packed::regs_down<72>();
    if (warp == kTmaWarp && n > 0) {
      // ------------------------------------------------------------ loads
      int issued = 0;
      if (lane == 0) {
        const uint32_t row_bytes = tile_tokens * s.G * kD * 2;
        for (int x = 0; x < 2; ++x) {
          if (n_tiles[x] == 0) continue;
          mbar_arrive_expect_tx(&bars[L::kQFull + x], row_bytes);
          for (int c = 0; c < kD / 64; ++c)
            packed::tma_load_4d(smem_u32(smem + x * kTile + c * 16384), &maps.q, c * 64, 0, h,
                                seq.q0 + t0 + x * tile_tokens, &bars[L::kQFull + x]);
        }
        for (; issued < 2 * n; ++issued) {
          const int st = issued % kStages;
          if (issued >= kStages && !mbar_wait(&bars[L::kEmpty + st], (issued / kStages - 1) & 1, s.status)) break;
          // A V tile to be looked through lands on a barrier of its own; its stage's only counts the turn.
          const int j = issued >> 1;
          uint64_t* bar = &bars[L::kFull + st];
          if ((issued & 1) && j >= partial) {
            mbar_arrive(bar);
            bar = &bars[L::kPartial + j - partial];
          }
          mbar_arrive_expect_tx(bar, kTile);
          for (int c = 0; c < kD / 64; ++c)
            packed::tma_load_3d(smem_u32(ring + st * kTile + c * 16384), issued & 1 ? &maps.v : &maps.k, c * 64,
                                seq.k0 + (j0 + j) * 128, h, bar);
        }
      }
      issued = __shfl_sync(0xffffffffu, issued, 0);
      // The CTA outlives its copies, also after a wait that gave up.  (The last copy
      // of a stage is its barrier's newest phase here.)
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait(&bars[L::kFull + i % kStages], (i / kStages) & 1, s.status);
      for (int j = looked; 2 * j + 1 < issued; ++j) mbar_wait(&bars[L::kPartial + j - partial], 0, s.status);
      for (int x = 0; x < 2; ++x)
        if (n_tiles[x] > 0) mbar_wait(&bars[L::kQFull + x], 0, s.status);
    } else if (warp >= kCheckWarp) {
      // ---------------------------------------------- V attended in part
      for (int j = looked; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars[L::kPartial + j - partial], 0, s.status))) break;
        packed::check_rows<kD, kFp16>(ring + (2 * j + 1) % kStages * kTile, warp - kCheckWarp,
                                      seq.n_k - (j0 + j) * 128, flags + 4 * (j - partial));
        if (lane == 0) mbar_arrive(&bars[L::kChecked + j - partial]);
      }
    } else if (warp == kMmaWarp && n > 0) {
      // --------------------------------------------------------- products
      constexpr uint32_t kIdS = packed::idesc<kFp16>(128, 128, 0, 0);
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t q_desc = packed::desc_rows(smem_u32(smem));
      const uint64_t k_desc = packed::desc_rows(smem_u32(ring));
      const uint64_t v_desc = packed::desc_cols(smem_u32(ring));
      const bool issuer = packed::elect_one();
      bool ok = true;
      auto wait = [&](int bar, int phase) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
        tc::fence_after_sync();
      };
      auto scores = [&](int x, int j) {   // S of half x and key tile j
        if (issuer) {
          packed::mma_rows<kD>(tmem + x * 128, q_desc + ((x * kTile) >> 4),
                               k_desc + (((2 * j) % kStages * kTile) >> 4), kIdS);
          tc::commit(&bars[L::kSFull + x]);
        }
        __syncwarp();
      };
      wait(L::kFull, 0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (n_tiles[x] == 0) continue;
        wait(L::kQFull + x, 0);
        if (ok) scores(x, 0);
      }
      if (ok && issuer) tc::commit(&bars[L::kEmpty]);
      __syncwarp();
      for (int j = 0; j < n && ok; ++j) {
        const int vi = 2 * j + 1, ki = 2 * j + 2;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (j >= n_tiles[x] || !ok) continue;
          if (j < partial) {
            wait(L::kFull + vi % kStages, vi / kStages);
          } else {
            wait(L::kChecked + j - partial, 0);
          }
          wait(L::kPFull + x, j);
          if (!ok) continue;
          if (issuer)
            packed::mma_cols(tmem + kColO + x * kD, tmem + x * 128, v_desc + ((vi % kStages * kTile) >> 4), kIdO,
                             j > 0);
          __syncwarp();
          if (j + 1 < n_tiles[x]) {
            wait(L::kFull + ki % kStages, ki / kStages);
            if (ok) scores(x, j + 1);
          } else {
            if (issuer) tc::commit(&bars[L::kODone + x]);
            __syncwarp();
          }
        }
        if (ok && issuer) {
          tc::commit(&bars[L::kEmpty + vi % kStages]);
          if (j + 1 < n) tc::commit(&bars[L::kEmpty + ki % kStages]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    packed::regs_up<216>();
    const int x = warp >> 2;
    const int r = tid & 127;
    const int token = t0 + x * tile_tokens + r / s.G;   // in the sequence
    const bool active = r < tile_tokens * s.G && token < seq.n_q;
    const int limit = active ? before + token + 1 - j0 * 128 : 0;   // keys 0 .. limit - 1, from tile j0 on
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + x * 128, o_addr = lane_addr + kColO + x * kD;
    const int mine = x ? n_tiles[1] : n_tiles[0];
    // Key tiles before this one need no mask in any row of the warp.
    const int whole = static_cast<int>(__reduce_min_sync(0xffffffffu, active ? max(limit, 0) : 0x7fffffff)) / 128;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < mine; ++j) {
      // (A warp whose wait gave up goes on without waiting; the status word has the error.)
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kSFull + x], j & 1, s.status));
      tc::fence_after_sync();
      uint32_t z[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
      tc::wait_ld();
      if (j >= whole) {
        const int keep = limit - j * 128;
#pragma unroll
        for (int i = 0; i < 128; ++i) z[i] = i < keep ? z[i] : 0xff800000u;   // -inf
      }
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = __uint_as_float(z[i]);
#pragma unroll
      for (int i = 4; i < 128; ++i) t[i & 3] = fmaxf(t[i & 3], __uint_as_float(z[i]));
      const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * s.scale2;
      // S of tile j was issued after P V of tile j - 1, so x may be rescaled now.
      const bool move = top > m + kLazy;
      if (__any_sync(0xffffffffu, move)) {
        const float alpha = move ? fast_exp2(m - top) : 1.f;   // 0 the first time
        if (move) {
          m = top;
          l *= alpha;
        }
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t w[32];
            tc::ld32(o_addr + 32 * c, w);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
            tc::st32(o_addr + 32 * c, w);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m - kTop<kFp16>;   // (a row that attends no key yet)
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = fast_exp2(fmaf(__uint_as_float(z[64 * c + 2 * i]), s.scale2, -base));
          const float d = fast_exp2(fmaf(__uint_as_float(z[64 * c + 2 * i + 1]), s.scale2, -base));
          sum[0] += a;
          sum[1] += d;
          p[i] = packed::pack2<kFp16>(a, d);
        }
        tc::st32(s_addr + 32 * c, p);
      }
      l += sum[0] + sum[1];
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kPFull + x]);
    }
    // (kSplit: of both halves, whose products read the ring that is written next.)
    for (int y = 0; y < 2; ++y)
      if ((kSplit || y == x) && n_tiles[y] > 0 && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kODone + y], 0, s.status));
    tc::fence_after_sync();
    // ---- x / l and the log sum ----
    const float inv = 1.f / l;
    const int head = h * s.G + r % s.G;
    const long long row = seq.q0 + token;
    const bool none = before + token < 0;   // the row attends no key
    uint16_t* out = static_cast<uint16_t*>(o.out) + row * o.st.token + head * o.st.head;
    const uint16_t* q_row = static_cast<const uint16_t*>(in.q) + row * in.q_st.token + head * in.q_st.head;
    uint32_t cleared = 0u;   // P V of the last tile is done, so every tile has been looked through
    for (int j = looked; j < mine && ok; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kChecked + j - partial], 0, s.status));
      for (int i = 0; i < 4; ++i) cleared |= flags[4 * (j - partial) + i];
    }
#pragma unroll 1
    for (int c = 0; c < kD / 32; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (mine > 0) {
        tc::ld32(o_addr + 32 * c, w);
        tc::wait_ld();
      }
      if (cleared && active) {
#pragma unroll 1
        for (int key = looked * 128; key < min(limit, mine * 128); ++key) {
          const int bit = key - partial * 128;
          if (!((flags[bit >> 5] >> (bit & 31)) & 1)) continue;
          const long long at = seq.k0 + j0 * 128 + key;
          const uint16_t* k_row = static_cast<const uint16_t*>(in.k) + at * in.k_st.token + h * in.k_st.head;
          const uint16_t* v_row = static_cast<const uint16_t*>(in.v) + at * in.v_st.token + h * in.v_st.head + 32 * c;
          const float p = fast_exp2(fmaf(dot<kD, kFp16>(q_row, k_row), s.scale2, kTop<kFp16> - m));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 v = packed::unpack2<kFp16>(reinterpret_cast<const uint32_t*>(v_row)[i]);
            w[2 * i] = __float_as_uint(fmaf(p, v.x, __uint_as_float(w[2 * i])));
            w[2 * i + 1] = __float_as_uint(fmaf(p, v.y, __uint_as_float(w[2 * i + 1])));
          }
        }
      }
      if (kSplit) {   // into this CTA's ring, which is free now
#pragma unroll
        for (int i = 0; i < 8; ++i)
          parts[packed::swizzled<kD>(x * 128 + r, 8 * c + i)] =
              make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]), __uint_as_float(w[4 * i + 2]),
                          __uint_as_float(w[4 * i + 3]));
      } else if (active) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = !none ? packed::pack2<kFp16>(__uint_as_float(w[8 * i + 2 * e]) * inv,
                                                    __uint_as_float(w[8 * i + 2 * e + 1]) * inv)
                             : 0u;
          *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    }
    if (kSplit) {
      sums[x * 128 + r] = make_float2(m, l);
    } else if (active && o.lse) {
      o.lse[row * (s.Hkv * s.G) + head] =
          !none ? (m - kTop<kFp16> + fast_log2(l)) * 0.69314718055994531f : -INFINITY;
    }
  }
  if (kSplit) {
    // ---- each CTA joins its share of the rows over the cluster: with M the largest m,
    // out = sum 2^(m - M) x / sum 2^(m - M) l ----
    __syncwarp();
    cluster_sync();
    if (warp < 8) {   // (the others have given registers away)
      const int share = 256 / ctas, row0 = rank * share;
      for (int e = tid; e < share; e += 256) {   // a row: its weights, over l, and log sum
        const int row = row0 + e, rr = row & 127;
        const int token = t0 + (row >> 7) * tile_tokens + rr / s.G;
        float top = -INFINITY, l = 0.f;
        for (int c = 0; c < ctas; ++c) top = fmaxf(top, ld_dsmem_f32(dsmem_addr(&sums[row].x, c)));
        const float base = top == -INFINITY ? 0.f : top;
        for (int c = 0; c < ctas; ++c) {
          const float2 ml = ld_dsmem_f32x2(dsmem_addr(&sums[row], c));
          const float weight = fast_exp2(ml.x - base);
          weights[e * 16 + c] = weight;
          l = fmaf(weight, ml.y, l);
        }
        const bool active = rr < tile_tokens * s.G && token < seq.n_q, none = before + token < 0;
        for (int c = 0; c < ctas; ++c) weights[e * 16 + c] *= none ? 0.f : 1.f / l;
        if (active && o.lse)
          o.lse[static_cast<long long>(seq.q0 + token) * (s.Hkv * s.G) + h * s.G + rr % s.G] =
              !none ? (top - kTop<kFp16> + fast_log2(l)) * 0.69314718055994531f : -INFINITY;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int e = tid; e < share * (kD / 4); e += 256) {
        const int local = e / (kD / 4), c4 = e % (kD / 4), row = row0 + local, rr = row & 127;
        const int token = t0 + (row >> 7) * tile_tokens + rr / s.G;
        if (rr >= tile_tokens * s.G || token >= seq.n_q) continue;
        const float4* mine = parts + packed::swizzled<kD>(row, c4);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll 4
        for (int c = 0; c < ctas; ++c) {
          const float weight = weights[local * 16 + c];
          const float4 v = packed::ld_dsmem_f32x4(dsmem_addr(mine, c));
          sum.x = fmaf(weight, v.x, sum.x);
          sum.y = fmaf(weight, v.y, sum.y);
          sum.z = fmaf(weight, v.z, sum.z);
          sum.w = fmaf(weight, v.w, sum.w);
        }
        uint16_t* out = static_cast<uint16_t*>(o.out) + static_cast<long long>(seq.q0 + token) * o.st.token +
                        (h * s.G + rr % s.G) * o.st.head + 4 * c4;
        *reinterpret_cast<uint2*>(out) =
            make_uint2(packed::pack2<kFp16>(sum.x, sum.y), packed::pack2<kFp16>(sum.z, sum.w));
      }
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while another reads its ring
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

constexpr int kMaxSplit = 16;

// Clusters of `ctas` CTAs that the current device runs at once (looked up once per device).
template <int kD, bool kFp16>
int clusters_at_once(int ctas) {
  static std::mutex mu;
  static int known[64][5];   // by log2 of ctas; what it is plus 1
  int dev = 0, i = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  while ((1 << i) < ctas) ++i;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev][i]) {
    const auto kernel = packed_attn_kernel<kD, kFp16, true>;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Layout<kD>::kBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<kD>::kBytes) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[dev][i] = n + 1;
  }
  return known[dev][i] - 1;
}

// CTAs per unit.  Units that fill half the SMs, or have few keys, are not split: a
// CTA's start and the join cost what a few key tiles do.  The lengths are on the
// device, so this goes by the average sequence.
template <int kD, bool kFp16>
int split(const PackedAttnShape& s, int step) {
  const long long each = (s.Tq + s.B - 1) / s.B;
  const long long units = (each + step - 1) / step * s.B * s.Hkv;
  const long long tiles = s.Tk / s.B / 128;
  if (2 * units > device_sm_count()) return 1;
  int ctas = kMaxSplit;
  while (ctas > 1 && (tiles / ctas < 4 || clusters_at_once<kD, kFp16>(ctas) < units)) ctas /= 2;
  return ctas;
}

template <int kD, bool kFp16>
cudaError_t launch(const PackedAttnShape& s, const PackedAttnMaps& maps, const PackedAttnIn& in, const PackedAttnOut& o,
                   cudaStream_t st) {
  // Units of two tiles: at most one partly filled one per sequence.
  const int step = 2 * packed_tile_tokens(s.G);
  const long long units = std::min<long long>(s.Tq, static_cast<long long>(s.Tq) / step + s.B);
  const int ctas = split<kD, kFp16>(s, step);
  const auto kernel = ctas > 1 ? packed_attn_kernel<kD, kFp16, true> : packed_attn_kernel<kD, kFp16, false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<kD>::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * s.Hkv * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<kD>::kBytes;
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
  return cudaLaunchKernelEx(&cfg, kernel, maps, s, in, o, ctas);
}

}  // namespace

cudaError_t launch_packed_attn(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                               const PackedAttnIn& in, const PackedAttnOut& o, cudaStream_t st) {
  if (D == 128) return fp16 ? launch<128, true>(s, maps, in, o, st) : launch<128, false>(s, maps, in, o, st);
  return fp16 ? launch<64, true>(s, maps, in, o, st) : launch<64, false>(s, maps, in, o, st);
}

}  // namespace infllmv2
