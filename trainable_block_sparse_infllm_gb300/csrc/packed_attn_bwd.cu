// Gradient of causal attention over packed sequences.  With z = scale q.k and the
// forward pass's lse,
//     P = exp(z - lse),  D = rowsum(dout * out),  dS = P * (dout . v - D),
//     dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout.
//
// Two kernels, so that every sum has one owner and one order: dq walks the keys
// for a tile of query rows, dk and dv walk the query rows for a tile of keys.
// Scores and dout . v are computed in both, seven products in all instead of the
// five that one kernel with atomic sums of dq would need.  Rows are (token, head
// of the group) pairs as in the forward pass, so a group's heads sum into their
// keys' gradients inside the product.
//
// D from the rounded `out` is off by up to half a step of |out| |dout|.  Where a row
// attends few keys, dout . v - D is a small difference of such numbers and the
// error shows in dq and dk (2% of them for documents of 7 tokens in bf16, against
// 0.3% past a thousand).  So rows of up to kExactTiles tiles of keys walk them twice
// and sum D = sum P (dout . v) first (one tile: it is all in registers); and every
// row ends with sum P (dout . v - D), which is what its D lacks, before D goes to
// the dk and dv kernel.
//
// In both kernels the operand that the second products take from the scores, dS (dq), or
// P^T and dS^T (dk, dv: scores are computed transposed, keys in rows), is the A
// operand in tensor memory: no product's input passes through shared memory but
// the tiles that TMA brought.  Two warpgroups share a tile's columns.
#include <algorithm>

#include "kernels.h"
#include "packed_attn.cuh"

namespace infllmv2 {

namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kRowsWarp = 10;
constexpr float kLog2e = 1.4426950408889634f;
// log2 of what P is multiplied by on its way to dv.  A probability of a long row is
// among fp16's subnormal numbers, where it would lose bits.
template <bool kFp16>
constexpr int kUp = kFp16 ? 8 : 0;
// Rows that attend at most so many tiles of keys get D from their scores.
constexpr int kExactTiles = 8;

// ------------------------------------------------------------------- dq ----

template <int kD>
struct DqLayout {
  static constexpr int kTile = kD / 64 * 16384;
  static constexpr int kStages = 163840 / kTile;
  static constexpr int kRing = 2 * kTile;   // Q and dout before it
  static constexpr int kBars = kRing + kStages * kTile;
  static constexpr int kQFull = 0, kFull = 1, kEmpty = kFull + kStages, kCleared = kEmpty + kStages,
                       kSFull = kCleared + 1, kDpFull = kSFull + 1, kFree = kDpFull + 1, kDsFull = kFree + 1,
                       kDqDone = kDsFull + 2, kNumBars = kDqDone + 2;
  static constexpr int kScratch = kBars + 8 * kNumBars;
  static constexpr int kSum = kScratch + 32;   // [2][128]: sums over the halves of a row
  static constexpr int kBytes = kSum + 1024 + 1024;
};
// Tensor memory: S, dout . v, two buffers of dS, dq.
constexpr uint32_t kDqS = 0, kDqDp = 128, kDqDs = 256, kDqAcc = 384;

template <int kD, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnGrads g) {
  using L = DqLayout<kD>;
  constexpr int kTile = L::kTile, kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int* scratch = reinterpret_cast<int*>(smem + L::kScratch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 4);
  uint8_t* ring = smem + L::kRing;
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;

  pdl_wait();
  pdl_trigger();
  const int tile_tokens = packed_tile_tokens(s.G);
  const int h = static_cast<int>(blockIdx.x) % s.Hkv;
  int b, tile;
  if (!packed::find_tile(s, static_cast<int>(blockIdx.x) / s.Hkv, tile_tokens, false, scratch, &b, &tile)) return;
  bool bad = false;
  const packed::Sequence seq = packed::sequence(s, b, &bad);
  const int t0 = tile * tile_tokens;
  const int before = seq.n_k - seq.n_q;
  const int last = min(t0 + tile_tokens, seq.n_q) - 1;
  const int n = (max(before + last + 1, 0) + 127) / 128;   // key tiles
  const bool clears = n * 128 > seq.n_k;
  const bool exact = n <= kExactTiles;
  const int steps = exact && n > 1 ? 2 * n : n;   // walks the keys twice, or once
  const int back = steps - n;                     // the first step of the walk that sums dq

  if (tid == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.dout);
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(&bars[i], i == L::kFree || i == L::kDsFull || i == L::kDsFull + 1 ? 8 : 1);
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
      int issued = 0;   // K_0, V_0, K_1, V_1, ...
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[L::kQFull], 2 * tile_tokens * s.G * kD * 2);
        for (int c = 0; c < kD / 64; ++c) {
          packed::tma_load_4d(smem_u32(smem + c * 16384), &maps.q, c * 64, 0, h, seq.q0 + t0, &bars[L::kQFull]);
          packed::tma_load_4d(smem_u32(smem + kTile + c * 16384), &maps.dout, c * 64, 0, h, seq.q0 + t0,
                              &bars[L::kQFull]);
        }
        for (; issued < 2 * steps; ++issued) {
          const int st = issued % kStages;
          if (issued >= kStages && !mbar_wait(&bars[L::kEmpty + st], (issued / kStages - 1) & 1, s.status)) break;
          mbar_arrive_expect_tx(&bars[L::kFull + st], kTile);
          for (int c = 0; c < kD / 64; ++c)
            packed::tma_load_3d(smem_u32(ring + st * kTile + c * 16384), issued & 1 ? &maps.v : &maps.k, c * 64,
                                seq.k0 + (issued >> 1) % n * 128, h, &bars[L::kFull + st]);
        }
      }
      issued = __shfl_sync(0xffffffffu, issued, 0);
      // The last copy of each stage: here its phase is the barrier's newest.  The
      // CTA outlives its copies, also after a wait that gave up.
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait(&bars[L::kFull + i % kStages], (i / kStages) & 1, s.status);
      if (clears && issued == 2 * steps) {   // K rows behind the sequence: they meet dS = 0
        packed::clear_rows<kD>(ring + (2 * steps - 2) % kStages * kTile, seq.n_k - (n - 1) * 128);
        if (lane == 0) mbar_arrive(&bars[L::kCleared]);
      }
      mbar_wait(&bars[L::kQFull], 0, s.status);
    } else if (warp == kMmaWarp && n > 0) {
      constexpr uint32_t kIdS = packed::idesc<kFp16>(128, 128, 0, 0);
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t q_desc = packed::desc_rows(smem_u32(smem));
      const uint64_t do_desc = packed::desc_rows(smem_u32(smem + kTile));
      const uint64_t rows_desc = packed::desc_rows(smem_u32(ring));
      const uint64_t cols_desc = packed::desc_cols(smem_u32(ring));
      const bool issuer = packed::elect_one();
      bool ok = true;
      auto wait = [&](int bar, int phase) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
        tc::fence_after_sync();
      };
      auto stage = [&](int i) { return static_cast<uint64_t>((i % kStages * kTile) >> 4); };
      auto scores = [&](int j) {   // S and dout . v of step j
        wait(L::kFull + (2 * j) % kStages, 2 * j / kStages);
        if (clears && j == steps - 1) wait(L::kCleared, 0);
        if (!ok) return;
        if (issuer) {
          packed::mma_rows<kD>(tmem + kDqS, q_desc, rows_desc + stage(2 * j), kIdS);
          tc::commit(&bars[L::kSFull]);
        }
        __syncwarp();
        wait(L::kFull + (2 * j + 1) % kStages, (2 * j + 1) / kStages);
        if (!ok) return;
        if (issuer) {
          packed::mma_rows<kD>(tmem + kDqDp, do_desc, rows_desc + stage(2 * j + 1), kIdS);
          tc::commit(&bars[L::kDpFull]);
          tc::commit(&bars[L::kEmpty + (2 * j + 1) % kStages]);
        }
        __syncwarp();
      };
      wait(L::kQFull, 0);
      if (ok) scores(0);
      for (int j = 0; j < steps && ok; ++j) {
        if (j < back && issuer) tc::commit(&bars[L::kEmpty + (2 * j) % kStages]);
        __syncwarp();
        if (j + 1 < steps) {
          wait(L::kFree, j);   // both score buffers are in registers
          if (ok) scores(j + 1);
        }
        if (j < back) continue;
        const int i = j - back;
        wait(L::kDsFull + (i & 1), i >> 1);
        if (!ok) break;
        if (issuer) {
          packed::mma_cols(tmem + kDqAcc, tmem + kDqDs + (i & 1) * 64, cols_desc + stage(2 * j), kIdO, i > 0);
          tc::commit(&bars[L::kDqDone + (i & 1)]);
          tc::commit(&bars[L::kEmpty + (2 * j) % kStages]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    packed::regs_up<216>();
    const int half = warp >> 2;   // columns 64 half .. 64 half + 63
    const int r = tid & 127;
    const int token = t0 + r / s.G;
    const bool active = r < tile_tokens * s.G && token < seq.n_q;
    const int limit = active ? before + token + 1 : 0;
    const int head = h * s.G + r % s.G;
    const long long row = seq.q0 + token;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* part = reinterpret_cast<float*>(smem + L::kSum);

    // The sum of the row's two halves, in both threads that share it.
    auto both = [&](float v) {
      asm volatile("bar.sync 1, 256;" ::: "memory");
      part[half * 128 + r] = v;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      return part[r] + part[128 + r];
    };
    float D = 0.f, lse2 = 0.f, rest = 0.f;
    if (active) {
      if (!exact) {
        const uint4* a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.out) + row * g.out_st.token +
                                                        head * g.out_st.head + half * (kD / 2));
        const uint4* c = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.dout) + row * g.dout_st.token +
                                                        head * g.dout_st.head + half * (kD / 2));
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          const uint4 u = __ldg(a + i), w = __ldg(c + i);
          const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = packed::unpack2<kFp16>(us[e]), q = packed::unpack2<kFp16>(ws[e]);
            D = fmaf(p.x, q.x, fmaf(p.y, q.y, D));
          }
        }
      }
      // A row that attends nothing has P = 0: no finite score reaches 2^+inf.
      lse2 = __ldg(g.lse + row * (s.Hkv * s.G) + head) * kLog2e;
      if (limit <= 0) lse2 = INFINITY;
    }
    if (!exact) D = both(D);

    const int whole = static_cast<int>(__reduce_min_sync(0xffffffffu, active ? max(limit, 0) : 0x7fffffff)) / 128;
    bool ok = true;
    auto wait = [&](int bar, int phase) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
      tc::fence_after_sync();
    };
    for (int j = 0; j < steps; ++j) {
      const int tile_j = j < back ? j : j - back;
      uint32_t z[64], dp[64];
      wait(L::kSFull, j);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tc::ld32(lane_addr + kDqS + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
      tc::wait_ld();
      const int keep = limit - tile_j * 128 - 64 * half;
      if (tile_j >= whole) {
#pragma unroll
        for (int i = 0; i < 64; ++i) z[i] = i < keep ? z[i] : 0xff800000u;
      }
#pragma unroll
      for (int i = 0; i < 64; ++i)
        z[i] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(z[i]), s.scale2, -lse2)));
      wait(L::kDpFull, j);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tc::ld32(lane_addr + kDqDp + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&dp[32 * c]));
      tc::wait_ld();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kFree]);
      if (tile_j >= whole) {   // a hidden value's infinity meets P = 0
#pragma unroll
        for (int i = 0; i < 64; ++i) dp[i] = i < keep ? dp[i] : 0u;
      }
      if (j < back || (exact && n == 1)) {
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          d0 = fmaf(__uint_as_float(z[i]), __uint_as_float(dp[i]), d0);
          d1 = fmaf(__uint_as_float(z[i + 1]), __uint_as_float(dp[i + 1]), d1);
        }
        D += d0 + d1;
        if (tile_j == n - 1) D = both(D);
        if (j < back) continue;
      }
      uint32_t ds[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float a = __uint_as_float(z[2 * i]) * (__uint_as_float(dp[2 * i]) - D);
        const float c = __uint_as_float(z[2 * i + 1]) * (__uint_as_float(dp[2 * i + 1]) - D);
        rest += a + c;
        ds[i] = packed::pack2<kFp16>(a, c);
      }
      if (tile_j >= 2) wait(L::kDqDone + (tile_j & 1), (tile_j - 2) >> 1);   // this buffer's last reader
      tc::st32(lane_addr + kDqDs + (tile_j & 1) * 64 + 32 * half, ds);
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kDsFull + (tile_j & 1)]);
    }
    // sum P (dout . v - D) is what D lacks.
    D += both(rest);
    if (half == 0 && active) g.rows[row * (s.Hkv * s.G) + head] = make_float2(lse2, D);
    if (n > 0) wait(L::kDqDone + ((n - 1) & 1), (n - 1) >> 1);
    uint16_t* dq = static_cast<uint16_t*>(g.dq) + row * g.dq_st.token + head * g.dq_st.head;
#pragma unroll 1
    for (int c = 0; c < kD / 64; ++c) {
      const int col = half * (kD / 2) + 32 * c;
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (n > 0) {
        tc::ld32(lane_addr + kDqAcc + col, w);
        tc::wait_ld();
      }
      if (active) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = limit > 0 ? packed::pack2<kFp16>(__uint_as_float(w[8 * i + 2 * e]) * s.scale,
                                                    __uint_as_float(w[8 * i + 2 * e + 1]) * s.scale)
                             : 0u;
          *reinterpret_cast<uint4*>(dq + col + 8 * i) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------- dk and dv ----

template <int kD>
struct DkvLayout {
  static constexpr int kTile = kD / 64 * 16384;
  static constexpr int kStages = 131072 / kTile;
  static constexpr int kRing = 2 * kTile;   // K and V before it
  static constexpr int kRows = kRing + kStages * kTile;   // two buffers of [128] lse log2(e), [128] D
  static constexpr int kBars = kRows + 2 * 1024;
  static constexpr int kKvFull = 0, kFull = 1, kEmpty = kFull + kStages, kRowsFull = kEmpty + kStages,
                       kRowsFree = kRowsFull + 2, kCleared = kRowsFree + 2, kSFull = kCleared + 2,
                       kPFull = kSFull + 1, kDpFull = kPFull + 1, kDsFull = kDpFull + 1, kDone = kDsFull + 1,
                       kNumBars = kDone + 1;
  static constexpr int kScratch = kBars + 8 * kNumBars;
  static constexpr int kBytes = kScratch + 32 + 1024;
};
// Tensor memory: S^T with P^T over it, (v . dout)^T with dS^T over it, dv, dk.  A
// warpgroup's 16-bit values lie over its own 64 columns' first 32.
constexpr uint32_t kKvS = 0, kKvDp = 128, kKvDv = 256, kKvDk = 384;

template <int kD, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkv_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnGrads g,
                      const int ctas) {
  using L = DkvLayout<kD>;
  constexpr int kTile = L::kTile, kStages = L::kStages;
  constexpr float kDown = 1.f / (1 << kUp<kFp16>);   // takes kUp off again: from dout . v - D for dS, from dv
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int* scratch = reinterpret_cast<int*>(smem + L::kScratch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 4);
  uint8_t* ring = smem + L::kRing;
  float* rows = reinterpret_cast<float*>(smem + L::kRows);
  float4* parts = reinterpret_cast<float4*>(ring);   // at the end: this CTA's dv and dk, 2 x 128 rows of kD
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;

  pdl_wait();
  pdl_trigger();
  const int tile_tokens = packed_tile_tokens(s.G), tile_rows = tile_tokens * s.G;
  const int rank = static_cast<int>(blockIdx.x) % ctas, unit = static_cast<int>(blockIdx.x) / ctas;
  const int h = unit % s.Hkv;
  int b, level;
  if (!packed::find_tile(s, unit / s.Hkv, 128, true, scratch, &b, &level)) return;   // the same for the whole cluster
  bool bad = false;
  const packed::Sequence seq = packed::sequence(s, b, &bad);
  const int key0 = ((seq.n_k + 127) / 128 - 1 - level) * 128;
  const int before = seq.n_k - seq.n_q;
  const int t0 = max(key0 - before, 0);   // the first query that attends the tile's first key
  // Row tiles: of all of them this CTA takes rank, rank + ctas, ...
  const int n_all = (max(seq.n_q - t0, 0) + tile_tokens - 1) / tile_tokens;
  const int n = (n_all - rank + ctas - 1) / ctas;
  auto tile_token = [&](int i) { return t0 + (rank + i * ctas) * tile_tokens; };   // of its i-th tile
  // Rows of the last tile that hold no query of the sequence meet P = dS = 0.
  const int last_rows = (seq.n_q - tile_token(n - 1)) * s.G;
  const bool clears = n > 0 && last_rows < tile_rows;

  if (tid == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.dout);
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool by_warps = i == L::kPFull || i == L::kDsFull || i == L::kRowsFree || i == L::kRowsFree + 1;
      mbar_init(&bars[i], by_warps ? 8 : 1);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  // Rows that no copy writes (G does not divide 128) are 0 in every stage.
  if (tile_rows < 128) {
    for (int st = warp; st < kStages; st += kThreads / 32) packed::clear_rows<kD>(ring + st * kTile, tile_rows);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    packed::regs_down<72>();
    if (warp == kTmaWarp && n > 0) {
      int issued = 0;   // Q_0, dout_0, Q_1, dout_1, ...
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[L::kKvFull], 2 * kTile);
        for (int c = 0; c < kD / 64; ++c) {
          packed::tma_load_3d(smem_u32(smem + c * 16384), &maps.k, c * 64, seq.k0 + key0, h, &bars[L::kKvFull]);
          packed::tma_load_3d(smem_u32(smem + kTile + c * 16384), &maps.v, c * 64, seq.k0 + key0, h,
                              &bars[L::kKvFull]);
        }
        for (; issued < 2 * n; ++issued) {
          const int st = issued % kStages;
          if (issued >= kStages && !mbar_wait(&bars[L::kEmpty + st], (issued / kStages - 1) & 1, s.status)) break;
          mbar_arrive_expect_tx(&bars[L::kFull + st], tile_rows * kD * 2);
          for (int c = 0; c < kD / 64; ++c)
            packed::tma_load_4d(smem_u32(ring + st * kTile + c * 16384), issued & 1 ? &maps.dout : &maps.q, c * 64, 0,
                                h, seq.q0 + tile_token(issued >> 1), &bars[L::kFull + st]);
        }
      }
      issued = __shfl_sync(0xffffffffu, issued, 0);
      for (int i = max(0, issued - kStages); i < issued; ++i)   // (as above)
        mbar_wait(&bars[L::kFull + i % kStages], (i / kStages) & 1, s.status);
      if (clears && issued == 2 * n) {
        for (int i = 2 * n - 2; i < 2 * n; ++i) {
          packed::clear_rows<kD>(ring + i % kStages * kTile, last_rows);
          if (lane == 0) mbar_arrive(&bars[L::kCleared + (i & 1)]);
        }
      }
      mbar_wait(&bars[L::kKvFull], 0, s.status);
    } else if (warp == kRowsWarp) {
      // Each row tile's (lse, D), +inf for a row of no query: its P is 0.
      for (int i = 0; i < n; ++i) {
        const int buf = i & 1;
        if (i >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bars[L::kRowsFree + buf], (i / 2 - 1) & 1, s.status))) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = lane + 32 * k, token = tile_token(i) + r / s.G;
          float2 v = make_float2(INFINITY, 0.f);
          if (r < tile_rows && token < seq.n_q)
            v = __ldg(g.rows + static_cast<long long>(seq.q0 + token) * (s.Hkv * s.G) + h * s.G + r % s.G);
          rows[buf * 256 + r] = v.x - kUp<kFp16>;
          rows[buf * 256 + 128 + r] = v.y * kDown;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kRowsFull + buf]);
      }
    } else if (warp == kMmaWarp && n > 0) {
      constexpr uint32_t kIdS = packed::idesc<kFp16>(128, 128, 0, 0);
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t k_desc = packed::desc_rows(smem_u32(smem));
      const uint64_t v_desc = packed::desc_rows(smem_u32(smem + kTile));
      const uint64_t rows_desc = packed::desc_rows(smem_u32(ring));
      const uint64_t cols_desc = packed::desc_cols(smem_u32(ring));
      const bool issuer = packed::elect_one();
      bool ok = true;
      auto wait = [&](int bar, int phase) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
        tc::fence_after_sync();
      };
      auto stage = [&](int i) { return static_cast<uint64_t>((i % kStages * kTile) >> 4); };
      auto loaded = [&](int i) {   // the i-th tile of the ring, cleared where it must be
        wait(L::kFull + i % kStages, i / kStages);
        if (clears && (i >> 1) == n - 1) wait(L::kCleared + (i & 1), 0);
        return ok;
      };
      auto scores = [&](int i) {
        if (!loaded(2 * i)) return;
        if (issuer) {
          packed::mma_rows<kD>(tmem + kKvS, k_desc, rows_desc + stage(2 * i), kIdS);
          tc::commit(&bars[L::kSFull]);
        }
        __syncwarp();
      };
      auto inner = [&](int i) {
        if (!loaded(2 * i + 1)) return;
        if (issuer) {
          packed::mma_rows<kD>(tmem + kKvDp, v_desc, rows_desc + stage(2 * i + 1), kIdS);
          tc::commit(&bars[L::kDpFull]);
        }
        __syncwarp();
      };
      wait(L::kKvFull, 0);
      if (ok) scores(0);
      if (ok) inner(0);
      for (int i = 0; i < n && ok; ++i) {
        wait(L::kPFull, i);
        if (!ok) break;
        if (issuer) {
          packed::mma_cols<64>(tmem + kKvDv, tmem + kKvS, cols_desc + stage(2 * i + 1), kIdO, i > 0);
          tc::commit(&bars[L::kEmpty + (2 * i + 1) % kStages]);
        }
        __syncwarp();
        if (i + 1 < n) scores(i + 1);
        wait(L::kDsFull, i);
        if (!ok) break;
        if (issuer) {
          packed::mma_cols<64>(tmem + kKvDk, tmem + kKvDp, cols_desc + stage(2 * i), kIdO, i > 0);
          tc::commit(&bars[L::kEmpty + (2 * i) % kStages]);
        }
        __syncwarp();
        if (i + 1 < n) inner(i + 1);
      }
      if (ok && issuer) tc::commit(&bars[L::kDone]);
    }
    __syncwarp();
  } else {
    packed::regs_up<216>();
    const int half = warp >> 2;   // query rows 64 half .. 64 half + 63 of a tile
    const int key = key0 + (tid & 127);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int warp_last = key0 + (warp & 3) * 32 + 31;
    bool ok = true;
    auto wait = [&](int bar, int phase) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
      tc::fence_after_sync();
    };
    for (int i = 0; i < n; ++i) {
      // Rows of tokens before key - before do not attend the key.
      const int token0 = tile_token(i);
      const int from = (key - before - token0) * s.G - 64 * half;
      const bool masked = warp_last - before > token0;
      const float4* lse2 = reinterpret_cast<const float4*>(rows + (i & 1) * 256 + 64 * half);
      const float4* D = reinterpret_cast<const float4*>(rows + (i & 1) * 256 + 128 + 64 * half);
      uint32_t z[64];
      wait(L::kRowsFull + (i & 1), i >> 1);
      wait(L::kSFull, i);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tc::ld32(lane_addr + kKvS + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
      tc::wait_ld();
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float4 m = lse2[c];
        z[4 * c] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(z[4 * c]), s.scale2, -m.x)));
        z[4 * c + 1] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(z[4 * c + 1]), s.scale2, -m.y)));
        z[4 * c + 2] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(z[4 * c + 2]), s.scale2, -m.z)));
        z[4 * c + 3] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(z[4 * c + 3]), s.scale2, -m.w)));
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; ++c) z[c] = c >= from ? z[c] : 0u;
      }
      uint32_t p[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) p[c] = packed::pack2<kFp16>(__uint_as_float(z[2 * c]), __uint_as_float(z[2 * c + 1]));
      tc::st32(lane_addr + kKvS + 64 * half, p);
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kPFull]);
      wait(L::kDpFull, i);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32];
        tc::ld32(lane_addr + kKvDp + 64 * half + 32 * c, dp);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 d = D[8 * c + e];
          const uint32_t* zz = &z[32 * c + 4 * e];
          p[16 * c + 2 * e] = packed::pack2<kFp16>(__uint_as_float(zz[0]) * fmaf(__uint_as_float(dp[4 * e]), kDown, -d.x),
                                                   __uint_as_float(zz[1]) * fmaf(__uint_as_float(dp[4 * e + 1]), kDown, -d.y));
          p[16 * c + 2 * e + 1] = packed::pack2<kFp16>(__uint_as_float(zz[2]) * fmaf(__uint_as_float(dp[4 * e + 2]), kDown, -d.z),
                                                       __uint_as_float(zz[3]) * fmaf(__uint_as_float(dp[4 * e + 3]), kDown, -d.w));
        }
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (2 * c + 1 < from) p[c] = 0u;
          if (2 * c < from) p[c] &= 0xffff0000u;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kRowsFree + (i & 1)]);
      tc::st32(lane_addr + kKvDp + 64 * half, p);
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kDsFull]);
    }
    if (n > 0) wait(L::kDone, 0);
    // ---- the first warpgroup has dv, the second dk ----
    const bool active = key < seq.n_k;
    const PackedStride st = half ? g.dk_st : g.dv_st;
    uint16_t* to = static_cast<uint16_t*>(half ? g.dk : g.dv) + static_cast<long long>(seq.k0 + key) * st.token +
                   h * st.head;
    const float scale = half ? s.scale : kDown;
#pragma unroll 1
    for (int c = 0; c < kD / 32; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (n > 0) {
        tc::ld32(lane_addr + (half ? kKvDk : kKvDv) + 32 * c, w);
        tc::wait_ld();
      }
      if (ctas > 1) {   // into this CTA's ring, which is free now
#pragma unroll
        for (int i = 0; i < 8; ++i)
          parts[packed::swizzled<kD>(half * 128 + (tid & 127), 8 * c + i)] =
              make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]), __uint_as_float(w[4 * i + 2]),
                          __uint_as_float(w[4 * i + 3]));
      } else if (active) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = packed::pack2<kFp16>(__uint_as_float(w[8 * i + 2 * e]) * scale,
                                        __uint_as_float(w[8 * i + 2 * e + 1]) * scale);
          *reinterpret_cast<uint4*>(to + 32 * c + 8 * i) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    }
  }
  if (ctas > 1) {
    // ---- every CTA sums its share of the rows over the cluster, in the order of the ranks ----
    __syncwarp();
    cluster_sync();
    if (warp < 8) {   // (the others have given registers away)
      const int share = 2 * 128 / ctas;   // rows of dv, then of dk
      for (int e = tid; e < share * (kD / 4); e += 256) {
        const int row = rank * share + e / (kD / 4), c4 = e % (kD / 4);
        const int which = row >> 7, key = key0 + (row & 127);
        if (key >= seq.n_k) continue;
        const float4* mine = parts + packed::swizzled<kD>(row, c4);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < ctas; ++c) {
          const float4 x = packed::ld_dsmem_f32x4(dsmem_addr(mine, static_cast<uint32_t>(c)));
          sum.x += x.x;
          sum.y += x.y;
          sum.z += x.z;
          sum.w += x.w;
        }
        const PackedStride st = which ? g.dk_st : g.dv_st;
        const float scale = which ? s.scale : kDown;
        uint16_t* to = static_cast<uint16_t*>(which ? g.dk : g.dv) + static_cast<long long>(seq.k0 + key) * st.token +
                       h * st.head + 4 * c4;
        *reinterpret_cast<uint2*>(to) = make_uint2(packed::pack2<kFp16>(sum.x * scale, sum.y * scale),
                                                   packed::pack2<kFp16>(sum.z * scale, sum.w * scale));
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

template <typename Kernel, typename... More>
cudaError_t launch_one(Kernel kernel, int bytes, long long units, int ctas, cudaStream_t st, const More&... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tiles of `step` tokens of B sequences with `tokens` in all: at most one partly filled one each.
long long most_tiles(int tokens, int step, int B) {
  return std::min<long long>(tokens, static_cast<long long>(tokens) / step + B);
}

template <int kD, bool kFp16>
cudaError_t launch(const PackedAttnShape& s, const PackedAttnMaps& maps, const PackedAttnGrads& g, cudaStream_t st) {
  const cudaError_t e =
      launch_one(packed_dq_kernel<kD, kFp16>, DqLayout<kD>::kBytes,
                 most_tiles(s.Tq, packed_tile_tokens(s.G), s.B) * s.Hkv, 1, st, maps, s, g);
  if (e != cudaSuccess) return e;
  // CTAs per tile of keys.  Causal tiles differ by the whole length of the sequence, so
  // units that are few leave SMs idle behind the longest: one 8K sequence with 2 KV
  // heads took 1.42 ms with clusters of 4, 1.53 with 2, 1.76 with 8 (which few SMs
  // of a GPC are left over for) and 2.52 alone.  16 documents (640 units) took
  // 0.57 ms alone and 0.62 with 2: enough units, and the join costs a few row tiles.
  const long long units = ((s.Tk + s.B - 1) / s.B + 127) / 128 * static_cast<long long>(s.B) * s.Hkv;
  const long long row_tiles = static_cast<long long>(s.Tq) * s.G / 128 / s.B;
  const int sms = device_sm_count();
  int ctas = 1;
  while (ctas < 4 && units * ctas < 2 * sms && row_tiles >= 12 * ctas) ctas *= 2;
  if (ctas == 4 && units * 8 <= sms && row_tiles >= 48) ctas = 8;
  return launch_one(packed_dkv_kernel<kD, kFp16>, DkvLayout<kD>::kBytes, most_tiles(s.Tk, 128, s.B) * s.Hkv, ctas, st,
                    maps, s, g, ctas);
}

}  // namespace

cudaError_t launch_packed_attn_bwd(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                                   const PackedAttnGrads& g, cudaStream_t st) {
  if (D == 128) return fp16 ? launch<128, true>(s, maps, g, st) : launch<128, false>(s, maps, g, st);
  return fp16 ? launch<64, true>(s, maps, g, st) : launch<64, false>(s, maps, g, st);
}

}  // namespace infllmv2
