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
// attends few keys, or one key takes most of its weight, or values and keys have large
// means, dout . v - D is a small difference of such numbers and the error shows in dq and
// dk.  So rows of up to kExactTiles tiles of keys walk them twice and sum
// D = sum P (dout . v) first (one tile: it is all in registers).  Longer ones walk them
// once, from the last to the first: sum P (dout . v - D) of all tiles is what D lacked
// (`moved`), so that the first tile's dS (the first tokens are what draws much of the
// attention in trained models) and the dk and dv kernel have D exactly.  dq of the other
// tiles is off by scale moved sum P k: with W their weight by moved W times the size of
// their keys at most, while rounding dS to 16 bits costs dq e sqrt(sum dS^2) times that size
// at most (e: half a step of the type).  A tile of rows is done once more, with the D that
// is known then, where the first passes the second (by sums of squares over the tile).  Where
// none of the cases above holds, their ratio is about 0.4, and 0.73 was the largest among 900
// tiles of 8192 keys with a sink at the first.  bf16, d 128, 2000 keys, key 1500 with
// 0.97 of the weight: dq 6.0% off before, 0.23% now; 3000 keys and values with means of 3
// deviations: 14.4% and 0.56%.  It costs those tiles twice their time.
//
// In both kernels the operand that the second products take from the scores, dS (dq), or
// P^T and dS^T (dk, dv: scores are computed transposed, keys in rows), is the A
// operand in tensor memory: no product's input passes through shared memory but
// the tiles that TMA brought.  Two warpgroups share a tile's columns.
//
// Measured (GB300): one sequence of 8192 tokens, 2 KV heads of 16, d 128, 1.07 ms
// (dq 475 us, tensor cores 79% busy; dk and dv 608, 86%; 1.19 ms in turn with other work):
// 1.28 PFLOP/s of five products, 1.80 of the seven that are issued, 94% of the measured
// library product.  16 documents of 17 to 2500 tokens, 4 heads of 5, d 64, fp16, 435 us (dq 262, 32%;
// dk and dv 178, 53%): the exponentials, the second walk of the rows that attend up to 1024
// keys and the start and end of short units.  96 sequences of 256, 4 heads of 5, d 64:
// 230 us in bf16, 243 in fp16.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "packed_attn.cuh"

namespace infllmv2 {

namespace {

constexpr int kThreads = 384;
constexpr int kPairWarp = 8, kTmaWarp = 9, kSumWarp = 10;   // dq
constexpr int kMmaWarp = 8, kRowsWarp = 10, kKvSumWarp = 11;   // dk and dv (and kTmaWarp)
constexpr float kLog2e = 1.4426950408889634f;
// log2 of what P is multiplied by on its way to dv.  A probability of a long row is
// among fp16's subnormal numbers, where it would lose bits.
template <bool kFp16>
constexpr int kUp = kFp16 ? 8 : 0;
// Half a step of the type, the most that one rounding costs.
template <bool kFp16>
constexpr float kHalfStep = kFp16 ? 0x1p-11f : 0x1p-8f;
// Rows that attend at most so many tiles of keys get D from their scores.
constexpr int kExactTiles = 8;

// fp16's dS.  Upstream gradients of 10^-3 to 10^-4 are ordinary (a mean over tokens), and dS, a probability times
// them, is then among fp16's subnormal numbers or below; with large ones it passes 65504.  So dS is formed times
// a power of two, which comes off the fp32 sums.  |dS| <= max |dout . v| + |D|, and what a bound is above the truth
// only costs bits of a range of 2^40, so norms will do.
//   * dq: one power per row, in the exponent of P.  Rows of up to kExactTiles tiles know |dout . v| and D before they
//     form dS: 8 times their sum, at most, goes to 2^15.  Longer ones take |dout| |out|, which is about |dS| where
//     a few keys have the weight and far above it where many have: at most 4 times that goes to 2^10.  A row whose
//     dS passes 2^15.5 all the same (values that cancel in out; by the sum of squares) has its unit done once more,
//     with the power from that sum.
//   * dk: one power per tile of keys, from the largest |dS| that dq found among the rows that attend it.
// 3000 keys, d 64, dout of 10^-3 (10^-4): dq 0.094% (0.90%) off without the powers, 0.034% (0.20%) with them, which
// is the rounding of the results; dout of 1000 and values of 50 gave infinities.  It costs 7% of the time of 16
// documents of 17 to 2500 tokens, d 64 (403 or 432 us), and 4% of a sequence of 8192's.
constexpr int kNoTop = -1000;   // of a row without a finite dS

// The power for values below 2^top: `to` is log2 of where they go.  From 2^-30 to 2^20, which is beyond what
// results in fp16 show, and keeps fp32 sums of squares finite.
__device__ __forceinline__ int power_for(int top, int to) { return top == kNoTop ? 0 : min(max(to - top, -30), 20); }
// The least `top` with 0 <= x < 2^top.
__device__ __forceinline__ int top_of(float x) {
  return x < INFINITY ? static_cast<int>(__float_as_uint(x) >> 23) - 126 : kNoTop;
}
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// ------------------------------------------------------------------- dq ----
//
// A CTA takes one tile of rows after another.  For step j (a tile of keys) the tensor
// cores form S and dout . v, the threads P and dS, the tensor cores add dS K.  Both
// scores go into registers at once and are replaced while the threads compute: S and
// dout . v of step j + 1 run beside P and dS of step j, whose exponentials and
// products overlap in turn.

template <int kD>
struct DqLayout {
  static constexpr int kTile = kD / 64 * 16384;
  static constexpr int kKs = 4 * 128 / kD, kVs = 2 * 128 / kD;   // stages of the K and the V ring
  static constexpr int kK = kTile, kV = kK + kKs * kTile;        // behind dout
  static constexpr int kBars = kV + kVs * kTile;
  static constexpr int kUnit = 0, kUnitFree = 2, kDoFull = 4, kDoFree = 5, kKFull = 6, kKEmpty = kKFull + kKs,
                       kVFull = kKEmpty + kKs, kVEmpty = kVFull + kVs, kTail = kVEmpty + kVs, kCleared = kTail + 2,
                       kPair = kCleared + 2, kFree = kPair + 1, kDsFull = kFree + 1, kDqDone = kDsFull + 1,
                       kAccFree = kDqDone + 1, kQIn = kAccFree + 1, kOutRead = kQIn + 1, kLse = kOutRead + 1,
                       kEnd = kLse + 2, kNumBars = kEnd + 2;
  static constexpr int kUnits = kBars + (8 * kNumBars + 15) / 16 * 16;   // two units, 32 bytes each
  static constexpr int kSlot = kUnits + 64;
  static constexpr int kSum = kSlot + 16;   // [2][128]: sums over the halves of a row
  static constexpr int kLses = kSum + 1024;   // of two units [128]: lse log2(e)
  static constexpr int kMost = kLses + 1024;   // [2][128] 16 bits: the larger of two halves
  static constexpr int kTops = kMost + 512;    // of two units: the largest top_of of their rows; and the first row
  static constexpr int kAgain = kTops + 16;    // a bit for each of kAgainUnits of the CTA's units: once more
  static constexpr int kBytes = kAgain + 128;   // (no slack: where the base is not aligned the kernel says so)
};
constexpr int kAgainUnits = 1024;   // (further units share the bits: some are done once more for nothing)
// Tensor memory: S, dout . v, dS, Q (16 bits: the A operand of S), dq.  Q comes through
// the K ring, as the element before K_0, and makes room there: a tile of K is read
// until its dS K is done, more than a step after its S.
constexpr uint32_t kDqS = 0, kDqDp = 128, kDqDs = 256, kDqQ = 320, kDqAcc = 384;

struct DqUnit {
  packed::Sequence seq;
  int t0, h, before;   // its first query, its KV head; query t attends keys 0 .. before + t
  int n;               // tiles of keys
  bool again;          // it has been done: D and the power of its dS are known
  bool exact, clears;  // D not from out; the last tile runs past the sequence
  int steps, back;     // tiles walked (twice where D comes from the scores), the first of the walk that sums dq
  int number;          // among the CTA's, modulo kAgainUnits
};

template <int kD, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnGrads g) {
  using L = DqLayout<kD>;
  constexpr int kTile = L::kTile, kKs = L::kKs, kVs = L::kVs;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) % 1024 != 0) {   // the whole grid: shared memory starts on 1024 bytes or it does not
    if (threadIdx.x == 0) atomicOr(s.status, kStatusBounds);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int4* units = reinterpret_cast<int4*>(smem + L::kUnits);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;
  const int tile_tokens = packed_tile_tokens(s.G);

  if (tid < L::kNumBars) {
    int count = 1;
    if (tid == L::kUnitFree || tid == L::kUnitFree + 1) count = 11;   // the warps but the one that finds units
    if (tid == L::kFree || tid == L::kDsFull || tid == L::kAccFree || tid == L::kQIn || tid == L::kOutRead) count = 8;
    mbar_init(&bars[tid], count);
    fence_barrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.out);
    prefetch_tensormap(&maps.dout);
  }
  // Tensor memory is taken once the kernel before has ended and before the next one may start: neither ever
  // waits for columns that the other holds.
  pdl_wait();
  packed::Walker walker;   // of the warp that finds the units
  bool bad = false;
  if (warp == kTmaWarp) walker.start(s, tile_tokens, false, &bad);
  if (warp == kPairWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  int* tops = reinterpret_cast<int*>(smem + L::kTops);
  uint32_t* again = reinterpret_cast<uint32_t*>(smem + L::kAgain);
  if (tid < 2) tops[tid] = kNoTop;
  if (tid < kAgainUnits / 32) again[tid] = 0u;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  // A unit from where it lies, (0, or 1 once more; -1: there is none; its tile, KV head and number), and its
  // sequence.
  auto unit_of = [&](int4 at, int4 rows) {
    DqUnit u;
    u.seq = {rows.x, rows.y, rows.z, rows.w};
    u.t0 = at.y * tile_tokens;
    u.h = at.z;
    u.before = u.seq.n_k - u.seq.n_q;
    const int last = min(u.t0 + tile_tokens, u.seq.n_q) - 1;
    u.n = (max(u.before + last + 1, 0) + 127) / 128;
    u.clears = u.n * 128 > u.seq.n_k;
    u.again = at.x > 0;
    u.exact = u.again || u.n <= kExactTiles;
    u.steps = u.exact && !u.again && u.n > 1 ? 2 * u.n : u.n;
    u.back = u.steps - u.n;
    u.number = at.w;
    return u;
  };
  auto next_unit = [&](int k, bool* ok, DqUnit* u) {
    if (*ok) *ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kUnit + (k & 1)], (k >> 1) & 1, s.status));
    if (!*ok) return false;
    int4 at = units[2 * (k & 1)];
    const int4 rows = units[2 * (k & 1) + 1];
    at.x = __shfl_sync(0xffffffffu, at.x, 0);   // (uniform for the compiler, so that the roles' loops are)
    if (at.x < 0) return false;
    *u = unit_of(at, rows);
    return true;
  };
  auto unit_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[L::kUnitFree + (k & 1)]);
  };
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  // Stage and phase of a ring, or a phase alone.
  struct Place {
    int stage, phase;
  };
  auto next = [](Place& p, int stages) {
    if (++p.stage == stages) {
      p.stage = 0;
      p.phase ^= 1;
    }
  };
  DqUnit u;
  bool ok = true;
  auto wait = [&](int bar, int phase) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
    tc::fence_after_sync();
  };

  if (warp >= 8) {
    packed::regs_down<72>();
    if (warp == kTmaWarp) {
      // ------------------------------------------------------ units and loads
      const int stride = static_cast<int>(gridDim.x);
      int k_copies = 0, v_copies = 0, tails[2] = {0, 0}, uses = 0;   // (tails: of units of each parity)
      // The next stage of the K ring, with a copy of `bytes` announced on `bar` (null: the stage's own).
      auto k_stage = [&](uint32_t bytes, uint64_t* bar) {
        const int st = k_copies % kKs;
        if (k_copies >= kKs) wait(L::kKEmpty + st, k_copies / kKs - 1);
        if (ok && lane == 0) {
          if (bar) mbar_arrive(&bars[L::kKFull + st]);   // only counts the turn
          mbar_arrive_expect_tx(bar ? bar : &bars[L::kKFull + st], bytes);
        }
        if (ok) ++k_copies;
        return st;
      };
      // Unit number n of the CTA.
      auto find_unit = [&](int n, int4* at, int4* rows) {
        // Down the order of all units and back, so that no CTA gets the longest of each round.
        int i = static_cast<int>(blockIdx.x);
        i = n * stride + (n & 1 ? stride - 1 - i : i);
        int b, level;
        if (!walker.find(s, i / s.Hkv, tile_tokens, false, &b, &level, &bad)) return false;
        *at = make_int4(0, level, i % s.Hkv, n % kAgainUnits);
        const packed::Sequence seq = packed::sequence(s, b, &bad);
        *rows = make_int4(seq.q0, seq.n_q, seq.k0, seq.n_k);
        return true;
      };
      bool repeats = false, may_repeat = false;   // past the last unit; there was one that may be done once more
      uint32_t wanted = 0u;                       // the lane's 32 bits of those that are
      for (int k = 0, number = 0;; ++k) {
        int4 at = make_int4(-1, 0, 0, 0), rows = make_int4(0, 0, 0, 0);
        bool found = !repeats && find_unit(number, &at, &rows);
        if (found) {
          ++number;
        } else if (!repeats && may_repeat) {
          // Once more: each unit says so before it is done with.
          repeats = true;
          for (int d = k >= 2 ? 2 : 1; d > 0 && ok; --d)
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&bars[L::kUnitFree + ((k - d) & 1)], ((k - d) >> 1) & 1, s.status));
          wanted = again[lane];
          number = 0;
          walker.start(s, tile_tokens, false, &bad);
        }
        if (repeats && __any_sync(0xffffffffu, wanted != 0u)) {
          while ((found = find_unit(number, &at, &rows))) {
            ++number;
            if ((__shfl_sync(0xffffffffu, wanted, at.w >> 5) >> (at.w & 31)) & 1) break;
          }
          at.x = found ? 1 : -1;
        }
        if (k >= 2 && ok)
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kUnitFree + (k & 1)], ((k >> 1) - 1) & 1, s.status));
        if (!ok) at.x = -1;
        if (lane == 0) {
          units[2 * (k & 1)] = at;
          units[2 * (k & 1) + 1] = rows;
          mbar_arrive(&bars[L::kUnit + (k & 1)]);
        }
        __syncwarp();
        if (at.x < 0) break;
        u = unit_of(at, rows);
        may_repeat |= !u.exact;
        const uint32_t row_bytes = tile_tokens * s.G * kD * 2;
        if (u.n > 0) {
          const int st = k_stage(row_bytes, nullptr);
          if (ok && lane == 0)
            for (int c = 0; c < kD / 64; ++c)
              packed::tma_load_4d(smem_u32(smem + L::kK + st * kTile + c * 16384), &maps.q, c * 64, 0, u.h,
                                  u.seq.q0 + u.t0, &bars[L::kKFull + st]);
        }
        for (int j = 0; j < u.steps && ok; ++j) {
          const int row = u.seq.k0 + (j < u.back ? j : u.steps - 1 - j) * 128;
          // The tile of K that is to be cleared behind the sequence lands on a barrier of its own (of two in
          // turn: the unit after next waits for this one's end).
          const bool tail = u.clears && j == u.back;
          uint64_t* own = tail ? &bars[L::kTail + (k & 1)] : nullptr;
          const int st = k_stage(kTile, own);
          if (!ok) break;
          if (lane == 0)
            for (int c = 0; c < kD / 64; ++c)
              packed::tma_load_3d(smem_u32(smem + L::kK + st * kTile + c * 16384), &maps.k, c * 64, row, u.h,
                                  own ? own : &bars[L::kKFull + st]);
          tails[0] += tail && !(k & 1);
          tails[1] += tail && (k & 1);
          if (j == 0) {
            if (uses > 0) wait(L::kDoFree, uses - 1);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars[L::kDoFull], row_bytes);
              for (int c = 0; c < kD / 64; ++c)
                packed::tma_load_4d(smem_u32(smem + c * 16384), &maps.dout, c * 64, 0, u.h, u.seq.q0 + u.t0,
                                    &bars[L::kDoFull]);
            }
            ++uses;
          }
          // Through the V ring, before V_0 where D is rowsum(dout * out): out.
          for (int first = j == 0 && !u.exact ? 0 : 1; first < 2; ++first) {
            const int vs = v_copies % kVs;
            if (v_copies >= kVs) wait(L::kVEmpty + vs, v_copies / kVs - 1);
            if (!ok) break;
            if (lane == 0) {
              const uint32_t to = smem_u32(smem + L::kV + vs * kTile);
              mbar_arrive_expect_tx(&bars[L::kVFull + vs], first ? kTile : row_bytes);
              for (int c = 0; c < kD / 64; ++c) {
                if (first) {
                  packed::tma_load_3d(to + c * 16384, &maps.v, c * 64, row, u.h, &bars[L::kVFull + vs]);
                } else {
                  packed::tma_load_4d(to + c * 16384, &maps.out, c * 64, 0, u.h, u.seq.q0 + u.t0,
                                      &bars[L::kVFull + vs]);
                }
              }
            }
            ++v_copies;
          }
          if (!ok) break;
        }
        __syncwarp();
      }
      if (bad && blockIdx.x == 0) atomicOr(s.status, kStatusBadKvLen);
      // The CTA outlives its copies, also after a wait that gave up.  (Each barrier's last copy is its
      // newest phase here.)
      for (int i = max(0, k_copies - kKs); i < k_copies; ++i)
        mbar_wait(&bars[L::kKFull + i % kKs], (i / kKs) & 1, s.status);
      for (int i = max(0, v_copies - kVs); i < v_copies; ++i)
        mbar_wait(&bars[L::kVFull + i % kVs], (i / kVs) & 1, s.status);
      for (int i = 0; i < 2; ++i)
        if (tails[i] > 0) mbar_wait(&bars[L::kTail + i], (tails[i] - 1) & 1, s.status);
      if (uses > 0) mbar_wait(&bars[L::kDoFull], (uses - 1) & 1, s.status);
    } else if (warp == kPairWarp) {
      // ------------------------------------------------- S and dout . v of a step
      constexpr uint32_t kIdS = packed::idesc<kFp16>(128, 128, 0, 0);
      const uint64_t do_desc = packed::desc_rows(smem_u32(smem));
      const uint64_t k_desc = packed::desc_rows(smem_u32(smem + L::kK));
      const uint64_t v_desc = packed::desc_rows(smem_u32(smem + L::kV));
      const bool issuer = packed::elect_one();
      Place pk = {0, 0}, pv = {0, 0};
      int pairs = 0, even = 0, odd = 0, ins = 0, uses = 0, outs = 0;   // (tails of units of each parity)
      for (int k = 0; next_unit(k, &ok, &u); ++k) {
        const int steps = uniform(u.steps), back = uniform(u.back), tail = uniform(u.clears) ? back : -1;
        const bool exact = uniform(u.exact);
        if (steps > 0) {
          wait(L::kQIn, ins++);
          if (issuer) mbar_arrive(&bars[L::kKEmpty + pk.stage]);   // Q's stage has been read
          __syncwarp();
          next(pk, kKs);
        }
        for (int t = 0; t < steps; ++t) {
          if (t == tail) {
            wait(L::kTail + (k & 1), k & 1 ? odd++ : even++);
          } else {
            wait(L::kKFull + pk.stage, pk.phase);
          }
          if (t > 0) wait(L::kVFull + pv.stage, pv.phase);
          if (pairs > 0) wait(L::kFree, pairs - 1);   // both have been read
          ++pairs;
          if (issuer) {
            packed::mma_rows_ts<kD>(tmem + kDqS, tmem + kDqQ,
                                    k_desc + static_cast<uint64_t>(pk.stage * (kTile >> 4)), kIdS);
            if (t < back) tc::commit(&bars[L::kKEmpty + pk.stage]);   // (otherwise dS K is its last reader)
          }
          __syncwarp();
          next(pk, kKs);
          if (t == 0) {
            wait(L::kDoFull, uses++);
            if (!exact) {   // out's stage: read by the threads before their first pair
              wait(L::kOutRead, outs++);
              if (issuer) mbar_arrive(&bars[L::kVEmpty + pv.stage]);
              __syncwarp();
              next(pv, kVs);
            }
            wait(L::kVFull + pv.stage, pv.phase);
          }
          if (issuer) {
            packed::mma_rows<kD>(tmem + kDqDp, do_desc, v_desc + static_cast<uint64_t>(pv.stage * (kTile >> 4)), kIdS);
            tc::commit(&bars[L::kPair]);
            tc::commit(&bars[L::kVEmpty + pv.stage]);
            if (t == steps - 1) tc::commit(&bars[L::kDoFree]);
          }
          __syncwarp();
          next(pv, kVs);
        }
        unit_done(k);
      }
      packed::products_end(&bars[L::kEnd], issuer, s.status);   // (nothing outlives the CTA)
    } else if (warp == kSumWarp) {
      // ---------------------------------------------------------- dq += dS K
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t k_desc = packed::desc_cols(smem_u32(smem + L::kK));
      const bool issuer = packed::elect_one();
      Place pk = {0, 0};
      int even = 0, odd = 0, used = 0, made = 0;
      for (int k = 0; next_unit(k, &ok, &u); ++k) {
        const int steps = uniform(u.steps), back = uniform(u.back), tail = uniform(u.clears) ? back : -1;
        if (steps > 0) next(pk, kKs);   // Q's stage
        for (int j = 0; j < steps; ++j) {
          if (j >= back) {
            if (j == tail)   // (dS says that the other tiles are there)
              wait(L::kCleared + (k & 1), k & 1 ? odd++ : even++);
            if (j == back && used++ > 0) wait(L::kAccFree, used - 2);   // the last unit's dq has been read
            wait(L::kDsFull, made++);
            if (issuer) {
              packed::mma_cols(tmem + kDqAcc, tmem + kDqDs,
                               k_desc + static_cast<uint64_t>(pk.stage * (kTile >> 4)), kIdO, j > back);
              tc::commit(&bars[L::kDqDone]);
              tc::commit(&bars[L::kKEmpty + pk.stage]);
            }
            __syncwarp();
          }
          next(pk, kKs);
        }
        unit_done(k);
      }
      packed::products_end(&bars[L::kEnd + 1], issuer, s.status);
    } else {
      // ----------- the rows' lse, and K rows behind the sequence: they meet dS = 0
      Place pk = {0, 0};
      int even = 0, odd = 0;
      float* lses = reinterpret_cast<float*>(smem + L::kLses);
      for (int k = 0; next_unit(k, &ok, &u); ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a unit ahead of who needs it
          const int r = lane + 32 * i, token = u.t0 + r / s.G;
          const long long at = (u.seq.q0 + token) * static_cast<long long>(s.Hkv * s.G) + u.h * s.G + r % s.G;
          // A row that attends nothing has P = 0: no finite score reaches 2^+inf.
          float lse2 = 0.f;
          if (r < tile_tokens * s.G && token < u.seq.n_q)
            lse2 = u.before + token >= 0 ? g.lse[at] * kLog2e : INFINITY;
          lses[(k & 1) * 128 + r] = lse2;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kLse + (k & 1)]);
        if (u.steps > 0) next(pk, kKs);   // Q's stage
        for (int j = 0; j < u.steps; ++j) {
          if (u.clears && j == u.back) {
            wait(L::kTail + (k & 1), k & 1 ? odd++ : even++);
            packed::clear_rows<kD>(smem + L::kK + pk.stage * kTile, u.seq.n_k - (u.n - 1) * 128);
            if (lane == 0) mbar_arrive(&bars[L::kCleared + (k & 1)]);
          }
          next(pk, kKs);
        }
        unit_done(k);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ P and dS
    packed::regs_up<216>();
    const int half = warp >> 2;   // columns 64 half .. 64 half + 63
    const int r = tid & 127, row_token = r / s.G, row_head = r % s.G;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + kDqS + 64 * half, dp_addr = lane_addr + kDqDp + 64 * half;
    float* part = reinterpret_cast<float*>(smem + L::kSum);
    uint16_t* larger = reinterpret_cast<uint16_t*>(smem + L::kMost);
    const uint64_t scale2 = packed::pair(s.scale2, s.scale2);
    const bool wide = packed::wide_rows(g.dq, g.dq_st);
    // The sum of a row's two halves, in both threads that share it.
    auto both = [&](float v) {
      asm volatile("bar.sync 1, 256;" ::: "memory");
      part[half * 128 + r] = v;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      return part[r] + part[128 + r];
    };
    // The same, and top_of of sqrt((x + x')(y + y')), rounded up, with other values x and y >= 0 of the two.  (Once
    // in a unit: no barrier keeps a second one from `larger`.)
    auto both_and_top = [&](float v, float x, float y, int* top) {
      larger[half * 128 + r] = static_cast<uint16_t>((__float_as_uint(x) >> 23) << 8 | __float_as_uint(y) >> 23);
      const float sum = both(v);
      const uint32_t both_tops = __vmaxu4(larger[r], larger[128 + r]);   // (biased exponents)
      const int tx = static_cast<int>(both_tops >> 8) - 125, ty = static_cast<int>(both_tops & 0xffu) - 125;
      *top = max(tx, ty) > 128 ? kNoTop : (tx + ty + 1) >> 1;   // (a sum is at most twice the larger)
      return sum;
    };
    // fp16: the largest top_of of a unit's rows lies beside its first row's, once all warps are past the unit.
    // (Thread 0 alone knows of it, and keeps the row's number and its own top_of beside the tops.)
    if (tid == 0) tops[2] = -1;
    auto tops_put = [&](int k) {
      if (tid != 0 || tops[2] < 0) return;
      g.rows[tops[2]].x =
          __uint_as_float((static_cast<uint32_t>(tops[k & 1]) << 16) | (static_cast<uint32_t>(tops[3]) & 0xffffu));
      tops[k & 1] = kNoTop;
      tops[2] = -1;
    };
    int pairs = 0, summed = 0, uses = 0;   // in all: pairs of scores read, dS written, units with keys
    Place pk = {0, 0}, pv = {0, 0};
    for (int k = 0;; ++k) {
      const bool more = packed::all_agree(next_unit(k, &ok, &u));
      if (kFp16) tops_put(k - 1);
      if (!more) break;
      const int token = u.t0 + row_token;
      const bool active = r < tile_tokens * s.G && token < u.seq.n_q;
      const int limit = active ? u.before + token + 1 : 0;
      const int head = u.h * s.G + row_head;
      const long long row = u.seq.q0 + token;
      float D = 0.f;
      int top = kNoTop;   // fp16: the row's |dS| < 2^top
      if (u.steps > 0) {
        // Q into tensor memory: S of the last unit has been read, so its Q has been.
        wait(L::kKFull + pk.stage, pk.phase);
        const uint8_t* q = smem + L::kK + pk.stage * kTile + r * 128;
        uint32_t w[kD / 4];   // half of the row's columns
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          const int c = half * (kD / 16) + i;
          const uint4 v = *reinterpret_cast<const uint4*>(q + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4));
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
        packed::st_words(lane_addr + kDqQ + half * (kD / 4), w);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kQIn]);
        for (int i = 0; i <= u.steps; ++i) next(pk, kKs);
        if (!u.exact) {   // D from dout and out, half of the columns each; fp16: |dout| |out| for the power
          float dd = 0.f, oo = 0.f;
          wait(L::kDoFull, uses);
          wait(L::kVFull + pv.stage, pv.phase);
          const uint8_t* x = smem + r * 128;
          const uint8_t* y = smem + L::kV + pv.stage * kTile + r * 128;
#pragma unroll
          for (int i = 0; i < kD / 16; ++i) {
            const int c = half * (kD / 16) + i, at = (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4);
            const uint4 v = *reinterpret_cast<const uint4*>(x + at), o = *reinterpret_cast<const uint4*>(y + at);
            const uint32_t vs[4] = {v.x, v.y, v.z, v.w}, os[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = packed::unpack2<kFp16>(vs[e]), b = packed::unpack2<kFp16>(os[e]);
              D = fmaf(a.x, b.x, fmaf(a.y, b.y, D));
              if (kFp16) {
                dd = fmaf(a.x, a.x, fmaf(a.y, a.y, dd));
                oo = fmaf(b.x, b.x, fmaf(b.y, b.y, oo));
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::kOutRead]);
          next(pv, kVs);
          D = kFp16 ? both_and_top(D, dd, oo, &top) : both(D);
        }
        for (int i = 0; i < u.steps; ++i) next(pv, kVs);
        ++uses;
      }
      const int whole = static_cast<int>(__reduce_min_sync(0xffffffffu, active ? max(limit, 0) : 0x7fffffff)) / 128;
      wait(L::kLse + (k & 1), k >> 1);
      const float lse2 = reinterpret_cast<const float*>(smem + L::kLses)[(k & 1) * 128 + r];
      uint64_t down = packed::pair(-lse2, -lse2);
      // Columns of tile j that the row attends, of this half's 64; 64 where no row of the warp needs a mask.
      auto attended = [&](int j) { return j >= whole ? limit - j * 128 - 64 * half : 64; };
      uint64_t rest = 0ull, squares = 0ull;   // the sums of dS and of its square, times the row's power
      int e = 0;                              // fp16: log2 of what P, and so dS, is multiplied by
      uint32_t z[64], dp[64];
      // P and dout . v of the next step, 64 columns each, of which the tensor cores then form the next.
      auto probs = [&](int j) {
        wait(L::kPair, pairs++);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tc::ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
          tc::ld32(dp_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&dp[32 * c]));
        }
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kFree]);
        const int keep = attended(j);
        if (keep < 64) {   // (a hidden value may be infinite)
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            z[i] = i < keep ? z[i] : 0xff800000u;
            dp[i] = i < keep ? dp[i] : 0u;
          }
        }
      };
      auto prob2 = [&](int i) {   // P of columns 2 i and 2 i + 1
        const float2 e = packed::unpair(
            packed::fma2(packed::pair(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1])), scale2, down));
        return packed::pair(fast_exp2(e.x), fast_exp2(e.y));
      };
      auto value2 = [&](int i) { return packed::pair(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])); };
      // Of the columns in registers: sum P (dout . v - x), and sum P into `weights`.
      uint64_t weights = 0ull;
      auto sum_p = [&](float x) {
        const uint64_t minus_x = packed::pair(-x, -x);
        uint64_t d = 0ull;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint64_t p = prob2(i);
          d = packed::fma2(p, packed::add2(value2(i), minus_x), d);
          weights = packed::add2(p, weights);
        }
        const float2 halves = packed::unpair(d);
        return halves.x + halves.y;
      };
      auto sum_values = [&](uint64_t d) {   // of the columns in registers: sum (dout . v)^2
        uint64_t c = 0ull;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          d = packed::fma2(value2(i), value2(i), d);
          c = packed::fma2(value2(i + 1), value2(i + 1), c);
        }
        return packed::add2(d, c);
      };
      // fp16: the row's D and top_of of its |dS|, for dk and for a unit that is done once more.
      auto put_row = [&](int top) {
        const int in_warp = __reduce_max_sync(0xffffffffu, active ? top : kNoTop);
        if (half == 0 && lane == 0) atomicMax(&tops[k & 1], in_warp);
        const int at = static_cast<int>(row) * (s.Hkv * s.G) + head;   // (heads * tokens < 2^31)
        if (half == 0 && active) g.rows[at] = make_float2(__uint_as_float(static_cast<uint32_t>(top) & 0xffffu), D);
        if (tid == 0) {
          tops[2] = at;
          tops[3] = top;
        }
      };
      // fp16: the row's power, which takes 2^top to 2^to.
      auto set_power = [&](int to) {
        e = power_for(top, to);
        down = packed::pair(e - lse2, e - lse2);
      };
      if (u.again) {
        if (active) {
          const float2 was = g.rows[row * (s.Hkv * s.G) + head];
          D = was.y;
          top = static_cast<int16_t>(__float_as_uint(was.x) & 0xffffu);
        }
        if (kFp16) set_power(14);
      } else if (kFp16 && !u.exact) {
        set_power(10);
      }
      // Both walks in one loop: what a unit runs through is short (the instruction cache).
      float part_of_d = 0.f, moved = 0.f;   // (moved: by how much the scores' D differs from that of out)
      uint64_t values = 0ull;   // fp16: sum (dout . v)^2
      for (int t = 0; t < u.steps; ++t) {
        const bool first_walk = t < u.back;
        probs(first_walk ? t : u.steps - 1 - t);
        // The last tile's sums complete D, where there is one walk (one tile: D and dS are from the same registers).
        const bool completes = t + 1 == u.steps && u.back == 0 && !u.again;
        if (first_walk || completes) {
          part_of_d += sum_p(D);   // (in the first walk D is 0)
          if (kFp16) values = sum_values(values);
          if (completes || t + 1 == u.back) {
            const float2 sums = packed::unpair(rest), squares_of = packed::unpair(values);
            part_of_d += sums.x + sums.y;
            if (kFp16 && u.exact) {   // (the top from all dout . v)
              D = both_and_top(part_of_d, squares_of.x + squares_of.y, 0.5f, &top);
              if (top != kNoTop) top = max(top, top_of(fabsf(D))) + 1;
              set_power(15);
            } else {
              moved = both(part_of_d) * (kFp16 ? power(-e) : 1.f);
              D += moved;
              // The first tile's weight.  (All have read `larger` before: products of several dS, which all warps
              // wait for, are between.)
              const float2 weight = packed::unpair(weights);
              if (!u.exact)
                larger[half * 128 + r] = static_cast<uint16_t>(
                    __float_as_uint((weight.x + weight.y) * (kFp16 ? power(-e) : 1.f)) >> 16);
            }
          }
          if (first_walk) continue;
        }
        const uint64_t minus_d = packed::pair(-D, -D);
        uint32_t ds[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint64_t v = packed::mul2(prob2(i), packed::add2(value2(i), minus_d));
          rest = packed::add2(rest, v);
          squares = packed::fma2(v, v, squares);   // (only long rows need it; a loop without it costs the same)
          const float2 w = packed::unpair(v);
          ds[i] = packed::pack2<kFp16>(w.x, w.y);
        }
        if (summed > 0) wait(L::kDqDone, summed - 1);   // the last dS has been read
        ++summed;
        tc::st32(lane_addr + kDqDs + 32 * half, ds);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kDsFull]);
      }
      if (!u.exact) {   // whether it has to be done once more
        const float2 halves = packed::unpair(squares);
        const float sum = both(halves.x + halves.y);
        const float size = sqrtf(sum) * (kFp16 ? power(-e) : 1.f);   // the norm of dS
        if (kFp16) top = top_of(size + fabsf(moved));   // (dk has the scores' D in all its tiles)
        const bool too_large = kFp16 && sum >= 0x1p31f && sum < INFINITY;
        if (active && too_large) atomicOr(&again[u.number >> 5], 1u << (u.number & 31));
        const float weight = 1.f - __uint_as_float(static_cast<uint32_t>(larger[r]) << 16) -
                             __uint_as_float(static_cast<uint32_t>(larger[128 + r]) << 16);
        float off_by = active ? moved * fmaxf(weight, 0.f) : 0.f, most = active ? size * kHalfStep<kFp16> : 0.f;
        off_by *= off_by;
        most *= most;
        if (!(off_by < INFINITY && most < INFINITY)) off_by = most = 0.f;   // (a row with one in dout has no say)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          off_by += __shfl_xor_sync(0xffffffffu, off_by, o);
          most += __shfl_xor_sync(0xffffffffu, most, o);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");   // (`part` has been read)
        if (half == 0 && lane == 0) {
          part[2 * warp] = off_by;
          part[2 * warp + 1] = most;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 0 && part[0] + part[2] + part[4] + part[6] > part[1] + part[3] + part[5] + part[7])
          atomicOr(&again[u.number >> 5], 1u << (u.number & 31));
      }
      if (kFp16 && !u.again) {
        put_row(top);
      } else if (!u.again && half == 0 && active) {
        g.rows[row * (s.Hkv * s.G) + head] = make_float2(lse2, D);
      }
      const float off = kFp16 ? power(-e) : 1.f;
      if (u.n > 0) wait(L::kDqDone, summed - 1);
      uint16_t* dq = static_cast<uint16_t*>(g.dq) + row * g.dq_st.token + head * g.dq_st.head;
#pragma unroll 1
      for (int c = 0; c < kD / 64; ++c) {
        const int col = half * (kD / 2) + 32 * c;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = 0u;
        if (u.n > 0) {
          tc::ld32(lane_addr + kDqAcc + col, w);
          tc::wait_ld();
        }
        if (active) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = limit > 0 ? packed::pack2<kFp16>(__uint_as_float(w[2 * i]) * off * s.scale,
                                                    __uint_as_float(w[2 * i + 1]) * off * s.scale)
                             : 0u;
          packed::store_row(dq + col, v, wide);
        }
      }
      if (u.n > 0) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kAccFree]);
      }
      unit_done(k);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kPairWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------- dk and dv ----
//
// A CTA (or a cluster, each CTA every ctas-th tile of rows) takes one tile of keys.
// D = 128: two scores and two accumulators fill tensor memory, so P^T lies over S^T
// and dS^T over (v . dout)^T, and the products go round: dv += P^T dout, the next S^T,
// dk += dS^T Q, the next (v . dout)^T, each pair beside the threads' other half step.
// D = 64 leaves room for P^T and dS^T of their own: both scores go into registers at
// once and the next ones are formed while the threads compute, as for dq.

template <int kD>
struct DkvLayout {
  static constexpr int kTile = kD / 64 * 16384;
  static constexpr int kStages = 163840 / kTile;
  static constexpr int kRing = 2 * kTile;   // K and V before it
  static constexpr int kRows = kRing + kStages * kTile;   // two buffers of [128] -lse log2(e), [128] -D
  static constexpr int kBars = kRows + 2 * 1024;
  static constexpr int kKvFull = 0, kFull = 1, kEmpty = kFull + kStages, kRowsFull = kEmpty + kStages,
                       kRowsFree = kRowsFull + 2, kCleared = kRowsFree + 2, kSFull = kCleared + 2,
                       kPFull = kSFull + 1, kDpFull = kPFull + 1, kDsFull = kDpFull + 1, kDone = kDsFull + 1,
                       kUsed = kDone + 1, kEnd = kUsed + 1, kNumBars = kEnd + 2;
  static constexpr int kScratch = kBars + 8 * kNumBars;
  static constexpr int kBytes = kScratch + 160 + 16;   // (no slack: where the base is not aligned the kernel says so)
};
// Tensor memory: S^T, (v . dout)^T, dv, dk and (D = 64) P^T and dS^T.  Over the scores a
// warpgroup's 16-bit values lie over its own 64 columns' first 32.
constexpr uint32_t kKvS = 0, kKvDp = 128, kKvDv = 256;
template <int kD>
constexpr uint32_t kKvDk = kKvDv + kD;
constexpr uint32_t kKvP = 384, kKvDs = 448;

template <int kD, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkv_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnGrads g,
                      const int ctas) {
  using L = DkvLayout<kD>;
  constexpr int kTile = L::kTile, kStages = L::kStages;
  constexpr bool kOwn = kD == 64;   // P^T and dS^T have columns of their own
  constexpr float kDown = 1.f / (1 << kUp<kFp16>);   // takes kUp off dv again
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) % 1024 != 0) {   // (as above)
    if (threadIdx.x == 0) atomicOr(s.status, kStatusBounds);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int* scratch = reinterpret_cast<int*>(smem + L::kScratch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 40);
  uint8_t* ring = smem + L::kRing;
  float* rows = reinterpret_cast<float*>(smem + L::kRows);
  float4* parts = reinterpret_cast<float4*>(ring);   // at the end: this CTA's dv and dk, 2 x 128 rows of kD
  int* top = scratch + 41;   // fp16: the largest top_of of the rows that attend the tile
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;

  pdl_wait();
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

  if (tid == 0) *top = kNoTop;
  if (tid < L::kNumBars) {
    // (D = 64: kSFull is both scores, kPFull that they have been read, kDsFull both of P^T and dS^T.)
    const bool by_warps = tid == L::kPFull || tid == L::kDsFull || tid == L::kRowsFree || tid == L::kRowsFree + 1;
    mbar_init(&bars[tid], by_warps ? 8 : 1);
    fence_barrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
    prefetch_tensormap(&maps.dout);
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
  pdl_trigger();
  bool ok = true;
  auto wait = [&](int bar, int phase) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[bar], phase & 1, s.status));
    tc::fence_after_sync();
  };
  // fp16: what dout . v - D is multiplied by for dS, beside P's 2^kUp, once the computing warps have found `top`.
  auto dp_power = [&]() { return power_for(*top, 14) - kUp<kFp16>; };
  auto top_found = [&]() {
    if (kFp16) asm volatile("bar.sync 1, 288;" ::: "memory");   // (the computing warps and kRowsWarp)
  };

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
      // Each row tile's (lse, D), +inf for a row of no query: its P is 0.  Two tiles are on their way in
      // registers while a buffer is waited for.
      int token_in[4];          // of rows lane, lane + 32, ...: their token in a tile
      long long from[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = lane + 32 * k;
        token_in[k] = r < tile_rows ? r / s.G : 0x40000000;   // (no such token)
        from[k] = static_cast<long long>(seq.q0 + t0 + r / s.G) * (s.Hkv * s.G) + h * s.G + r % s.G;
      }
      const long long step = static_cast<long long>(tile_tokens) * s.Hkv * s.G;
      auto load = [&](int i, float2 (&v)[4]) {
        const int tile = rank + i * ctas, left = seq.n_q - t0 - tile * tile_tokens;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = make_float2(INFINITY, 0.f);
          if (i < n && token_in[k] < left) {
            const long long at = from[k] + tile * step;
            v[k] = kFp16 ? make_float2(g.lse[at], g.rows[at].y) : g.rows[at];   // (fp16: lse as it is, see put)
          }
        }
      };
      float d_power = 1.f;
      auto put = [&](int i, const float2 (&v)[4]) {
        float* to = rows + (i & 1) * 256 + lane;
        if (i >= 2) wait(L::kRowsFree + (i & 1), i / 2 - 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          to[32 * k] = kUp<kFp16> - (kFp16 ? v[k].x * kLog2e : v[k].x);   // negated: what is added
          to[128 + 32 * k] = -v[k].y * d_power;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kRowsFull + (i & 1)]);
      };
      float2 even[4], odd[4];
      load(0, even);
      load(1, odd);
      if (kFp16 && n > 0) {
        top_found();
        d_power = power(dp_power());
      }
      for (int i = 0; i < n && ok; i += 2) {
        put(i, even);
        load(i + 2, even);
        if (i + 1 < n) put(i + 1, odd);
        load(i + 3, odd);
      }
    } else if (warp == kMmaWarp && n > 0) {
      constexpr uint32_t kIdS = packed::idesc<kFp16>(128, 128, 0, 0);
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t k_desc = packed::desc_rows(smem_u32(smem));
      const uint64_t v_desc = packed::desc_rows(smem_u32(smem + kTile));
      const uint64_t rows_desc = packed::desc_rows(smem_u32(ring));
      const uint64_t cols_desc = packed::desc_cols(smem_u32(ring));
      const bool issuer = packed::elect_one();
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
      if constexpr (kOwn) {
        for (int i = 0; i < n && ok; ++i) {
          if (!loaded(2 * i) || !loaded(2 * i + 1)) break;
          if (i > 0) wait(L::kPFull, i - 1);   // both scores have been read
          if (issuer) {
            packed::mma_rows<kD>(tmem + kKvS, k_desc, rows_desc + stage(2 * i), kIdS);
            packed::mma_rows<kD>(tmem + kKvDp, v_desc, rows_desc + stage(2 * i + 1), kIdS);
            tc::commit(&bars[L::kSFull]);
          }
          __syncwarp();
        }
        packed::products_end(&bars[L::kEnd], issuer, s.status);
      } else {
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
            packed::mma_cols<64>(tmem + kKvDk<kD>, tmem + kKvDp, cols_desc + stage(2 * i), kIdO, i > 0);
            tc::commit(&bars[L::kEmpty + (2 * i) % kStages]);
          }
          __syncwarp();
          if (i + 1 < n) inner(i + 1);
        }
        if (ok && issuer) tc::commit(&bars[L::kDone]);
        packed::products_end(&bars[L::kEnd], issuer, s.status);
      }
    } else if (kOwn && warp == kKvSumWarp && n > 0) {
      constexpr uint32_t kIdO = packed::idesc<kFp16>(128, kD, 0, 1);
      const uint64_t cols_desc = packed::desc_cols(smem_u32(ring));
      const bool issuer = packed::elect_one();
      int at = 0;   // the stage of Q_i; dout_i is in the next
      for (int i = 0; i < n && ok; ++i) {
        const uint64_t q = cols_desc + static_cast<uint64_t>(at * (kTile >> 4));
        const uint64_t dout = cols_desc + static_cast<uint64_t>((at + 1) * (kTile >> 4));
        wait(L::kDsFull, i);
        if (!ok) break;
        if (issuer) {
          packed::mma_cols(tmem + kKvDv, tmem + kKvP, dout, kIdO, i > 0);
          packed::mma_cols(tmem + kKvDk<kD>, tmem + kKvDs, q, kIdO, i > 0);
          tc::commit(&bars[L::kUsed]);
          tc::commit(&bars[L::kEmpty + at]);
          tc::commit(&bars[L::kEmpty + at + 1]);
        }
        __syncwarp();
        at += 2;   // (an even number of stages)
        if (at == kStages) at = 0;
      }
      if (ok && issuer) tc::commit(&bars[L::kDone]);
      packed::products_end(&bars[L::kEnd + 1], issuer, s.status);
    }
    __syncwarp();
  } else {
    packed::regs_up<216>();
    const int half = warp >> 2;   // query rows 64 half .. 64 half + 63 of a tile
    const int key = key0 + (tid & 127);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int warp_last = key0 + (warp & 3) * 32 + 31;
    const uint64_t scale2 = packed::pair(s.scale2, s.scale2);
    float d_power = 1.f;
    if (kFp16 && n > 0) {   // (while the first tiles are on their way)
      const int tiles = (seq.n_q + tile_tokens - 1) / tile_tokens;
      int mine = kNoTop;
      for (int i = t0 / tile_tokens + tid; i < tiles; i += 256) {
        const float2* first = g.rows + (seq.q0 + static_cast<long long>(i) * tile_tokens) * (s.Hkv * s.G) + h * s.G;
        mine = max(mine, static_cast<int>(__float_as_uint(first->x)) >> 16);
      }
      mine = __reduce_max_sync(0xffffffffu, mine);
      if (lane == 0) atomicMax(top, mine);
      top_found();
      d_power = power(dp_power());
    }
    const uint64_t up = packed::pair(d_power, d_power);
    for (int i = 0; i < n; ++i) {
      // Rows of tokens before key - before do not attend the key.
      const int token0 = tile_token(i);
      const int from = (key - before - token0) * s.G - 64 * half;
      const bool masked = warp_last - before > token0;
      const float4* lse2 = reinterpret_cast<const float4*>(rows + (i & 1) * 256 + 64 * half);
      const float4* D = reinterpret_cast<const float4*>(rows + (i & 1) * 256 + 128 + 64 * half);
      wait(L::kRowsFull + (i & 1), i >> 1);
      if constexpr (kOwn) {
        uint32_t z[64], dp[64];
        wait(L::kSFull, i);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tc::ld32(lane_addr + kKvS + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
          tc::ld32(lane_addr + kKvDp + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&dp[32 * c]));
        }
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kPFull]);
        uint32_t p[32], ds[32];
        auto compute = [&](auto masks) {
          constexpr bool kMasks = decltype(masks)::value;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 m = lse2[c], d = D[c];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = 4 * c + 2 * e;
              const uint64_t minus_m = e ? packed::pair(m.z, m.w) : packed::pair(m.x, m.y);
              const uint64_t minus_d = e ? packed::pair(d.z, d.w) : packed::pair(d.x, d.y);
              float2 x = packed::unpair(packed::fma2(
                  packed::pair(__uint_as_float(z[at]), __uint_as_float(z[at + 1])), scale2, minus_m));
              x.x = fast_exp2(x.x);
              x.y = fast_exp2(x.y);
              if (kMasks) {
                x.x = at >= from ? x.x : 0.f;
                x.y = at + 1 >= from ? x.y : 0.f;
              }
              p[at / 2] = packed::pack2<kFp16>(x.x, x.y);
              const uint64_t v = packed::pair(__uint_as_float(dp[at]), __uint_as_float(dp[at + 1]));
              const float2 y = packed::unpair(packed::mul2(
                  packed::pair(x.x, x.y), kFp16 ? packed::fma2(v, up, minus_d) : packed::add2(v, minus_d)));
              ds[at / 2] = packed::pack2<kFp16>(y.x, y.y);
              if (kMasks) {   // a hidden row's 0 stays 0 beside an infinity
                if (at + 1 < from) ds[at / 2] = 0u;
                if (at < from) ds[at / 2] &= 0xffff0000u;
              }
            }
          }
        };
        if (masked) {
          compute(std::true_type());
        } else {
          compute(std::false_type());
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kRowsFree + (i & 1)]);
        if (i > 0) wait(L::kUsed, i - 1);   // the last P^T and dS^T have been read
        tc::st32(lane_addr + kKvP + 32 * half, p);
        tc::st32(lane_addr + kKvDs + 32 * half, ds);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kDsFull]);
      } else {
        uint32_t z[64];
        wait(L::kSFull, i);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tc::ld32(lane_addr + kKvS + 64 * half + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&z[32 * c]));
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 m = lse2[c];
          const float2 a = packed::unpair(packed::fma2(
              packed::pair(__uint_as_float(z[4 * c]), __uint_as_float(z[4 * c + 1])), scale2, packed::pair(m.x, m.y)));
          const float2 e = packed::unpair(packed::fma2(
              packed::pair(__uint_as_float(z[4 * c + 2]), __uint_as_float(z[4 * c + 3])), scale2,
              packed::pair(m.z, m.w)));
          z[4 * c] = __float_as_uint(fast_exp2(a.x));
          z[4 * c + 1] = __float_as_uint(fast_exp2(a.y));
          z[4 * c + 2] = __float_as_uint(fast_exp2(e.x));
          z[4 * c + 3] = __float_as_uint(fast_exp2(e.y));
        }
        if (masked) {
#pragma unroll
          for (int c = 0; c < 64; ++c) z[c] = c >= from ? z[c] : 0u;
        }
        uint32_t p[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
          p[c] = packed::pack2<kFp16>(__uint_as_float(z[2 * c]), __uint_as_float(z[2 * c + 1]));
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
            const uint64_t v0 = packed::pair(__uint_as_float(dp[4 * e]), __uint_as_float(dp[4 * e + 1]));
            const uint64_t v1 = packed::pair(__uint_as_float(dp[4 * e + 2]), __uint_as_float(dp[4 * e + 3]));
            const uint64_t d0 = packed::pair(d.x, d.y), d1 = packed::pair(d.z, d.w);
            const float2 a = packed::unpair(packed::mul2(packed::pair(__uint_as_float(zz[0]), __uint_as_float(zz[1])),
                                                         kFp16 ? packed::fma2(v0, up, d0) : packed::add2(v0, d0)));
            const float2 b = packed::unpair(packed::mul2(packed::pair(__uint_as_float(zz[2]), __uint_as_float(zz[3])),
                                                         kFp16 ? packed::fma2(v1, up, d1) : packed::add2(v1, d1)));
            p[16 * c + 2 * e] = packed::pack2<kFp16>(a.x, a.y);
            p[16 * c + 2 * e + 1] = packed::pack2<kFp16>(b.x, b.y);
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
    }
    if (n > 0) wait(L::kDone, 0);
    // ---- the first warpgroup has dv, the second dk ----
    const bool active = key < seq.n_k;
    const PackedStride st = half ? g.dk_st : g.dv_st;
    uint16_t* to = static_cast<uint16_t*>(half ? g.dk : g.dv) + static_cast<long long>(seq.k0 + key) * st.token +
                   h * st.head;
    const float scale = half ? s.scale : kDown;
    const float off = kFp16 && n > 0 ? power(-dp_power() - kUp<kFp16>) : 1.f;   // takes dS's power off dk
    const bool wide = packed::wide_rows(half ? g.dk : g.dv, st);
#pragma unroll 1
    for (int c = 0; c < kD / 32; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0u;
      if (n > 0) {
        tc::ld32(lane_addr + (half ? kKvDk<kD> : kKvDv) + 32 * c, w);
        tc::wait_ld();
        if (kFp16 && half) {
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * off);
        }
      }
      if (ctas > 1) {   // into this CTA's ring, which is free now
#pragma unroll
        for (int i = 0; i < 8; ++i)
          parts[packed::swizzled<kD>(half * 128 + (tid & 127), 8 * c + i)] =
              make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]), __uint_as_float(w[4 * i + 2]),
                          __uint_as_float(w[4 * i + 3]));
      } else if (active) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          p[i] = packed::pack2<kFp16>(__uint_as_float(w[2 * i]) * scale, __uint_as_float(w[2 * i + 1]) * scale);
        packed::store_row(to + 32 * c, p, wide);
      }
    }
  }
  if (ctas > 1) {
    // ---- every CTA sums its share of the rows over the cluster, in the order of the ranks ----
    __syncwarp();
    cluster_sync();
    if (warp < 8) {   // (the others have given registers away)
      const int row0 = rank * 256 / ctas, share = (rank + 1) * 256 / ctas - row0;   // rows of dv, then of dk
      for (int e = tid; e < share * (kD / 4); e += 256) {
        const int row = row0 + e / (kD / 4), c4 = e % (kD / 4);
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
cudaError_t launch_one(packed::SharedMemory& shared, Kernel kernel, int bytes, long long units, int ctas,
                       cudaStream_t st, const More&... args) {
  const cudaError_t e = shared.allow(kernel, bytes);
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
  const long long tiles = most_tiles(s.Tq, packed_tile_tokens(s.G), s.B) * s.Hkv;
  static packed::SharedMemory shared[2];   // of each kernel
  const cudaError_t e = launch_one(shared[0], packed_dq_kernel<kD, kFp16>, DqLayout<kD>::kBytes,
                                   std::min<long long>(tiles, device_sm_count()), 1, st, maps, s, g);
  if (e != cudaSuccess) return e;
  // CTAs per tile of keys.  Causal tiles differ by the whole length of the sequence, so
  // units that are few leave SMs idle behind the longest: with kernels before these the gradient
  // of one 8K sequence with 2 KV heads took 1.13 ms with clusters of 4 (which find 144 of the
  // 152 SMs), 1.16 with 2, 1.35 with 7 (105 SMs) and 1.72 alone.  That of 16 documents (640
  // units) took 0.47 ms alone and 0.52 with 2: enough units, and the join costs a few row
  // tiles.  Clusters of 8 where all their units run at once: both kernels 41 us instead of 50 (10 units
  // of 1200 tokens, group 8, d 128), 45 instead of 58 (18 of 1100, group 16, d 64); with 32
  // units (2000 tokens, group 4) 63 instead of 50.
  const long long units = ((s.Tk + s.B - 1) / s.B + 127) / 128 * static_cast<long long>(s.B) * s.Hkv;
  const long long row_tiles = static_cast<long long>(s.Tq) * s.G / 128 / s.B;
  const int sms = device_sm_count();
  int ctas = 1;
  while (ctas < 4 && units * ctas < 2 * sms && row_tiles >= 12 * ctas) ctas *= 2;
  if (ctas == 4 && units * 8 <= sms && row_tiles >= 48) ctas = 8;
  return launch_one(shared[1], packed_dkv_kernel<kD, kFp16>, DkvLayout<kD>::kBytes, most_tiles(s.Tk, 128, s.B) * s.Hkv,
                    ctas, st, maps, s, g, ctas);
}

}  // namespace

cudaError_t launch_packed_attn_bwd(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                                   const PackedAttnGrads& g, cudaStream_t st) {
  if (D == 128) return fp16 ? launch<128, true>(s, maps, g, st) : launch<128, false>(s, maps, g, st);
  return fp16 ? launch<64, true>(s, maps, g, st) : launch<64, false>(s, maps, g, st);
}

}  // namespace infllmv2
