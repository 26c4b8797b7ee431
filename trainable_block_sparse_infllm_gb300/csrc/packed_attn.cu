// Causal attention over packed sequences: out = softmax(scale q k^T) v.
//
// The group's heads share their keys, so the rows of a tile are (token, head of
// the group) pairs, token by token: 128 / G tokens of G heads fill a 128-row
// product whatever the group, and a short prompt wastes few rows.  Online softmax
// in base 2: with m >= the row's scores (up to 2^8, see below), x = sum 2^(z - m) v
// and l = sum 2^(z - m) are kept per row, and out = x / l.  One pass over the keys.
//
// A unit is two adjacent tiles (256 rows) of one sequence and KV head; it walks the
// keys in tiles of 128 up to the last one that a row attends.  A CTA stays on its SM
// and takes one unit after another, the longest first; while a unit's last tiles are
// finished the next one's copies and first scores are under way.
//   warps 0-3, 4-7  softmax of the first and second tile; a thread is a row.  S
//              comes from tensor memory, P (16 bits) goes back over it, which makes
//              it the A operand of P V.  The running maximum moves only when it
//              grows by more than 2^8, which is rare, so x is rarely rescaled.
//   warp 8     issues the products of both tiles in turn: while one tile's softmax
//              runs, the other's P V and next Q K^T keep the tensor cores busy.
//   warp 9     finds the units; TMA: both Q tiles, then K_0, V_0, K_1, V_1, ...
//              through a ring that goes on from unit to unit.
//   warps 10, 11 (D = 64: 11; 10 issues the scores, 8 the P V)  look through the V
//              tiles that some row attends in part (at most three): a zero
//              probability must meet no infinity or NaN.  Rows behind the
//              sequence's end are cleared; a row of the sequence that holds one is
//              cleared too, and the rows that attend it add it at the end, one by one.
// Jobs (a tile's scores for one tile of keys, then P V) go through the score buffers
// in tensor memory in turn, columns of 128: two for D = 128 and three for D = 64,
// beside two accumulators of D.  S of job k overwrites P of job k - 2 or k - 3, so it goes
// out behind that P V.  With three buffers the next scores of a tile are there before
// its softmax ends.  An issuer that waits or computes addresses leaves the tensor
// cores idle (their queue is short): the jobs of D = 64 are so small that two warps
// share them, and the loop of D = 128 has its halves unrolled.
// Few queries against many keys (drafted tokens, a short chunk after a long past)
// leave most SMs without a unit: its key tiles are then divided over a cluster,
// whose CTAs join their (m, l, x) through distributed shared memory.
//
// Measured (GB300): one prompt of 16,384 tokens, 2 KV heads of 16, d 128, 1.24 to 1.36 ms,
// 1.62 to 1.78 PFLOP/s, 85 to 93% of the measured library product: the tensor cores
// (72% busy at 8K, the rest goes to the handing over of S and P).  24 prompts of up to
// 2047 tokens, 8 heads of 4, d 64, 170 us (177 in turn with other work): the softmax warps' chain of a tile (1.9
// thousand cycles, two warps of a scheduler, a quarter of it waiting for S) and 2.2
// thousand cycles at the end of units of five tiles.  12 tokens after 32,000 in 4
// sequences 47 us: the 8 units' clusters have 12 CTAs, 96 SMs.  One prompt of 301
// tokens 8.7 us in a graph.  With the products issued by lane 0 of a diverged warp the
// first took 1.92 ms, with a CTA for each unit the second took 283 us.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "kernels.h"
#include "packed_attn.cuh"

namespace infllmv2 {

namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kCheckWarp = 10;
constexpr int kMaxPartial = 3;   // V tiles that rows attend in part: 256 queries' own keys lie in three tiles at most
constexpr float kLazy = 8.0f;   // log2 of how far scores may pass the running maximum
// log2 of P at the running maximum.  fp16 loses what is below 2^-25, which many
// small probabilities could add up to; its largest value leaves room for 2^(6 + 8).
template <bool kFp16>
constexpr float kTop = kFp16 ? 6.0f : 0.0f;

// kTiles: CTAs have more than one unit; whole tiles of out go through shared memory and
// TMA, since a warp's stores of 32 rows at once, 32 bytes of each, take twice the time
// of whole lines (24 prompts of up to 2047 tokens, d 64: 177 us or 170; 48 of 512,
// d 128: 149 or 142).  kFew: they have one, and leave that out, for each SM meets the code
// only once (one prompt of 301 tokens: 11.3 us or 10.6).  kSplit: one unit per cluster,
// among whose CTAs its key tiles are divided.
enum class Form { kFew, kTiles, kSplit };

template <int kD, Form kForm>
struct Layout {
  static constexpr int kTile = kD / 64 * 16384;   // 128 rows of kD
  static constexpr int kRing = kD == 128 && kForm == Form::kTiles ? 131072 : 163840;   // bytes of the K / V ring
  static constexpr int kStages = kRing / kTile;
  static constexpr int kBuffers = kD == 64 ? 3 : 2;   // of scores
  // V tiles that may be looked through at once, as many as the ring holds: each has barriers of its own, so
  // that none is two phases ahead of who waits for it.
  static constexpr int kLooks = (kStages + 1) / 2;
  static constexpr uint32_t kColO = 128 * kBuffers;
  static constexpr int kOut = 2 * kTile + kRing;   // kTiles: 64 columns of out for each half
  static constexpr int kBars = kOut + (kForm == Form::kTiles ? 2 * 16384 : 0);
  // Barriers: a unit found and done with; Q of each tile full and free; ring full and empty; V tiles
  // attended in part, before and after they were looked through; of each tile S (three buffers: three, in
  // turn); of each score buffer P; of each tile P V (three, in turn) and x read; kSplit: all products; of each
  // score buffer P V once more, for who issues scores; and all that each issuer issued.
  static constexpr int kUnit = 0, kUnitFree = kUnit + 2, kQFull = kUnitFree + 2, kQFree = kQFull + 2,
                       kFull = kQFree + 2, kEmpty = kFull + kStages, kPartial = kEmpty + kStages,
                       kChecked = kPartial + kLooks, kSFull = kChecked + kLooks,
                       kPFull = kSFull + (kBuffers == 3 ? 6 : 2), kPvDone = kPFull + kBuffers,
                       kOFree = kPvDone + 6, kAllDone = kOFree + 2, kReused = kAllDone + 1,
                       kEnd = kReused + kBuffers, kNumBars = kEnd + 2;
  static constexpr int kUnits = kBars + (8 * kNumBars + 15) / 16 * 16;   // two units, 32 bytes each
  static constexpr int kFlags = kUnits + 2 * 32;   // of each unit [kMaxPartial][4]: rows that were cleared
  static constexpr int kSlot = kFlags + 2 * kMaxPartial * 16;
  static constexpr int kBytes = kSlot + 16 + 1024;   // and slack to align the tiles
};

// What the roles need to know of a unit.  All tile indexes count from key tile j0.
struct Unit {
  packed::Sequence seq;
  int t0, h;             // its first query and its KV head
  int before;            // query t attends keys 0 .. before + t
  int j0, n_tiles[2], n;
  int partial, looked;   // the first key tile that some row attends in part, and that is looked through
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

template <int kD, bool kFp16, Form kForm>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attn_kernel(const __grid_constant__ PackedAttnMaps maps, const PackedAttnShape s, const PackedAttnIn in,
                       const PackedAttnOut o, const int ctas, const int halves) {
  using L = Layout<kD, kForm>;
  constexpr bool kSplit = kForm == Form::kSplit, kTiles = kForm == Form::kTiles;
  constexpr int kTile = L::kTile, kStages = L::kStages, kBuffers = L::kBuffers;
  constexpr uint32_t kColO = L::kColO;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int4* units = reinterpret_cast<int4*>(smem + L::kUnits);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + L::kFlags);
  uint8_t* ring = smem + 2 * kTile;
  // kSplit, at the end, over the ring: x of this CTA's 256 rows, their (m, l), and the weights of the share it joins.
  float4* parts = reinterpret_cast<float4*>(ring);
  float2* sums = reinterpret_cast<float2*>(ring + 256 * kD * 4);
  float* weights = reinterpret_cast<float*>(sums + 256);   // [rows of the share][16]
  const int tid = threadIdx.x, warp = packed::warp_index(), lane = tid & 31;
  const int tile_tokens = packed_tile_tokens(s.G);
  const int rank = kSplit ? static_cast<int>(blockIdx.x) % ctas : 0;

  if (tid < L::kNumBars) {
    int count = 1;
    if (tid == L::kUnitFree || tid == L::kUnitFree + 1) count = 11;   // the warps but the one that finds units
    if ((tid >= L::kPFull && tid < L::kPFull + kBuffers) || (tid >= L::kOFree && tid < L::kOFree + 2)) count = 4;
    if (tid >= L::kChecked && tid < L::kChecked + L::kLooks) count = kBuffers == 2 ? 2 : 1;
    mbar_init(&bars[tid], count);
    fence_barrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  // Tensor memory is taken once the kernel before has ended and before the next one may start: neither ever
  // waits for columns that the other holds.
  pdl_wait();
  packed::Walker walker;   // of the warp that finds the units
  bool bad = false;
  if (warp == kTmaWarp) walker.start(s, halves * tile_tokens, false, &bad);
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  // A unit from where it lies, (whether there is one, index of its two tiles, KV head), and its sequence.
  auto unit_of = [&](int4 at, int4 rows) {
    Unit u;
    u.seq = {rows.x, rows.y, rows.z, rows.w};
    u.t0 = at.y * halves * tile_tokens;
    u.h = at.z;
    u.before = u.seq.n_k - u.seq.n_q;
    u.j0 = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {   // each half: up to its last query's own key
      const int first = u.t0 + x * tile_tokens, last = min(first + tile_tokens, u.seq.n_q) - 1;
      u.n_tiles[x] = x >= halves || last < first ? 0 : (max(u.before + last + 1, 0) + 127) / 128;
    }
    if (kSplit) {
      const int all = max(u.n_tiles[0], u.n_tiles[1]), j1 = (rank + 1) * all / ctas;
      u.j0 = rank * all / ctas;
      u.n_tiles[0] = max(min(u.n_tiles[0], j1) - u.j0, 0);
      u.n_tiles[1] = max(min(u.n_tiles[1], j1) - u.j0, 0);
    }
    u.n = max(u.n_tiles[0], u.n_tiles[1]);
    u.partial = max(u.before + u.t0 + 1, 0) / 128 - u.j0;
    u.looked = max(u.partial, 0);
    return u;
  };
  // The next unit, for the warps that do not find it: false past the last one, or after a wait that gave up.
  auto next_unit = [&](int k, bool* ok, Unit* u) {
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
  Unit u;
  bool any = false;   // a softmax warp: the CTA had a unit (kSplit: its only one)

  if (warp >= 8) {
    packed::regs_down<72>();
    if (warp == kTmaWarp) {
      // ---------------------------------------------------- units and loads
      bool ok = true;
      int issued = 0, seen = 0, q_uses[2] = {0, 0};   // ring copies, V tiles looked through, Q tiles
      const int stride = kSplit ? 1 : static_cast<int>(gridDim.x);
      for (int k = 0;; ++k) {
        // Unit number k of this CTA: down the order of all and back, so that none gets the longest of each round.
        int i = kSplit ? static_cast<int>(blockIdx.x) / ctas : static_cast<int>(blockIdx.x);
        if (!kSplit) i = k * stride + (k & 1 ? stride - 1 - i : i);
        int4 at = make_int4(-1, 0, i % s.Hkv, 0), rows = make_int4(0, 0, 0, 0);
        int b, level;
        if (!(kSplit && k > 0) && walker.find(s, i / s.Hkv, halves * tile_tokens, false, &b, &level, &bad)) {
          at.x = 0;
          at.y = level;
          const packed::Sequence seq = packed::sequence(s, b, &bad);
          rows = make_int4(seq.q0, seq.n_q, seq.k0, seq.n_k);
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
        const uint32_t row_bytes = tile_tokens * s.G * kD * 2;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (u.n_tiles[x] == 0) continue;
          if (q_uses[x] > 0 && ok)
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kQFree + x], (q_uses[x] - 1) & 1, s.status));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars[L::kQFull + x], row_bytes);
            for (int c = 0; c < kD / 64; ++c)
              packed::tma_load_4d(smem_u32(smem + x * kTile + c * 16384), &maps.q, c * 64, 0, u.h,
                                  u.seq.q0 + u.t0 + x * tile_tokens, &bars[L::kQFull + x]);
          }
          ++q_uses[x];
        }
        for (int i2 = 0; i2 < 2 * u.n && ok; ++i2) {
          const int st = issued % kStages, j = i2 >> 1;
          if (issued >= kStages)
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kEmpty + st], (issued / kStages - 1) & 1, s.status));
          if (!ok) break;
          // A V tile to be looked through lands on a barrier of its own; its stage's only counts the turn.
          uint64_t* bar = &bars[L::kFull + st];
          const bool looks = (i2 & 1) && j >= u.looked;
          if (lane == 0) {
            if (looks) {
              mbar_arrive(bar);
              bar = &bars[L::kPartial + seen % L::kLooks];
            }
            mbar_arrive_expect_tx(bar, kTile);
            for (int c = 0; c < kD / 64; ++c)
              packed::tma_load_3d(smem_u32(ring + st * kTile + c * 16384), i2 & 1 ? &maps.v : &maps.k, c * 64,
                                  u.seq.k0 + (u.j0 + j) * 128, u.h, bar);
          }
          seen += looks;
          ++issued;
        }
        __syncwarp();
      }
      if (kSplit && blockIdx.x == 0) {   // (its only unit is behind it: on to the end, where bad starts may be)
        int b, level;
        walker.find(s, 0x7fffffff, halves * tile_tokens, false, &b, &level, &bad);
      }
      if (bad && blockIdx.x == 0) atomicOr(s.status, kStatusBadKvLen);
      // The CTA outlives its copies, also after a wait that gave up.  (Each barrier's last copy is its
      // newest phase here.)
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait(&bars[L::kFull + i % kStages], (i / kStages) & 1, s.status);
      for (int i = max(0, seen - L::kLooks); i < seen; ++i)
        mbar_wait(&bars[L::kPartial + i % L::kLooks], (i / L::kLooks) & 1, s.status);
      for (int x = 0; x < 2; ++x)
        if (q_uses[x] > 0) mbar_wait(&bars[L::kQFull + x], (q_uses[x] - 1) & 1, s.status);
    } else if (warp > kCheckWarp || (kBuffers == 2 && warp == kCheckWarp)) {
      // ---------------------------------------------- V attended in part
      bool ok = true;
      int copies = 0, seen = 0;
      for (int k = 0; next_unit(k, &ok, &u); ++k) {
        for (int j = u.looked; j < u.n && ok; ++j, ++seen) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kPartial + seen % L::kLooks], (seen / L::kLooks) & 1,
                                                 s.status));
          if (!ok) break;
          for (int half = 0; half < 2; ++half)   // (two warps share a tile, or one has all of it)
            if (kBuffers == 3 || half == warp - kCheckWarp)
              packed::check_rows<kD, kFp16>(ring + (copies + 2 * j + 1) % kStages * kTile, half,
                                            u.seq.n_k - (u.j0 + j) * 128,
                                            flags + ((k & 1) * kMaxPartial + j - u.looked) * 4);
          if (lane == 0) mbar_arrive(&bars[L::kChecked + seen % L::kLooks]);
        }
        copies += 2 * u.n;
        unit_done(k);
      }
    } else {
      // ----------------- products (three buffers: scores by warp 10, P V by warp 8)
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
      auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      // Where the scores' and the P V stream are: stage and phase in the ring (every other place is a K),
      // score buffer and phase.  They go on from unit to unit.
      struct Stream {
        int stage, stage_phase, buffer, buffer_phase;
      };
      Stream ss = {0, 0, 0, 0}, sv = {1, 0, 0, 0};
      auto next_tile = [](Stream& t) {
        t.stage += 2;
        if (t.stage >= kStages) {
          t.stage -= kStages;
          t.stage_phase ^= 1;
        }
      };
      auto next_buffer = [](Stream& t) {
        if (++t.buffer == kBuffers) {
          t.buffer = 0;
          t.buffer_phase ^= 1;
        }
      };
      // Of each half: its units and the turn of its barriers (of P V, or of S); and V tiles looked through.
      // (After a wait that gave up nothing waits any more; what is issued then stays within this CTA's memory.)
      int used[2] = {0, 0}, turn[2] = {0, 0}, look = 0, look_phase = 0, jobs = 0;
      auto next_turn = [&](int& t) { t = t == 2 ? 0 : t + 1; };
      auto values = [&](bool checked) {   // this tile's V is there
        if (!checked) {
          wait(L::kFull + sv.stage, sv.stage_phase);
          return;
        }
        wait(L::kChecked + look, look_phase);
        if (++look == L::kLooks) {
          look = 0;
          look_phase ^= 1;
        }
      };
      for (int k = 0; next_unit(k, &ok, &u); ++k) {
        const int n0 = uniform(u.n_tiles[0]), n1 = uniform(u.n_tiles[1]), looked = uniform(u.looked);
        const int n = max(n0, n1);
        if constexpr (kBuffers == 2) {
          // A buffer for each half; both in turn, each P V followed by the half's next scores.
          auto scores = [&](auto half, bool first, bool last) {
            constexpr int x = decltype(half)::value;
            if (first) wait(L::kQFull + x, used[x]);
            if (issuer) {
              packed::mma_rows<kD>(tmem + x * 128, q_desc + (x * kTile >> 4),
                                   k_desc + static_cast<uint64_t>(ss.stage * (kTile >> 4)), kIdS);
              tc::commit(&bars[L::kSFull + x]);
              if (last) tc::commit(&bars[L::kQFree + x]);
            }
            __syncwarp();
          };
          auto job = [&](auto half, int j, int mine) {
            constexpr int x = decltype(half)::value;
            if (j == 0 && used[x] > 0) wait(L::kOFree + x, used[x] - 1);   // the last unit's x has been read
            wait(L::kPFull + x, x ? ss.buffer_phase : sv.buffer_phase);
            if (x) {
              ss.buffer_phase ^= 1;
            } else {
              sv.buffer_phase ^= 1;
            }
            if (issuer) {
              packed::mma_cols(tmem + kColO + x * kD, tmem + x * 128,
                               v_desc + static_cast<uint64_t>(sv.stage * (kTile >> 4)), kIdO, j > 0);
              if (j + 1 == mine) tc::commit(&bars[L::kPvDone + 3 * x + turn[x]]);
            }
            __syncwarp();
            if (j + 1 < mine) scores(half, false, j + 2 == mine);
          };
          using Half0 = std::integral_constant<int, 0>;
          using Half1 = std::integral_constant<int, 1>;
          if (n > 0) wait(L::kFull + ss.stage, ss.stage_phase);
          if (n0 > 0) scores(Half0(), true, n0 == 1);
          if (n1 > 0) scores(Half1(), true, n1 == 1);
          for (int j = 0; j < n; ++j) {
            if (issuer) tc::commit(&bars[L::kEmpty + ss.stage]);   // K of tile j
            __syncwarp();
            next_tile(ss);
            values(j >= looked);
            if (j + 1 < n) wait(L::kFull + ss.stage, ss.stage_phase);
            if (j < n0) job(Half0(), j, n0);
            if (j < n1) job(Half1(), j, n1);
            if (issuer) tc::commit(&bars[L::kEmpty + sv.stage]);
            __syncwarp();
            next_tile(sv);
          }
          if (n0 > 0) next_turn(turn[0]);
          if (n1 > 0) next_turn(turn[1]);
        } else {
          // The unit's jobs: the halves in turn, then what the longer one has more.
          const int both = min(n0, n1), total = n0 + n1, longer = n1 > n0 ? 1 : 0;
          int xs = both > 0 ? 0 : longer, js = 0, xv = xs, jv = 0;
          auto next_job = [&](int& x, int& j) {   // true where the tile of keys changes
            if (x == 0 && j < both) {
              x = 1;
              return false;
            }
            ++j;
            x = j < both ? 0 : longer;
            return true;
          };
          for (int i = 0; i < total && warp == kCheckWarp; ++i) {
            const int x = xs, j = js;
            if (j == 0) wait(L::kQFull + x, x ? used[1] : used[0]);
            if (i == 0 || x == 0 || j >= both) wait(L::kFull + ss.stage, ss.stage_phase);
            const bool q_free = j + 1 == (x ? n1 : n0);
            const bool changes = next_job(xs, js) || i + 1 == total;   // K's last reader
            if (jobs >= kBuffers) wait(L::kReused + ss.buffer, ss.buffer_phase ^ 1);
            ++jobs;
            if (issuer) {
              packed::mma_rows<kD>(tmem + ss.buffer * 128, q_desc + (x ? kTile >> 4 : 0),
                                   k_desc + static_cast<uint64_t>(ss.stage * (kTile >> 4)), kIdS);
              tc::commit(&bars[L::kSFull + (x ? 3 + turn[1] : turn[0])]);
              if (changes) tc::commit(&bars[L::kEmpty + ss.stage]);
              if (q_free) tc::commit(&bars[L::kQFree + x]);
            }
            __syncwarp();
            next_buffer(ss);
            if (x) {
              next_turn(turn[1]);
            } else {
              next_turn(turn[0]);
            }
            if (changes) next_tile(ss);
          }
          bool opens = true;   // a tile whose V has not been waited for
          for (int i = 0; i < total && warp == kMmaWarp; ++i) {
            const int x = xv, j = jv;
            if (opens) values(j >= looked);
            opens = next_job(xv, jv) || i + 1 == total;   // V's last reader
            if (j == 0 && (x ? used[1] : used[0]) > 0) wait(L::kOFree + x, (x ? used[1] : used[0]) - 1);
            wait(L::kPFull + sv.buffer, sv.buffer_phase);
            if (issuer) {
              packed::mma_cols(tmem + kColO + (x ? kD : 0), tmem + sv.buffer * 128,
                               v_desc + static_cast<uint64_t>(sv.stage * (kTile >> 4)), kIdO, j > 0);
              tc::commit(&bars[L::kReused + sv.buffer]);
              tc::commit(&bars[L::kPvDone + (x ? 3 + turn[1] : turn[0])]);
              if (opens) tc::commit(&bars[L::kEmpty + sv.stage]);
            }
            __syncwarp();
            next_buffer(sv);
            if (x) {
              next_turn(turn[1]);
            } else {
              next_turn(turn[0]);
            }
            if (opens) next_tile(sv);
          }
        }
        if (kSplit && issuer && warp == kMmaWarp) tc::commit(&bars[L::kAllDone]);
        __syncwarp();
        used[0] += n0 > 0;
        used[1] += n1 > 0;
        unit_done(k);
      }
      // Nothing that was issued outlives the CTA, also after a wait that gave up.
      packed::products_end(&bars[L::kEnd + (warp == kMmaWarp ? 0 : 1)], issuer, s.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    packed::regs_up<216>();
    const int x = warp >> 2;
    const int r = tid & 127, row_token = r / s.G, row_head = r % s.G;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t o_addr = lane_addr + kColO + x * kD;
    const uint64_t scale2 = packed::pair(s.scale2, s.scale2);
    const bool wide = packed::wide_rows(o.out, o.st);
    bool ok = true;
    int jobs = 0, done = 0, used = 0;   // of all units before: jobs, this half's, and its units
    for (int k = 0;; ++k) {
      const bool more = next_unit(k, &ok, &u);
      if (kTiles ? !packed::all_agree(more, 2 + x, 128) : !more) break;
      any = true;
      const int token = u.t0 + x * tile_tokens + row_token;   // in the sequence
      const bool active = x < halves && r < tile_tokens * s.G && token < u.seq.n_q;
      const int limit = active ? u.before + token + 1 - u.j0 * 128 : 0;   // keys 0 .. limit - 1, from tile j0 on
      const int mine = x ? u.n_tiles[1] : u.n_tiles[0], both = min(u.n_tiles[0], u.n_tiles[1]);
      // Key tiles before this one need no mask in any row of the warp.
      const int whole = static_cast<int>(__reduce_min_sync(0xffffffffu, active ? max(limit, 0) : 0x7fffffff)) / 128;
      // P V number i of the half is done (two buffers: the last of its unit i).  With three buffers S of a tile
      // may be there before its last three P V are done, but no more: with a barrier for every third one,
      // none is two phases off.
      auto product_done = [&](int i) {
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kPvDone + 3 * x + i % 3], (i / 3) & 1, s.status));
        tc::fence_after_sync();
      };
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < mine; ++j) {
        const int job = kBuffers == 2 ? 2 * (done + j) + x : jobs + (j < both ? 2 * j + x : both + j);
        const int buffer = job % kBuffers;
        const uint32_t s_addr = lane_addr + buffer * 128;
        // S of the half's tile number done + j.  (Not by buffer: a half without tiles in a unit is a unit ahead,
        // and a buffer's barrier may then be any number of phases behind.)
        const int full = kBuffers == 2 ? L::kSFull + x : L::kSFull + 3 * x + (done + j) % 3;
        const int phase = kBuffers == 2 ? done + j : (done + j) / 3;
        // (A warp whose wait gave up goes on without waiting; the status word has the error.)
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars[full], phase & 1, s.status));
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
        for (int i = 0; i < 4; ++i) t[i] = fmaxf(__uint_as_float(z[i]), __uint_as_float(z[i + 4]));
#pragma unroll
        for (int i = 8; i < 128; i += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            t[e] = packed::max3(t[e], __uint_as_float(z[i + e]), __uint_as_float(z[i + e + 4]));
        }
        const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * s.scale2;
        const bool move = top > m + kLazy;
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? fast_exp2(m - top) : 1.f;   // 0 the first time
          if (move) {
            m = top;
            l *= alpha;
          }
          if (j > 0) {   // x of the tiles before, once their P V is done
            // (Two buffers: S of this tile was issued after that P V.)
            if (kBuffers == 3) product_done(done + j - 1);
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
        const uint64_t down = packed::pair(-base, -base);
        uint64_t sum = 0ull;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int at = 64 * c + 2 * i;
            const float2 e = packed::unpair(
                packed::fma2(packed::pair(__uint_as_float(z[at]), __uint_as_float(z[at + 1])), scale2, down));
            const float a = fast_exp2(e.x), d = fast_exp2(e.y);
            sum = packed::add2(sum, packed::pair(a, d));
            p[i] = packed::pack2<kFp16>(a, d);
          }
          tc::st32(s_addr + 32 * c, p);
        }
        const float2 halves = packed::unpair(sum);
        l += halves.x + halves.y;
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kPFull + buffer]);
      }
      // ---- x / l and the log sum ----
      if (mine > 0) product_done(kBuffers == 3 ? done + mine - 1 : used);
      if (kSplit && ok)   // the other half's too: they read the ring, which is written next
        ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::kAllDone], 0, s.status));
      tc::fence_after_sync();
      const float inv = 1.f / l;
      const int head = u.h * s.G + row_head;
      const long long row = u.seq.q0 + token;
      const bool none = u.before + token < 0;   // the row attends no key
      uint16_t* out = static_cast<uint16_t*>(o.out) + row * o.st.token + head * o.st.head;
      // Rows that were cleared.  (P V of each tile is done, so each has been looked through.)
      const uint32_t* gone = flags + (k & 1) * kMaxPartial * 4;
      uint32_t cleared = 0u;
      for (int j = u.looked; j < mine && ok; ++j) {
        const uint4 four = *reinterpret_cast<const uint4*>(gone + 4 * (j - u.looked));
        cleared |= four.x | four.y | four.z | four.w;
      }
      constexpr int kPart = kTiles ? 64 : 32;   // columns at a time
#pragma unroll 1
      for (int c0 = 0; c0 < kD; c0 += kPart) {
        uint32_t w[kPart];
#pragma unroll
        for (int i = 0; i < kPart; ++i) w[i] = 0u;
        if (mine > 0) {
#pragma unroll
          for (int c = 0; c < kPart; c += 32) tc::ld32(o_addr + c0 + c, *reinterpret_cast<uint32_t(*)[32]>(&w[c]));
          tc::wait_ld();
          if (c0 + kPart == kD) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::kOFree + x]);
          }
        }
        if (cleared && active) {
          const uint16_t* q_row = static_cast<const uint16_t*>(in.q) + row * in.q_st.token + head * in.q_st.head;
#pragma unroll 1
          for (int key = u.looked * 128; key < min(limit, mine * 128); ++key) {
            const int bit = key - u.looked * 128;
            if (!((gone[bit >> 5] >> (bit & 31)) & 1)) continue;
            const long long at = u.seq.k0 + u.j0 * 128 + key;
            const uint16_t* k_row = static_cast<const uint16_t*>(in.k) + at * in.k_st.token + u.h * in.k_st.head;
            const uint16_t* v_row = static_cast<const uint16_t*>(in.v) + at * in.v_st.token + u.h * in.v_st.head + c0;
            const float p = fast_exp2(fmaf(dot<kD, kFp16>(q_row, k_row), s.scale2, kTop<kFp16> - m));
#pragma unroll
            for (int i = 0; i < kPart / 2; ++i) {
              const float2 v = packed::unpack2<kFp16>(reinterpret_cast<const uint32_t*>(v_row)[i]);
              w[2 * i] = __float_as_uint(fmaf(p, v.x, __uint_as_float(w[2 * i])));
              w[2 * i + 1] = __float_as_uint(fmaf(p, v.y, __uint_as_float(w[2 * i + 1])));
            }
          }
        }
        if (kSplit) {   // into this CTA's ring, which is free now
#pragma unroll
          for (int i = 0; i < kPart; i += 4)
            parts[packed::swizzled<kD>(x * 128 + r, (c0 + i) / 4)] =
                make_float4(__uint_as_float(w[i]), __uint_as_float(w[i + 1]), __uint_as_float(w[i + 2]),
                            __uint_as_float(w[i + 3]));
          continue;
        }
        uint32_t p[kPart / 2];
#pragma unroll
        for (int i = 0; i < kPart / 2; ++i)
          p[i] = !none ? packed::pack2<kFp16>(__uint_as_float(w[2 * i]) * inv, __uint_as_float(w[2 * i + 1]) * inv)
                       : 0u;
        if (kTiles && x < halves && u.t0 + (x + 1) * tile_tokens <= u.seq.n_q) {
          // Every row of the tile is a query's.
          uint8_t* tile = smem + L::kOut + x * 16384;
          if (r == 0) packed::stores_read();
          asm volatile("bar.sync %0, 128;" ::"r"(2 + x) : "memory");
#pragma unroll
          for (int c = 0; c < kPart / 8; ++c)
            *reinterpret_cast<uint4*>(tile + r * 128 + ((c ^ (r & 7)) << 4)) =
                make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
          fence_proxy_async_smem();
          asm volatile("bar.sync %0, 128;" ::"r"(2 + x) : "memory");
          if (r == 0)
            packed::tma_store_4d(&maps.out, smem_u32(tile), c0, 0, u.h, u.seq.q0 + u.t0 + x * tile_tokens);
        } else if (active) {
#pragma unroll
          for (int c = 0; c < kPart; c += 32)
            packed::store_row(out + c0 + c, *reinterpret_cast<uint32_t(*)[16]>(&p[c / 2]), wide);
        }
      }
      if (kSplit) {
        sums[x * 128 + r] = make_float2(m, l);
      } else if (active && o.lse) {
        o.lse[row * (s.Hkv * s.G) + head] =
            !none ? (m - kTop<kFp16> + fast_log2(l)) * 0.69314718055994531f : -INFINITY;
      }
      jobs += u.n_tiles[0] + u.n_tiles[1];
      done += mine;
      used += mine > 0;
      unit_done(k);
      if (kSplit) break;
    }
    if (kTiles && r == 0) packed::stores_done();
  }
  if (kSplit) {
    // ---- each CTA joins its share of the rows over the cluster: with M the largest m,
    // out = sum 2^(m - M) x / sum 2^(m - M) l ----
    __syncwarp();
    cluster_sync();
    if (warp < 8 && packed::all_agree(any)) {   // (the softmax warps: the others have given registers away)
      const int row0 = rank * 256 / ctas, share = (rank + 1) * 256 / ctas - row0;
      for (int e = tid; e < share; e += 256) {   // a row: its weights, over l, and log sum
        const int row = row0 + e, rr = row & 127;
        const int token = u.t0 + (row >> 7) * tile_tokens + rr / s.G;
        float top = -INFINITY, l = 0.f;
        for (int c = 0; c < ctas; ++c) top = fmaxf(top, ld_dsmem_f32(dsmem_addr(&sums[row].x, c)));
        const float base = top == -INFINITY ? 0.f : top;
        for (int c = 0; c < ctas; ++c) {
          const float2 ml = ld_dsmem_f32x2(dsmem_addr(&sums[row], c));
          const float weight = fast_exp2(ml.x - base);
          weights[e * 16 + c] = weight;
          l = fmaf(weight, ml.y, l);
        }
        const bool active = rr < tile_tokens * s.G && token < u.seq.n_q, none = u.before + token < 0;
        for (int c = 0; c < ctas; ++c) weights[e * 16 + c] *= none ? 0.f : 1.f / l;
        if (active && o.lse)
          o.lse[static_cast<long long>(u.seq.q0 + token) * (s.Hkv * s.G) + u.h * s.G + rr % s.G] =
              !none ? (top - kTop<kFp16> + fast_log2(l)) * 0.69314718055994531f : -INFINITY;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int e = tid; e < share * (kD / 4); e += 256) {
        const int local = e / (kD / 4), c4 = e % (kD / 4), row = row0 + local, rr = row & 127;
        const int token = u.t0 + (row >> 7) * tile_tokens + rr / s.G;
        if (rr >= tile_tokens * s.G || token >= u.seq.n_q) continue;
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
        uint16_t* out = static_cast<uint16_t*>(o.out) + static_cast<long long>(u.seq.q0 + token) * o.st.token +
                        (u.h * s.G + rr % s.G) * o.st.head + 4 * c4;
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
  static int known[64][kMaxSplit + 1];   // what it is plus 1
  const int i = ctas;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev][i]) {
    const auto kernel = packed_attn_kernel<kD, kFp16, Form::kSplit>;
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Layout<kD, Form::kSplit>::kBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<kD, Form::kSplit>::kBytes) != cudaSuccess ||
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
  while (ctas > 1 && (tiles / ctas < 4 || clusters_at_once<kD, kFp16>(ctas) < units)) --ctas;
  return ctas;
}

template <int kD, bool kFp16>
cudaError_t launch(const PackedAttnShape& s, const PackedAttnMaps& maps, const PackedAttnIn& in, const PackedAttnOut& o,
                   cudaStream_t st) {
  // Units of two tiles: at most one partly filled one per sequence.
  // While single tiles fill no more than the SMs, each is a unit of its own: its softmax then shares the SM
  // with no other (one prompt of 301 tokens, 38 units or 76: 12.4 or 11.3 us a call when that was measured).
  const int one = packed_tile_tokens(s.G);
  auto most = [&](int step) { return std::min<long long>(s.Tq, static_cast<long long>(s.Tq) / step + s.B); };
  const int ctas = split<kD, kFp16>(s, 2 * one);
  const int halves = ctas == 1 && most(one) * s.Hkv <= device_sm_count() ? 1 : 2;
  const long long units = most(halves * one);
  const auto kernel = ctas > 1    ? packed_attn_kernel<kD, kFp16, Form::kSplit>
                      : o.by_tile ? packed_attn_kernel<kD, kFp16, Form::kTiles>
                                  : packed_attn_kernel<kD, kFp16, Form::kFew>;
  const int bytes = ctas > 1    ? Layout<kD, Form::kSplit>::kBytes
                    : o.by_tile ? Layout<kD, Form::kTiles>::kBytes
                                : Layout<kD, Form::kFew>::kBytes;
  static packed::SharedMemory shared[3];   // of each of the three kernels
  const cudaError_t e = shared[ctas > 1 ? 2 : o.by_tile].allow(kernel, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // A CTA per SM, or a cluster per unit.
  const long long grid = ctas > 1 ? units * s.Hkv * ctas : std::min<long long>(units * s.Hkv, device_sm_count());
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
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
  return cudaLaunchKernelEx(&cfg, kernel, maps, s, in, o, ctas, halves);
}

}  // namespace

// Where a CTA has more than one unit (see Form::kTiles).
bool packed_attn_by_tile(const PackedAttnShape& s) {
  return static_cast<long long>(s.Tq) * s.Hkv > 2ll * packed_tile_tokens(s.G) * device_sm_count();
}

cudaError_t launch_packed_attn(const PackedAttnShape& s, int D, bool fp16, const PackedAttnMaps& maps,
                               const PackedAttnIn& in, const PackedAttnOut& o, cudaStream_t st) {
  if (D == 128) return fp16 ? launch<128, true>(s, maps, in, o, st) : launch<128, false>(s, maps, in, o, st);
  return fp16 ? launch<64, true>(s, maps, in, o, st) : launch<64, false>(s, maps, in, o, st);
}

}  // namespace infllmv2
