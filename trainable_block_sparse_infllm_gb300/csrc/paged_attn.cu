// Attention of one new token per sequence over a paged cache, split over the
// cache's length and joined.
//
//   z[h, s] = scale q_h . k_s            m_h = max_s z   l_h = sum_s exp(z - m)
//   out_h   = sum_s exp(z - m) v_s / l   lse_h = m + ln l
//   weights[s] += sum_{h in the group} exp(z[h, s] - lse_h)      (optional)
//
// Bound by memory: 4 d FLOPs per head for 4 d bytes of a key and a value, so
// even 32 heads to a KV head give 32 FLOPs per byte.  The aim is one pass over
// the pages at the copy rate, whatever the lengths.
//
// Split.  The work is all tiles (64 or 128 slots) of all (sequence, KV head)
// units, in that order, each unit with a fixed cost before its tiles.  That line is cut
// into chunks whatever the units' borders: one equal chunk for every CTA, so
// that those of any ragged batch carry the same load and one long sequence
// spreads over all SMs.  SMs do not read at one rate, though (a 32 x 32K batch
// in equal shares took the CTAs 442 to 535 us): of a long line every CTA gets
// four fifths of its share, and the rest goes in small chunks to whoever is
// done, from a counter.  A unit inside one chunk is finished there; of a unit
// that borders cut, each piece leaves (m, l, sum of exp(z - m) v) in the
// workspace, at a place that goes by the chunk and not by the CTA, and
// paged_join_kernel joins them in the line's order.  The host needs no lengths.
//
// Where the capacity is small the second launch costs more than the balance
// gives.  Then each unit goes to a cluster of 4 or 8 CTAs, which joins its
// pieces itself behind the cluster's barrier (cluster_size has the rule), or,
// of many caches of up to 256 slots, whole to one CTA.
//
// A CTA.  One warp loads: per page piece (16, 32 or 64 rows of one page) it
// issues one TMA box per 64 columns of K and of V, through a ring of tiles; the
// queries of a piece come with its first tile, and what a tile is (whose, which
// rows of it hold slots, whether a piece ends) stands beside it.  Four warps
// (eight for 17 to 32 heads: four per half) compute, each on its own quarter of
// every tile's slots with its own running maximum and sum, so that nothing but
// the ring's barriers is shared until the piece's end.  The heads are the 16 rows
// of mma.m16n8k16: at these intensities the tensor pipe idles and a tcgen05
// tile (128 rows) would be seven eighths empty.
//
// Types.  z, maxima, sums and accumulators are fp32.  Maxima are those of the
// unscaled scores, and a score is scaled after the maximum is taken off: of the
// largest that leaves 0, whatever its size.  (exp2(z scale - m), with m the rounded
// product, is 2^(half a step of m), which passes fp16's range from scores of 2^25
// and fp32's from 2^31.)  A probability feeds the product with V as two 16-bit
// parts (hi + lo, to 2^-16 of it or better): one rounding of it to bf16 would cost
// as much again as the output's own, and against 2^-16 the output's own is all that
// is seen: bf16 outputs are 0.00167 (relative 2-norm) from the formula in 64 bits
// with 24-bit probabilities and with these, and 0.3% of them are the neighbouring
// value.  With up to 8 heads the lo parts fill the rows 8..15 that would be empty;
// with more they are a second product (a unit of 256 slots, d 128, cut over the
// SMs: 7.9 us a call with 8 heads, 8.8 with 16).  fp16 probabilities are scaled by
// 2^14, so that the long tail of a sharp softmax stays above fp16's smallest number.
//
// Measured (GB300, bf16 unless said): 32 sequences of 16K to 32K, 8 KV heads of
// 8, with weights: the pass 500 us (3.3 GB: 6.6 TB/s, 99% of the copy rate, its
// scores' 0.2 GB included), the join and weights 46 us.  64 ragged of up to 8K,
// fp16, token-major pages of 16, with weights: 179 us (6.4 TB/s) and 21 us.  One
// of 128K, 2 KV heads of 16, with weights: 30 us (134 MB; 4 us until the first
// tiles land, and CTAs of 13 or 14 tiles) and 9 us.
#include <atomic>

#include "paged.cuh"
#include "kernels.h"
#include "paged_rules.h"

namespace infllmv2 {

namespace {

// Slots per tile: 32 KB of keys and values, so that a tile's fixed cost (its
// barriers, maxima and their exchange) is shared by as many bytes at either d:
// 96 short sequences at d 64 took 84 us with 64 slots and 70 with 128.  With two
// groups (17 to 32 heads) 128 slots at either: each warp then has two
// independent parts to overlap; 4 x 60K slots, 8 KV heads of 32, d 128, took
// 248 us with 64 slots and 168 with 128 (where 48 bytes of a thread spill).
template <int kDim, int kGroups>
constexpr int kTileOf = kGroups == 2 ? 128 : 8192 / kDim;

struct PagedAttnArgs {
  int B, Hkv, G, ps, P, maxp, cap, box;
  PagedMapOrder ko, vo;
  float scale2;   // scale * log2(e)
  const void* q;
  const int32_t* table;
  const int32_t* kv_lens;
  void* out;
  float* lse;
  float* weights;    // null: not accumulated
  float* part_o;     // [2 chunks][G][D]: pieces of cut units, relative to their m
  float2* part_ml;   // [2 chunks][32]: (m of the unscaled scores, l)
  // Cut units, (unit or -1, chunk of the second piece, last chunk, first
  // piece's place).  unit_cut, by unit, is kept where there are no more units
  // than chunks or weights are summed; chunk_cut, by the chunk that the second
  // piece starts, where there are more units.  The join goes by the shorter list.
  int4* unit_cut;
  int4* chunk_cut;
  int* chunks;       // number of chunks, for the join
  int most;          // chunks that the workspace has room for
  int* next;         // chunks handed out beyond the CTAs' first ones; null: none are
  float2* unit_ml;   // [B Hkv G] (m, 1 / l) of units that no border cut (weights only)
  float* scores;     // [B Hkv G][cap64] z, unscaled (weights only)
  int cap64;         // scores of a head: cap rounded up to whole tiles
  int whole;         // no unit is cut: one launch
  int cluster;       // CTAs of a cluster per unit, which join their pieces themselves: one launch; 0: none
  int tile_shift;    // log2 of the slots per tile
  uint32_t* status;
};

// ---- the split of the tiles over the CTAs ----------------------------------

// The units lie one after the other on a line, each `cost` positions for its
// fixed work (merge, output) and then one for every tile; empty sequences take
// none.  Chunk k < n is [k A / n, (k + 1) A / n), and the chunks behind those
// have `small` positions each.
struct Split {
  long long W;        // positions
  long long A;        // of them in the first n chunks
  int n, chunks;      // n: min(CTAs, W)
  int small;
  int cost;
  bool whole;         // units go whole to the chunk that has their first position
  int b, h;           // the unit of this CTA's first chunk's first position
  long long unit0;    // where that unit begins
};

// a / b for a >= 0, b > 0: in 32 bits where that does (a 64-bit division is a
// hundred instructions, and every CTA starts with a few).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ long long chunk_begin(const Split& s, int k) {
  return k <= s.n ? quotient(k * s.A, s.n) : min(s.W, s.A + static_cast<long long>(k - s.n) * s.small);
}
// The chunk that a position belongs to.
__device__ __forceinline__ int chunk_of(const Split& s, long long at) {
  return static_cast<int>(at < s.A ? quotient((at + 1) * s.n - 1, s.A) : s.n + quotient(at - s.A, s.small));
}

__device__ __forceinline__ int unit_tiles(const PagedAttnArgs& a, int len) {
  return (len + (1 << a.tile_shift) - 1) >> a.tile_shift;
}

// Positions of one unit of sequence b.
__device__ __forceinline__ int unit_width(const PagedAttnArgs& a, int b, int cost) {
  const int tiles = unit_tiles(a, paged_len(a.kv_lens, b, a.cap, a.status));
  return tiles ? tiles + cost : 0;
}

// All threads of the CTA.  Each sums a run of sequences; the one whose run
// holds the CTA's first position says where that is.  before[t]: positions of
// one KV head before thread t's run; before[kThreads]: of all.
template <int kThreads>
__device__ __forceinline__ Split make_split(const PagedAttnArgs& a, int cta, int ctas, int cost, long long* before,
                                            int* shared) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  int sum = 0;   // at most 26 sequences of 2^24 tiles (4096 sequences, 2^30 slots)
  for (int b = b0; b < b1; ++b) sum += unit_width(a, b, cost);
  long long pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += up;
  }
  long long* totals = reinterpret_cast<long long*>(shared);   // [kWarps]
  if (lane == 31) totals[warp] = pre;
  __syncthreads();
  long long all = 0, earlier = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) earlier = all;
    all += totals[w];
  }
  pre += earlier - sum;
  before[tid] = pre;
  if (tid == 0) before[kThreads] = all;
  Split s;
  s.W = all * a.Hkv;
  s.n = static_cast<int>(min(static_cast<long long>(ctas), s.W));
  s.cost = cost;
  s.whole = a.whole != 0;
  const bool shares = a.next != nullptr && s.n > 0 && s.W >= 32LL * s.n;
  s.A = s.W;
  s.small = 8;
  s.chunks = s.n;
  if (shares) {
    s.A -= s.W / 5;
    s.small = max(8, static_cast<int>((s.W - s.A + 6LL * s.n - 1) / (6LL * s.n)));
    s.chunks += static_cast<int>((s.W - s.A + s.small - 1) / s.small);
  }
  s.b = s.h = 0;
  s.unit0 = 0;
  int* where = shared + 2 * kWarps;
  if (cta < s.n) {
    const long long begin = chunk_begin(s, cta);
    if (begin >= pre * a.Hkv && begin < (pre + sum) * a.Hkv) {
      long long rest = begin - pre * a.Hkv;
      for (int b = b0; b < b1; ++b) {
        const int w = unit_width(a, b, cost);
        if (rest < static_cast<long long>(w) * a.Hkv) {
          where[0] = b;
          where[1] = static_cast<int>(quotient(rest, w));
          where[2] = static_cast<int>(rest - static_cast<long long>(where[1]) * w);
          break;
        }
        rest -= static_cast<long long>(w) * a.Hkv;
      }
    }
  }
  __syncthreads();
  if (cta < s.n) {
    s.b = where[0];
    s.h = where[1];
    s.unit0 = chunk_begin(s, cta) - where[2];
  }
  return s;
}

// One warp: the unit of position `at`, into s.b, s.h and s.unit0.
template <int kThreads>
__device__ __forceinline__ void locate(Split& s, const PagedAttnArgs& a, long long at, const long long* before) {
  const int lane = threadIdx.x & 31, run = (a.B + kThreads - 1) / kThreads;
  int r = 0;
  for (int r0 = 0; r0 < kThreads; r0 += 32) {   // the run of sequences that holds it
    const bool here = before[r0 + lane] * a.Hkv <= at && at < before[r0 + lane + 1] * a.Hkv;
    const uint32_t hit = __ballot_sync(0xffffffffu, here);
    if (hit) {
      r = r0 + __ffs(hit) - 1;
      break;
    }
  }
  const int b = r * run + lane;   // a run has at most 26 sequences
  const int w = lane < run && b < a.B ? unit_width(a, b, s.cost) : 0;
  const int upto = warp_inclusive_scan(w);
  const long long rest = at - before[r] * a.Hkv;
  const bool here = static_cast<long long>(upto - w) * a.Hkv <= rest && rest < static_cast<long long>(upto) * a.Hkv;
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  const int width = __shfl_sync(0xffffffffu, w, src), first = __shfl_sync(0xffffffffu, upto - w, src);
  const long long in = rest - static_cast<long long>(first) * a.Hkv;
  s.b = r * run + src;
  s.h = static_cast<int>(quotient(in, width));
  s.unit0 = at - (in - static_cast<long long>(s.h) * width);
}

// The tiles of one unit in a chunk [begin, end).
struct Piece {
  int b, h, len, tiles;      // the unit: its sequence, KV head, slots and tiles
  int tile0, tile1;          // the piece
  long long unit0;           // where the unit begins
};

__device__ __forceinline__ long long tile_at(const Split& s, const Piece& p, int tile) { return p.unit0 + s.cost + tile; }

// Both: false where the chunk holds no (further) tile.
__device__ __forceinline__ bool next_piece(Piece& p, const Split& s, const PagedAttnArgs& a, long long end) {
  p.unit0 = tile_at(s, p, p.tiles);
  if (p.unit0 >= end) return false;
  if (++p.h == a.Hkv) {
    p.h = 0;
    do {
      ++p.b;
      p.len = paged_len(a.kv_lens, p.b, a.cap, a.status);
    } while (p.len == 0);   // positions are left, so a sequence with slots is
    p.tiles = unit_tiles(a, p.len);
  }
  p.tile0 = 0;
  p.tile1 = s.whole ? p.tiles : static_cast<int>(min(static_cast<long long>(p.tiles), end - tile_at(s, p, 0)));
  return p.tile1 > 0;
}

__device__ __forceinline__ bool first_piece(Piece& p, const Split& s, const PagedAttnArgs& a, long long begin,
                                            long long end) {
  p.b = s.b;
  p.h = s.h;
  p.len = paged_len(a.kv_lens, p.b, a.cap, a.status);
  p.tiles = unit_tiles(a, p.len);
  p.unit0 = s.unit0;
  p.tile0 = max(0, static_cast<int>(begin - p.unit0) - s.cost);
  p.tile1 = static_cast<int>(min(static_cast<long long>(p.tiles), end - tile_at(s, p, 0)));
  if (s.whole) {
    if (p.unit0 < begin) return next_piece(p, s, a, end);
    p.tile1 = p.tiles;
  }
  return p.tile1 > p.tile0;
}

// A cluster's unit and the piece of CTA `cta` in it; false where it has no tile.
__device__ __forceinline__ bool cluster_piece(Piece& p, const PagedAttnArgs& a, int cta) {
  const int unit = cta / a.cluster, rank = cta % a.cluster;
  p.b = unit / a.Hkv;
  p.h = unit % a.Hkv;
  p.len = paged_len(a.kv_lens, p.b, a.cap, a.status);
  p.tiles = unit_tiles(a, p.len);
  p.tile0 = p.tiles * rank / a.cluster;
  p.tile1 = p.tiles * (rank + 1) / a.cluster;
  p.unit0 = 0;
  return p.tile1 > p.tile0;
}

// Workspace place of a cut unit's piece in chunk k whose first tile is at `at`:
// 2 k for a piece that starts the chunk, 2 k + 1 for one that starts later (and
// so is the chunk's last).
__device__ __forceinline__ int piece_place(int k, long long begin, long long at) { return 2 * k + (at > begin ? 1 : 0); }

// ---- types ------------------------------------------------------------------

template <bool kFp16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFp16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    mma_bf16_16816(d, a, b0, b1);
  }
}

// Two probabilities as 16-bit parts, x = hi + lo to 2^-16 (bf16) or 2^-19 (fp16).
// Both parts of a positive x are positive: with hi the nearest, lo would be zero
// or negative as often as not, and an infinite v in an attended row would end as
// 0 * inf or inf - inf.  (In fp16 lo is positive from x = 2^-14 on, a probability
// of 2^-28; in bf16 from 2^-110 on.)
template <bool kFp16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (kFp16) {
    const __half2 h = __hmul2(__floats2half2_rn(x, y), __float2half2_rn(1.f - 0x1p-9f));   // 1 to 5 steps below x
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const uint32_t bx = __float_as_uint(x), by = __float_as_uint(y);
    hi = __byte_perm(bx, by, 0x7632);   // cut off
    constexpr float kAbove = 1.f + 0x1p-23f;
    lo = pack_bf16x2(fmaf(x, kAbove, -__uint_as_float(bx & 0xffff0000u)),
                     fmaf(y, kAbove, -__uint_as_float(by & 0xffff0000u)));
  }
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
  if constexpr (kFp16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(x, y);
  }
}

// lse of a sum relative to the maximum m of the unscaled scores.  fp16
// probabilities, and so their sum, carry a factor 2^14.
template <bool kFp16>
__device__ __forceinline__ float lse_of(float m, float sum, float scale2) {
  return fmaf(m, scale2, log2f(sum) - (kFp16 ? 14.f : 0.f)) * 0.6931471805599453f;
}

// Merges the sum l2 relative to the maximum m2 (of unscaled scores; -inf where
// nothing was attended) into (m, l); returns what the two sides' other sums are to
// be multiplied by.
__device__ __forceinline__ float2 merge_ml(float& m, float& l, float m2, float l2, float scale2) {
  const float top = fmaxf(m, m2), use = top == -INFINITY ? 0.f : top;
  const float f = fast_exp2((m - use) * scale2), f2 = fast_exp2((m2 - use) * scale2);
  m = top;
  l = l * f + l2 * f2;
  return make_float2(f, f2);
}
__device__ __forceinline__ void merge_sums(float& m, float& l, float4& x, float m2, float l2, const float4& x2,
                                           float scale2) {
  const float2 f = merge_ml(m, l, m2, l2, scale2);
  x.x = x.x * f.x + x2.x * f.y;
  x.y = x.y * f.x + x2.y * f.y;
  x.z = x.z * f.x + x2.z * f.y;
  x.w = x.w * f.x + x2.w * f.y;
}

// What add_weights needs of a head; nothing attended weighs nothing.
template <bool kFp16>
__device__ __forceinline__ float2 m_and_inverse(float m, float sum) {
  return make_float2(m == -INFINITY ? 0.f : m, sum == 0.f ? 0.f : (kFp16 ? 16384.f : 1.f) / sum);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ int by_order(PagedMapOrder o, int dim, int token, int head, int page) {
  return o.token == dim ? token : (o.head == dim ? head : page);
}


// Adds the weights of slots `first`, + `step`, ... (four each) of a unit, from
// the z of its heads and their (m, 1 / l): exp(scale (z - m)) / l as for the
// output.  (exp2(z - lse) with an lse of one float loses what lse's size takes
// from it: at |lse| = 4000 every weight of a head was off by up to 1.7e-4.)
__device__ __forceinline__ void add_weights(const PagedAttnArgs& a, long long unit, int b, int kv_head, int len, int first,
                                            int step, const float2* ml) {
  const int32_t* table = a.table + static_cast<long long>(b) * a.maxp;
  for (int slot = first; slot < len; slot += step) {   // the four share a page (pages hold multiples of 16)
    const int page = __ldg(table + slot / a.ps);
    const float* z = a.scores + unit * a.G * a.cap64 + slot;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < a.G; ++h) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(z + static_cast<long long>(h) * a.cap64));
      const float2 y = ml[h];
      w.x += fast_exp2((x.x - y.x) * a.scale2) * y.y;
      w.y += fast_exp2((x.y - y.x) * a.scale2) * y.y;
      w.z += fast_exp2((x.z - y.x) * a.scale2) * y.y;
      w.w += fast_exp2((x.w - y.x) * a.scale2) * y.y;
    }
    if (page < 0 || page >= a.P) continue;
    // One add per slot of a call, so that a cache's own pages sum in a fixed
    // order; pages that sequences share are summed in the order of arrival.
    float* to = a.weights + paged_meta(page, kv_head, slot % a.ps, a.Hkv, a.ps);
    if (slot + 4 <= len) {
      asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(w.x), "f"(w.y), "f"(w.z),
                   "f"(w.w)
                   : "memory");
    } else {
      atomicAdd(to, w.x);
      if (slot + 1 < len) atomicAdd(to + 1, w.y);
      if (slot + 2 < len) atomicAdd(to + 2, w.z);
    }
  }
}

// ---- the pass over the pages -------------------------------------------------

// CTAs of a cluster, at most (cluster_size picks 8 or 4).
constexpr int kMaxCluster = 8;

// A unit's merge and output cost a CTA about as much as this many tiles.
constexpr int kUnitCost = 2;

// What a stage of the ring holds.
struct __align__(16) StageInfo {
  uint2 valid;      // rows of each 16 that hold slots, 8 bits each
  uint32_t flags;
  int unit;         // b * Hkv + h
  int place;        // where the piece's sums go if the unit is cut
  int len, tile, b;
};
constexpr uint32_t kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8;   // of a piece; its unit is not cut; no more tiles

// kGroups: groups of four warps, one per 16 heads.  kStack: at most 8 heads,
// the lo parts of the probabilities in rows 8..15.
template <int kDim, int kGroups, bool kStack>
struct AttnCfg {
  static constexpr int kTile = kTileOf<kDim, kGroups>;
  static constexpr int kSub = kTile / 64;               // 16-slot parts of a tile per warp
  static constexpr int kStage = kTile * kDim * 4;       // K and V of a tile
  static constexpr int kQRow = kDim * 2 + 16;           // a query row, so padded that 8 rows meet all banks
  static constexpr int kQ = 16 * kGroups * kQRow;       // the queries beside it
  // Two CTAs of at most 113 KB per SM for one group, one of at most 227 KB for two.
  static constexpr int kStages = (kGroups == 1 ? 98304 : 196608) / kStage;
  static constexpr int kThreads = 32 + 128 * kGroups;
  static constexpr int kPerSm = kGroups == 1 ? 2 : 1;
  static constexpr int kCost = kUnitCost;
  static constexpr int kQOff = kStages * kStage;
  static constexpr int kInfoOff = kQOff + kStages * kQ;
  static constexpr int kMlOff = kInfoOff + kStages * static_cast<int>(sizeof(StageInfo));
  static constexpr int kUnitOff = kMlOff + kGroups * 4 * 16 * 8;     // a whole unit's (m, 1 / l)
  static constexpr int kBeforeOff = kUnitOff + kPagedMaxGroup * 8;
  static constexpr int kSplitOff = kBeforeOff + (kThreads + 1) * 8;
  static constexpr int kBarOff = kSplitOff + 128;
  static constexpr int kSmem = 1024 + kBarOff + (2 * kStages + kGroups + 1) * 8;
  static_assert(kPerSm * (kSmem + 1024) <= 233472 && kSmem <= 232448, "shared memory of an SM");
};

template <bool kFp16, int kDim, int kGroups, bool kStack>
__global__ void __launch_bounds__(AttnCfg<kDim, kGroups, kStack>::kThreads, AttnCfg<kDim, kGroups, kStack>::kPerSm)
    paged_attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const PagedAttnArgs a) {
  using C = AttnCfg<kDim, kGroups, kStack>;
  constexpr int kTile = C::kTile, kSub = C::kSub;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* group_bar = empty + C::kStages;   // [kGroups], then one for all computing warps
  StageInfo* info = reinterpret_cast<StageInfo*>(smem + C::kInfoOff);
  long long* before = reinterpret_cast<long long*>(smem + C::kBeforeOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4 * kGroups);
    }
    for (int i = 0; i < kGroups; ++i) mbar_init(group_bar + i, 4);
    mbar_init(group_bar + kGroups, 4 * kGroups);
    fence_barrier_init();
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  pdl_wait();
  pdl_trigger();
  Split s = {};
  if (a.cluster)
    __syncthreads();   // the barriers are set up
  else
    s = make_split<C::kThreads>(a, cta, ctas, C::kCost, before, reinterpret_cast<int*>(smem + C::kSplitOff));
  if (cta == 0 && tid == 0 && a.chunks) *a.chunks = s.chunks;

  // Empty sequences attend nothing: a zero row, lse = -inf.
  const long long heads = static_cast<long long>(a.Hkv) * a.G;
  for (int b = cta; b < a.B; b += ctas) {
    if (paged_len(a.kv_lens, b, a.cap, a.status) != 0) continue;
    uint32_t* out = static_cast<uint32_t*>(a.out) + b * heads * (kDim / 2);
    for (int e = tid; e < heads * (kDim / 2); e += C::kThreads) out[e] = 0;
    if (a.lse)
      for (int e = tid; e < heads; e += C::kThreads) a.lse[b * heads + e] = -INFINITY;
    if (a.unit_cut)
      for (int h = tid; h < a.Hkv; h += C::kThreads) a.unit_cut[b * a.Hkv + h] = make_int4(-1, 0, 0, 0);
  }
  if (cta >= s.n && !a.cluster) return;

  if (warp == 4 * kGroups) {
    // ------------------------------------------------ the loading warp -------
    fence_proxy_async_global();   // rows that earlier kernels stored are read by TMA
    const int boxes = kTile / a.box;
    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    uint32_t issued = 0;
    int chunk = cta;
    while (true) {
      long long begin = 0, end = 0;
      Piece p;
      bool have;
      if (a.cluster) {
        have = cluster_piece(p, a, cta);
      } else {
        begin = chunk_begin(s, chunk);
        end = chunk_begin(s, chunk + 1);
        have = first_piece(p, s, a, begin, end);
      }
      // Does the chunk before hold the first piece of the unit that starts this one?
      const bool later = have && p.tile0 > 0;
      const int cut_unit = p.b * a.Hkv + p.h, cut_tiles = p.tiles;
      const long long cut_at = tile_at(s, p, 0);
      while (have && !dead) {
        const int unit = p.b * a.Hkv + p.h;
        const bool whole = p.tile0 == 0 && p.tile1 == p.tiles;
        if (lane == 0 && a.unit_cut && whole) a.unit_cut[unit] = make_int4(-1, 0, 0, 0);
        const int32_t* row = a.table + static_cast<long long>(p.b) * a.maxp;
        // Lane i handles box i of a tile; its page is fetched one tile ahead.
        auto fetch = [&](int tile) {
          const int slot = tile * kTile + lane * a.box;
          return (lane < boxes && tile < p.tile1 && slot < p.len) ? __ldg(row + slot / a.ps) : -1;
        };
        int page_next = fetch(p.tile0);
        // The unit's queries, 16 bytes per lane and step, on their way while the
        // first page entry is.
        constexpr int kQSteps = kGroups * kDim / 16;
        uint4 qv[kQSteps];
        {
          const uint4* q = static_cast<const uint4*>(a.q) + static_cast<long long>(unit) * a.G * (kDim / 8);
#pragma unroll
          for (int i = 0; i < kQSteps; ++i)
            if (i * 32 + lane < a.G * (kDim / 8)) qv[i] = __ldg(q + i * 32 + lane);
        }
        const int place = a.cluster ? cta : piece_place(chunk, begin, tile_at(s, p, p.tile0));
        for (int t = p.tile0; t < p.tile1; ++t) {
          const int page = page_next;
          page_next = fetch(t + 1);
          const int slot = t * kTile + lane * a.box;
          const bool ok = page >= 0 && page < a.P;
          // The slots of an entry that names no page count as absent.
          if (!ok && lane < boxes && slot < p.len) atomicOr(a.status, kStatusBadPage);
          const uint32_t oks = __ballot_sync(0xffffffffu, ok);
          if (!mbar_wait(empty + stage, phase ^ 1, a.status)) {
            dead = true;
            break;
          }
          uint8_t* dst = smem + stage * C::kStage;
          if (lane == 0) {
            StageInfo x;
            uint32_t valid[2] = {0, 0};
            const int box_shift = 31 - __clz(a.box);
#pragma unroll
            for (int w = 0; w < kTile / 16; ++w) {
              const int left = p.len - (t * kTile + w * 16);
              if ((oks >> (w * 16 >> box_shift)) & 1u)
                valid[w >> 2] |= static_cast<uint32_t>(max(0, min(16, left))) << (8 * (w & 3));
            }
            x.valid = make_uint2(valid[0], valid[1]);
            x.flags = (t == p.tile0 ? kFirst : 0) | (t + 1 == p.tile1 ? kLast : 0) | (whole ? kWhole : 0);
            x.unit = unit;
            x.place = place;
            x.len = p.len;
            x.tile = t;
            x.b = p.b;
            info[stage] = x;
          }
          if (t == p.tile0) {
#pragma unroll
            for (int i = 0; i < kQSteps; ++i) {
              const int e = i * 32 + lane;
              if (e < a.G * (kDim / 8))
                *reinterpret_cast<uint4*>(smem + C::kQOff + stage * C::kQ + e / (kDim / 8) * C::kQRow +
                                          e % (kDim / 8) * 16) = qv[i];
            }
          }
          __syncwarp();   // the arrival releases what every lane has written
          if (lane == 0) mbar_arrive_expect_tx(full + stage, __popc(oks) * a.box * kDim * 4);
          __syncwarp();
          if (ok) {
            const int in_page = slot % a.ps;
            const int k1 = by_order(a.ko, 1, in_page, p.h, page), k2 = by_order(a.ko, 2, in_page, p.h, page),
                      k3 = by_order(a.ko, 3, in_page, p.h, page);
            const int v1 = by_order(a.vo, 1, in_page, p.h, page), v2 = by_order(a.vo, 2, in_page, p.h, page),
                      v3 = by_order(a.vo, 3, in_page, p.h, page);
#pragma unroll
            for (int c = 0; c < kDim / 64; ++c) {
              tma_load_4d(dst + c * kTile * 128 + lane * a.box * 128, &k_map, c * 64, k1, k2, k3, full + stage);
              tma_load_4d(dst + kTile * kDim * 2 + c * kTile * 128 + lane * a.box * 128, &v_map, c * 64, v1, v2, v3,
                          full + stage);
            }
          }
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!dead) have = !a.cluster && next_piece(p, s, a, end);
      }
      if (a.cluster) break;
      if (lane == 0) {   // the chunk's loads are on their way: note the cut
        int4 c = make_int4(-1, 0, 0, 0);
        if (later && cut_at < begin && chunk_of(s, cut_at) == chunk - 1)
          c = make_int4(cut_unit, chunk, chunk_of(s, cut_at + cut_tiles - 1),
                        piece_place(chunk - 1, chunk_begin(s, chunk - 1), cut_at));
        if (a.chunk_cut) a.chunk_cut[chunk] = c;
        if (a.unit_cut && c.x >= 0) a.unit_cut[c.x] = c;
      }
      if (dead || s.chunks == s.n) break;
      int next = 0;
      if (lane == 0) next = s.n + atomicAdd(a.next, 1);
      chunk = __shfl_sync(0xffffffffu, next, 0);
      if (chunk >= s.chunks) break;
      locate<C::kThreads>(s, a, chunk_begin(s, chunk), before);
    }
    if (!dead && !mbar_wait(empty + stage, phase ^ 1, a.status)) dead = true;
    if (!dead && lane == 0) {
      info[stage].flags = kEnd;
      mbar_arrive(full + stage);
    }
    // Whatever gave up, here or in the computing warps, this warp does not leave
    // before the copies in flight have landed (or as long a wait for them).
    for (uint32_t i = first_in_flight(issued, C::kStages, !dead); i < issued; ++i)
      mbar_wait(full + i % C::kStages, (i / C::kStages) & 1, a.status);
    __syncwarp();
    if (a.cluster) cluster_sync();   // with the computing warps' below
    return;
  }

  // -------------------------------------------------- the computing warps -----
  const int group = kGroups == 1 ? 0 : warp >> 2, w = warp & 3;       // 16 heads; 16 slots of a tile
  const int g = lane >> 2, t4 = lane & 3;          // rows g and g + 8; columns 2 t4, 2 t4 + 1
  const int head0 = group * 16;                    // first head of the group within the KV head's
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff) + group * 64;   // [4 warps][16 rows]
  float2* unit_ml = reinterpret_cast<float2*>(smem + C::kUnitOff);
  const bool row0 = head0 + g < a.G, row1 = !kStack && head0 + g + 8 < a.G;
  int stage = 0;
  uint32_t phase = 0, group_phase = 0, all_phase = 0;
  // Barriers of warps, bounded like every wait: a warp that gave up is missed
  // for a while, not for ever.
  auto sync = [&](uint64_t* bar, uint32_t& parity) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    const bool ok = mbar_wait(bar, parity, a.status);
    parity ^= 1;
    return ok;
  };
  uint32_t qf[kDim / 16][4];
  float o[kDim / 8][4];
  float m[2], l[2];

  while (mbar_wait(full + stage, phase, a.status)) {
    const uint4 head = *reinterpret_cast<const uint4*>(&info[stage]);   // valid, flags, unit
    const uint32_t flags = head.z;
    if (flags & kEnd) break;
    if (flags & kFirst) {
      // The group's queries as A fragments, rows beyond G zero.
      const uint8_t* q = smem + C::kQOff + stage * C::kQ + (head0 + g) * C::kQRow + t4 * 4;
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        qf[kk][0] = row0 ? *reinterpret_cast<const uint32_t*>(q + kk * 32) : 0u;
        qf[kk][1] = row1 ? *reinterpret_cast<const uint32_t*>(q + 8 * C::kQRow + kk * 32) : 0u;
        qf[kk][2] = row0 ? *reinterpret_cast<const uint32_t*>(q + kk * 32 + 16) : 0u;
        qf[kk][3] = row1 ? *reinterpret_cast<const uint32_t*>(q + 8 * C::kQRow + kk * 32 + 16) : 0u;
      }
#pragma unroll
      for (int i = 0; i < kDim / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    // This warp's parts of the tile: slots (w kSub + sub) 16 .. + 15.
    int valid[kSub];
    bool any = false;
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
      const int part = w * kSub + sub;
      valid[sub] = static_cast<int>(((part < 4 ? head.x : head.y) >> (8 * (part & 3))) & 0xffu);
      any = any || valid[sub] > 0;
    }
    if (any) {
      const uint32_t ks = smem_u32(smem + stage * C::kStage);
      const uint32_t vs = ks + kTile * kDim * 2;
      const int row0w = w * kSub * 16;
      float z[kSub][2][4];
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        float even[2][4] = {}, odd[2][4] = {};   // two sums each: half the dependent products
        const int row = row0w + sub * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int kk = 0; kk < kDim / 16; kk += 2) {
          uint32_t r[4];
          ldmatrix_x4(r, ks + swz128_offset(row, kk * 2 + ((lane >> 3) & 1), kTile));
          mma_16816<kFp16>(even[0], qf[kk], r[0], r[1]);
          mma_16816<kFp16>(even[1], qf[kk], r[2], r[3]);
          ldmatrix_x4(r, ks + swz128_offset(row, kk * 2 + 2 + ((lane >> 3) & 1), kTile));
          mma_16816<kFp16>(odd[0], qf[kk + 1], r[0], r[1]);
          mma_16816<kFp16>(odd[1], qf[kk + 1], r[2], r[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[sub][j][e] = even[j][e] + odd[j][e];   // unscaled
      }
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        if (valid[sub] == 16) continue;
        // Slots past `valid` hold nothing: their probability is to be 0, and
        // their V rows, whatever the page (or the stage, where no page was
        // loaded) holds there, have to read as 0.
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j * 8 + 2 * t4 + (e & 1) >= valid[sub]) z[sub][j][e] = -INFINITY;
        for (int e = lane; e < (16 - valid[sub]) * (kDim / 8); e += 32) {
          const int row = row0w + sub * 16 + valid[sub] + e / (kDim / 8);
          *reinterpret_cast<uint4*>(smem + stage * C::kStage + kTile * kDim * 2 +
                                    swz128_offset(row, e % (kDim / 8), kTile)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();   // before the stage is loaded again
        __syncwarp();
      }
      if (a.weights) {
        float* sc = a.scores + (static_cast<long long>(head.w) * a.G + head0) * a.cap64 + info[stage].tile * kTile +
                    row0w + 2 * t4;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (r == 0 ? row0 : row1) {
              float* to = sc + static_cast<long long>(g + 8 * r) * a.cap64 + sub * 16;
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float2*>(to + 8 * j) = make_float2(z[sub][j][2 * r], z[sub][j][2 * r + 1]);
            }
      }
      float alpha[2];
      float base[2];
#pragma unroll
      for (int r = 0; r < (kStack ? 1 : 2); ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
          mx = fmaxf(mx, fmaxf(fmaxf(z[sub][0][2 * r], z[sub][0][2 * r + 1]),
                               fmaxf(z[sub][1][2 * r], z[sub][1][2 * r + 1])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m[r]);
        base[r] = mx == -INFINITY ? 0.f : mx;
        alpha[r] = fast_exp2((m[r] - base[r]) * a.scale2);
        m[r] = mx;
        l[r] *= alpha[r];
      }
      if constexpr (kStack) alpha[1] = alpha[0];
      const bool changed = alpha[0] != 1.f || alpha[1] != 1.f;
      if (__any_sync(0xffffffffu, changed)) {
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int r = 0; r < (kStack ? 1 : 2); ++r) {
          constexpr float kUp = kFp16 ? 14.f : 0.f;   // fp16: probabilities times 2^14
          const float p0 = fast_exp2(fmaf(z[sub][0][2 * r] - base[r], a.scale2, kUp));
          const float p1 = fast_exp2(fmaf(z[sub][0][2 * r + 1] - base[r], a.scale2, kUp));
          const float p2 = fast_exp2(fmaf(z[sub][1][2 * r] - base[r], a.scale2, kUp));
          const float p3 = fast_exp2(fmaf(z[sub][1][2 * r + 1] - base[r], a.scale2, kUp));
          l[r] += (p0 + p1) + (p2 + p3);
          split_pair<kFp16>(p0, p1, hi[r], lo[r]);
          split_pair<kFp16>(p2, p3, hi[2 + r], lo[2 + r]);
        }
        if constexpr (kStack) {
          hi[1] = lo[0];
          hi[3] = lo[2];
        }
        const int row = row0w + sub * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int dn = 0; dn < kDim / 16; ++dn) {
          uint32_t r[4];
          ldmatrix_x4_trans(r, vs + swz128_offset(row, dn * 2 + (lane >> 4), kTile));
          mma_16816<kFp16>(o[2 * dn], hi, r[0], r[1]);
          mma_16816<kFp16>(o[2 * dn + 1], hi, r[2], r[3]);
          if constexpr (!kStack) {
            mma_16816<kFp16>(o[2 * dn], lo, r[0], r[1]);
            mma_16816<kFp16>(o[2 * dn + 1], lo, r[2], r[3]);
          }
        }
      }
    }
    if (!(flags & kLast)) {   // the piece's last stage is held: it is the merge's scratch
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
      continue;
    }

    // ---- the four warps' partials merge in the last stage's memory ----------
    // [4 warps][16 rows (8 stacked)][kDim] fp32, 256 kDim bytes at most: a stage or half of one.
    if constexpr (kStack) {
#pragma unroll
      for (int i = 0; i < kDim / 8; ++i) {
        o[i][0] += o[i][2];
        o[i][1] += o[i][3];
      }
    }
#pragma unroll
    for (int r = 0; r < (kStack ? 1 : 2); ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t4 == 0) ml[w * 16 + g + 8 * r] = make_float2(m[r], l[r]);
    }
    const bool whole = (flags & kWhole) != 0;
    constexpr int kRows = kStack ? 8 : 16;
    float* buf = reinterpret_cast<float*>(smem + stage * C::kStage);
    bool ok = sync(group_bar + kGroups, all_phase);   // every warp is done with the stage; ml is written
    const long long unit = info[stage].unit;
    const int place = info[stage].place;
#pragma unroll
    for (int turn = 0; turn < kGroups; ++turn) {
      if (turn == group) {
#pragma unroll
        for (int r = 0; r < (kStack ? 1 : 2); ++r) {
          const int row = g + 8 * r;
          float mx = fmaxf(fmaxf(ml[row].x, ml[16 + row].x), fmaxf(ml[32 + row].x, ml[48 + row].x));
          if (mx == -INFINITY) mx = 0.f;
          const float f = fast_exp2((m[r] - mx) * a.scale2);
          float* to = buf + (w * kRows + row) * kDim;
          // Columns are permuted by row so that the 8 rows of a store meet
          // different banks.
#pragma unroll
          for (int i = 0; i < kDim / 8; ++i)
            *reinterpret_cast<float2*>(to + ((i * 8 + 2 * t4) ^ ((row & 3) << 3))) =
                make_float2(o[i][2 * r] * f, o[i][2 * r + 1] * f);
        }
        ok = sync(group_bar + group, group_phase) && ok;
        const int gt = tid - group * 128;
        const int rows = min(kRows, a.G - head0);
        for (int e = gt; e < rows * (kDim / 4); e += 128) {
          const int row = e / (kDim / 4), c = (e % (kDim / 4)) * 4;
          const float* from = buf + row * kDim + (c ^ ((row & 3) << 3));
          float4 y = *reinterpret_cast<const float4*>(from);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            const float4 z = *reinterpret_cast<const float4*>(from + i * kRows * kDim);
            y.x += z.x;
            y.y += z.y;
            y.z += z.z;
            y.w += z.w;
          }
          float mx = fmaxf(fmaxf(ml[row].x, ml[16 + row].x), fmaxf(ml[32 + row].x, ml[48 + row].x));
          const float use = mx == -INFINITY ? 0.f : mx;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += ml[i * 16 + row].y * fast_exp2((ml[i * 16 + row].x - use) * a.scale2);
          const long long head = unit * a.G + head0 + row;
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint2 z;
            z.x = pack_pair<kFp16>(y.x * inv, y.y * inv);
            z.y = pack_pair<kFp16>(y.z * inv, y.w * inv);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + head * kDim + c) = z;
            if (c == 0) {
              if (a.lse) a.lse[head] = lse_of<kFp16>(use, sum, a.scale2);
              if (a.whole || a.cluster)
                unit_ml[head0 + row] = m_and_inverse<kFp16>(mx, sum);
              else if (a.weights)
                a.unit_ml[head] = m_and_inverse<kFp16>(mx, sum);
            }
          } else {
            *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(place) * a.G + head0 + row) * kDim + c) = y;
            if (c == 0) a.part_ml[place * kPagedMaxGroup + head0 + row] = make_float2(mx, sum);
          }
        }
        fence_proxy_async_smem();   // the next tile lands here through the async proxy
      }
      if (kGroups > 1) ok = sync(group_bar + kGroups, all_phase) && ok;
    }
    if (kGroups == 1) ok = sync(group_bar + group, group_phase) && ok;   // ml is read before the next piece writes it
    // (The barrier also orders the z that every warp has stored and the lse.)
    if (a.whole && a.weights)
      add_weights(a, unit, info[stage].b, info[stage].unit - info[stage].b * a.Hkv, info[stage].len, 4 * tid,
                  4 * 128 * kGroups, unit_ml);
    if (!ok) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + stage);
    if (++stage == C::kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (a.cluster == 0) return;

  // ---- a cluster joins its unit ---------------------------------------------
  // The pieces lie in the workspace; the cluster's barrier orders them.
  cluster_sync();
  Piece p;
  const bool mine = cluster_piece(p, a, cta);
  const int unit = cta / a.cluster, rank = cta % a.cluster;
  int pieces = 0;
  for (int r = 0; r < a.cluster; ++r)
    pieces += p.tiles * (r + 1) / a.cluster > p.tiles * r / a.cluster ? 1 : 0;
  if (pieces > 1) {
    auto has = [&](int r) { return p.tiles * (r + 1) / a.cluster > p.tiles * r / a.cluster; };
    // Head rank + C i is joined by warp i of CTA `rank`.
    for (int h = rank + a.cluster * warp; h < a.G; h += a.cluster * 4 * kGroups) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float mx = -INFINITY, sum = 0.f;
      float2 v[kMaxCluster];   // all pieces in flight
      float4 y[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        v[r] = make_float2(-INFINITY, 0.f);
        y[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < a.cluster && has(r)) {
          const long long at = unit * a.cluster + r;
          v[r] = __ldcg(a.part_ml + at * kPagedMaxGroup + h);
          if (lane < kDim / 4) y[r] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (at * a.G + h) * kDim) + lane);
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) merge_sums(mx, sum, x, v[r].x, v[r].y, y[r], a.scale2);
      const float use = mx == -INFINITY ? 0.f : mx;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long head = static_cast<long long>(unit) * a.G + h;
      if (lane < kDim / 4) {
        uint2 y;
        y.x = pack_pair<kFp16>(x.x * inv, x.y * inv);
        y.y = pack_pair<kFp16>(x.z * inv, x.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + head * kDim + lane * 4) = y;
      }
      if (lane == 0 && a.lse) a.lse[head] = lse_of<kFp16>(use, sum, a.scale2);
    }
    if (a.weights && tid < a.G) {
      float mx = -INFINITY, sum = 0.f;
      for (int r = 0; r < a.cluster; ++r) {
        if (!has(r)) continue;
        const float2 v = __ldcg(a.part_ml + static_cast<long long>(unit * a.cluster + r) * kPagedMaxGroup + tid);
        merge_ml(mx, sum, v.x, v.y, a.scale2);
      }
      unit_ml[tid] = m_and_inverse<kFp16>(mx, sum);
    }
  }
  if (a.weights && mine && sync(group_bar + kGroups, all_phase))
    add_weights(a, unit, p.b, p.h, min(p.len, p.tile1 * kTile), p.tile0 * kTile + 4 * tid, 4 * 128 * kGroups, unit_ml);
}

// ---- the join -----------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kChunk = 4 * kJoinThreads;   // slots that a CTA of the weights' part takes at once

// The first `jobs` CTAs (weights only), as many for every unit, add each slot's
// weight, from the z that the pass left and the unit's (m, l): CTA y of a unit
// takes chunks y, y + jobs / units, ... of it.  The CTAs behind them join `hp`
// heads (a power of two up to 8) of one cut unit each.
template <bool kFp16, int kDim>
__global__ void __launch_bounds__(kJoinThreads, 4) paged_join_kernel(const PagedAttnArgs a, int jobs, int hp) {
  __shared__ float red_m[8], red_l[8];
  __shared__ float4 red_o[8][kDim / 4];
  __shared__ float2 unit_ml[kPagedMaxGroup];
  __shared__ float2 red_ml[kJoinThreads / 32][kPagedMaxGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) >= jobs) {
    const int per_cut = (a.G + hp - 1) / hp, job = blockIdx.x - jobs;
    const int at = job / per_cut;
    if (a.chunk_cut && at >= *a.chunks) return;
    const int4 c = (a.chunk_cut ? a.chunk_cut : a.unit_cut)[at];
    if ((a.chunk_cut ? c.y : c.x) != at || !cut_in_range(c.x, c.y, c.z, c.w, a.B * a.Hkv, a.most)) return;
    const int warps = 8 / hp, warp0 = warp / warps * warps;   // a head's warps
    const int h = job % per_cut * hp + warp / warps;
    const int i = c.y, t = tid - warp0 * 32;
    // Chunks i - 1 .. c.z hold a piece; a head past the last one joins none.
    const int pieces = h < a.G ? c.z - i + 2 : 0;
    auto slot_of = [&](int j) { return j == 0 ? c.w : 2 * (i - 1 + j); };
    constexpr int kLanes = kDim / 4;            // threads of a row
    const int par = warps * 32 / kLanes;        // rows at once
    const int col = t % kLanes, part = t / kLanes;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, sum = 0.f;
    constexpr int kAhead = 8;   // rows in flight
    for (int j0 = part; j0 < pieces; j0 += kAhead * par) {
      float2 v[kAhead];
      float4 y[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int j = j0 + e * par;
        v[e] = make_float2(-INFINITY, 0.f);
        y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < pieces) {
          const int sl = slot_of(j);
          v[e] = a.part_ml[sl * kPagedMaxGroup + h];
          y[e] = *reinterpret_cast<const float4*>(a.part_o + (static_cast<long long>(sl) * a.G + h) * kDim + col * 4);
        }
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) merge_sums(mx, sum, x, v[e].x, v[e].y, y[e], a.scale2);
    }
    if constexpr (kLanes == 16) {   // two rows per warp
      const float m2 = __shfl_xor_sync(0xffffffffu, mx, 16), s2 = __shfl_xor_sync(0xffffffffu, sum, 16);
      const float4 x2 = make_float4(__shfl_xor_sync(0xffffffffu, x.x, 16), __shfl_xor_sync(0xffffffffu, x.y, 16),
                                    __shfl_xor_sync(0xffffffffu, x.z, 16), __shfl_xor_sync(0xffffffffu, x.w, 16));
      merge_sums(mx, sum, x, m2, s2, x2, a.scale2);
    }
    if (lane < kLanes) red_o[warp][lane] = x;
    if (lane == 0) {
      red_m[warp] = mx;
      red_l[warp] = sum;
    }
    __syncthreads();
    if (t < kLanes && h < a.G) {
      for (int j = warp0 + 1; j < warp0 + warps; ++j)
        merge_sums(mx, sum, x, red_m[j], red_l[j], red_o[j][t], a.scale2);
      const float use = mx == -INFINITY ? 0.f : mx;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long head = static_cast<long long>(c.x) * a.G + h;
      uint2 y;
      y.x = pack_pair<kFp16>(x.x * inv, x.y * inv);
      y.y = pack_pair<kFp16>(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + head * kDim + t * 4) = y;
      if (t == 0 && a.lse) a.lse[head] = lse_of<kFp16>(use, sum, a.scale2);
    }
    return;
  }

  // -------------------------------------------------------------- weights ------
  const int units = a.B * a.Hkv;
  const int y = blockIdx.x / units, unit_i = blockIdx.x % units, step = jobs / units;
  const int b = unit_i / a.Hkv, kv_head = unit_i % a.Hkv;
  const int len = paged_len(a.kv_lens, b, a.cap, a.status);
  if (y * kChunk >= len) return;
  const long long unit = unit_i;
  {
    const int4 c = a.unit_cut[unit];
    if (c.x < 0) {
      if (tid < a.G) unit_ml[tid] = a.unit_ml[unit * a.G + tid];
    } else if (c.x != unit_i || !cut_in_range(c.x, c.y, c.z, c.w, units, a.most)) {
      return;
    } else {
      // The pieces' (m, l): `wide` lanes read a piece's heads, 8 loads in flight.
      const int pieces = c.z - c.y + 2;
      const int wide = a.G > 16 ? 32 : (a.G > 8 ? 16 : 8), rows = kJoinThreads / wide;
      const int head = tid % wide;
      float mx = -INFINITY, sum = 0.f;
      for (int j0 = tid / wide; j0 < pieces; j0 += 8 * rows) {
        float2 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + e * rows;
          v[e] = make_float2(-INFINITY, 0.f);
          if (j < pieces && head < a.G) v[e] = a.part_ml[(j == 0 ? c.w : 2 * (c.y - 1 + j)) * kPagedMaxGroup + head];
        }
        float nm = mx;
#pragma unroll
        for (int e = 0; e < 8; ++e) nm = fmaxf(nm, v[e].x);
        const float use = nm == -INFINITY ? 0.f : nm;
        sum *= fast_exp2((mx - use) * a.scale2);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e].y * fast_exp2((v[e].x - use) * a.scale2);
        mx = nm;
      }
      for (int o = wide; o < 32; o <<= 1) {   // rows within the warp
        const float m2 = __shfl_xor_sync(0xffffffffu, mx, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        merge_ml(mx, sum, m2, s2, a.scale2);
      }
      red_ml[warp][lane] = make_float2(mx, sum);
      __syncthreads();
      if (warp == 0 && lane < a.G) {
        float all = mx;
#pragma unroll
        for (int j = 1; j < kJoinThreads / 32; ++j) all = fmaxf(all, red_ml[j][lane].x);
        const float use = all == -INFINITY ? 0.f : all;
        float l = 0.f;
#pragma unroll
        for (int j = 0; j < kJoinThreads / 32; ++j) l += red_ml[j][lane].y * fast_exp2((red_ml[j][lane].x - use) * a.scale2);
        unit_ml[lane] = m_and_inverse<kFp16>(all, l);
      }
    }
    __syncthreads();
  }
  add_weights(a, unit, b, kv_head, len, y * kChunk + 4 * tid, step * kChunk, unit_ml);
}

// The count of chunks handed out starts at 0.
__global__ void paged_counter_kernel(int* next) {
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) *next = 0;
}

// ---- host side -------------------------------------------------------------------

// Where clusters do not serve, caches of up to this many slots are attended
// without cuts, in one launch (256 units of 128 to 256 slots, 16 heads, d 128:
// 11.4 us without cuts, 17.5 with them; of 256 to 512 slots 21.4 and 22.7, and
// with fewer units of those cuts win).
constexpr int kWholeCap = 256;

int tile_shift_of(const PagedShape& s, int G) {
  static_assert(kTileOf<128, 1> == 64 && kTileOf<64, 1> == 128 && kTileOf<128, 2> == 128 && kTileOf<64, 2> == 128, "");
  return s.D == 128 && G <= 16 ? 6 : 7;
}

int unit_tiles_of(const PagedShape& s, int G) {
  const int shift = tile_shift_of(s, G);
  return (s.cap + (1 << shift) - 1) >> shift;
}

int attn_ctas(const PagedShape& s, int G) {
  const long long positions = static_cast<long long>(s.B) * s.Hkv * (unit_tiles_of(s, G) + kUnitCost);
  const long long most = static_cast<long long>(device_sm_count()) * (G > 16 ? 1 : 2);
  return static_cast<int>(positions < most ? positions : most);
}

// CTAs of a cluster for each unit, or 0 where the line is split over all CTAs.
// A cluster joins its unit itself, which saves the second launch, but its few
// CTAs have to suffice.  With 8 or 4 CTAs, d 128, 16 heads, calls from Python,
// clusters against the split: 2 units of 512 / 1024 / 2048 / 4096 slots 8.0 / 8.6 /
// 10.1 / 12.9 us against 9.6 / 9.8 / 9.8 / 10.2; 16 units of 512 / 2048 / 4096 / 8192
// slots 8.6 / 11.0 / 15.0 / 22.5 against 11.6 / 13.2 / 17.2 / 22.9; so two tiles per
// CTA, or eight where half the SMs have a CTA.  Clusters that fill more than half
// of the GPU's CTAs do not all fit its processing clusters at once (32 units of
// 512 slots: 11.2 us with 8 CTAs each, 8.9 with 4).
int cluster_size(const PagedShape& s, int G) {
  const int tiles = unit_tiles_of(s, G), sms = device_sm_count();
  const long long units = static_cast<long long>(s.B) * s.Hkv;
  if (tiles < 3) return 0;
  for (int c = kMaxCluster; c >= 4; c /= 2) {
    const long long ctas = units * c;
    if (2 * tiles <= c || 2 * ctas > sms * (G > 16 ? 1 : 2)) continue;
    return tiles <= c * (2 * ctas >= sms ? 8 : 2) ? c : 0;
  }
  return 0;
}

// Scores of a head: the capacity in whole tiles.
size_t score_row(const PagedShape& s, int G) {
  return static_cast<size_t>(unit_tiles_of(s, G)) << tile_shift_of(s, G);
}

// Small chunks are handed out where the line is long enough for the SMs' rates
// to matter more than the counter's launch: 128 tiles of the capacity for every
// CTA.  32 x 32K (430 tiles per CTA): 572 us in equal shares, 552 handed out; 64
// ragged (215): 205 and 201; 96 short (81): 70.5 and 70.9, and 2 us of the host.
bool hands_out(const PagedShape& s, int G, int ctas) {
  return static_cast<long long>(s.B) * s.Hkv * unit_tiles_of(s, G) >= 128LL * ctas;
}

// Chunks at most: see make_split.
int most_chunks(const PagedShape& s, int G, int ctas) { return hands_out(s, G, ctas) ? 7 * ctas : ctas; }

struct WsLayout {
  size_t counts, unit_cut, chunk_cut, ml, o, unit_ml, scores, total;
};

WsLayout ws_layout(const PagedShape& s, int G) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t n = most_chunks(s, G, attn_ctas(s, G)), units = static_cast<size_t>(s.B) * s.Hkv, heads = units * G;
  const size_t row = score_row(s, G);
  WsLayout w;
  w.counts = 0;
  w.unit_cut = 256;
  w.chunk_cut = w.unit_cut + up(units * sizeof(int4));
  w.ml = w.chunk_cut + up(n * sizeof(int4));
  w.o = w.ml + up(2 * n * kPagedMaxGroup * sizeof(float2));
  w.unit_ml = w.o + up(2 * n * G * s.D * sizeof(float));
  w.scores = w.unit_ml + (s.weights ? up(heads * sizeof(float2)) : 0);
  w.total = w.scores + (s.weights ? up(heads * row * sizeof(float)) : 0);
  return w;
}

// CTAs of the weights' part: about 8 per SM, the same number for every unit
// and no more than its chunks.  Their loads are short, and latency is what they
// wait for.
int weight_jobs(const PagedAttnArgs& a) {
  const int units = a.B * a.Hkv, chunks = (a.cap + kChunk - 1) / kChunk;
  const int want = (8 * device_sm_count() + units - 1) / units;
  return units * (want < chunks ? want : chunks);
}

template <typename F, typename... A>
cudaError_t launch_pdl(F kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool kFp16, int kDim, int kGroups, bool kStack>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas, int most,
                   cudaStream_t st) {
  using C = AttnCfg<kDim, kGroups, kStack>;
  auto kernel = paged_attn_kernel<kFp16, kDim, kGroups, kStack>;
  static std::atomic<uint64_t> allowed{0};   // devices whose copy of the kernel has the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (a.next) {
    e = launch_pdl(paged_counter_kernel, dim3(1), 32, 0, st, 0, a.next);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(kernel, dim3(a.cluster ? a.B * a.Hkv * a.cluster : ctas), C::kThreads, C::kSmem, st, a.cluster, km, vm,
                 a);
  if (e != cudaSuccess || a.whole || a.cluster) return e;
  const int jobs = a.weights ? weight_jobs(a) : 0;
  // One CTA per head of a cut unit while that fills no more than the SMs twice
  // (a long sequence's unit has hundreds of pieces), else up to 8 heads each.
  const int cuts = a.chunk_cut ? most : a.B * a.Hkv;
  int hp = 1;
  while (hp < 8 && cuts * ((a.G + hp - 1) / hp) > 2 * device_sm_count()) hp *= 2;
  return launch_pdl(paged_join_kernel<kFp16, kDim>, dim3(static_cast<unsigned>(jobs + cuts * ((a.G + hp - 1) / hp))),
                    kJoinThreads, 0, st, 0, a, jobs, hp);
}

template <bool kFp16, int kDim>
cudaError_t launch_g(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas, int most,
                     cudaStream_t st) {
  if (a.G > 16) return launch<kFp16, kDim, 2, false>(km, vm, a, ctas, most, st);
  if (a.G > 8) return launch<kFp16, kDim, 1, false>(km, vm, a, ctas, most, st);
  return launch<kFp16, kDim, 1, true>(km, vm, a, ctas, most, st);
}

}  // namespace

size_t paged_attn_workspace_bytes(const PagedShape& s, int G) { return ws_layout(s, G).total; }

cudaError_t launch_paged_attn(const PagedShape& s, int G, const CUtensorMap& k_map, PagedMapOrder k_order,
                              const CUtensorMap& v_map, PagedMapOrder v_order, int box_rows, const void* q,
                              float scale2, bool accumulate, void* out, float* lse, void* ws, cudaStream_t st) {
  const WsLayout w = ws_layout(s, G);
  char* base = static_cast<char*>(ws);
  PagedAttnArgs a;
  a.B = s.B;
  a.Hkv = s.Hkv;
  a.G = G;
  a.ps = s.ps;
  a.P = s.P;
  a.maxp = s.maxp;
  a.cap = s.cap;
  a.box = box_rows;
  a.ko = k_order;
  a.vo = v_order;
  a.scale2 = scale2;
  a.q = q;
  a.table = s.table;
  a.kv_lens = s.kv_lens;
  a.out = out;
  a.lse = lse;
  a.weights = accumulate ? s.weights : nullptr;
  a.part_ml = reinterpret_cast<float2*>(base + w.ml);
  a.part_o = reinterpret_cast<float*>(base + w.o);
  a.unit_ml = reinterpret_cast<float2*>(base + w.unit_ml);
  a.scores = reinterpret_cast<float*>(base + w.scores);
  a.cap64 = static_cast<int>(score_row(s, G));
  a.tile_shift = tile_shift_of(s, G);
  a.status = s.status;
  const int ctas = attn_ctas(s, G), most = most_chunks(s, G, ctas);
  const bool by_unit = s.B * s.Hkv <= most;
  a.most = most;
  a.cluster = cluster_size(s, G);
  a.whole = !a.cluster && s.cap <= kWholeCap;   // then nothing is cut and nothing joined
  const bool joins = !a.whole && !a.cluster;   // a second launch does
  a.unit_cut = joins && (by_unit || accumulate) ? reinterpret_cast<int4*>(base + w.unit_cut) : nullptr;
  a.chunk_cut = joins && !by_unit ? reinterpret_cast<int4*>(base + w.chunk_cut) : nullptr;
  a.chunks = !joins ? nullptr : reinterpret_cast<int*>(base + w.counts);
  a.next = joins && hands_out(s, G, ctas) ? reinterpret_cast<int*>(base + w.counts) + 1 : nullptr;
  if (s.fp16)
    return s.D == 128 ? launch_g<true, 128>(k_map, v_map, a, ctas, most, st)
                      : launch_g<true, 64>(k_map, v_map, a, ctas, most, st);
  return s.D == 128 ? launch_g<false, 128>(k_map, v_map, a, ctas, most, st)
                    : launch_g<false, 64>(k_map, v_map, a, ctas, most, st);
}

}  // namespace infllmv2
