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
// Split.  The work is all 64-slot tiles of all (sequence, KV head) units, in
// that order, each unit with a fixed cost before its tiles; the CTAs take
// equal shares of that line, so those of any ragged batch carry the same load,
// and one long sequence spreads over all SMs.  A unit inside one CTA is finished there; of a unit that CTA borders
// cut, each piece leaves (m, l, sum of exp(z - m) v) in the workspace and
// paged_join_kernel joins them.  The host needs no lengths.
//
// A CTA.  One warp loads: per page piece (16, 32 or 64 rows of one page) it
// issues one TMA box per 64 columns of K and of V, through a ring of tiles.
// Four warps (eight for 17 to 32 heads: four per half) compute, each on its
// own 16 slots of every tile with its own running maximum and sum, so that
// nothing but the ring's barriers is shared until the unit's end.  The heads
// are the 16 rows of mma.m16n8k16: at these intensities the tensor pipe idles
// and a tcgen05 tile (128 rows) would be seven eighths empty.
//
// Types.  z, maxima, sums and accumulators are fp32.  A probability feeds the
// product with V as two 16-bit parts (hi + lo, 16 to 22 significant bits): one
// rounding of it to bf16 would cost as much again as the output's own.  With
// up to 8 heads the lo parts fill the rows 8..15 that would be empty; with
// more they are a second product.  fp16 probabilities are scaled by 2^14, so
// that the long tail of a sharp softmax stays above fp16's smallest number.
#include <atomic>

#include "paged.cuh"
#include "kernels.h"

namespace infllmv2 {

namespace {

constexpr int kTile = 64;   // slots per tile

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
  float* part_o;     // [2 n][G][D]: pieces of cut units, relative to their m
  float2* part_ml;   // [2 n][32]: (m in log2 units, l)
  // Cut units, (unit or -1, CTA of the second piece, last CTA, first piece's
  // slot).  unit_cut, by unit, is kept where there are no more units than CTAs
  // or weights are summed; cta_cut, by the CTA that the second piece starts,
  // where there are more units than CTAs.  The join goes by the shorter list.
  int4* unit_cut;
  int4* cta_cut;
  float* lse2;       // [B Hkv G] lse in log2 units, of units that no border cut (weights only)
  float* scores;     // [B Hkv G][cap64] z in log2 units (weights only)
  int cap64;         // cap rounded up to whole tiles
  int whole;         // no unit is cut: one launch
  uint32_t* status;
};

// ---- the split of the tiles over the CTAs ----------------------------------

// The units lie one after the other on a line, each `cost` positions for its
// fixed work (queries, merge, output) and then one for every tile; empty
// sequences take none.  CTA i has positions [i W / n, (i + 1) W / n) and the
// tiles in them.
struct Split {
  long long W;           // positions
  int n;                 // CTAs that have positions: min(CTAs, W)
  int cost;
  bool whole;            // units go whole to the CTA that has their first position
  long long begin, end;  // this CTA's positions
  int b, h;              // the unit of the first one
  long long unit0;       // where that unit begins
};

__device__ __forceinline__ long long split_begin(const Split& s, int i) { return i * s.W / s.n; }
// The CTA that a position belongs to.
__device__ __forceinline__ int split_owner(const Split& s, long long at) {
  return static_cast<int>(((at + 1) * s.n - 1) / s.W);
}

__device__ __forceinline__ int unit_tiles(int len) { return (len + kTile - 1) / kTile; }

// All threads of the CTA.  Each sums a run of sequences; the one whose run
// holds the CTA's first position says where that is.
template <int kThreads>
__device__ __forceinline__ Split make_split(const PagedAttnArgs& a, int cta, int ctas, int cost, int* shared) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
  auto width = [&](int b) {   // of one unit of sequence b
    const int tiles = unit_tiles(paged_len(a.kv_lens, b, a.cap, a.status));
    return tiles ? tiles + cost : 0;
  };
  int sum = 0;   // at most 32 sequences of 2^24 tiles (4096 sequences, 2^30 slots)
  for (int b = b0; b < b1; ++b) sum += width(b);
  long long pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += up;
  }
  long long* totals = reinterpret_cast<long long*>(shared);   // [kWarps]
  if (lane == 31) totals[warp] = pre;
  __syncthreads();
  long long all = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all += totals[w];
  }
  pre += before - sum;   // positions of one KV head before this thread's run
  Split s;
  s.W = all * a.Hkv;
  s.n = static_cast<int>(min(static_cast<long long>(ctas), s.W));
  s.cost = cost;
  s.whole = a.whole != 0;
  s.begin = s.end = s.unit0 = 0;
  s.b = s.h = 0;
  int* where = shared + 2 * kWarps;
  if (cta < s.n) {
    s.begin = split_begin(s, cta);
    s.end = split_begin(s, cta + 1);
    if (s.begin >= pre * a.Hkv && s.begin < (pre + sum) * a.Hkv) {
      long long rest = s.begin - pre * a.Hkv;
      for (int b = b0; b < b1; ++b) {
        const int w = width(b);
        if (rest < static_cast<long long>(w) * a.Hkv) {
          where[0] = b;
          where[1] = static_cast<int>(rest / w);
          where[2] = static_cast<int>(rest % w);
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
    s.unit0 = s.begin - where[2];
  }
  return s;
}

// The tiles of one unit in a CTA's positions.
struct Piece {
  int b, h, len, tiles;      // the unit: its sequence, KV head, slots and tiles
  int tile0, tile1;          // the piece
  long long unit0;           // where the unit begins
};

__device__ __forceinline__ long long tile_at(const Split& s, const Piece& p, int tile) { return p.unit0 + s.cost + tile; }

__device__ __forceinline__ bool next_piece(Piece& p, const Split& s, const PagedAttnArgs& a);

// Both: false where the CTA's positions hold no (further) tile.
__device__ __forceinline__ bool first_piece(Piece& p, const Split& s, const PagedAttnArgs& a) {
  if (s.end == s.begin) return false;
  p.b = s.b;
  p.h = s.h;
  p.len = paged_len(a.kv_lens, p.b, a.cap, a.status);
  p.tiles = unit_tiles(p.len);
  p.unit0 = s.unit0;
  p.tile0 = max(0, static_cast<int>(s.begin - p.unit0) - s.cost);
  p.tile1 = static_cast<int>(min(static_cast<long long>(p.tiles), s.end - tile_at(s, p, 0)));
  if (s.whole) {
    if (p.unit0 < s.begin) return next_piece(p, s, a);
    p.tile1 = p.tiles;
  }
  return p.tile1 > p.tile0;
}

__device__ __forceinline__ bool next_piece(Piece& p, const Split& s, const PagedAttnArgs& a) {
  p.unit0 = tile_at(s, p, p.tiles);
  if (p.unit0 >= s.end) return false;
  if (++p.h == a.Hkv) {
    p.h = 0;
    do {
      ++p.b;
      p.len = paged_len(a.kv_lens, p.b, a.cap, a.status);
    } while (p.len == 0);   // positions are left, so a sequence with slots is
    p.tiles = unit_tiles(p.len);
  }
  p.tile0 = 0;
  p.tile1 = s.whole ? p.tiles : static_cast<int>(min(static_cast<long long>(p.tiles), s.end - tile_at(s, p, 0)));
  return p.tile1 > 0;
}

// Workspace slot of a cut unit's piece in CTA i: 2 i for a piece that starts at
// the CTA's first position, 2 i + 1 for one that starts later (and so is its last).
__device__ __forceinline__ int piece_slot(const Split& s, int cta, long long at) {
  return 2 * cta + (at > split_begin(s, cta) ? 1 : 0);
}

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

// Two floats as 16-bit parts: hi = their roundings, lo = the rest's.
template <bool kFp16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (kFp16) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    hi = pack_bf16x2(x, y);
    lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
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

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Adds the weights of slots `first`, + `step`, ... (four each) of a unit, from
// the z of its heads and their lse.
__device__ __forceinline__ void add_weights(const PagedAttnArgs& a, long long unit, int b, int kv_head, int len, int first,
                                            int step, const float* lse2) {
  const int32_t* table = a.table + static_cast<long long>(b) * a.maxp;
  for (int slot = first; slot < len; slot += step) {   // the four share a page (pages hold multiples of 16)
    const int page = __ldg(table + slot / a.ps);
    const float* z = a.scores + unit * a.G * a.cap64 + slot;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < a.G; ++h) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(z + static_cast<long long>(h) * a.cap64));
      const float l = lse2[h];
      w.x += fast_exp2(x.x - l);
      w.y += fast_exp2(x.y - l);
      w.z += fast_exp2(x.z - l);
      w.w += fast_exp2(x.w - l);
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

// A unit's queries, merge and output cost a CTA about as much as this many tiles.
template <int kDim>
constexpr int kUnitCost = kDim == 64 ? 2 : 1;

// kGroups: groups of four warps, one per 16 heads.  kStack: at most 8 heads,
// the lo parts of the probabilities in rows 8..15.
template <int kDim, int kGroups, bool kStack>
struct AttnCfg {
  static constexpr int kStage = kTile * kDim * 4;   // K and V of a tile
  // Two CTAs of at most 113 KB per SM for one group, one of at most 227 KB for two.
  static constexpr int kStages = (kGroups == 1 ? 98304 : 196608) / kStage;
  static constexpr int kThreads = 32 + 128 * kGroups;
  static constexpr int kPerSm = kGroups == 1 ? 2 : 1;
  static constexpr int kCost = kUnitCost<kDim>;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kInfoOff = kBarOff + 2 * kStages * 8;
  static constexpr int kMlOff = kInfoOff + ((kStages * 4 + 15) & ~15);
  static constexpr int kLseOff = kMlOff + kGroups * 4 * 16 * 8;      // a whole unit's lse in log2 units
  static constexpr int kSplitOff = kLseOff + kPagedMaxGroup * 4;
  static constexpr int kSmem = 1024 + kSplitOff + 128;
};

template <bool kFp16, int kDim, int kGroups, bool kStack>
__global__ void __launch_bounds__(AttnCfg<kDim, kGroups, kStack>::kThreads, AttnCfg<kDim, kGroups, kStack>::kPerSm)
    paged_attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const PagedAttnArgs a) {
  using C = AttnCfg<kDim, kGroups, kStack>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint32_t* info = reinterpret_cast<uint32_t*>(smem + C::kInfoOff);   // per stage: valid rows of each 16, 8 bits each
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4 * kGroups);
    }
    fence_barrier_init();
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  pdl_wait();
  pdl_trigger();
  const Split s = make_split<C::kThreads>(a, cta, ctas, C::kCost, reinterpret_cast<int*>(smem + C::kSplitOff));

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
  Piece p;
  if (!first_piece(p, s, a)) {
    if (tid == 0 && a.cta_cut) a.cta_cut[cta] = make_int4(-1, 0, 0, 0);
    return;
  }

  if (warp == 4 * kGroups) {
    // ------------------------------------------------ the loading warp -------
    if (lane == 0) {
      // Does the previous CTA hold the first piece of the unit that starts this one?
      const long long first = tile_at(s, p, 0);
      const bool second = p.tile0 > 0 && split_owner(s, first) == cta - 1;
      const int unit = p.b * a.Hkv + p.h;
      int4 c = make_int4(-1, 0, 0, 0);
      if (second)
        c = make_int4(unit, cta, split_owner(s, tile_at(s, p, p.tiles - 1)), piece_slot(s, cta - 1, first));
      if (a.cta_cut) a.cta_cut[cta] = c;
      if (a.unit_cut && second) a.unit_cut[unit] = c;
    }
    const int boxes = kTile / a.box;
    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    uint32_t issued = 0;
    do {
      if (lane == 0 && a.unit_cut && p.tile0 == 0 && p.tile1 == p.tiles)
        a.unit_cut[p.b * a.Hkv + p.h] = make_int4(-1, 0, 0, 0);
      const int32_t* row = a.table + static_cast<long long>(p.b) * a.maxp;
      // Lane i handles box i of a tile; its page is fetched one tile ahead.
      auto fetch = [&](int tile) {
        const int slot = tile * kTile + lane * a.box;
        return (lane < boxes && tile < p.tile1 && slot < p.len) ? __ldg(row + slot / a.ps) : -1;
      };
      int page_next = fetch(p.tile0);
      for (int t = p.tile0; t < p.tile1 && !dead; ++t) {
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
          uint32_t v = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int left = p.len - (t * kTile + w * 16);
            if ((oks >> (w * 16 / a.box)) & 1u) v |= static_cast<uint32_t>(max(0, min(16, left))) << (8 * w);
          }
          info[stage] = v;
          mbar_arrive_expect_tx(full + stage, __popc(oks) * a.box * kDim * 4);
        }
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
    } while (!dead && next_piece(p, s, a));
    if (dead) {
      // A wait gave up: nothing more is issued, and the copies in flight land
      // (or are waited for as long) before this warp leaves.
      const uint32_t from = issued > C::kStages ? issued - C::kStages : 0;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait(full + i % C::kStages, (i / C::kStages) & 1, a.status);
    }
    return;
  }

  // -------------------------------------------------- the computing warps -----
  const int group = kGroups == 1 ? 0 : warp >> 2, w = warp & 3;       // 16 heads; 16 slots of a tile
  const int g = lane >> 2, t4 = lane & 3;          // rows g and g + 8; columns 2 t4, 2 t4 + 1
  const int head0 = group * 16;                    // first head of the group within the KV head's
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff) + group * 64;   // [4 warps][16 rows]
  float* unit_lse2 = reinterpret_cast<float*>(smem + C::kLseOff);
  const bool row0 = head0 + g < a.G, row1 = !kStack && head0 + g + 8 < a.G;
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;
  bool more = true;
  while (more) {
    const long long unit = static_cast<long long>(p.b) * a.Hkv + p.h;
    // The group's queries as A fragments, rows beyond G zero.
    uint32_t qf[kDim / 16][4];
    {
      const uint32_t* q = static_cast<const uint32_t*>(a.q) + (unit * a.G + head0) * (kDim / 2);
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        const int c = kk * 8 + t4;
        qf[kk][0] = row0 ? __ldg(q + g * (kDim / 2) + c) : 0u;
        qf[kk][1] = row1 ? __ldg(q + (g + 8) * (kDim / 2) + c) : 0u;
        qf[kk][2] = row0 ? __ldg(q + g * (kDim / 2) + c + 4) : 0u;
        qf[kk][3] = row1 ? __ldg(q + (g + 8) * (kDim / 2) + c + 4) : 0u;
      }
    }
    float o[kDim / 8][4];
#pragma unroll
    for (int i = 0; i < kDim / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int t = p.tile0; t < p.tile1; ++t) {
      if (!dead) dead = !mbar_wait(full + stage, phase, a.status);
      const int valid = dead ? 0 : static_cast<int>((info[stage] >> (8 * w)) & 0xffu);
      const uint32_t ks = smem_u32(smem + stage * C::kStage);
      const uint32_t vs = ks + kTile * kDim * 2;
      if (valid > 0) {
        if (valid < 16) {
          // Slots past `valid` hold nothing: their probability will be 0, and
          // their V rows, whatever the page holds there, have to read as 0.
          for (int e = lane; e < (16 - valid) * (kDim / 8); e += 32) {
            const int row = w * 16 + valid + e / (kDim / 8);
            *reinterpret_cast<uint4*>(smem + stage * C::kStage + kTile * kDim * 2 +
                                      swz128_offset(row, e % (kDim / 8), kTile)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();   // before the stage is loaded again
          __syncwarp();
        }
        float z[2][4];
        {
          float even[2][4] = {}, odd[2][4] = {};   // two sums each: half the dependent products
          const int row = w * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
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
            for (int e = 0; e < 4; ++e) z[j][e] = even[j][e] + odd[j][e];   // unscaled
        }
        if (valid < 16) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j * 8 + 2 * t4 + (e & 1) >= valid) z[j][e] = -INFINITY;
        }
        if (a.weights) {
          float* sc = a.scores + (unit * a.G + head0) * a.cap64 + t * kTile + w * 16 + 2 * t4;
          if (row0) {
            float* r = sc + static_cast<long long>(g) * a.cap64;
            *reinterpret_cast<float2*>(r) = make_float2(z[0][0] * a.scale2, z[0][1] * a.scale2);
            *reinterpret_cast<float2*>(r + 8) = make_float2(z[1][0] * a.scale2, z[1][1] * a.scale2);
          }
          if (row1) {
            float* r = sc + static_cast<long long>(g + 8) * a.cap64;
            *reinterpret_cast<float2*>(r) = make_float2(z[0][2] * a.scale2, z[0][3] * a.scale2);
            *reinterpret_cast<float2*>(r + 8) = make_float2(z[1][2] * a.scale2, z[1][3] * a.scale2);
          }
        }
        float alpha[2];
        float base[2];
#pragma unroll
        for (int r = 0; r < (kStack ? 1 : 2); ++r) {
          float mx = fmaxf(fmaxf(z[0][2 * r], z[0][2 * r + 1]), fmaxf(z[1][2 * r], z[1][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx = fmaxf(mx * a.scale2, m[r]);
          const float use = mx == -INFINITY ? 0.f : mx;
          alpha[r] = fast_exp2(m[r] - use);
          m[r] = mx;
          base[r] = kFp16 ? use - 14.f : use;   // fp16: probabilities times 2^14
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
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int r = 0; r < (kStack ? 1 : 2); ++r) {
          const float p0 = fast_exp2(fmaf(z[0][2 * r], a.scale2, -base[r]));
          const float p1 = fast_exp2(fmaf(z[0][2 * r + 1], a.scale2, -base[r]));
          const float p2 = fast_exp2(fmaf(z[1][2 * r], a.scale2, -base[r]));
          const float p3 = fast_exp2(fmaf(z[1][2 * r + 1], a.scale2, -base[r]));
          l[r] = l[r] * alpha[r] + ((p0 + p1) + (p2 + p3));
          split_pair<kFp16>(p0, p1, hi[r], lo[r]);
          split_pair<kFp16>(p2, p3, hi[2 + r], lo[2 + r]);
        }
        if constexpr (kStack) {
          hi[1] = lo[0];
          hi[3] = lo[2];
        }
        {
          const int row = w * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
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
      if (t + 1 < p.tile1) {   // the piece's last stage is held: it is the merge's scratch
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + stage);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }

    // ---- the four warps' partials merge in the last stage's memory ----------
    // [4 warps][16 rows (8 stacked)][kDim] fp32, 64 kDim * 4 bytes at most: a stage.
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
    const bool whole = p.tile0 == 0 && p.tile1 == p.tiles;
    const int slot = piece_slot(s, cta, tile_at(s, p, p.tile0));
    constexpr int kRows = kStack ? 8 : 16;
    float* buf = reinterpret_cast<float*>(smem + stage * C::kStage);
    named_sync(1 + kGroups, 128 * kGroups);   // every warp is done with the stage; ml is written
#pragma unroll
    for (int turn = 0; turn < kGroups; ++turn) {
      if (turn == group) {
#pragma unroll
        for (int r = 0; r < (kStack ? 1 : 2); ++r) {
          const int row = g + 8 * r;
          float mx = fmaxf(fmaxf(ml[row].x, ml[16 + row].x), fmaxf(ml[32 + row].x, ml[48 + row].x));
          if (mx == -INFINITY) mx = 0.f;
          const float f = fast_exp2(m[r] - mx);
          float* to = buf + (w * kRows + row) * kDim;
          // Columns are permuted by row so that the 8 rows of a store meet
          // different banks.
#pragma unroll
          for (int i = 0; i < kDim / 8; ++i)
            *reinterpret_cast<float2*>(to + ((i * 8 + 2 * t4) ^ ((row & 3) << 3))) =
                make_float2(o[i][2 * r] * f, o[i][2 * r + 1] * f);
        }
        named_sync(1 + group, 128);
        const int gt = tid - group * 128;
        const int rows = min(kRows, a.G - head0);
        for (int e = gt; e < rows * (kDim / 4); e += 128) {
          const int row = e / (kDim / 4), c = (e % (kDim / 4)) * 4;
          const float* from = buf + row * kDim + (c ^ ((row & 3) << 3));
          float4 x = *reinterpret_cast<const float4*>(from);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(from + i * kRows * kDim);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
          }
          float mx = fmaxf(fmaxf(ml[row].x, ml[16 + row].x), fmaxf(ml[32 + row].x, ml[48 + row].x));
          const float use = mx == -INFINITY ? 0.f : mx;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += ml[i * 16 + row].y * fast_exp2(ml[i * 16 + row].x - use);
          const long long head = unit * a.G + head0 + row;
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint2 y;
            y.x = pack_pair<kFp16>(x.x * inv, x.y * inv);
            y.y = pack_pair<kFp16>(x.z * inv, x.w * inv);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + head * kDim + c) = y;
            if (c == 0) {
              // fp16 probabilities, and so the sum, carry a factor 2^14.
              const float lse2 = use + log2f(sum) - (kFp16 ? 14.f : 0.f);
              if (a.lse) a.lse[head] = lse2 * 0.6931471805599453f;
              if (a.whole)
                unit_lse2[head0 + row] = lse2;
              else if (a.weights)
                a.lse2[head] = lse2;
            }
          } else {
            *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(slot) * a.G + head0 + row) * kDim + c) = x;
            if (c == 0) a.part_ml[slot * kPagedMaxGroup + head0 + row] = make_float2(mx, sum);
          }
        }
        fence_proxy_async_smem();   // the next tile lands here through the async proxy
      }
      if (kGroups > 1) named_sync(1 + kGroups, 128 * kGroups);
    }
    if (kGroups == 1) named_sync(1 + group, 128);   // ml is read before the next piece writes it
    // (The barrier also orders the z that every warp has stored and the lse.)
    if (a.whole && a.weights)
      add_weights(a, unit, p.b, p.h, p.len, 4 * tid, 4 * 128 * kGroups, unit_lse2);
    if (lane == 0) mbar_arrive(empty + stage);
    if (++stage == C::kStages) {
      stage = 0;
      phase ^= 1;
    }
    more = next_piece(p, s, a);
  }
}

// ---- the join -----------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kChunk = 4 * kJoinThreads;   // slots that a CTA of the weights' part takes at once

// The first `jobs` CTAs (weights only), as many for every unit, add each slot's
// weight, from the z that the pass left and the unit's lse: CTA y of a unit
// takes chunks y, y + jobs / units, ... of it.  The CTAs behind them join `hp`
// heads (a power of two up to 8) of one cut unit each.
template <bool kFp16, int kDim>
__global__ void __launch_bounds__(kJoinThreads, 4) paged_join_kernel(const PagedAttnArgs a, int jobs, int hp) {
  __shared__ float red_m[8], red_l[8];
  __shared__ float4 red_o[8][kDim / 4];
  __shared__ float unit_lse2[kPagedMaxGroup];
  __shared__ float2 red_ml[kJoinThreads / 32][kPagedMaxGroup];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) >= jobs) {
    const int per_cut = (a.G + hp - 1) / hp, job = blockIdx.x - jobs;
    const int4 c = (a.cta_cut ? a.cta_cut : a.unit_cut)[job / per_cut];
    if (c.x < 0) return;
    const int warps = 8 / hp, warp0 = warp / warps * warps;   // a head's warps
    const int h = job % per_cut * hp + warp / warps;
    const int i = c.y, t = tid - warp0 * 32;
    // CTAs i - 1 .. c.z hold a piece; a head past the last one joins none.
    const int pieces = h < a.G ? c.z - i + 2 : 0;
    auto slot_of = [&](int j) { return j == 0 ? c.w : 2 * (i - 1 + j); };
    float mx = -INFINITY;
    for (int j = t; j < pieces; j += warps * 32) mx = fmaxf(mx, a.part_ml[slot_of(j) * kPagedMaxGroup + h].x);
    mx = warp_max(mx);
    if (lane == 0) red_m[warp] = mx;
    __syncthreads();
    for (int j = 0; j < warps; ++j) mx = fmaxf(mx, red_m[warp0 + j]);
    const float use = mx == -INFINITY ? 0.f : mx;
    constexpr int kLanes = kDim / 4;            // threads of a row
    const int par = warps * 32 / kLanes;        // rows at once
    const int col = t % kLanes, part = t / kLanes;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int j0 = part; j0 < pieces; j0 += 4 * par) {   // 4 rows in flight
      float2 v[4];
      float4 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
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
      for (int e = 0; e < 4; ++e) {
        const float f = fast_exp2(v[e].x - use);
        sum += v[e].y * f;
        x.x += y[e].x * f;
        x.y += y[e].y * f;
        x.z += y[e].z * f;
        x.w += y[e].w * f;
      }
    }
    if constexpr (kLanes == 16) {   // two rows per warp
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      x.x += __shfl_xor_sync(0xffffffffu, x.x, 16);
      x.y += __shfl_xor_sync(0xffffffffu, x.y, 16);
      x.z += __shfl_xor_sync(0xffffffffu, x.z, 16);
      x.w += __shfl_xor_sync(0xffffffffu, x.w, 16);
    }
    if (lane < kLanes) red_o[warp][lane] = x;
    if (lane == 0) red_l[warp] = sum;
    __syncthreads();
    if (t < kLanes && h < a.G) {
      sum = 0.f;
      x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j = warp0; j < warp0 + warps; ++j) {
        const float4 y = red_o[j][t];
        sum += red_l[j];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long head = static_cast<long long>(c.x) * a.G + h;
      uint2 y;
      y.x = pack_pair<kFp16>(x.x * inv, x.y * inv);
      y.y = pack_pair<kFp16>(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + head * kDim + t * 4) = y;
      if (t == 0 && a.lse) a.lse[head] = (use + log2f(sum) - (kFp16 ? 14.f : 0.f)) * 0.6931471805599453f;
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
      if (tid < a.G) unit_lse2[tid] = a.lse2[unit * a.G + tid];
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
        sum *= fast_exp2(mx - use);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e].y * fast_exp2(v[e].x - use);
        mx = nm;
      }
      for (int o = wide; o < 32; o <<= 1) {   // rows within the warp
        const float m2 = __shfl_xor_sync(0xffffffffu, mx, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        const float nm = fmaxf(mx, m2), use = nm == -INFINITY ? 0.f : nm;
        sum = sum * fast_exp2(mx - use) + s2 * fast_exp2(m2 - use);
        mx = nm;
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
        for (int j = 0; j < kJoinThreads / 32; ++j) l += red_ml[j][lane].y * fast_exp2(red_ml[j][lane].x - use);
        unit_lse2[lane] = use + log2f(l) - (kFp16 ? 14.f : 0.f);
      }
    }
    __syncthreads();
  }
  add_weights(a, unit, b, kv_head, len, y * kChunk + 4 * tid, step * kChunk, unit_lse2);
}

// ---- host side -------------------------------------------------------------------

// Caches of up to this many slots are attended without cuts, in one launch.  Two
// KV heads of 256 slots (16 heads each, d 128): 9.0 us a call from Python and
// 8.4 us on the GPU without cuts, 9.8 and 8.2 us with them; 512 slots: 12.4 and
// 12.1 against 10.1 and 8.5 us.
constexpr int kWholeCap = 256;

int attn_ctas(const PagedShape& s, int G) {
  const int cost = s.D == 64 ? kUnitCost<64> : kUnitCost<128>;
  const long long positions = static_cast<long long>(s.B) * s.Hkv * ((s.cap + kTile - 1) / kTile + cost);
  const long long most = static_cast<long long>(device_sm_count()) * (G > 16 ? 1 : 2);
  return static_cast<int>(positions < most ? positions : most);
}

struct WsLayout {
  size_t unit_cut, cta_cut, ml, o, lse2, scores, total;
};

WsLayout ws_layout(const PagedShape& s, int G) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t n = attn_ctas(s, G), heads = static_cast<size_t>(s.B) * s.Hkv * G;
  const size_t cap64 = static_cast<size_t>((s.cap + kTile - 1) / kTile) * kTile;
  WsLayout w;
  const size_t units = static_cast<size_t>(s.B) * s.Hkv;
  w.unit_cut = 0;
  w.cta_cut = up(units * sizeof(int4));
  w.ml = w.cta_cut + up(n * sizeof(int4));
  w.o = w.ml + up(2 * n * kPagedMaxGroup * sizeof(float2));
  w.lse2 = w.o + up(2 * n * G * s.D * sizeof(float));
  w.scores = w.lse2 + (s.weights ? up(heads * sizeof(float)) : 0);
  w.total = w.scores + (s.weights ? up(heads * cap64 * sizeof(float)) : 0);
  return w;
}

// CTAs of the weights' part: about 16 per SM, the same number for every unit
// and no more than its chunks.  Their loads are short, and latency is what they
// wait for.
int weight_jobs(const PagedAttnArgs& a) {
  const int units = a.B * a.Hkv, chunks = (a.cap + kChunk - 1) / kChunk;
  const int want = (16 * device_sm_count() + units - 1) / units;
  return units * (want < chunks ? want : chunks);
}

template <typename F, typename... A>
cudaError_t launch_pdl(F kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool kFp16, int kDim, int kGroups, bool kStack>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas, cudaStream_t st) {
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
  e = launch_pdl(kernel, dim3(ctas), C::kThreads, C::kSmem, st, km, vm, a);
  if (e != cudaSuccess || a.whole) return e;
  const int jobs = a.weights ? weight_jobs(a) : 0;
  // One CTA per head of a cut unit while that fills no more than the SMs twice
  // (a long sequence's unit has hundreds of pieces), else up to 8 heads each.
  const int cuts = a.cta_cut ? ctas : a.B * a.Hkv;
  int hp = 1;
  while (hp < 8 && cuts * ((a.G + hp - 1) / hp) > 2 * device_sm_count()) hp *= 2;
  return launch_pdl(paged_join_kernel<kFp16, kDim>, dim3(static_cast<unsigned>(jobs + cuts * ((a.G + hp - 1) / hp))),
                    kJoinThreads, 0, st, a, jobs, hp);
}

template <bool kFp16, int kDim>
cudaError_t launch_g(const CUtensorMap& km, const CUtensorMap& vm, const PagedAttnArgs& a, int ctas, cudaStream_t st) {
  if (a.G > 16) return launch<kFp16, kDim, 2, false>(km, vm, a, ctas, st);
  if (a.G > 8) return launch<kFp16, kDim, 1, false>(km, vm, a, ctas, st);
  return launch<kFp16, kDim, 1, true>(km, vm, a, ctas, st);
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
  a.lse2 = reinterpret_cast<float*>(base + w.lse2);
  a.scores = reinterpret_cast<float*>(base + w.scores);
  a.cap64 = (s.cap + kTile - 1) / kTile * kTile;
  a.status = s.status;
  const int ctas = attn_ctas(s, G);
  const bool by_unit = s.B * s.Hkv <= ctas;
  // Short caches are not cut: see kWholeCap.
  a.whole = s.cap <= kWholeCap;
  a.unit_cut = a.whole ? nullptr : by_unit || accumulate ? reinterpret_cast<int4*>(base + w.unit_cut) : nullptr;
  a.cta_cut = a.whole || by_unit ? nullptr : reinterpret_cast<int4*>(base + w.cta_cut);
  if (s.fp16)
    return s.D == 128 ? launch_g<true, 128>(k_map, v_map, a, ctas, st) : launch_g<true, 64>(k_map, v_map, a, ctas, st);
  return s.D == 128 ? launch_g<false, 128>(k_map, v_map, a, ctas, st) : launch_g<false, 64>(k_map, v_map, a, ctas, st);
}

}  // namespace infllmv2
