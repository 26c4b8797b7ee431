// C-ABI layer of the packed step: rotary positions, packed attention and its
// gradient.  Argument checks, tensor maps and launches.  See include/infllmv2.h.
#include <cmath>

#include "api_common.h"
#include "packed.h"
#include "packed_attn.h"

using namespace infllmv2;

namespace {

constexpr int kMaxRotary = 512;

// Strides between tokens and heads of [tokens, heads, d]: whole 16-byte units,
// and 0 for a dimension of one entry.
int check_rows(const int64_t st[2], int64_t tokens, int64_t heads, int bytes, const char* what, PackedRows* r) {
  const int64_t n[2] = {tokens, heads};
  long long got[2];
  for (int i = 0; i < 2; ++i) {
    got[i] = n[i] > 1 ? st[i] : 0;
    if (got[i] < 0) return fail(INFLLMV2_INVALID_ARGUMENT, "%s: strides must be >= 0", what);
    if (got[i] * bytes % 16 != 0) return fail(INFLLMV2_UNSUPPORTED, "%s: strides must be multiples of 16 bytes", what);
    if (got[i] > (1ll << 56) / n[i]) return fail(INFLLMV2_UNSUPPORTED, "%s: strides span too much", what);
  }
  r->token = got[0];
  r->head = got[1];
  return INFLLMV2_OK;
}

// Rows of an output must not overlap: one dimension steps over the other's extent.
int check_apart(const PackedRows& r, int64_t tokens, int64_t heads, int d, const char* what) {
  const bool ok = (tokens == 1 || heads == 1)
                      ? (tokens == 1 || r.token >= d) && (heads == 1 || r.head >= d)
                      : (r.head >= d && r.token >= r.head * (heads - 1) + d) ||
                            (r.token >= d && r.head >= r.token * (tokens - 1) + d);
  return ok ? INFLLMV2_OK : fail(INFLLMV2_INVALID_ARGUMENT, "%s: rows overlap (strides)", what);
}

int check_rotary_rows(const void* in, void* out, const int64_t in_strides[2], const int64_t out_strides[2],
                      int64_t tokens, int64_t heads, int d, int bytes, const char* what, PackedRows* from,
                      PackedRows* to) {
  if (heads > 4096) return fail(INFLLMV2_UNSUPPORTED, "%s: at most 4096 heads (got %d)", what, (int)heads);
  if (!in || !out) return fail(INFLLMV2_INVALID_ARGUMENT, "%s or its output is NULL", what);
  if (!aligned16(in) || !aligned16(out))
    return fail(INFLLMV2_UNSUPPORTED, "%s: pointers must be 16-byte aligned", what);
  int rc;
  if ((rc = check_rows(in_strides, tokens, heads, bytes, what, from)) ||
      (rc = check_rows(out_strides, tokens, heads, bytes, what, to)) ||
      (rc = check_apart(*to, tokens, heads, d, what)))
    return rc;
  if (in == out && (from->token != to->token || from->head != to->head))
    return fail(INFLLMV2_INVALID_ARGUMENT, "%s: in place takes the same strides for input and output", what);
  from->x = const_cast<void*>(in);
  to->x = out;
  return INFLLMV2_OK;
}

// Tokens, heads and type of an attention call; the strides of its inputs.
struct AttnCall {
  PackedAttnShape s;
  int D;
  bool fp16;
  PackedRows q, k, v;
};

int check_tensor(const int64_t st[2], int64_t tokens, int64_t heads, int d, const char* what, PackedRows* r) {
  int rc = check_rows(st, tokens, heads, 2, what, r);
  if (rc || (rc = check_apart(*r, tokens, heads, d, what))) return rc;
  if (r->token >= (1ll << 39) || r->head >= (1ll << 34))
    return fail(INFLLMV2_UNSUPPORTED, "%s: a stride is too large", what);
  return INFLLMV2_OK;
}

int check_attn(const infllmv2_packed_attn_args* a, AttnCall* c) {
  if (!a) return fail(INFLLMV2_INVALID_ARGUMENT, "args is NULL");
  if (a->dtype != INFLLMV2_BF16 && a->dtype != INFLLMV2_FP16)
    return fail(INFLLMV2_UNSUPPORTED, "dtype must be INFLLMV2_BF16 or INFLLMV2_FP16 (got %d)", a->dtype);
  if (a->head_dim != 64 && a->head_dim != 128)
    return fail(INFLLMV2_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", a->head_dim);
  if (a->batch < 1 || a->n_kv_heads < 1 || a->group_size < 1 || a->q_tokens < 1 || a->k_tokens < 1)
    return fail(INFLLMV2_INVALID_ARGUMENT, "batch, n_kv_heads, group_size, q_tokens and k_tokens must be >= 1");
  if (a->batch > kPackedMaxBatch)
    return fail(INFLLMV2_UNSUPPORTED, "at most %d sequences (got %d)", kPackedMaxBatch, a->batch);
  if (a->group_size > kPackedMaxGroup)
    return fail(INFLLMV2_UNSUPPORTED, "at most %d query heads per KV head (got %d)", kPackedMaxGroup, a->group_size);
  if (a->n_kv_heads > 1024) return fail(INFLLMV2_UNSUPPORTED, "at most 1024 KV heads (got %d)", a->n_kv_heads);
  const int64_t heads = static_cast<int64_t>(a->n_kv_heads) * a->group_size;
  if (heads * a->q_tokens >= 0x7fffffffLL || heads * a->k_tokens >= 0x7fffffffLL)
    return fail(INFLLMV2_UNSUPPORTED, "heads * tokens must be < 2^31");
  if (!a->q || !a->k || !a->v || !a->q_starts) return fail(INFLLMV2_INVALID_ARGUMENT, "q, k, v or q_starts is NULL");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v))
    return fail(INFLLMV2_UNSUPPORTED, "q, k and v must be 16-byte aligned");
  const float scale2 = a->scale * 1.4426950408889634f;
  if (!(std::isfinite(scale2) && scale2 > 0.f && a->scale > 0.f))
    return fail(INFLLMV2_INVALID_ARGUMENT, "scale must be > 0 and finite, also times log2(e)");
  int rc;
  if ((rc = check_tensor(a->q_strides, a->q_tokens, heads, a->head_dim, "q", &c->q)) ||
      (rc = check_tensor(a->k_strides, a->k_tokens, a->n_kv_heads, a->head_dim, "k", &c->k)) ||
      (rc = check_tensor(a->v_strides, a->k_tokens, a->n_kv_heads, a->head_dim, "v", &c->v)))
    return rc;
  c->D = a->head_dim;
  c->fp16 = a->dtype == INFLLMV2_FP16;
  c->s = PackedAttnShape{a->batch, a->n_kv_heads, a->group_size, a->q_tokens, a->k_tokens, a->scale, scale2,
                         a->q_starts, a->k_starts ? a->k_starts : a->q_starts, status_ptr()};
  if (!a->k_starts && a->q_tokens != a->k_tokens)
    return fail(INFLLMV2_INVALID_ARGUMENT, "without k_starts, q and k must hold the same tokens (%d and %d)",
                a->q_tokens, a->k_tokens);
  return INFLLMV2_OK;
}

int check_status(const AttnCall& c) {
  return c.s.status ? INFLLMV2_OK : fail(INFLLMV2_CUDA_ERROR, "no device status word (no current CUDA device?)");
}

int encode(CUtensorMap* map, const AttnCall& c, const void* base, int rank, const cuuint64_t* dims,
           const long long* stride, const cuuint32_t* box, const char* what) {
  auto enc = encode_fn();
  if (!enc) return fail(INFLLMV2_CUDA_ERROR, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t bytes[3];
  cuuint32_t es[4] = {1u, 1u, 1u, 1u};
  // A dimension of one entry is never stepped over.
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = 2 * static_cast<cuuint64_t>(dims[i + 1] > 1 ? stride[i] : c.D);
  const CUresult r = enc(map, c.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                         const_cast<void*>(base), dims, bytes, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B,
                         c.D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(INFLLMV2_CUDA_ERROR, "tensor map for %s failed (CUresult %d)", what, (int)r);
  return INFLLMV2_OK;
}

// [d, group, KV head, token], boxes of one tile's rows.
int row_map(CUtensorMap* map, const AttnCall& c, const void* base, const PackedRows& r, const char* what) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.s.G),
                              static_cast<cuuint64_t>(c.s.Hkv), static_cast<cuuint64_t>(c.s.Tq)};
  const long long stride[3] = {r.head, r.head * c.s.G, r.token};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(c.s.G), 1u,
                             static_cast<cuuint32_t>(packed_tile_tokens(c.s.G))};
  return encode(map, c, base, 4, dims, stride, box, what);
}

// [d, token, KV head], boxes of 128 tokens.
int key_map(CUtensorMap* map, const AttnCall& c, const void* base, const PackedRows& r, const char* what) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.s.Tk),
                              static_cast<cuuint64_t>(c.s.Hkv)};
  const long long stride[2] = {r.token, r.head};
  const cuuint32_t box[3] = {64u, 128u, 1u};
  return encode(map, c, base, 3, dims, stride, box, what);
}

int attn_maps(PackedAttnMaps* m, const infllmv2_packed_attn_args* a, const AttnCall& c) {
  int rc;
  if ((rc = row_map(&m->q, c, a->q, c.q, "q")) || (rc = key_map(&m->k, c, a->k, c.k, "k"))) return rc;
  return key_map(&m->v, c, a->v, c.v, "v");
}

}  // namespace

extern "C" {

int infllmv2_rotary_frequencies(const infllmv2_rotary_config* c, uint64_t* turns, float* scale) {
  INFLLMV2_GUARD({
    if (!c || !turns || !scale) return fail(INFLLMV2_INVALID_ARGUMENT, "config, turns or scale is NULL");
    const int d = c->rotary_dim;
    const int half = d / 2;
    if (d < 2 || d % 2 != 0) return fail(INFLLMV2_INVALID_ARGUMENT, "rotary_dim must be even and >= 2 (got %d)", d);
    if (d > kMaxRotary) return fail(INFLLMV2_UNSUPPORTED, "rotary_dim must be <= %d (got %d)", kMaxRotary, d);
    if (c->scaling < INFLLMV2_ROTARY_PLAIN || c->scaling > INFLLMV2_ROTARY_FACTORS)
      return fail(INFLLMV2_UNSUPPORTED, "scaling must be one of INFLLMV2_ROTARY_* (got %d)", c->scaling);
    if (!(std::isfinite(c->base) && c->base > 1.0)) return fail(INFLLMV2_INVALID_ARGUMENT, "base must be > 1");
    const bool scaled = c->scaling != INFLLMV2_ROTARY_PLAIN;
    if (scaled && !(std::isfinite(c->factor) && c->factor >= 1.0))
      return fail(INFLLMV2_INVALID_ARGUMENT, "factor must be >= 1");
    const bool long_context = c->scaling == INFLLMV2_ROTARY_PARTS || c->scaling == INFLLMV2_ROTARY_FACTORS;
    if (long_context && c->original_len <= 1)
      return fail(INFLLMV2_INVALID_ARGUMENT, "original_len must be > 1 (got %d)", c->original_len);
    const double kTurn = 6.283185307179586476925;   // radians of a whole turn
    double base = c->base;
    if (c->scaling == INFLLMV2_ROTARY_BASE) {
      if (d == 2) return fail(INFLLMV2_INVALID_ARGUMENT, "INFLLMV2_ROTARY_BASE needs rotary_dim > 2");
      base *= std::pow(c->factor, static_cast<double>(d) / (d - 2));
    }
    double low = 0;
    double high = 0;
    double size = 1.0;
    if (c->scaling == INFLLMV2_ROTARY_PARTS) {
      if (!(c->slow_turns > 0 && c->fast_turns > c->slow_turns && std::isfinite(c->fast_turns)))
        return fail(INFLLMV2_INVALID_ARGUMENT, "fast_turns > slow_turns > 0 must hold");
      // The pair that turns n times in original_len positions: base^(-2 i / d) original_len = 2 pi n.
      const double per = half / std::log(base);
      low = std::fmax(std::floor(per * std::log(c->original_len / (kTurn * c->fast_turns))), 0.0);
      high = std::fmin(std::ceil(per * std::log(c->original_len / (kTurn * c->slow_turns))), d - 1.0);
      size = 0.1 * std::log(c->factor) + 1.0;
    } else if (c->scaling == INFLLMV2_ROTARY_FACTORS) {
      if (!c->factors) return fail(INFLLMV2_INVALID_ARGUMENT, "factors is NULL");
      for (int i = 0; i < half; ++i)
        if (!(std::isfinite(c->factors[i]) && c->factors[i] >= 1.0))
          return fail(INFLLMV2_INVALID_ARGUMENT, "factors must be >= 1");
      size = std::sqrt(1.0 + std::log(c->factor) / std::log(static_cast<double>(c->original_len)));
    }
    for (int i = 0; i < half; ++i) {
      double f = std::pow(base, -2.0 * i / d);
      if (c->scaling == INFLLMV2_ROTARY_LINEAR) f /= c->factor;
      if (c->scaling == INFLLMV2_ROTARY_FACTORS) f /= c->factors[i];
      if (c->scaling == INFLLMV2_ROTARY_PARTS) {
        const double slowed = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
        f = f / c->factor * slowed + f * (1.0 - slowed);
      }
      // f <= 1 radian, so the turn is below 2^-2 and 2^64 times it fits.
      turns[i] = static_cast<uint64_t>(std::ldexp(f / kTurn, 64));
    }
    *scale = static_cast<float>(size);
    return INFLLMV2_OK;
  });
}

int infllmv2_rotary(const infllmv2_rotary_args* r, void* stream) {
  INFLLMV2_GUARD({
    if (!r) return fail(INFLLMV2_INVALID_ARGUMENT, "args is NULL");
    if (r->dtype != INFLLMV2_BF16 && r->dtype != INFLLMV2_FP16 && r->dtype != INFLLMV2_FP32)
      return fail(INFLLMV2_UNSUPPORTED, "dtype must be bf16, fp16 or fp32 (got %d)", r->dtype);
    if (r->tokens < 1) return fail(INFLLMV2_INVALID_ARGUMENT, "tokens must be >= 1 (got %d)", r->tokens);
    if (r->tokens > kPackedMaxTokens)
      return fail(INFLLMV2_UNSUPPORTED, "tokens must be <= 2^30 (got %d)", r->tokens);
    if (r->q_heads < 1 || r->k_heads < 0)
      return fail(INFLLMV2_INVALID_ARGUMENT, "q_heads must be >= 1 and k_heads >= 0");
    const int d = r->head_dim;
    if (d < 16 || d % 16 != 0 || d > kMaxRotary)
      return fail(INFLLMV2_UNSUPPORTED, "head_dim must be a multiple of 16 up to %d (got %d)", kMaxRotary, d);
    if (r->rotary_dim < 16 || r->rotary_dim % 16 != 0 || r->rotary_dim > d)
      return fail(INFLLMV2_UNSUPPORTED, "rotary_dim must be a multiple of 16 up to head_dim (got %d)", r->rotary_dim);
    if (!r->positions || !r->turns) return fail(INFLLMV2_INVALID_ARGUMENT, "positions or turns is NULL");
    if (!(std::isfinite(r->scale) && r->scale > 0.f))
      return fail(INFLLMV2_INVALID_ARGUMENT, "scale must be > 0 and finite");
    if ((r->interleaved != 0 && r->interleaved != 1) || (r->transpose != 0 && r->transpose != 1))
      return fail(INFLLMV2_INVALID_ARGUMENT, "interleaved and transpose must be 0 or 1");
    RotaryArgs a = {};
    const int bytes = r->dtype == INFLLMV2_FP32 ? 4 : 2;
    int rc = check_rotary_rows(r->q, r->q_out, r->q_strides, r->q_out_strides, r->tokens, r->q_heads, d, bytes, "q",
                               &a.q_in, &a.q_out);
    if (rc) return rc;
    if (r->k_heads > 0 && (rc = check_rotary_rows(r->k, r->k_out, r->k_strides, r->k_out_strides, r->tokens,
                                                  r->k_heads, d, bytes, "k", &a.k_in, &a.k_out)))
      return rc;
    if (r->k_heads > 0 && (r->k_out == r->q_out || r->k_out == r->q || r->q_out == r->k))
      return fail(INFLLMV2_INVALID_ARGUMENT, "q and k must be apart from each other's output");
    a.positions = r->positions;
    a.turns = r->turns;
    a.scale = r->scale;
    a.tokens = r->tokens;
    a.q_heads = r->q_heads;
    a.k_heads = r->k_heads;
    a.dim = d;
    a.part = r->rotary_dim;
    a.interleaved = r->interleaved != 0;
    a.transpose = r->transpose != 0;
    a.in_place = r->q == r->q_out && (r->k_heads == 0 || r->k == r->k_out);
    const RotaryType type = r->dtype == INFLLMV2_BF16   ? RotaryType::kBf16
                            : r->dtype == INFLLMV2_FP16 ? RotaryType::kFp16
                                                        : RotaryType::kFp32;
    const cudaError_t e = launch_rotary(a, type, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "rotary");
    return INFLLMV2_OK;
  });
}

int infllmv2_packed_attn(const infllmv2_packed_attn_args* args, void* out, const int64_t* out_strides, float* lse,
                         void* stream) {
  INFLLMV2_GUARD({
    AttnCall c = {};
    int rc = check_attn(args, &c);
    if (rc) return rc;
    if (!out || !out_strides) return fail(INFLLMV2_INVALID_ARGUMENT, "out or out_strides is NULL");
    if (!aligned16(out)) return fail(INFLLMV2_UNSUPPORTED, "out must be 16-byte aligned");
    if (out == args->q || out == args->k || out == args->v)
      return fail(INFLLMV2_INVALID_ARGUMENT, "out must be apart from q, k and v");
    PackedRows o = {};
    if ((rc = check_tensor(out_strides, c.s.Tq, static_cast<int64_t>(c.s.Hkv) * c.s.G, c.D, "out", &o))) return rc;
    if ((rc = check_status(c))) return rc;
    PackedAttnMaps maps = {};
    if ((rc = attn_maps(&maps, args, c))) return rc;
    const bool by_tile = packed_attn_by_tile(c.s);
    if (by_tile && (rc = row_map(&maps.out, c, out, o, "out"))) return rc;
    const PackedAttnOut to{out, {o.token, o.head}, lse, by_tile};
    const PackedAttnIn in{args->q, args->k, args->v, {c.q.token, c.q.head}, {c.k.token, c.k.head},
                          {c.v.token, c.v.head}};
    const cudaError_t e = launch_packed_attn(c.s, c.D, c.fp16, maps, in, to, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "packed_attn");
    return INFLLMV2_OK;
  });
}

size_t infllmv2_packed_workspace_size(const infllmv2_packed_attn_args* args) {
  try {
    AttnCall c = {};
    if (check_attn(args, &c)) return 0;
    return sizeof(float2) * c.s.Tq * c.s.Hkv * c.s.G;
  } catch (...) {
  }
  return 0;
}

int infllmv2_packed_attn_backward(const infllmv2_packed_attn_args* args, const void* out, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, const int64_t* grad_strides,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  INFLLMV2_GUARD({
    AttnCall c = {};
    int rc = check_attn(args, &c);
    if (rc) return rc;
    if (!out || !lse || !dout || !dq || !dk || !dv || !grad_strides)
      return fail(INFLLMV2_INVALID_ARGUMENT, "out, lse, dout, a gradient or grad_strides is NULL");
    if (!aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
      return fail(INFLLMV2_UNSUPPORTED, "out, dout and the gradients must be 16-byte aligned");
    const void* read[6] = {args->q, args->k, args->v, out, lse, dout};
    const void* written[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
      bool apart = written[i] != written[(i + 1) % 3];
      for (const void* x : read) apart = apart && x != written[i];
      if (!apart) return fail(INFLLMV2_INVALID_ARGUMENT, "the gradients must be apart from each other and the inputs");
    }
    const int64_t heads = static_cast<int64_t>(c.s.Hkv) * c.s.G;
    const size_t need = sizeof(float2) * c.s.Tq * heads;
    if (!workspace || workspace_bytes < need)
      return fail(INFLLMV2_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes (got %zu)", need, workspace_bytes);
    if (!aligned16(workspace)) return fail(INFLLMV2_UNSUPPORTED, "workspace must be 16-byte aligned");
    PackedRows r[5] = {};
    const char* names[5] = {"out", "dout", "dq", "dk", "dv"};
    for (int i = 0; i < 5; ++i)
      if ((rc = check_tensor(grad_strides + 2 * i, i < 3 ? c.s.Tq : c.s.Tk, i < 3 ? heads : c.s.Hkv, c.D, names[i],
                             &r[i])))
        return rc;
    if ((rc = check_status(c))) return rc;
    PackedAttnMaps maps = {};
    if ((rc = attn_maps(&maps, args, c)) || (rc = row_map(&maps.out, c, out, r[0], "out")) ||
        (rc = row_map(&maps.dout, c, dout, r[1], "dout")))
      return rc;
    PackedAttnGrads g = {};
    g.lse = lse;
    g.dq = dq;
    g.dk = dk;
    g.dv = dv;
    g.dq_st = {r[2].token, r[2].head};
    g.dk_st = {r[3].token, r[3].head};
    g.dv_st = {r[4].token, r[4].head};
    g.rows = static_cast<float2*>(workspace);
    const cudaError_t e = launch_packed_attn_bwd(c.s, c.D, c.fp16, maps, g, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "packed_attn_backward");
    return INFLLMV2_OK;
  });
}

}  // extern "C"
