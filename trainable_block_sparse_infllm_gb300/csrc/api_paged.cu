// C-ABI layer of the paged cache: argument checks, tensor maps of the page
// pools, workspace accounting and launches.  See include/infllmv2.h.
#include <cmath>

#include "api_common.h"
#include "packed.h"
#include "paged.h"

using namespace infllmv2;

namespace {

constexpr int kMaxCap = 1 << 30;

// Strides of a pool dimension (elements): positive where the dimension has
// more than one entry, and whole 16-byte units.
int check_strides(const int64_t st[3], const int64_t n[3], const char* what) {
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] <= 0) return fail(INFLLMV2_INVALID_ARGUMENT, "%s: strides must be > 0", what);
    if (st[i] % 8 != 0) return fail(INFLLMV2_UNSUPPORTED, "%s: strides must be multiples of 8 elements", what);
    if (st[i] >= (1ll << 39)) return fail(INFLLMV2_UNSUPPORTED, "%s: a stride is too large", what);
  }
  return INFLLMV2_OK;
}

// No two of the pool's rows overlap: sorted by stride, each dimension steps
// over the extent of the ones below it.  Extents past 2^56 elements, which no
// address space holds, are refused before they could wrap around.
int check_layout(const int64_t st[3], const int64_t n[3], int d, const char* what) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[order[j]] < st[order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  int64_t extent = d;
  for (int i = 0; i < 3; ++i) {
    const int x = order[i];
    if (n[x] <= 1) continue;
    if (st[x] < extent) return fail(INFLLMV2_INVALID_ARGUMENT, "%s: rows overlap (strides)", what);
    if (st[x] > ((1ll << 56) - extent) / (n[x] - 1))
      return fail(INFLLMV2_UNSUPPORTED, "%s: strides span too much", what);
    extent = st[x] * (n[x] - 1) + extent;
  }
  return INFLLMV2_OK;
}

int check_cache(const infllmv2_paged_cache* c, int32_t batch, int32_t max_pages, PagedShape* s) {
  if (!c) return fail(INFLLMV2_INVALID_ARGUMENT, "cache is NULL");
  if (c->dtype != INFLLMV2_BF16 && c->dtype != INFLLMV2_FP16)
    return fail(INFLLMV2_UNSUPPORTED, "dtype must be INFLLMV2_BF16 or INFLLMV2_FP16 (got %d)", c->dtype);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(INFLLMV2_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", c->head_dim);
  if (c->n_kv_heads < 1 || c->num_pages < 1 || c->page_size < 1)
    return fail(INFLLMV2_INVALID_ARGUMENT, "n_kv_heads, num_pages and page_size must be >= 1");
  if (c->page_size % 16 != 0 || c->page_size > 65536)
    return fail(INFLLMV2_UNSUPPORTED, "page_size must be a multiple of 16 up to 65536 (got %d)", c->page_size);
  if (c->n_kv_heads > 1024) return fail(INFLLMV2_UNSUPPORTED, "at most 1024 KV heads (got %d)", c->n_kv_heads);
  if (batch < 1 || max_pages < 1) return fail(INFLLMV2_INVALID_ARGUMENT, "batch and max_pages must be >= 1");
  if (batch > kPagedMaxBatch) return fail(INFLLMV2_UNSUPPORTED, "at most %d sequences (got %d)", kPagedMaxBatch, batch);
  if (static_cast<int64_t>(batch) * c->n_kv_heads > 65535)
    return fail(INFLLMV2_UNSUPPORTED, "batch * n_kv_heads must be <= 65535");
  if (static_cast<int64_t>(max_pages) * c->page_size > kMaxCap)
    return fail(INFLLMV2_UNSUPPORTED, "max_pages * page_size must be <= 2^30");
  if (static_cast<int64_t>(c->num_pages) * c->page_size > 0x7fffffffLL)
    return fail(INFLLMV2_UNSUPPORTED, "num_pages * page_size must be < 2^31");
  if (!c->k_pages || !c->v_pages) return fail(INFLLMV2_INVALID_ARGUMENT, "k_pages or v_pages is NULL");
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned16(c->weights) || !aligned16(c->positions))
    return fail(INFLLMV2_UNSUPPORTED, "k_pages, v_pages, weights and positions must be 16-byte aligned");
  const int64_t n[3] = {c->num_pages, c->n_kv_heads, c->page_size};
  int rc;
  if ((rc = check_strides(c->k_strides, n, "k_pages")) || (rc = check_strides(c->v_strides, n, "v_pages"))) return rc;
  if ((rc = check_layout(c->k_strides, n, c->head_dim, "k_pages")) ||
      (rc = check_layout(c->v_strides, n, c->head_dim, "v_pages")))
    return rc;
  s->B = batch;
  s->Hkv = c->n_kv_heads;
  s->D = c->head_dim;
  s->ps = c->page_size;
  s->P = c->num_pages;
  s->maxp = max_pages;
  s->cap = max_pages * c->page_size;
  s->fp16 = c->dtype == INFLLMV2_FP16;
  for (int i = 0; i < 3; ++i) {
    s->kst[i] = n[i] > 1 ? c->k_strides[i] : 0;
    s->vst[i] = n[i] > 1 ? c->v_strides[i] : 0;
  }
  s->k = c->k_pages;
  s->v = c->v_pages;
  s->weights = c->weights;
  s->positions = c->positions;
  return INFLLMV2_OK;
}

// 4D view [d, x, y, z] of a pool with x, y, z = tokens, heads and pages by
// ascending stride, in boxes of 64 columns x box_rows tokens of one head and
// page, 128-byte swizzle.  L2 is told to fetch whole rows and no more: with 256
// bytes for rows of 128 a token-major pool is read twice (16 KV heads, d 64: 114
// against 86 us), with 128 for rows of 256 in two boxes 178 against 168 us.
int make_pool_map(CUtensorMap* map, PagedMapOrder* order, const PagedShape& s, const void* base, const long long st[3],
                  int box_rows, const char* what) {
  auto enc = encode_fn();
  if (!enc) return fail(INFLLMV2_CUDA_ERROR, "cuTensorMapEncodeTiled is unavailable");
  const long long n[3] = {s.P, s.Hkv, s.ps};
  long long stride[3];
  // A dimension of one entry is never stepped over: it goes last.
  for (int i = 0; i < 3; ++i) stride[i] = n[i] > 1 ? st[i] : (1ll << 39) - 8;
  int x[3] = {2, 1, 0};   // token, head, page
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[x[j]] < stride[x[i]]) {
        const int t = x[i];
        x[i] = x[j];
        x[j] = t;
      }
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(s.D)};
  cuuint64_t strides[3];
  cuuint32_t box[4] = {64u, 1u, 1u, 1u};
  cuuint32_t es[4] = {1u, 1u, 1u, 1u};
  long long extent = s.D;
  for (int i = 0; i < 3; ++i) {
    if (n[x[i]] == 1) stride[x[i]] = extent;
    dims[i + 1] = static_cast<cuuint64_t>(n[x[i]]);
    strides[i] = static_cast<cuuint64_t>(stride[x[i]]) * 2;
    extent = stride[x[i]] * n[x[i]];
    if (x[i] == 2) {
      order->token = i + 1;
      box[i + 1] = static_cast<cuuint32_t>(box_rows);
    } else if (x[i] == 1) {
      order->head = i + 1;
    } else {
      order->page = i + 1;
    }
  }
  const CUresult r = enc(map, s.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                         const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B,
                         s.D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(INFLLMV2_CUDA_ERROR, "tensor map for %s failed (CUresult %d)", what, (int)r);
  return INFLLMV2_OK;
}

int check_group(int32_t G) {
  if (G < 1) return fail(INFLLMV2_INVALID_ARGUMENT, "group_size must be >= 1");
  if (G > kPagedMaxGroup)
    return fail(INFLLMV2_UNSUPPORTED, "at most %d query heads per KV head (got %d)", kPagedMaxGroup, G);
  return INFLLMV2_OK;
}

int check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (!workspace || bytes < need)
    return fail(INFLLMV2_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes (got %zu)", need, bytes);
  if (!aligned16(workspace)) return fail(INFLLMV2_UNSUPPORTED, "workspace must be 16-byte aligned");
  return INFLLMV2_OK;
}

int check_tables(const int32_t* page_table, const int32_t* kv_lens, PagedShape* s) {
  if (!page_table || !kv_lens) return fail(INFLLMV2_INVALID_ARGUMENT, "page_table or kv_lens is NULL");
  s->table = page_table;
  s->kv_lens = kv_lens;
  s->status = status_ptr();
  if (!s->status) return fail(INFLLMV2_CUDA_ERROR, "no device status word (no current CUDA device?)");
  return INFLLMV2_OK;
}

}  // namespace

extern "C" {

size_t infllmv2_paged_workspace_size(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                                     int32_t group_size, int32_t op) {
  try {
    PagedShape s;
    if (check_cache(cache, batch, max_pages, &s)) return 0;
    if (op == INFLLMV2_OP_PAGED_DECODE) return check_group(group_size) ? 0 : paged_attn_workspace_bytes(s, group_size);
    if (op == INFLLMV2_OP_PAGED_EVICT) return paged_evict_supported(s) ? paged_evict_workspace_bytes(s) : 0;
  } catch (...) {
  }
  return 0;
}

int infllmv2_paged_append_kv(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages, int32_t n_q,
                             const void* k_new, const void* v_new, const int64_t* new_strides,
                             const int32_t* page_table, const int32_t* kv_lens, const int32_t* n_new,
                             const int32_t* seq_lens, void* stream) {
  INFLLMV2_GUARD({
    PagedShape s;
    int rc = check_cache(cache, batch, max_pages, &s);
    if (rc) return rc;
    if (n_q < 1 || n_q > s.cap)
      return fail(INFLLMV2_INVALID_ARGUMENT, "n_q = %d outside [1, max_pages * page_size = %d]", n_q, s.cap);
    if (!k_new || !v_new) return fail(INFLLMV2_INVALID_ARGUMENT, "k_new or v_new is NULL");
    if (!aligned16(k_new) || !aligned16(v_new))
      return fail(INFLLMV2_UNSUPPORTED, "k_new and v_new must be 16-byte aligned");
    PagedRows r;
    r.k = k_new;
    r.v = v_new;
    const int64_t n[3] = {batch, s.Hkv, n_q};
    const long long whole[3] = {static_cast<long long>(s.Hkv) * n_q * s.D, static_cast<long long>(n_q) * s.D, s.D};
    for (int i = 0; i < 3; ++i) {
      r.kst[i] = new_strides ? new_strides[i] : whole[i];
      r.vst[i] = new_strides ? new_strides[3 + i] : whole[i];
      if (n[i] > 1 && (r.kst[i] < 0 || r.vst[i] < 0))
        return fail(INFLLMV2_INVALID_ARGUMENT, "new_strides must be >= 0");
      if (n[i] > 1 && (r.kst[i] % 8 != 0 || r.vst[i] % 8 != 0))
        return fail(INFLLMV2_UNSUPPORTED, "new_strides must be multiples of 8 elements");
      if (n[i] == 1) r.kst[i] = r.vst[i] = 0;
    }
    if ((rc = check_tables(page_table, kv_lens, &s))) return rc;
    const cudaError_t e = launch_paged_append(s, n_q, r, n_new, seq_lens, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_append_kv");
    return INFLLMV2_OK;
  });
}

int infllmv2_paged_attn_decode(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                               int32_t group_size, const void* q, const int32_t* page_table, const int32_t* kv_lens,
                               float attn_scale, int32_t accumulate, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  INFLLMV2_GUARD({
    PagedShape s;
    int rc = check_cache(cache, batch, max_pages, &s);
    if (rc) return rc;
    if ((rc = check_group(group_size))) return rc;
    if (!q || !out) return fail(INFLLMV2_INVALID_ARGUMENT, "q or out is NULL");
    if (!aligned16(q) || !aligned16(out)) return fail(INFLLMV2_UNSUPPORTED, "q and out must be 16-byte aligned");
    const float scale2 = attn_scale * 1.4426950408889634f;
    if (!(std::isfinite(scale2) && scale2 > 0.f))
      return fail(INFLLMV2_INVALID_ARGUMENT, "attn_scale must be > 0 and finite, also times log2(e)");
    if (accumulate != 0 && accumulate != 1) return fail(INFLLMV2_INVALID_ARGUMENT, "accumulate must be 0 or 1");
    if (accumulate && !s.weights) return fail(INFLLMV2_INVALID_ARGUMENT, "accumulate needs the cache's weights");
    if ((rc = check_workspace(paged_attn_workspace_bytes(s, group_size), workspace, workspace_bytes))) return rc;
    if ((rc = check_tables(page_table, kv_lens, &s))) return rc;
    // Rows of a page that one copy fetches: a tile of 64, or what divides both.
    const int box = s.ps % 64 == 0 ? 64 : (s.ps % 32 == 0 ? 32 : 16);
    CUtensorMap km, vm;
    PagedMapOrder ko, vo;
    if ((rc = make_pool_map(&km, &ko, s, s.k, s.kst, box, "k_pages"))) return rc;
    if ((rc = make_pool_map(&vm, &vo, s, s.v, s.vst, box, "v_pages"))) return rc;
    const cudaError_t e = launch_paged_attn(s, group_size, km, ko, vm, vo, box, q, scale2, accumulate != 0, out, lse,
                                            workspace, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_attn_decode");
    return INFLLMV2_OK;
  });
}

int infllmv2_paged_evict(const infllmv2_paged_cache* cache, int32_t batch, int32_t max_pages,
                         const int32_t* page_table, const int32_t* kv_lens, int32_t budget, int32_t n_init,
                         int32_t n_local, const int32_t* seq_lens, int32_t* new_lens, void* workspace,
                         size_t workspace_bytes, void* stream) {
  INFLLMV2_GUARD({
    PagedShape s;
    int rc = check_cache(cache, batch, max_pages, &s);
    if (rc) return rc;
    if (!s.weights || !s.positions)
      return fail(INFLLMV2_INVALID_ARGUMENT, "eviction needs the cache's weights and positions");
    if (budget < 1 || n_init < 0 || n_local < 0)
      return fail(INFLLMV2_INVALID_ARGUMENT, "budget must be >= 1, n_init and n_local >= 0");
    if (static_cast<int64_t>(n_init) + n_local > budget)
      return fail(INFLLMV2_INVALID_ARGUMENT, "budget %d < n_init %d + n_local %d", budget, n_init, n_local);
    if (!new_lens) return fail(INFLLMV2_INVALID_ARGUMENT, "new_lens is NULL");
    if (new_lens == seq_lens) return fail(INFLLMV2_INVALID_ARGUMENT, "new_lens must not be seq_lens");
    if (!paged_evict_supported(s))
      return fail(INFLLMV2_UNSUPPORTED, "eviction takes max_pages * page_size <= 524288 (got %d)", s.cap);
    if ((rc = check_workspace(paged_evict_workspace_bytes(s), workspace, workspace_bytes))) return rc;
    if ((rc = check_tables(page_table, kv_lens, &s))) return rc;
    const cudaError_t e = launch_paged_evict(s, budget, n_init, n_local, seq_lens, new_lens, workspace,
                                             static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_evict");
    return INFLLMV2_OK;
  });
}

int infllmv2_paged_append_packed(const infllmv2_paged_cache* cache, int32_t tokens, const void* k_new,
                                 const void* v_new, const int64_t* strides, const int32_t* slots,
                                 const int32_t* positions, void* stream) {
  INFLLMV2_GUARD({
    PagedShape s = {};
    int rc = check_cache(cache, 1, 1, &s);
    if (rc) return rc;
    if (tokens < 1) return fail(INFLLMV2_INVALID_ARGUMENT, "tokens must be >= 1 (got %d)", tokens);
    if (tokens > kPackedMaxTokens) return fail(INFLLMV2_UNSUPPORTED, "tokens must be <= 2^30 (got %d)", tokens);
    if (!k_new || !v_new || !slots) return fail(INFLLMV2_INVALID_ARGUMENT, "k_new, v_new or slots is NULL");
    if (!aligned16(k_new) || !aligned16(v_new))
      return fail(INFLLMV2_UNSUPPORTED, "k_new and v_new must be 16-byte aligned");
    if (s.positions && !positions)
      return fail(INFLLMV2_INVALID_ARGUMENT, "a cache with positions needs those of the new tokens");
    const int64_t n[2] = {tokens, s.Hkv};
    const long long whole[2] = {static_cast<long long>(s.Hkv) * s.D, s.D};
    long long st[4];
    for (int i = 0; i < 4; ++i) {
      st[i] = n[i & 1] > 1 ? (strides ? strides[i] : whole[i & 1]) : 0;
      if (st[i] < 0) return fail(INFLLMV2_INVALID_ARGUMENT, "strides must be >= 0");
      if (st[i] % 8 != 0) return fail(INFLLMV2_UNSUPPORTED, "strides must be multiples of 8 elements");
      if (st[i] > (1ll << 56) / n[i & 1]) return fail(INFLLMV2_UNSUPPORTED, "strides span too much");
    }
    s.status = status_ptr();
    if (!s.status) return fail(INFLLMV2_CUDA_ERROR, "no device status word (no current CUDA device?)");
    const PackedAppend a{k_new, v_new, st[0], st[1], st[2], st[3], tokens, slots, positions};
    const cudaError_t e = launch_paged_append_packed(s, a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_append_packed");
    return INFLLMV2_OK;
  });
}

int infllmv2_paged_reserve(const infllmv2_reserve_args* r, void* stream) {
  INFLLMV2_GUARD({
    if (!r) return fail(INFLLMV2_INVALID_ARGUMENT, "args is NULL");
    if (r->page_size < 1 || r->num_pages < 1 || r->batch < 1 || r->max_pages < 1)
      return fail(INFLLMV2_INVALID_ARGUMENT, "page_size, num_pages, batch and max_pages must be >= 1");
    if (r->batch > kPagedMaxBatch)
      return fail(INFLLMV2_UNSUPPORTED, "at most %d sequences (got %d)", kPagedMaxBatch, r->batch);
    if (r->page_size > 65536) return fail(INFLLMV2_UNSUPPORTED, "page_size must be <= 65536 (got %d)", r->page_size);
    if (static_cast<int64_t>(r->max_pages) * r->page_size > kMaxCap)
      return fail(INFLLMV2_UNSUPPORTED, "max_pages * page_size must be <= 2^30");
    if (static_cast<int64_t>(r->num_pages) * r->page_size > 0x7fffffffLL)
      return fail(INFLLMV2_UNSUPPORTED, "num_pages * page_size must be < 2^31");
    if (r->max_tokens < 0) return fail(INFLLMV2_INVALID_ARGUMENT, "max_tokens must be >= 0 (got %d)", r->max_tokens);
    if (r->max_tokens > kMaxCap)
      return fail(INFLLMV2_UNSUPPORTED, "max_tokens must be <= 2^30 (got %d)", r->max_tokens);
    if (!r->page_table || !r->held || !r->free_pages || !r->n_free || !r->kv_lens || !r->n_new || !r->new_lens ||
        !r->starts || !r->missing)
      return fail(INFLLMV2_INVALID_ARGUMENT, "a required array is NULL");
    if (r->new_lens == r->seq_lens || r->new_lens == r->held || r->starts == r->kv_lens || r->starts == r->n_new ||
        r->starts == r->seq_lens || r->starts == r->new_lens || r->starts == r->held)
      return fail(INFLLMV2_INVALID_ARGUMENT, "new_lens and starts must be apart from seq_lens, held and the lengths");
    uint32_t* status = status_ptr();
    if (!status) return fail(INFLLMV2_CUDA_ERROR, "no device status word (no current CUDA device?)");
    const ReserveArgs a{r->batch, r->max_pages, r->page_size, r->num_pages, r->max_tokens, r->page_table, r->held,
                        r->free_pages, r->n_free, r->kv_lens, r->n_new, r->seq_lens, r->new_lens, r->starts,
                        r->slots, r->positions, r->missing, status};
    const cudaError_t e = launch_paged_reserve(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_reserve");
    return INFLLMV2_OK;
  });
}

}  // extern "C"
