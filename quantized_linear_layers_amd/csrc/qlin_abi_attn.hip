// C ABI of the attention operators: argument validation, device check, dispatch, as
// qlin_abi.hip for the linears (whose hardware counters are kept with a hash of that
// file: it does not change with these).
#include <mutex>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "qlin_internal.h"

namespace qlin {

namespace {

// Once-per-device check that the current device is gfx950.
int device_ok() {
  static std::mutex mu;
  static signed char state[64] = {0};  // 0 unknown, 1 ok, -1 unsupported
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(mu);
  if (state[dev] == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_fail(e);
    state[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
  }
  return state[dev] == 1 ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

bool a16(const void* p) { return aligned16(p); }

// An array of n int32; no two of some share memory (NULL is none).
struct Ints {
  const int32_t* p;
  int64_t n;
};
template <int N>
bool apart(const Ints (&x)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j) {
      const uintptr_t a = (uintptr_t)x[i].p, b = (uintptr_t)x[j].p;
      if (a && b && a < b + 4 * (uintptr_t)x[j].n && b < a + 4 * (uintptr_t)x[i].n) return false;
    }
  return true;
}

}  // namespace

}  // namespace qlin

using namespace qlin;

#define QLIN_CHECK(cond, code) \
  do {                         \
    if (!(cond)) return (code); \
  } while (0)

extern "C" {

int qlin_rope_turns(int64_t rot, double base, int rule, double factor, double trained_len, double low,
                    double high, double* out) {
  QLIN_CHECK(out && rule >= QLIN_ROPE_PLAIN && rule <= QLIN_ROPE_RAMP, QLIN_ERR_ARG);
  QLIN_CHECK(rot >= 16 && rot % 16 == 0 && rot <= 1024, QLIN_ERR_SHAPE);
  QLIN_CHECK(std::isfinite(base) && base > 1.0, QLIN_ERR_ARG);
  QLIN_CHECK(rule == QLIN_ROPE_PLAIN || (std::isfinite(factor) && factor > 0.0), QLIN_ERR_ARG);
  QLIN_CHECK(rule != QLIN_ROPE_RAMP || (std::isfinite(trained_len) && trained_len > 0.0 && low >= 0.0 &&
                                        std::isfinite(high) && high > low),
             QLIN_ERR_ARG);
  if (rule == QLIN_ROPE_BASE) base *= std::pow(factor, (double)rot / (double)(rot - 2));
  for (int64_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot) / 6.283185307179586476925286766559;
    if (rule == QLIN_ROPE_LINEAR) f /= factor;
    if (rule == QLIN_ROPE_RAMP) {
      const double keep = std::min(1.0, std::max(0.0, (trained_len * f - low) / (high - low)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    QLIN_CHECK(std::isfinite(f), QLIN_ERR_ARG);
    out[i] = f;
  }
  return QLIN_OK;
}

// A rotation plan for heads of D values.
static int rope_plan_args(const qlin_rope_plan* r, int64_t D) {
  QLIN_CHECK(r->rot >= 16 && r->rot % 16 == 0 && r->rot <= D, QLIN_ERR_SHAPE);
  QLIN_CHECK(r->turns && std::isfinite(r->magnitude), QLIN_ERR_ARG);
  QLIN_CHECK(((uintptr_t)r->turns & 7) == 0, QLIN_ERR_ALIGN);
  return QLIN_OK;
}

int qlin_rope(const qlin_bf16* x, int64_t ldx, int64_t T, int64_t H, int64_t D,
              const int32_t* positions, const qlin_rope_plan* rope, int inverse, qlin_bf16* y,
              int64_t ldy, qlin_stream_t stream) {
  QLIN_CHECK(rope, QLIN_ERR_ARG);
  QLIN_CHECK(T >= 0 && H >= 0 && D >= 16 && D % 16 == 0 && D <= 1024 && T <= 0x7FFFFFFF && H <= 0xFFFF &&
                 ldx >= H * D && ldy >= H * D && (x != y || ldx == ldy) && rope_grid_ok(T, H, D),
             QLIN_ERR_SHAPE);
  int rc = rope_plan_args(rope, D);
  if (rc) return rc;
  if (T == 0 || H == 0) return QLIN_OK;
  QLIN_CHECK(x && y && positions, QLIN_ERR_ARG);
  QLIN_CHECK(a16(x) && a16(y) && ldx % 8 == 0 && ldy % 8 == 0 && ((uintptr_t)positions & 3) == 0,
             QLIN_ERR_ALIGN);
  rc = device_ok();
  if (rc) return rc;
  return launch_rope(x, ldx, T, H, D, nullptr, positions, rope, inverse, y, ldy, as_stream(stream));
}

static int head_norm_args(const qlin_head_norm* n) {
  QLIN_CHECK(n && n->eps >= 0x1p-100f && n->eps <= 0x1p+100f && std::isfinite(n->offset), QLIN_ERR_ARG);
  QLIN_CHECK(a16(n->q_weight) && a16(n->k_weight) && a16(n->v_weight), QLIN_ERR_ALIGN);
  return QLIN_OK;
}

int qlin_norm_rope(const qlin_bf16* x, int64_t ldx, int64_t T, int64_t H, int64_t D, const qlin_head_norm* norm,
                   const int32_t* positions, const qlin_rope_plan* rope, qlin_bf16* y, int64_t ldy,
                   qlin_stream_t stream) {
  int rc = head_norm_args(norm);
  if (rc) return rc;
  QLIN_CHECK(T >= 0 && H >= 0 && D >= 16 && D <= 1024 && (D & (D - 1)) == 0 && T <= 0x7FFFFFFF && H <= 0xFFFF &&
                 ldx >= H * D && ldy >= H * D && (x != y || ldx == ldy) && rope_grid_ok(T, H, D),
             QLIN_ERR_SHAPE);
  if (rope) {
    rc = rope_plan_args(rope, D);
    if (rc) return rc;
  }
  if (T == 0 || H == 0) return QLIN_OK;
  QLIN_CHECK(x && y && (positions || !rope), QLIN_ERR_ARG);
  QLIN_CHECK(a16(x) && a16(y) && ldx % 8 == 0 && ldy % 8 == 0 && ((uintptr_t)positions & 3) == 0,
             QLIN_ERR_ALIGN);
  rc = device_ok();
  if (rc) return rc;
  return launch_rope(x, ldx, T, H, D, norm, positions, rope, 0, y, ldy, as_stream(stream));
}

static bool kv_shape_ok(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t T) {
  return (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) && c->page_size >= 16 &&
         c->page_size <= 256 && (c->page_size & (c->page_size - 1)) == 0 && c->pages >= 1 &&
         c->pages <= 0x7FFFFFFF && c->kv_heads >= 1 && c->kv_heads <= 0xFFFF &&
         c->pages * c->kv_heads <= 0x7FFFFFFF && T >= 0 && T <= 0x7FFFFFFF && b->batch >= 0 &&
         b->batch <= 0xFFFF && b->max_q >= 0 && b->table_cols >= 0 &&
         b->table_cols <= (0x7FFFFFFF - 65536) / c->page_size;
}

// The cache and batch of a call with T rows; the arrays of an empty call (T == 0
// or no sequence) may be NULL.
static int kv_args(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t T) {
  QLIN_CHECK(c && b, QLIN_ERR_ARG);
  QLIN_CHECK(c->fmt == QLIN_KV_BF16 || c->fmt == QLIN_KV_E4M3, QLIN_ERR_ARG);
  QLIN_CHECK(kv_shape_ok(c, b, T), QLIN_ERR_SHAPE);
  if (T == 0 || b->batch == 0) return QLIN_OK;
  QLIN_CHECK(b->table_cols >= 1 && b->max_q >= 1, QLIN_ERR_SHAPE);
  QLIN_CHECK(c->k && c->v && b->q_start && b->kv_len && b->page_table, QLIN_ERR_ARG);
  QLIN_CHECK((c->fmt == QLIN_KV_E4M3) == (c->k_scale != nullptr) &&
                 (c->fmt == QLIN_KV_E4M3) == (c->v_scale != nullptr),
             QLIN_ERR_ARG);
  QLIN_CHECK(a16(c->k) && a16(c->v) && ((uintptr_t)c->k_scale & 3) == 0 && ((uintptr_t)c->v_scale & 3) == 0 &&
                 ((uintptr_t)b->q_start & 3) == 0 && ((uintptr_t)b->kv_len & 3) == 0 &&
                 ((uintptr_t)b->page_table & 3) == 0,
             QLIN_ERR_ALIGN);
  return QLIN_OK;
}

static int kv_append(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, const qlin_bf16* k,
                     int64_t ldk, const qlin_bf16* v, int64_t ldv, const qlin_head_norm* norm,
                     const qlin_rope_plan* rope, const int32_t* positions, const qlin_bf16* q, int64_t ldq,
                     int64_t q_heads, qlin_bf16* q_out, int64_t ldqo, qlin_stream_t stream) {
  int rc = kv_args(cache, batch, T);
  if (rc) return rc;
  const int64_t D = cache->head_dim, kvd = cache->kv_heads * D;
  if (rope) {
    rc = rope_plan_args(rope, D);
    if (rc) return rc;
  }
  QLIN_CHECK((q == nullptr) == (q_out == nullptr), QLIN_ERR_ARG);
  QLIN_CHECK(ldk >= kvd && ldv >= kvd, QLIN_ERR_SHAPE);
  if (q)
    QLIN_CHECK(q_heads >= 1 && q_heads <= 0xFFFF && ldq >= q_heads * D && ldqo >= q_heads * D &&
                   (q != q_out || ldq == ldqo),
               QLIN_ERR_SHAPE);
  QLIN_CHECK(rope_grid_ok(T, (q ? q_heads : 0) + 2 * cache->kv_heads, D), QLIN_ERR_SHAPE);
  if (T == 0 || batch->batch == 0) return QLIN_OK;
  QLIN_CHECK(k && v, QLIN_ERR_ARG);
  QLIN_CHECK(a16(k) && a16(v) && ldk % 8 == 0 && ldv % 8 == 0 && ((uintptr_t)positions & 3) == 0,
             QLIN_ERR_ALIGN);
  if (q) QLIN_CHECK(a16(q) && a16(q_out) && ldq % 8 == 0 && ldqo % 8 == 0, QLIN_ERR_ALIGN);
  rc = device_ok();
  if (rc) return rc;
  return launch_kv_append(*cache, *batch, T, k, ldk, v, ldv, norm, rope, positions, q, ldq, q_heads, q_out, ldqo,
                          as_stream(stream));
}

int qlin_kv_append(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                   const qlin_bf16* k, int64_t ldk, const qlin_bf16* v, int64_t ldv,
                   const qlin_rope_plan* rope, const int32_t* positions, const qlin_bf16* q,
                   int64_t ldq, int64_t q_heads, qlin_bf16* q_out, int64_t ldqo,
                   qlin_stream_t stream) {
  return kv_append(cache, batch, T, k, ldk, v, ldv, nullptr, rope, positions, q, ldq, q_heads, q_out, ldqo, stream);
}

int qlin_kv_append_norm(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                        const qlin_bf16* k, int64_t ldk, const qlin_bf16* v, int64_t ldv,
                        const qlin_head_norm* norm, const qlin_rope_plan* rope, const int32_t* positions,
                        const qlin_bf16* q, int64_t ldq, int64_t q_heads, qlin_bf16* q_out, int64_t ldqo,
                        qlin_stream_t stream) {
  const int rc = head_norm_args(norm);
  if (rc) return rc;
  return kv_append(cache, batch, T, k, ldk, v, ldv, norm, rope, positions, q, ldq, q_heads, q_out, ldqo, stream);
}

static bool attn_shape_ok(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t T, int64_t q_heads) {
  return q_heads >= 1 && q_heads <= 0xFFFF && q_heads % c->kv_heads == 0 && T * q_heads <= 0x3FFFFFFF &&
         b->max_q <= 0x7FFFFFFF && b->batch * c->kv_heads <= 0xFFFFFF && attn_grid_ok(*c, *b, T, q_heads);
}

static bool attn_has_work(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, int64_t q_heads) {
  return cache && batch && kv_shape_ok(cache, batch, T) && T != 0 && batch->batch != 0 && batch->table_cols != 0 &&
         batch->max_q != 0 && attn_shape_ok(cache, batch, T, q_heads);
}

size_t qlin_attn_workspace_bytes(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                                 int64_t q_heads) {
  return attn_has_work(cache, batch, T, q_heads) ? attn_workspace_bytes(*cache, *batch, T, q_heads) : 0;
}

size_t qlin_attn_tree_workspace_bytes(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                                      int64_t q_heads) {
  return attn_has_work(cache, batch, T, q_heads) ? attn_tree_workspace_bytes(*cache, *batch, T, q_heads) : 0;
}

static int attn_paged(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                      const qlin_bf16* q, int64_t ldq, int64_t q_heads, float scale, int causal,
                      int64_t window, const qlin_tree* tree, qlin_bf16* out, int64_t ldo, float* lse, void* ws,
                      size_t ws_bytes, qlin_stream_t stream) {
  int rc = kv_args(cache, batch, T);
  if (rc) return rc;
  QLIN_CHECK(std::isfinite(attn_factor(scale)) && window >= 0 && (window == 0 || causal), QLIN_ERR_ARG);
  QLIN_CHECK(attn_shape_ok(cache, batch, T, q_heads) && ldq >= q_heads * cache->head_dim &&
                 ldo >= q_heads * cache->head_dim,
             QLIN_ERR_SHAPE);
  if (T == 0 || batch->batch == 0) return QLIN_OK;
  QLIN_CHECK(q && out, QLIN_ERR_ARG);
  QLIN_CHECK(a16(q) && a16(out) && ldq % 8 == 0 && ldo % 8 == 0 && ((uintptr_t)lse & 3) == 0, QLIN_ERR_ALIGN);
  const size_t need = tree ? attn_tree_workspace_bytes(*cache, *batch, T, q_heads)
                           : attn_workspace_bytes(*cache, *batch, T, q_heads);
  QLIN_CHECK(ws_bytes >= need && (need == 0 || ws), QLIN_ERR_WORKSPACE);
  QLIN_CHECK(need == 0 || ((uintptr_t)ws & 255) == 0, QLIN_ERR_ALIGN);
  rc = device_ok();
  if (rc) return rc;
  return launch_attn(*cache, *batch, T, q, ldq, q_heads, scale, causal, window, tree, out, ldo, lse, ws,
                     ws_bytes, as_stream(stream));
}

int qlin_attn_paged(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                    const qlin_bf16* q, int64_t ldq, int64_t q_heads, float scale, int causal,
                    int64_t window, qlin_bf16* out, int64_t ldo, float* lse, void* ws,
                    size_t ws_bytes, qlin_stream_t stream) {
  return attn_paged(cache, batch, T, q, ldq, q_heads, scale, causal, window, nullptr, out, ldo, lse, ws, ws_bytes,
                    stream);
}

static bool tree_words_ok(const qlin_kv_batch* b, int64_t words) {
  return words >= 1 && words <= 8 && b->max_q <= 64 * words;
}

int qlin_attn_tree(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                   const qlin_bf16* q, int64_t ldq, int64_t q_heads, float scale, const qlin_tree* tree,
                   int64_t window, qlin_bf16* out, int64_t ldo, float* lse, void* ws,
                   size_t ws_bytes, qlin_stream_t stream) {
  QLIN_CHECK(cache && batch && tree, QLIN_ERR_ARG);
  QLIN_CHECK(tree_words_ok(batch, tree->words), QLIN_ERR_SHAPE);
  QLIN_CHECK(window >= 0 && (window == 0 || window >= batch->max_q), QLIN_ERR_ARG);
  if (T > 0 && batch->batch > 0) {
    QLIN_CHECK(tree->mask && (window == 0 || tree->positions), QLIN_ERR_ARG);
    QLIN_CHECK(((uintptr_t)tree->mask & 7) == 0 && ((uintptr_t)tree->positions & 3) == 0, QLIN_ERR_ALIGN);
  }
  return attn_paged(cache, batch, T, q, ldq, q_heads, scale, 1, window, tree, out, ldo, lse, ws, ws_bytes, stream);
}

int qlin_tree_plan(const qlin_kv_batch* batch, int64_t T, const int32_t* parents, int64_t words, uint64_t* mask,
                   int32_t* positions, qlin_stream_t stream) {
  QLIN_CHECK(batch, QLIN_ERR_ARG);
  QLIN_CHECK(T >= 0 && T <= 0x7FFFFFFF && batch->batch >= 0 && batch->batch <= 0xFFFF && batch->max_q >= 0 &&
                 tree_words_ok(batch, words),
             QLIN_ERR_SHAPE);
  if (T == 0 || batch->batch == 0) return QLIN_OK;
  QLIN_CHECK(batch->max_q >= 1, QLIN_ERR_SHAPE);
  QLIN_CHECK(batch->q_start && batch->kv_len && parents && mask, QLIN_ERR_ARG);
  QLIN_CHECK(((uintptr_t)mask & 7) == 0 && (((uintptr_t)batch->q_start | (uintptr_t)batch->kv_len |
                                             (uintptr_t)parents | (uintptr_t)positions) & 3) == 0,
             QLIN_ERR_ALIGN);
  const Ints bits = {(const int32_t*)mask, 2 * T * words}, at = {positions, T};
  const Ints start = {batch->q_start, batch->batch + 1};
  QLIN_CHECK(apart<3>({bits, at, start}) && apart<3>({bits, at, {batch->kv_len, batch->batch}}) &&
                 apart<3>({bits, positions == parents ? Ints{} : at, {parents, T}}),
             QLIN_ERR_ARG);
  const int rc = device_ok();
  if (rc) return rc;
  return launch_tree_plan(*batch, T, parents, words, mask, positions, as_stream(stream));
}

static int tables_args(const qlin_kv_pool* p, const qlin_kv_tables* t) {
  QLIN_CHECK(p && t, QLIN_ERR_ARG);
  QLIN_CHECK(p->page_size >= 16 && p->page_size <= 256 && (p->page_size & (p->page_size - 1)) == 0 && p->pages >= 1 &&
                 p->pages <= 0x7FFFFFFF / p->page_size && t->batch >= 0 && t->batch <= 0xFFFF && t->table_cols >= 1 &&
                 t->table_cols <= (0x7FFFFFFF - 65536) / p->page_size,
             QLIN_ERR_SHAPE);
  if (t->batch == 0) return QLIN_OK;
  QLIN_CHECK(p->free_pages && p->count && t->page_table && t->kv_len, QLIN_ERR_ARG);
  QLIN_CHECK((((uintptr_t)p->free_pages | (uintptr_t)p->count | (uintptr_t)t->page_table | (uintptr_t)t->kv_len |
               (uintptr_t)t->q_start | (uintptr_t)t->slots | (uintptr_t)t->positions) & 3) == 0,
             QLIN_ERR_ALIGN);
  return QLIN_OK;
}

int qlin_kv_reserve(const qlin_kv_pool* pool, const qlin_kv_tables* tables, int64_t T, const int32_t* lengths,
                    const int32_t* new_tokens, qlin_stream_t stream) {
  int rc = tables_args(pool, tables);
  if (rc) return rc;
  QLIN_CHECK(T >= 0 && T <= 0x7FFFFFFF, QLIN_ERR_SHAPE);
  if (tables->batch == 0) return QLIN_OK;
  QLIN_CHECK(tables->q_start && lengths && new_tokens, QLIN_ERR_ARG);
  QLIN_CHECK((((uintptr_t)lengths | (uintptr_t)new_tokens) & 3) == 0, QLIN_ERR_ALIGN);
  const qlin_kv_tables& t = *tables;
  QLIN_CHECK(apart<9>({{t.page_table, t.batch * t.table_cols}, {t.q_start, t.batch + 1}, {t.kv_len, t.batch},
                       {t.slots, T}, {t.positions, T}, {pool->free_pages, pool->pages}, {pool->count, 2},
                       {lengths == t.kv_len || lengths == new_tokens ? nullptr : lengths, t.batch},
                       {new_tokens, t.batch}}),
             QLIN_ERR_ARG);
  rc = device_ok();
  if (rc) return rc;
  return launch_reserve(*pool, *tables, lengths, new_tokens, T, as_stream(stream));
}

int qlin_kv_release(const qlin_kv_pool* pool, const qlin_kv_tables* tables, const int32_t* lengths,
                    qlin_stream_t stream) {
  int rc = tables_args(pool, tables);
  if (rc) return rc;
  if (tables->batch == 0) return QLIN_OK;
  QLIN_CHECK(lengths, QLIN_ERR_ARG);
  QLIN_CHECK(((uintptr_t)lengths & 3) == 0, QLIN_ERR_ALIGN);
  const qlin_kv_tables& t = *tables;
  const Ints list = {pool->free_pages, pool->pages}, count = {pool->count, 2};
  QLIN_CHECK(apart<3>({list, count, {t.page_table, t.batch * t.table_cols}}) &&
                 apart<3>({list, count, {t.kv_len, t.batch}}) && apart<3>({list, count, {lengths, t.batch}}),
             QLIN_ERR_ARG);
  rc = device_ok();
  if (rc) return rc;
  return launch_release(*pool, *tables, lengths, as_stream(stream));
}

int qlin_kv_keep(const qlin_kv_cache* caches, int64_t n_caches, const qlin_kv_batch* batch, const int32_t* path,
                 int64_t path_cols, const int32_t* kept, int32_t* lengths, qlin_stream_t stream) {
  QLIN_CHECK(caches && batch, QLIN_ERR_ARG);
  QLIN_CHECK(n_caches >= 1 && n_caches <= 65535 && path_cols >= 0 && path_cols <= 0x7FFFFFFF, QLIN_ERR_SHAPE);
  const bool empty = batch->batch == 0;
  for (int64_t i = 0; i < n_caches; ++i) {
    const qlin_kv_cache& c = caches[i];
    // (the batch's max_q is not used; a sequence may have any number of new tokens)
    qlin_kv_batch b = *batch;
    b.max_q = 1;
    const int rc = kv_args(&c, &b, 1);
    if (rc) return rc;
    QLIN_CHECK(c.pages == caches->pages && c.kv_heads == caches->kv_heads && c.page_size == caches->page_size &&
                   c.head_dim == caches->head_dim && c.fmt == caches->fmt,
               QLIN_ERR_SHAPE);
  }
  if (empty) return QLIN_OK;
  QLIN_CHECK((path || path_cols == 0) && kept && lengths, QLIN_ERR_ARG);
  QLIN_CHECK((((uintptr_t)path | (uintptr_t)kept | (uintptr_t)lengths) & 3) == 0, QLIN_ERR_ALIGN);
  const int64_t B = batch->batch;
  const Ints out = {lengths, B};
  QLIN_CHECK(apart<2>({out, {batch->kv_len, B}}) && apart<2>({out, {batch->q_start, B + 1}}) &&
                 apart<2>({out, {batch->page_table, B * batch->table_cols}}) && apart<2>({out, {kept, B}}) &&
                 apart<2>({out, {path, B * path_cols}}),
             QLIN_ERR_ARG);
  const int rc = device_ok();
  if (rc) return rc;
  return launch_keep(caches, n_caches, *batch, path, path_cols, kept, lengths, as_stream(stream));
}

static int plan_call(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, int64_t q_heads,
                     int64_t window, bool tree, int64_t plan[3]) {
  QLIN_CHECK(cache && batch && plan && window >= 0, QLIN_ERR_ARG);
  QLIN_CHECK(cache->fmt == QLIN_KV_BF16 || cache->fmt == QLIN_KV_E4M3, QLIN_ERR_ARG);
  QLIN_CHECK(kv_shape_ok(cache, batch, T) && attn_shape_ok(cache, batch, T, q_heads), QLIN_ERR_SHAPE);
  plan[0] = plan[1] = plan[2] = 0;
  if (T == 0 || batch->batch == 0) return QLIN_OK;
  QLIN_CHECK(batch->table_cols >= 1 && batch->max_q >= 1, QLIN_ERR_SHAPE);
  attn_plan(*cache, *batch, T, q_heads, window, tree, plan);
  return QLIN_OK;
}

int qlin_attn_plan(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, int64_t q_heads,
                   int64_t window, int64_t plan[3]) {
  return plan_call(cache, batch, T, q_heads, window, false, plan);
}

int qlin_attn_tree_plan(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, int64_t q_heads,
                        int64_t window, int64_t plan[3]) {
  QLIN_CHECK(batch && batch->max_q <= 512, batch ? QLIN_ERR_SHAPE : QLIN_ERR_ARG);
  return plan_call(cache, batch, T, q_heads, window, true, plan);
}

}  // extern "C"
