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
  return launch_rope(x, ldx, T, H, D, positions, *rope, inverse, y, ldy, as_stream(stream));
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

int qlin_kv_append(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                   const qlin_bf16* k, int64_t ldk, const qlin_bf16* v, int64_t ldv,
                   const qlin_rope_plan* rope, const int32_t* positions, const qlin_bf16* q,
                   int64_t ldq, int64_t q_heads, qlin_bf16* q_out, int64_t ldqo,
                   qlin_stream_t stream) {
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
  return launch_kv_append(*cache, *batch, T, k, ldk, v, ldv, rope, positions, q, ldq, q_heads, q_out, ldqo,
                          as_stream(stream));
}

static bool attn_shape_ok(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t T, int64_t q_heads) {
  return q_heads >= 1 && q_heads <= 0xFFFF && q_heads % c->kv_heads == 0 && T * q_heads <= 0x3FFFFFFF &&
         b->max_q <= 0x7FFFFFFF && b->batch * c->kv_heads <= 0xFFFFFF && attn_grid_ok(*c, *b, T, q_heads);
}

size_t qlin_attn_workspace_bytes(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                                 int64_t q_heads) {
  if (!cache || !batch || !kv_shape_ok(cache, batch, T) || T == 0 || batch->batch == 0 ||
      batch->table_cols == 0 || batch->max_q == 0 || !attn_shape_ok(cache, batch, T, q_heads))
    return 0;
  return attn_workspace_bytes(*cache, *batch, T, q_heads);
}

int qlin_attn_paged(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T,
                    const qlin_bf16* q, int64_t ldq, int64_t q_heads, float scale, int causal,
                    int64_t window, qlin_bf16* out, int64_t ldo, float* lse, void* ws,
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
  const size_t need = attn_workspace_bytes(*cache, *batch, T, q_heads);
  QLIN_CHECK(ws_bytes >= need && (need == 0 || ws), QLIN_ERR_WORKSPACE);
  QLIN_CHECK(need == 0 || ((uintptr_t)ws & 255) == 0, QLIN_ERR_ALIGN);
  rc = device_ok();
  if (rc) return rc;
  return launch_attn(*cache, *batch, T, q, ldq, q_heads, scale, causal, window, out, ldo, lse, ws,
                     ws_bytes, as_stream(stream));
}

int qlin_attn_plan(const qlin_kv_cache* cache, const qlin_kv_batch* batch, int64_t T, int64_t q_heads,
                   int64_t window, int64_t plan[3]) {
  QLIN_CHECK(cache && batch && plan && window >= 0, QLIN_ERR_ARG);
  QLIN_CHECK(cache->fmt == QLIN_KV_BF16 || cache->fmt == QLIN_KV_E4M3, QLIN_ERR_ARG);
  QLIN_CHECK(kv_shape_ok(cache, batch, T) && attn_shape_ok(cache, batch, T, q_heads), QLIN_ERR_SHAPE);
  plan[0] = plan[1] = plan[2] = 0;
  if (T == 0 || batch->batch == 0) return QLIN_OK;
  QLIN_CHECK(batch->table_cols >= 1 && batch->max_q >= 1, QLIN_ERR_SHAPE);
  attn_plan(*cache, *batch, T, q_heads, window, plan);
  return QLIN_OK;
}

}  // extern "C"
