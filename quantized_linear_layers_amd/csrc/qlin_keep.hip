// Accepted tokens' rows of a paged cache moved together: after a tree of drafted tokens
// has been verified, the keys and values of the accepted path, which lie among those of
// all drafted tokens, become the sequence's next tokens.
//
// A workgroup moves one sequence's rows of one pool (a layer's keys or values) for some
// of its heads. A path ascends, so its i-th token never lies before the i-th place:
// in passes of as many tokens as the workgroup's registers hold, read, then written, a
// pass overwrites nothing that a later one reads. All layers go in one launch.
//
// Bound by latency: four loads that each need the one before (starts and lengths, path,
// pages, rows), then the store.
#include "qlin_internal.h"
#include "qlin_device.h"

namespace qlin {

namespace {

constexpr int kKeepThreads = 256;
constexpr int kKeepChunks = 8;    // 16-byte chunks of a thread, in flight together
constexpr int kKeepScales = 2;    // and scales (a row has 4 chunks at least)
constexpr int kKeepCaches = 32;   // caches of a launch (their addresses are kernel arguments)

struct KeepArgs {
  uint8_t* pool[2 * kKeepCaches];
  float* scale[2 * kKeepCaches];
  const int32_t *q_start, *kv_len, *table, *path, *kept;
  int32_t* lengths;
  int64_t cols, pages, heads;
  int width;        // of the path
  int page_shift, row_shift;  // tokens of a page; chunks of a row
  int wg_heads, wg_tokens;    // heads of a workgroup, tokens of a pass
};

__global__ __launch_bounds__(kKeepThreads) void keep_kernel(const KeepArgs a) {
  const int b = blockIdx.x;
  const int64_t n = (int64_t)a.q_start[b + 1] - a.q_start[b], len = max(a.kv_len[b], 0);
  const int64_t first = len - max(n, (int64_t)0);
  const int count = (int)max(min(min((int64_t)a.kept[b], n), (int64_t)a.width), (int64_t)0);
  if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) a.lengths[b] = (int32_t)max(first + count, (int64_t)0);
  const int64_t h0 = (int64_t)blockIdx.z * a.wg_heads;
  const int heads = (int)min((int64_t)a.wg_heads, a.heads - h0);
  uint8_t* pool = a.pool[blockIdx.y];
  float* scale = a.scale[blockIdx.y];
  // the row of a head and token in the pool, -1: none
  auto row_of = [&](int64_t token, int h) -> int64_t {
    const int64_t at = first + token, col = at >> a.page_shift;
    if (at < 0 || col >= a.cols) return -1;
    const int64_t page = a.table[b * a.cols + col];
    if (page < 0 || page >= a.pages) return -1;
    return ((page * a.heads + h0 + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
  };
  // item (i, h) of a pass: where its row comes from and goes (from -1: it stays)
  auto move_of = [&](int i, int h, int64_t& from, int64_t& to) {
    from = to = -1;
    if (i >= count) return;
    const int32_t u = a.path[(int64_t)b * a.width + i];
    if (u < 0 || u >= n || u == i) return;
    to = row_of(i, h);
    if (to >= 0) from = row_of(u, h);
  };
  for (int i0 = 0; i0 < count; i0 += a.wg_tokens) {
    const int items = min(a.wg_tokens, count - i0) * heads;  // (token, head), heads fastest
    uint4 x[kKeepChunks];
    int64_t dst[kKeepChunks];
#pragma unroll
    for (int k = 0; k < kKeepChunks; ++k) {
      const int e = k * kKeepThreads + threadIdx.x, item = e >> a.row_shift;
      const int c = e & ((1 << a.row_shift) - 1);
      int64_t from = -1;
      dst[k] = -1;
      if (item < items) move_of(i0 + item / heads, item % heads, from, dst[k]);
      if (from < 0)
        dst[k] = -1;
      else
        x[k] = ldg16(pool + (((from << a.row_shift) + c) << 4));
      if (dst[k] >= 0) dst[k] = (((dst[k] << a.row_shift) + c) << 4);
    }
    float s[kKeepScales];
    int64_t sdst[kKeepScales];
#pragma unroll
    for (int k = 0; k < kKeepScales; ++k) {
      const int item = k * kKeepThreads + threadIdx.x;
      int64_t from = -1;
      sdst[k] = -1;
      if (scale && item < items) move_of(i0 + item / heads, item % heads, from, sdst[k]);
      if (from < 0)
        sdst[k] = -1;
      else
        s[k] = scale[from];
    }
    __syncthreads();  // every row of the pass has been read
#pragma unroll
    for (int k = 0; k < kKeepChunks; ++k)
      if (dst[k] >= 0) *reinterpret_cast<uint4*>(pool + dst[k]) = x[k];
#pragma unroll
    for (int k = 0; k < kKeepScales; ++k)
      if (sdst[k] >= 0) scale[sdst[k]] = s[k];
    __syncthreads();  // and written, before the next pass reads
  }
}

}  // namespace

int launch_keep(const qlin_kv_cache* caches, int64_t n, const qlin_kv_batch& batch, const int32_t* path,
                int64_t width, const int32_t* kept, int32_t* lengths, hipStream_t st) {
  const qlin_kv_cache& c = caches[0];
  const bool f8 = c.fmt == QLIN_KV_E4M3;
  KeepArgs a = {};
  a.q_start = batch.q_start;
  a.kv_len = batch.kv_len;
  a.table = batch.page_table;
  a.path = path;
  a.kept = kept;
  a.lengths = lengths;
  a.cols = batch.table_cols;
  a.pages = c.pages;
  a.heads = c.kv_heads;
  a.width = (int)width;
  a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  a.row_shift = __builtin_ctzll((unsigned long long)c.head_dim) - (f8 ? 4 : 3);
  // a pass holds 2048 chunks: of at most 512 / (a row's chunks) heads four tokens or more
  const int64_t chunks = (int64_t)1 << a.row_shift;
  a.wg_heads = (int)(c.kv_heads < 512 / chunks ? c.kv_heads : 512 / chunks);
  a.wg_tokens = (int)(kKeepChunks * kKeepThreads / (a.wg_heads * chunks));
  const unsigned z = (unsigned)((c.kv_heads + a.wg_heads - 1) / a.wg_heads);
  for (int64_t at = 0; at < n; at += kKeepCaches) {
    const int here = (int)(n - at < kKeepCaches ? n - at : kKeepCaches);
    for (int i = 0; i < here; ++i) {
      const qlin_kv_cache& x = caches[at + i];
      a.pool[2 * i] = (uint8_t*)x.k;
      a.pool[2 * i + 1] = (uint8_t*)x.v;
      a.scale[2 * i] = x.k_scale;
      a.scale[2 * i + 1] = x.v_scale;
    }
    keep_kernel<<<dim3((unsigned)batch.batch, (unsigned)(2 * here), z), kKeepThreads, 0, st>>>(a);
    const int rc = launch_status();
    if (rc) return rc;
  }
  return QLIN_OK;
}

}  // namespace qlin
