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
// pages, rows), then the store. One request's 16 tokens in 16 layers 4.2 us (8.4 with the
// host's part); 64 requests' up to 48 of E4M3 in 16 layers 8.6 us (2.5 TB/s).
#include "qlin_internal.h"
#include "qlin_device.h"

namespace qlin {

namespace {

constexpr int kKeepThreads = 256;
constexpr int kKeepRows = 8;      // rows that a thread has a chunk of, in flight together
constexpr int kKeepCaches = 32;   // caches of a launch (their addresses are kernel arguments)

struct KeepArgs {
  uint8_t* pool[2 * kKeepCaches];
  float* scale[2 * kKeepCaches];
  const int32_t *q_start, *kv_len, *table, *path, *kept;
  int32_t* lengths;
  int64_t cols, pages, heads;
  int width;        // of the path
  int page_shift, row_shift;  // tokens of a page; chunks of a row
  int wg_heads, step;         // heads of a workgroup; tokens that its threads cover at once
};

__global__ __launch_bounds__(kKeepThreads) void keep_kernel(const KeepArgs a) {
  __shared__ int64_t from[kKeepThreads], to[kKeepThreads];  // a token's row of head 0; from -1: it stays
  const int b = blockIdx.x, tid = threadIdx.x;
  // (the path's first numbers are on their way while it is not yet known how many count)
  int32_t u = tid < a.width ? a.path[(int64_t)b * a.width + tid] : -1;
  const int64_t n = (int64_t)a.q_start[b + 1] - a.q_start[b], len = max(a.kv_len[b], 0);
  const int64_t first = len - max(n, (int64_t)0);
  const int count = (int)max(min(min((int64_t)a.kept[b], n), (int64_t)a.width), (int64_t)0);
  if (blockIdx.y == 0 && blockIdx.z == 0 && tid == 0) a.lengths[b] = (int32_t)max(first + count, (int64_t)0);
  const int64_t h0 = (int64_t)blockIdx.z * a.wg_heads;
  uint8_t* pool = a.pool[blockIdx.y];
  float* scale = a.scale[blockIdx.y];
  // this thread's chunk of a head, and which of the tokens that are covered at once
  const int c = tid & ((1 << a.row_shift) - 1), per = a.wg_heads << a.row_shift;
  const int token = tid / per;
  const int64_t h = (tid - token * per) >> a.row_shift;
  const bool busy = token < a.step && h0 + h < a.heads;
  auto row_of = [&](int64_t x) -> int64_t {
    const int64_t at = first + x, col = at >> a.page_shift;
    if (at < 0 || col >= a.cols) return -1;
    const int64_t page = a.table[b * a.cols + col];
    if (page < 0 || page >= a.pages) return -1;
    return ((page * a.heads + h0) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
  };
  const int pass = kKeepRows * a.step;  // (at most 256 tokens: a chunk is a row's fourth at least)
  for (int i0 = 0; i0 < count; i0 += pass) {
    const int here = min(pass, count - i0);
    if (i0) u = tid < here ? a.path[(int64_t)b * a.width + i0 + tid] : -1;
    if (tid < here) {
      const bool moves = u >= 0 && u < n && u != i0 + tid;
      const int64_t x = moves ? row_of(u) : -1, y = moves ? row_of(i0 + tid) : -1;
      from[tid] = y < 0 ? -1 : x;
      to[tid] = y;
    }
    __syncthreads();
    uint4 x[kKeepRows];
    float s[kKeepRows];
    int64_t dst[kKeepRows];
#pragma unroll
    for (int k = 0; k < kKeepRows; ++k) {
      const int i = k * a.step + token;
      dst[k] = -1;
      if (!busy || i >= here || from[i] < 0) continue;
      const int64_t src = from[i] + (h << a.page_shift);
      dst[k] = to[i] + (h << a.page_shift);
      x[k] = ldg16(pool + (((src << a.row_shift) + c) << 4));
      if (scale && c == 0) s[k] = scale[src];
    }
    __syncthreads();  // every row of the pass has been read
#pragma unroll
    for (int k = 0; k < kKeepRows; ++k) {
      if (dst[k] < 0) continue;
      *reinterpret_cast<uint4*>(pool + (((dst[k] << a.row_shift) + c) << 4)) = x[k];
      if (scale && c == 0) scale[dst[k]] = s[k];
    }
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
  // all heads if their chunks are no more than the threads, and as many tokens beside
  const int64_t chunks = (int64_t)1 << a.row_shift;
  a.wg_heads = (int)(c.kv_heads < kKeepThreads / chunks ? c.kv_heads : kKeepThreads / chunks);
  a.step = (int)(kKeepThreads / (a.wg_heads * chunks));
  a.step = a.step < kKeepThreads / kKeepRows ? a.step : kKeepThreads / kKeepRows;
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
