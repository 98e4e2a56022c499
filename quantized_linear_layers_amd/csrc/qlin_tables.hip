// Tables of a step over the paged cache, built on the device from what the requests'
// state and a drafting model leave there.
//
// tree_plan_kernel: the masks of a tree of drafted tokens from its parents. A
// workgroup has one sequence, a thread one token. By pointer jumping: every token
// knows its ancestors up to a distance and the one at that distance; taking that one's
// ancestors and its jump doubles the distance, so the deepest chain of 512 takes nine
// rounds through LDS, a tree of eight three.
//
// reserve_kernel, slots_kernel, release_kernel: the tables of a step from the requests'
// lengths. Which page a request gets depends on the pages of all before it, so one
// workgroup scans the requests, 1024 at a time; the pages themselves (entries, numbered
// over all requests) are spread evenly over its threads, which find an entry's request by
// bisection of the scanned counts in LDS. All inputs are read before what replaces
// them is written, so state is updated in place. Tokens' slots are written by the same
// workgroup where there are few, by a launch of their own else.
#include "qlin_internal.h"
#include "qlin_device.h"

namespace qlin {

namespace {

constexpr int kTreeWords = 8;  // 64-bit words of a mask, at most

struct TreePlanArgs {
  const int32_t *q_start, *kv_len, *parents;
  int64_t T;
  int words;
  uint64_t* mask;
  int32_t* positions;
};

__global__ __launch_bounds__(64 * kTreeWords) void tree_plan_kernel(const TreePlanArgs a) {
  __shared__ uint64_t seen[64 * kTreeWords * kTreeWords];  // [token][word]
  __shared__ int jumps[64 * kTreeWords];
  const int i = threadIdx.x, b = blockIdx.x;
  const int64_t s0 = a.q_start[b], s1 = a.q_start[b + 1];
  if (s0 < 0 || s1 > a.T || s1 <= s0) return;
  const int64_t first = (int64_t)a.kv_len[b] - (s1 - s0);
  const int n = (int)min(s1 - s0, (int64_t)blockDim.x);  // (tokens beyond have no bits)
  const int words = a.words;
  int jump = -1;
  if (i < n) {
    const int p = a.parents[s0 + i];
    jump = p >= 0 && p < i ? p : -1;
    jumps[i] = jump;
    for (int w = 0; w < words; ++w) seen[i * words + w] = w == i / 64 ? 1ull << (i % 64) : 0;
  }
  // (a jump goes to an earlier token: after at most ten rounds none is left)
  while (__syncthreads_or(jump >= 0)) {
    uint64_t more[kTreeWords];
    int next = -1;
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) more[w] = w < words ? seen[jump * words + w] : 0;
      next = jumps[jump];
    }
    __syncthreads();
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        if (w < words) seen[i * words + w] |= more[w];
      jumps[i] = jump = next;
    }
  }
  if (i < n && a.positions) {
    int depth = -1;
    for (int w = 0; w < words; ++w) depth += __popcll(seen[i * words + w]);
    a.positions[s0 + i] = (int32_t)(first + depth);
  }
  for (int e = i; e < n * words; e += blockDim.x) a.mask[s0 * words + e] = seen[e];
}

// ---------------------------------------------------------------- reserve, release
constexpr int kScan = 1024;   // requests that are scanned at a time: the workgroup's threads
constexpr int kEntries = 4;   // neighbouring entries of a thread

struct TablesArgs {
  const int32_t *cached, *fresh;  // release: the lengths kept, (none)
  int64_t B, cols, pages, T;
  int32_t* table;
  int32_t* free_pages;
  int32_t* count;                 // [2]: pages in the list; lacking
  int32_t *q_start, *kv_len;
  int32_t *slots, *positions;
  int page_shift, write_slots;
};

// Sums of x over the workgroup's threads before this one; their total.
__device__ __forceinline__ int64_t scan_before(int64_t x, int64_t& total, int64_t* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t sum = x;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t y = __shfl_up(sum, o, kWave);
    if (lane >= o) sum += y;
  }
  if (lane == 63) waves[wave] = sum;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kScan / 64; ++w) {
    const int64_t y = waves[w];
    before += w < wave ? y : 0;
    total += y;
  }
  __syncthreads();  // (the next scan may write)
  return before + sum - x;
}

__device__ __forceinline__ int32_t clamp_int(int64_t x) { return (int32_t)min(x, (int64_t)0x7FFFFFFF); }
__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// The last of n requests whose first entry is at or before `entry`: the one it belongs to.
__device__ __forceinline__ int request_of(const int64_t* first, int n, int64_t entry) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= entry)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Token t's slot and position, its sequence being one of [lo, hi).
__device__ __forceinline__ void place_token(const TablesArgs& a, int64_t t, int64_t lo, int64_t hi) {
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t s0 = a.q_start[lo], s1 = a.q_start[lo + 1];
  if (t >= s1) return;  // behind the last sequence: left as it is
  const int64_t at = (int64_t)a.kv_len[lo] - (s1 - s0) + (t - s0);
  const int64_t col = at >> a.page_shift;
  int64_t page = -1;
  if (at >= 0 && col < a.cols) page = a.table[lo * a.cols + col];
  if (a.slots)
    a.slots[t] = page >= 0 && page < a.pages
                     ? (int32_t)((page << a.page_shift) + (at & ((1 << a.page_shift) - 1)))
                     : -1;
  if (a.positions) a.positions[t] = (int32_t)at;
}

__global__ __launch_bounds__(kScan) void reserve_kernel(const TablesArgs a) {
  __shared__ int64_t waves[kScan / 64], first[kScan], column[kScan];
  const int i = threadIdx.x;
  const int64_t have = max(min((int64_t)a.count[0], a.pages), (int64_t)0);
  int64_t tokens = 0, taken = 0;  // of the requests before this chunk
  for (int64_t b0 = 0; b0 < a.B; b0 += kScan) {
    const int64_t b = b0 + i;
    int64_t len = 0, n = 0;
    if (b < a.B) {
      len = max(a.cached[b], 0);
      n = min((int64_t)max(a.fresh[b], 0), 0x7FFFFFFF - len);
    }
    const int64_t c0 = pages_of(len, a.page_shift), c1 = min(pages_of(len + n, a.page_shift), a.cols);
    int64_t all_tokens, all;
    const int64_t start = tokens + scan_before(n, all_tokens, waves);
    first[i] = scan_before(max(c1 - c0, (int64_t)0), all, waves);
    column[i] = c0;
    if (b < a.B) {
      a.q_start[b] = clamp_int(start);
      a.kv_len[b] = (int32_t)(len + n);
    }
    __syncthreads();
    const int here = (int)min((int64_t)kScan, a.B - b0);
    for (int64_t e0 = (int64_t)i * kEntries; e0 < all; e0 += kScan * kEntries) {
      int r = request_of(first, here, e0);
      int32_t page[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int64_t at = have - 1 - (taken + e0 + k);
        page[k] = e0 + k < all && at >= 0 ? a.free_pages[at] : -1;
      }
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int64_t e = e0 + k;
        if (e >= all) break;
        while (r + 1 < here && first[r + 1] <= e) ++r;
        a.table[(b0 + r) * a.cols + column[r] + (e - first[r])] = page[k];
      }
    }
    tokens += all_tokens;
    taken += all;
    __syncthreads();  // (also: the chunk's entries before the tokens below)
  }
  if (i == 0) {
    a.q_start[a.B] = clamp_int(tokens);
    a.count[0] = (int32_t)max(have - taken, (int64_t)0);
    a.count[1] = clamp_int(max(taken - have, (int64_t)0));
  }
  if (!a.write_slots) return;
  __syncthreads();
  for (int64_t t = i; t < min(a.T, tokens); t += kScan) place_token(a, t, 0, a.B);
}

// (a workgroup's tokens lie in few sequences: found once, from its first and last token)
constexpr int kSlotThreads = 256, kSlotTokens = 1024;
__global__ __launch_bounds__(kSlotThreads) void slots_kernel(const TablesArgs a) {
  const int64_t t0 = (int64_t)blockIdx.x * kSlotTokens, t1 = min(t0 + kSlotTokens, min(a.T, (int64_t)a.q_start[a.B]));
  if (t0 >= t1) return;
  const int lane = threadIdx.x & 63;
  // the last sequence that starts at or before t: 64 places tried at a time
  auto find = [&](int64_t t) {
    int64_t lo = 0, n = a.B;
    while (n > 1) {
      const int64_t part = (n + 63) / 64, at = lo + lane * part;
      const int k = __popcll(__ballot(lane * part < n && a.q_start[at] <= t)) - 1;
      lo += max(k, 0) * part;
      n = min(part, a.B - lo);
    }
    return lo;
  };
  const int64_t lo = find(t0), hi = find(t1 - 1) + 1;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kSlotThreads) place_token(a, t, lo, hi);
}

__global__ __launch_bounds__(kScan) void release_kernel(const TablesArgs a) {
  __shared__ int64_t waves[kScan / 64], first[kScan], column[kScan];
  const int i = threadIdx.x;
  int64_t have = max(min((int64_t)a.count[0], a.pages), (int64_t)0);
  // from the last request's last page to the first's first: a list that is given back
  // what was just taken from it is as before
  for (int64_t b0 = (a.B - 1) / kScan * kScan; b0 >= 0; b0 -= kScan) {
    const int64_t b = b0 + i;
    int64_t keep = 0, len = 0;
    if (b < a.B) {
      keep = max(a.cached[b], 0);
      len = max(a.kv_len[b], 0);
    }
    const int64_t c0 = pages_of(keep, a.page_shift), c1 = min(pages_of(len, a.page_shift), a.cols);
    int64_t all;
    first[i] = scan_before(max(c1 - c0, (int64_t)0), all, waves);
    column[i] = c0;
    __syncthreads();
    const int here = (int)min((int64_t)kScan, a.B - b0);
    for (int64_t x0 = 0; x0 < all; x0 += kScan * kEntries) {
      int32_t page[kEntries];
      int good = 0;
      const int64_t mine = x0 + (int64_t)i * kEntries;  // from the end
      int r = mine < all ? request_of(first, here, all - 1 - mine) : 0;
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int64_t e = all - 1 - (mine + k);
        page[k] = -1;
        if (e < 0) continue;
        while (first[r] > e) --r;
        page[k] = a.table[(b0 + r) * a.cols + column[r] + (e - first[r])];
        if (page[k] >= a.pages) page[k] = -1;
      }
#pragma unroll
      for (int k = 0; k < kEntries; ++k) good += page[k] >= 0;
      int64_t pushed;
      int64_t at = have + scan_before(good, pushed, waves);
#pragma unroll
      for (int k = 0; k < kEntries; ++k)
        if (page[k] >= 0) {
          if (at < a.pages) a.free_pages[at] = page[k];
          ++at;
        }
      have += pushed;
    }
    __syncthreads();
  }
  if (i == 0) a.count[0] = (int32_t)min(have, a.pages);
}

}  // namespace

int launch_reserve(const qlin_kv_pool& pool, const qlin_kv_tables& t, const int32_t* lengths,
                   const int32_t* new_tokens, int64_t T, hipStream_t st) {
  TablesArgs a = {};
  a.cached = lengths;
  a.fresh = new_tokens;
  a.B = t.batch;
  a.cols = t.table_cols;
  a.pages = pool.pages;
  a.T = t.slots || t.positions ? T : 0;
  a.table = t.page_table;
  a.free_pages = pool.free_pages;
  a.count = pool.count;
  a.q_start = t.q_start;
  a.kv_len = t.kv_len;
  a.slots = t.slots;
  a.positions = t.positions;
  a.page_shift = __builtin_ctzll((unsigned long long)pool.page_size);
  a.write_slots = a.T <= 4 * kScan;
  reserve_kernel<<<1, kScan, 0, st>>>(a);
  if (!a.write_slots) slots_kernel<<<(unsigned)((a.T + kSlotTokens - 1) / kSlotTokens), kSlotThreads, 0, st>>>(a);
  return launch_status();
}

int launch_release(const qlin_kv_pool& pool, const qlin_kv_tables& t, const int32_t* lengths, hipStream_t st) {
  TablesArgs a = {};
  a.cached = lengths;
  a.B = t.batch;
  a.cols = t.table_cols;
  a.pages = pool.pages;
  a.table = t.page_table;
  a.free_pages = pool.free_pages;
  a.count = pool.count;
  a.kv_len = t.kv_len;
  a.page_shift = __builtin_ctzll((unsigned long long)pool.page_size);
  release_kernel<<<1, kScan, 0, st>>>(a);
  return launch_status();
}

int launch_tree_plan(const qlin_kv_batch& batch, int64_t T, const int32_t* parents, int64_t words,
                     uint64_t* mask, int32_t* positions, hipStream_t st) {
  const TreePlanArgs a = {batch.q_start, batch.kv_len, parents, T, (int)words, mask, positions};
  tree_plan_kernel<<<(unsigned)batch.batch, (unsigned)(64 * words), 0, st>>>(a);
  return launch_status();
}

}  // namespace qlin
