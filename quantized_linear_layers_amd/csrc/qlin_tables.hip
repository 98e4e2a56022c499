// Tables of a step over the paged cache, built on the device from what the requests'
// state and a drafting model leave there.
//
// tree_plan_kernel: the masks of a tree of drafted tokens from its parents. A
// workgroup has one sequence, a thread one token. By pointer jumping: every token
// knows its ancestors up to a distance and the one at that distance; taking that one's
// ancestors and its jump doubles the distance, so the deepest chain of 512 takes nine
// rounds through LDS, a tree of eight three.
//
// scan_kernel, fill_kernel, release_kernel: the tables of a step from the requests'
// lengths. Which page a request gets depends on the pages of all before it: a workgroup
// scans the requests. A request's new entries and its tokens' slots then follow from its
// own sums and the free list alone (of its older pages only one can hold a new token), so
// a few neighbouring threads write them for each request, and no one waits for what
// another has written. All inputs are read before what replaces them is written, so
// state is updated in place. Where there are more tokens than one workgroup should write,
// it scans only, and a second launch of many workgroups fills, from the sums that the
// first one left.
//
// Bound by latency: the launch (1.8 us) and loads that each need the one before. A tree of 8
// 2.0 us, 256 of up to 256 tokens 5.6 (two barriers a round, eight rounds for a chain of
// 256, and masks of 1.7 MB); the tables of 64
// requests with up to 16 new tokens 3.5 and, back, 3.0; 64 prompts of up to 8192 tokens, 17000
// pages of 16, 1.9 + 4.7 and 8.3.
#include "qlin_internal.h"
#include "qlin_device.h"

namespace qlin {

namespace {

struct TreePlanArgs {
  const int32_t *q_start, *kv_len, *parents;
  int64_t T;
  int words;
  uint64_t* mask;
  int32_t* positions;
};

// W: words of a mask in LDS, a power of two from words on. Masks lie there word by word,
// so that neighbouring tokens' touch neighbouring banks.
template <int W>
__global__ __launch_bounds__(64 * W) void tree_plan_kernel(const TreePlanArgs a) {
  __shared__ uint64_t seen[W][64 * W];
  __shared__ int jumps[64 * W];
  const int i = threadIdx.x, b = blockIdx.x;
  const int64_t s0 = a.q_start[b], s1 = a.q_start[b + 1];
  const int64_t first = (int64_t)a.kv_len[b] - (s1 - s0);
  if (s0 < 0 || s1 > a.T || s1 <= s0) return;
  const int n = (int)min(s1 - s0, (int64_t)64 * a.words);  // (tokens beyond have no bits)
  int jump = -1;
  if (i < n) {
    const int p = a.parents[s0 + i];
    jump = p >= 0 && p < i ? p : -1;
    jumps[i] = jump;
  }
  uint64_t mine[W];
#pragma unroll
  for (int w = 0; w < W; ++w) seen[w][i] = mine[w] = w == i / 64 ? 1ull << (i % 64) : 0;
  // (a jump goes to an earlier token: after at most ten rounds none is left)
  while (__syncthreads_or(jump >= 0)) {
    int next = -1;
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) mine[w] |= seen[w][jump];
      next = jumps[jump];
    }
    __syncthreads();
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) seen[w][i] = mine[w];
      jumps[i] = jump = next;
    }
  }
  if (i < n && a.positions) {
    int depth = -1;
#pragma unroll
    for (int w = 0; w < W; ++w) depth += __popcll(mine[w]);
    a.positions[s0 + i] = (int32_t)(first + depth);
  }
  for (int e = i; e < n * a.words; e += 64 * W) a.mask[s0 * a.words + e] = seen[e % a.words][e / a.words];
}

// ---------------------------------------------------------------- reserve, release
struct TablesArgs {
  const int32_t *cached, *fresh;  // release: the lengths kept, (none)
  int64_t B, cols, pages, T;
  int32_t* table;
  int32_t* free_pages;
  int32_t* count;                 // [2]: pages in the list; lacking
  int32_t *q_start, *kv_len;
  int32_t *slots, *positions;
  int page_shift;
  int share;                      // threads of a request, as a power of two
};

__device__ __forceinline__ int32_t clamp_int(int64_t x) { return (int32_t)min(x, (int64_t)0x7FFFFFFF); }

// The sum of x over the wave's lanes up to this one. Small numbers (below 2^24: all but
// those of absurd lengths) are added in 32 bits within the vector unit, others by
// shuffles of 64.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
  if (!__any(x >> 24)) {
    int y = (int)x;
    y = dpp_add<0x111, 0xF>(y);  // from 1, 2, 4 and 8 lanes before, within a row of 16
    y = dpp_add<0x112, 0xF>(y);
    y = dpp_add<0x114, 0xF>(y);
    y = dpp_add<0x118, 0xF>(y);
    y = dpp_add<0x142, 0xA>(y);  // the row's before it, to rows 1 and 3
    y = dpp_add<0x143, 0xC>(y);  // the first two rows', to the last two
    return y;
  }
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t y = __shfl_up(x, o, kWave);
    if (lane >= o) x += y;
  }
  return x;
}

// Two sums at once.
struct Sums {
  int64_t a, b;
};
// Sums of x over the workgroup's NT threads before this one; their totals.
template <int NT>
__device__ __forceinline__ Sums scan_before(const Sums& x, Sums& total, Sums* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Sums sum = {wave_scan(x.a), wave_scan(x.b)};
  if (lane == 63) waves[wave] = sum;
  __syncthreads();
  Sums before = {0, 0};
  total = {0, 0};
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    const Sums y = waves[w];
    before.a += w < wave ? y.a : 0;
    before.b += w < wave ? y.b : 0;
    total.a += y.a;
    total.b += y.b;
  }
  __syncthreads();  // (the next scan may write)
  return {before.a + sum.a - x.a, before.b + sum.b - x.b};
}

// A request: cached and new tokens, its first column with a new page, how many such.
struct Request {
  int32_t len, n, col, pages;
};
__device__ __forceinline__ Request request(const TablesArgs& a, int32_t len, int32_t n) {
  const uint32_t round = (1u << a.page_shift) - 1;
  Request r;
  r.len = max(len, 0);
  r.n = min(max(n, 0), 0x7FFFFFFF - r.len);
  r.col = (int32_t)(((uint32_t)r.len + round) >> a.page_shift);
  const int32_t end = min((int32_t)(((uint32_t)(r.len + r.n) + round) >> a.page_shift), (int32_t)a.cols);
  r.pages = max(end - r.col, 0);
  return r;
}
// The page that a request's first new tokens share with cached ones, -1: none.
__device__ __forceinline__ int32_t old_page(const TablesArgs& a, const Request& r, int64_t b) {
  int32_t page = -1;
  if (r.n > 0 && (r.len & ((1 << a.page_shift) - 1)) && r.col <= a.cols) page = a.table[b * a.cols + r.col - 1];
  return page;
}
// What the threads that write a request's entries and tokens know of it.
struct Known {
  Request r;
  int32_t old;
  int32_t top;    // where in the free list its first new page is (the next ones below), below 0: nowhere
  int32_t start;  // its first token
};
__device__ __forceinline__ Known known_of(const Request& r, int32_t old, int64_t end, int64_t start) {
  return {r, old, (int32_t)max(end - 1, (int64_t)-1), clamp_int(start)};
}

// Entries and tokens of request b by thread `mine` of its `share` threads (four at a time,
// whose pages' loads overlap).
__device__ __forceinline__ void fill(const TablesArgs& a, int64_t b, const Known& s, int mine, int share) {
  auto page_at = [&](int k) { return k < s.r.pages && k <= s.top ? a.free_pages[s.top - k] : -1; };
  int32_t* row = a.table + b * a.cols + s.r.col;
  for (int64_t e0 = mine; e0 < s.r.pages; e0 += 4 * share) {
    int32_t page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = page_at((int)e0 + k * share);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (e0 + k * share < s.r.pages) row[e0 + k * share] = page[k];
  }
  const int n = s.start < a.T ? (int)min((int64_t)s.r.n, a.T - s.start) : 0;
  int32_t* slots = a.slots + s.start;
  int32_t* positions = a.positions + s.start;
  for (int64_t i0 = mine; i0 < n; i0 += 4 * share) {
    int32_t page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int col = (int)(((uint32_t)s.r.len + (uint32_t)i0 + k * share) >> a.page_shift) - s.r.col;
      page[k] = col < 0 ? s.old : page_at(col);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + k * share;
      const int32_t at = s.r.len + (int)i;
      if (i >= n) break;
      if (a.slots)
        slots[i] = (uint32_t)page[k] < (uint32_t)a.pages
                       ? (page[k] << a.page_shift) + (at & ((1 << a.page_shift) - 1))
                       : -1;
      if (a.positions) positions[i] = at;
    }
  }
}

// The scan, NT requests at a time; with FILL, of as many tokens as one workgroup should
// write, all of it.
template <int NT, bool FILL>
__global__ __launch_bounds__(NT) void scan_kernel(const TablesArgs a) {
  __shared__ Sums waves[NT / 64];
  __shared__ Known known[FILL ? NT : 1];
  const int i = threadIdx.x;
  const int64_t have = max(min((int64_t)a.count[0], a.pages), (int64_t)0);
  Sums done = {0, 0};  // tokens and pages of the requests before this chunk
  for (int64_t b0 = 0; b0 < a.B; b0 += NT) {
    const int64_t b = b0 + i;
    const Request r = b < a.B ? request(a, a.cached[b], a.fresh[b]) : request(a, 0, 0);
    const int32_t old = FILL && b < a.B ? old_page(a, r, b) : -1;
    Sums all;
    const Sums at = scan_before<NT>({r.n, r.pages}, all, waves);
    if (b < a.B) {
      if (FILL) known[i] = known_of(r, old, have - (done.b + at.b), done.a + at.a);
      a.q_start[b] = clamp_int(done.a + at.a);
      a.kv_len[b] = r.len + r.n;
    }
    if (FILL) {
      __syncthreads();
      const int here = (int)min((int64_t)NT, a.B - b0) << a.share;
      for (int x = i; x < here; x += NT)
        fill(a, b0 + (x >> a.share), known[x >> a.share], x & ((1 << a.share) - 1), 1 << a.share);
      __syncthreads();
    }
    done.a += all.a;
    done.b += all.b;
  }
  if (i == 0) {
    a.q_start[a.B] = clamp_int(done.a);
    a.count[0] = (int32_t)max(have - done.b, (int64_t)0);
    a.count[1] = clamp_int(max(done.b - have, (int64_t)0));
  }
}

// After scan_kernel<NT, false>: each workgroup's requests, 1 << a.share threads each.
constexpr int kFill = 256;
__global__ __launch_bounds__(kFill) void fill_kernel(const TablesArgs a) {
  __shared__ Sums waves[kFill / 64];
  __shared__ Known known[kFill];
  const int i = threadIdx.x;
  const int64_t x = (int64_t)blockIdx.x * kFill + i, mine = x >> a.share;
  const int64_t first = ((int64_t)blockIdx.x * kFill) >> a.share;  // the workgroup's requests
  const int64_t last = min((((int64_t)blockIdx.x + 1) * kFill - 1) >> a.share, a.B - 1);
  // what the requests had before, from what the scan left: lengths less new tokens
  auto was = [&](int64_t b) {
    const int32_t n = a.q_start[b + 1] - a.q_start[b];
    return request(a, a.kv_len[b] - n, n);
  };
  // Where a request's pages are in the list is what the list has left (less what it
  // lacked) and the pages of this request and the later ones: own ones in descending
  // order, and the sum of all behind.
  const int64_t b = last - i;
  const bool own = b >= first;
  const Request r = own ? was(b) : request(a, 0, 0);
  const int32_t old = own ? old_page(a, r, b) : -1;
  const int64_t start = own ? a.q_start[b] : 0;
  const int32_t left = a.count[0], lacking = a.count[1];
  int64_t after = 0;
  for (int64_t y = last + 1 + i; y < a.B; y += kFill) after += was(y).pages;
  Sums all;
  const Sums at = scan_before<kFill>({r.pages, after}, all, waves);
  // (below the list's length, also where absurd sums have passed 32 bits)
  const int64_t end = min((int64_t)left - lacking + all.b + at.a + r.pages, a.pages);
  if (own) known[b - first] = known_of(r, old, end, start);
  __syncthreads();
  if (mine < a.B) fill(a, mine, known[mine - first], (int)(x & ((1 << a.share) - 1)), 1 << a.share);
}

// Four entries of any alignment, one instruction each way.
struct __attribute__((packed, aligned(4))) Four {
  int32_t x[4];
};

// Pages back, from the last request's last page to the first's first: a list that is
// given back what was just taken from it is as before. All of them are looked at first;
// as a rule each is a page of the pool, and its place in the list follows from the scan.
template <int NT>
__global__ __launch_bounds__(NT) void release_kernel(const TablesArgs a) {
  __shared__ Sums waves[NT / 64];
  __shared__ int64_t to[NT];              // where a request's pages go in the list
  __shared__ int32_t end[NT], count[NT];  // its last column, and how many columns
  const int i = threadIdx.x;
  const uint32_t round = (1u << a.page_shift) - 1;
  int64_t have = max(min((int64_t)a.count[0], a.pages), (int64_t)0);
  for (int64_t b1 = a.B; b1 > 0; b1 -= NT) {
    const int64_t b = b1 - 1 - i;  // descending
    int32_t n = 0;
    if (b >= 0) {
      const int32_t c0 = (int32_t)(((uint32_t)max(a.cached[b], 0) + round) >> a.page_shift);
      const int32_t c1 = min((int32_t)(((uint32_t)max(a.kv_len[b], 0) + round) >> a.page_shift), (int32_t)a.cols);
      n = max(c1 - c0, 0);
      end[i] = c1 - 1;
    }
    count[i] = n;
    Sums all;
    const Sums at = scan_before<NT>({n, 0}, all, waves);
    if (all.a == 0) continue;
    to[i] = have + at.a;
    __syncthreads();
    // all requests at once, on as many threads each as there are
    const int here = (int)min((int64_t)NT, b1);
    const int share = 31 - __clz(NT / here), lanes = 1 << share, g = i & (lanes - 1), r = i >> share;
    // a thread's entries, e counted from its request's last: whole fours (four of them on
    // their way together), and what is left singly
    const int entries = r < here ? count[r] : 0, whole = entries & ~3;
    const int32_t* row = a.table + (entries ? (b1 - 1 - r) * a.cols + end[r] : 0);
    const int64_t at0 = entries ? to[r] : 0;
    auto load = [&](int64_t e0, Four (&p)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e0 + 4 * k * lanes < whole) p[k] = *reinterpret_cast<const Four*>(row - (e0 + 4 * k * lanes) - 3);
    };
    bool bad = false;
    const uint32_t pages = (uint32_t)a.pages;
    auto look = [&](int64_t e0, const Four (&p)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e0 + 4 * k * lanes < whole)
          bad |= (uint32_t)p[k].x[0] >= pages || (uint32_t)p[k].x[1] >= pages || (uint32_t)p[k].x[2] >= pages ||
                 (uint32_t)p[k].x[3] >= pages;
    };
    auto write = [&](int64_t e0, const Four (&p)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t e = e0 + 4 * k * lanes, slot = at0 + e;
        if (e >= whole) break;
        if (slot + 3 < a.pages) {
          *reinterpret_cast<Four*>(a.free_pages + slot) = Four{{p[k].x[3], p[k].x[2], p[k].x[1], p[k].x[0]}};
        } else {
          for (int j = 0; j < 4; ++j)
            if (slot + j < a.pages) a.free_pages[slot + j] = p[k].x[3 - j];
        }
      }
    };
    Four kept[4], p[4];  // (the first sixteen stay in registers between the two passes)
    const int left = whole + g < entries ? row[-(whole + g)] : 0;
    load(4 * g, kept);
    look(4 * g, kept);
    for (int64_t e0 = 4 * g + 16 * lanes; e0 < whole; e0 += 16 * lanes) {
      load(e0, p);
      look(e0, p);
    }
    // (less than four are left: a lane has one, or all with one or two lanes)
    for (int e = whole + g; e < entries; e += lanes) bad |= (uint32_t)row[-e] >= pages;
    if (!__syncthreads_or(bad)) {
      write(4 * g, kept);
      for (int64_t e0 = 4 * g + 16 * lanes; e0 < whole; e0 += 16 * lanes) {
        load(e0, p);
        write(e0, p);
      }
      for (int e = whole + g; e < entries; e += lanes)
        if (at0 + e < a.pages) a.free_pages[at0 + e] = e == whole + g ? left : row[-e];
      have += all.a;
    } else {  // (entries that are no page are passed over: a thread a request counts first)
      row = a.table + (b1 - 1 - i) * a.cols + (n ? end[i] : 0);
      int64_t good = 0;
      for (int e = 0; e < n; ++e) good += (uint32_t)row[-e] < pages;
      Sums pushed;
      int64_t slot = have + scan_before<NT>({good, 0}, pushed, waves).a;
      for (int e = 0; e < n; ++e) {
        const int32_t page = row[-e];
        if ((uint32_t)page >= pages) continue;
        if (slot < a.pages) a.free_pages[slot] = page;
        ++slot;
      }
      have += pushed.a;
    }
    __syncthreads();
  }
  if (i == 0) a.count[0] = (int32_t)min(have, a.pages);
}

// Tokens that one workgroup writes beside the scan (of at most 1024 requests).
constexpr int64_t kFillAlone = 4096;

}  // namespace

// Workgroups of 256 threads for few requests: the scan's instructions are issued for
// every wave, and four waves have a SIMD each.
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
  const bool few = a.B <= 256;
  if (T <= kFillAlone && a.B <= 1024) {
    while (a.B << (a.share + 1) <= (few ? 256 : 1024)) ++a.share;  // all of the workgroup's threads
    if (few)
      scan_kernel<256, true><<<1, 256, 0, st>>>(a);
    else
      scan_kernel<1024, true><<<1, 1024, 0, st>>>(a);
  } else {
    // a third of the tokens that a request has on average, 16 workgroups' at most
    while (a.share < 12 && a.B << (a.share + 2) <= T) ++a.share;
    if (few)
      scan_kernel<256, false><<<1, 256, 0, st>>>(a);
    else
      scan_kernel<1024, false><<<1, 1024, 0, st>>>(a);
    fill_kernel<<<(unsigned)(((a.B << a.share) + kFill - 1) / kFill), kFill, 0, st>>>(a);
  }
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
  // (many pages of few requests: more threads to read them)
  if (a.B <= 256 && a.cols <= 64)
    release_kernel<256><<<1, 256, 0, st>>>(a);
  else
    release_kernel<1024><<<1, 1024, 0, st>>>(a);
  return launch_status();
}

int launch_tree_plan(const qlin_kv_batch& batch, int64_t T, const int32_t* parents, int64_t words,
                     uint64_t* mask, int32_t* positions, hipStream_t st) {
  const TreePlanArgs a = {batch.q_start, batch.kv_len, parents, T, (int)words, mask, positions};
  const unsigned grid = (unsigned)batch.batch;
  if (words == 1)
    tree_plan_kernel<1><<<grid, 64, 0, st>>>(a);
  else if (words == 2)
    tree_plan_kernel<2><<<grid, 128, 0, st>>>(a);
  else if (words <= 4)
    tree_plan_kernel<4><<<grid, 256, 0, st>>>(a);
  else
    tree_plan_kernel<8><<<grid, 512, 0, st>>>(a);
  return launch_status();
}

}  // namespace qlin
