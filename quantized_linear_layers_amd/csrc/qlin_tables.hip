// Tables of a step over the paged cache, built on the device from what the requests'
// state and a drafting model leave there.
//
// tree_plan_kernel: the masks of a tree of drafted tokens from its parents. A
// workgroup has one sequence, a thread one token. By pointer jumping: every token
// knows its ancestors up to a distance and the one at that distance; taking that one's
// ancestors and its jump doubles the distance, so the deepest chain of 512 takes nine
// rounds through LDS, a tree of eight three.
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

}  // namespace

int launch_tree_plan(const qlin_kv_batch& batch, int64_t T, const int32_t* parents, int64_t words,
                     uint64_t* mask, int32_t* positions, hipStream_t st) {
  const TreePlanArgs a = {batch.q_start, batch.kv_len, parents, T, (int)words, mask, positions};
  tree_plan_kernel<<<(unsigned)batch.batch, (unsigned)(64 * words), 0, st>>>(a);
  return launch_status();
}

}  // namespace qlin
