// Rotary positions and the paged key/value cache's append.
//
// One kernel does both: a token's row of heads (queries, keys, values) is cut
// into pieces of 16 values, one a thread. A thread keeps its piece of the
// head over all heads that it handles, so its eight sines and cosines are
// computed once and used for every one of them.
//
// Bound by memory from about 1000 tokens on: 8192 tokens of 32 heads of 128 26.5 us
// (5.07 TB/s read and written); queries, keys and values of eight prompts of up to 1024
// tokens into a bf16 cache 30.2 us (4.81 TB/s). E4M3 rows are short of that (2249 tokens,
// heads of 256: 14.0 us, 3.61 TB/s): absmax, quotients that equal the per-token
// quantiser's, and encoding take the vector unit as long. A decode step takes 3.7 us (8
// tokens) to 5.2 (64 with the append): the launch and its loads, which are waited for one
// after the other (positions or lengths and page, frequencies, heads) although of these
// only the page needs the one before.
#include "qlin_internal.h"
#include "qlin_device.h"
#include "qlin_quant_row.h"

namespace qlin {

namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  // rows of heads: queries (or the tensor of qlin_rope), keys, values
  const uint16_t* x[3];
  int64_t ld[3];
  int heads[3];
  uint16_t* y;  // where rows of x[0] go
  int64_t ldy;
  int64_t T;
  int D;
  // pieces of a head that turn (rot / 16), 0: none
  int rot16;
  int interleaved;
  float magnitude;  // negative sine for the inverse rotation is in `sign`
  float sign;
  const double* turns;
  const int32_t* positions;  // NULL: from the batch
  // the cache and the batch (append only)
  uint8_t *kc, *vc;
  float *ks, *vs;
  int64_t pages, page_heads;
  int page_shift;
  const int32_t *q_start, *kv_len, *table;
  int64_t B, cols;
  int slots;  // heads of one token that a workgroup handles at a time
  int toks;   // tokens of a workgroup
};

// The sequence of token t: the number of sequences that end at or before it.
// One load a wave for 64 sequences.
__device__ __forceinline__ int64_t sequence_of(const int32_t* q_start, int64_t B, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t n = 0;
  for (int64_t b0 = 0; b0 < B; b0 += 64) {
    const int64_t b = b0 + lane;
    const bool before = b < B && (int64_t)q_start[b + 1] <= t;
    n += __popcll(__ballot(before));
  }
  return n;
}

// 16 values of a head: the pair halves (or the two 8-value runs) lo and hi.
struct Piece {
  float lo[8], hi[8];
};

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// p / sc, each quotient rounded to nearest as a division's: with y the rounded
// reciprocal and q = x y, the remainder q sc - x is exact and q - (q sc - x) y rounds to
// the quotient (Markstein). The remainder is taken in this order because a zero then keeps
// its sign, and with it its code (x - q sc is +0 for either; copysignf costs 0.4 us).
// Three instructions in place of a division's ten: 14.1 us for the 15.3 of the E4M3 call
// above. Unlike in divide8 the rows are not bf16 but use all of fp32's bits: where a code
// is not zero the remainders are multiples of 2^-57 sc, exact for every sc from 2^-92 on.
// Scales outside 2^-80 .. 2^90, the range that was compared with division (equal
// quotients and signs in 8e9 random pairs), are divided.
__device__ __forceinline__ void divide(Piece& p, float sc) {
  if (sc >= 0x1p-80f && sc <= 0x1p+90f) {
    const float y = 1.0f / sc;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = p.lo[i] * y;
      p.lo[i] = fmaf(-fmaf(q, sc, -p.lo[i]), y, q);
      q = p.hi[i] * y;
      p.hi[i] = fmaf(-fmaf(q, sc, -p.hi[i]), y, q);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.lo[i] = p.lo[i] / sc;
    p.hi[i] = p.hi[i] / sc;
  }
}

// APPEND: keys and values go to the cache; FP8: as E4M3 codes with a scale.
template <bool APPEND, bool FP8>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const RopeArgs a) {
  const int per_head = a.D / 16;
  const int c = threadIdx.x % per_head;       // this thread's piece of a head
  const int g = threadIdx.x / per_head;
  const int slot = g % a.slots;
  const int64_t t0 = (int64_t)blockIdx.x * a.toks;
  const int64_t t = t0 + g / a.slots;
  // every lane takes part in the sequence search before any leaves
  int64_t b = APPEND ? sequence_of(a.q_start, a.B, t0) : 0;
  if (g / a.slots >= a.toks || t >= a.T) return;

  int64_t index = 0;      // the token's place in its sequence
  int64_t page = -1;      // its page; -1: not stored
  if (APPEND) {
    while (b < a.B && (int64_t)a.q_start[b + 1] <= t) ++b;
    if (b >= a.B || t < (int64_t)a.q_start[b]) return;  // padding: left as it is
    const int64_t s0 = a.q_start[b], s1 = a.q_start[b + 1];
    index = a.kv_len[b] - (s1 - s0) + (t - s0);
    const int64_t col = index >> a.page_shift;
    if (index >= 0 && col < a.cols) {
      page = a.table[b * a.cols + col];
      if (page >= a.pages) page = -1;
    }
  }

  // Angles. pos * turns is exact to 2^-53 of its value in fp64, so its part of a
  // turn is right to 2^-22 up to the whole int32 range; sine and cosine are fp32.
  const bool turning = c < a.rot16;
  float cs[8], sn[8];
  if (turning) {
    const double pos = (double)(a.positions ? (int64_t)a.positions[t] : index);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double w = pos * a.turns[8 * c + i];
      const float r = (float)(w - __builtin_rint(w));
      float s, co;
      sincospif(2.0f * r, &s, &co);
      cs[i] = co * a.magnitude;
      sn[i] = s * a.magnitude * a.sign;
    }
  }
  // Offsets of the piece's two 16-byte runs in a head. Half layout: values
  // 8c.. and rot/2 + 8c..; else 16 values in a row.
  const bool halves = turning && !a.interleaved;
  const int o0 = halves ? 8 * c : 16 * c;
  const int o1 = halves ? 8 * c + 8 * a.rot16 : 16 * c + 8;

  const int h_all = a.heads[0] + a.heads[1] + a.heads[2];
  auto part_of = [&](int h) { return !APPEND || h < a.heads[0] ? 0 : h < a.heads[0] + a.heads[1] ? 1 : 2; };
  auto head_of = [&](int h, int part) {
    return h - (part > 0 ? a.heads[0] : 0) - (part > 1 ? a.heads[1] : 0);
  };
  uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
  auto next = [&](int h) {  // the head after this one is read before this one is worked on
    if (h >= h_all) return;
    const int part = part_of(h);
    const uint16_t* src = a.x[part] + t * a.ld[part] + (int64_t)head_of(h, part) * a.D;
    n0 = ldg16(src + o0);
    n1 = ldg16(src + o1);
  };
  const int step = gridDim.y * a.slots;
  int h = blockIdx.y * a.slots + slot;
  next(h);
  for (; h < h_all; h += step) {
    const int part = part_of(h), hh = head_of(h, part);
    uint4 r0 = n0, r1 = n1;
    next(h + step);
    if (part > 0 && page < 0) continue;
    Piece p;
    unpack_bf16x8(r0, p.lo);
    unpack_bf16x8(r1, p.hi);
    if (turning && part < 2) {
      if (halves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = p.lo[i], y = p.hi[i];
          p.lo[i] = fmaf(x, cs[i], -(y * sn[i]));
          p.hi[i] = fmaf(y, cs[i], x * sn[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = p.lo[2 * i], y = p.lo[2 * i + 1];
          p.lo[2 * i] = fmaf(x, cs[i], -(y * sn[i]));
          p.lo[2 * i + 1] = fmaf(y, cs[i], x * sn[i]);
          x = p.hi[2 * i];
          y = p.hi[2 * i + 1];
          p.hi[2 * i] = fmaf(x, cs[4 + i], -(y * sn[4 + i]));
          p.hi[2 * i + 1] = fmaf(y, cs[4 + i], x * sn[4 + i]);
        }
      }
      r0 = pack8(p.lo);
      r1 = pack8(p.hi);
    }
    if (part == 0) {
      uint16_t* dst = a.y + t * a.ldy + (int64_t)hh * a.D;
      *reinterpret_cast<uint4*>(dst + o0) = r0;
      *reinterpret_cast<uint4*>(dst + o1) = r1;
      continue;
    }
    const int in_page = (int)(index & ((1 << a.page_shift) - 1));
    const int64_t row = ((page * a.page_heads + hh) << a.page_shift) + in_page;
    uint8_t* pool = part == 1 ? a.kc : a.vc;
    if (!FP8) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + row * a.D;
      *reinterpret_cast<uint4*>(dst + o0) = r0;
      *reinterpret_cast<uint4*>(dst + o1) = r1;
      continue;
    }
    // the row's threads (4, 8 or 16 neighbours of one wave) share its absmax
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(p.lo[i]), fabsf(p.hi[i])));
    for (int o = per_head / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    const float sc = m > 0.0f ? m / 448.0f : 0.0f;
    uint2 q0 = make_uint2(0, 0), q1 = make_uint2(0, 0);
    if (sc > 0.0f) {
      divide(p, sc);
      q0 = encode8<QLIN_E4M3>(p.lo);
      q1 = encode8<QLIN_E4M3>(p.hi);
    }
    uint8_t* dst = pool + row * a.D;
    *reinterpret_cast<uint2*>(dst + o0) = q0;
    *reinterpret_cast<uint2*>(dst + o1) = q1;
    if (c == 0) (part == 1 ? a.ks : a.vs)[row] = sc;
  }
}

// Heads of one token that a workgroup handles at a time, and its tokens: a
// small call spreads a token's heads over all threads (latency), a large one
// lets each thread do four or eight heads that share the sines and cosines, as
// long as four (eight) workgroups a CU remain. 2249 tokens of 16 + 8 heads of 256
// into an E4M3 cache: 21.2 us with one head a thread, 15.6 with four; 5911 tokens
// of 32 + 16 heads of 128 in bf16: 31.8 with four, 29.5 with eight.
void rope_shape(RopeArgs& a, dim3& grid) {
  const int groups = kRopeThreads / (a.D / 16);
  const int h_all = a.heads[0] + a.heads[1] + a.heads[2];
  const int64_t blocks = a.T * h_all / groups;  // with one head a thread
  const int fold = blocks > 8192 ? 8 : blocks > 1024 ? 4 : 1;
  int slots = (h_all + fold - 1) / fold;
  slots = slots < groups ? slots : groups;
  a.slots = slots;
  a.toks = groups / slots;
  const int passes = (h_all + slots - 1) / slots;
  const int y = fold == 1 ? passes : (passes + fold - 1) / fold;
  grid = dim3((unsigned)((a.T + a.toks - 1) / a.toks), (unsigned)y);
}

}  // namespace

bool rope_grid_ok(int64_t T, int64_t heads, int64_t D) {
  RopeArgs a = {};
  a.T = T;
  a.D = (int)D;
  a.heads[0] = (int)heads;
  if (T == 0 || heads == 0) return true;
  dim3 grid;
  rope_shape(a, grid);
  return (int64_t)grid.x * kRopeThreads <= 0xFFFFFFFF && grid.y <= 0xFFFF;
}

int launch_rope(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, int64_t D,
                const int32_t* positions, const qlin_rope_plan& rope, int inverse, uint16_t* y,
                int64_t ldy, hipStream_t st) {
  RopeArgs a = {};
  a.x[0] = x;
  a.ld[0] = ldx;
  a.heads[0] = (int)H;
  a.y = y;
  a.ldy = ldy;
  a.T = T;
  a.D = (int)D;
  a.rot16 = (int)(rope.rot / 16);
  a.interleaved = rope.interleaved;
  a.magnitude = rope.magnitude;
  a.sign = inverse ? -1.0f : 1.0f;
  a.turns = rope.turns;
  a.positions = positions;
  dim3 grid;
  rope_shape(a, grid);
  rope_kernel<false, false><<<grid, kRopeThreads, 0, st>>>(a);
  return launch_status();
}

int launch_kv_append(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T,
                     const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                     const qlin_rope_plan* rope, const int32_t* positions, const uint16_t* q,
                     int64_t ldq, int64_t q_heads, uint16_t* q_out, int64_t ldqo, hipStream_t st) {
  RopeArgs a = {};
  a.x[0] = q;
  a.x[1] = k;
  a.x[2] = v;
  a.ld[0] = ldq;
  a.ld[1] = ldk;
  a.ld[2] = ldv;
  a.heads[0] = q ? (int)q_heads : 0;
  a.heads[1] = a.heads[2] = (int)cache.kv_heads;
  a.y = q_out;
  a.ldy = ldqo;
  a.T = T;
  a.D = (int)cache.head_dim;
  if (rope) {
    a.rot16 = (int)(rope->rot / 16);
    a.interleaved = rope->interleaved;
    a.magnitude = rope->magnitude;
    a.turns = rope->turns;
  }
  a.sign = 1.0f;
  a.positions = positions;
  a.kc = (uint8_t*)cache.k;
  a.vc = (uint8_t*)cache.v;
  a.ks = cache.k_scale;
  a.vs = cache.v_scale;
  a.pages = cache.pages;
  a.page_heads = cache.kv_heads;
  a.page_shift = __builtin_ctzll((unsigned long long)cache.page_size);
  a.q_start = batch.q_start;
  a.kv_len = batch.kv_len;
  a.table = batch.page_table;
  a.B = batch.batch;
  a.cols = batch.table_cols;
  dim3 grid;
  rope_shape(a, grid);
  if (cache.fmt == QLIN_KV_E4M3)
    rope_kernel<true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else
    rope_kernel<true, false><<<grid, kRopeThreads, 0, st>>>(a);
  return launch_status();
}

}  // namespace qlin
