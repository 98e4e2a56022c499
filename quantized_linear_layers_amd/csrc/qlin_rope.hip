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
// heads of 256: 13.5 us, 3.74 TB/s): absmax, quotients that equal the per-token
// quantiser's, and encoding take the vector unit as long. A decode step takes 3.7 us (8
// tokens) to 5.2 (64 with the append): the launch and its loads, which are waited for one
// after the other (positions or lengths and page, frequencies, heads) although of these
// only the page needs the one before.
//
// Head norms (NORM) cost nothing where memory bounds the call: 8192 tokens of 32 heads of 128
// 28.4 us (4.73 TB/s, 97% of a large copy's rate). E4M3 rows, bound by the vector unit, take
// 15.3 us for 13.5 (2250 tokens of 16 + 8 heads of 256). A decode step takes 4.7.
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
  // head norms: weights of queries, keys and values (NULL: 1), parts that are
  // normalised (bit 0 queries, 1 keys, 2 values)
  const uint16_t* w[3];
  float eps, offset, inv_d;
  int normed;
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
// Three instructions in place of a division's ten: the E4M3 call above takes 13.5 us, 14.5
// with divisions. Unlike in divide8 the rows are not bf16 but use all of fp32's bits: where a code
// is not zero the remainders are multiples of 2^-57 sc, exact for every sc from 2^-92 on.
// Scales outside 2^-80 .. 2^90, the range that was compared with division (equal
// quotients and signs in 8e9 random pairs), are divided.
// REST: by sc + rest, what a scale was before it was rounded (rest is below 2^-24 sc):
// the remainder is that much larger.
// (true: by the reciprocal)
template <bool REST>
__device__ __forceinline__ bool divide(Piece& p, float sc, float rest) {
  if (sc >= 0x1p-80f && sc <= 0x1p+90f) {
    const float y = 1.0f / sc;
    auto one = [&](float& x) {
      const float q = x * y;
      float r = fmaf(q, sc, -x);
      if (REST) r = fmaf(q, rest, r);
      x = fmaf(-r, y, q);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      one(p.lo[i]);
      one(p.hi[i]);
    }
    return true;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.lo[i] = p.lo[i] / sc;
    p.hi[i] = p.hi[i] / sc;
  }
  return false;
}

// Eight E4M3 codes of values up to a row's largest over its scale: a quotient exceeds 448
// by less than its rounding to a code forgives, so nothing is clamped. (Of scales below
// fp32's normal range it may exceed it by more: those rows are clamped, by encode8.)
__device__ __forceinline__ uint2 codes8(const float (&v)[8]) {
  int w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w[h], true);
  }
  return make_uint2((uint32_t)w[0], (uint32_t)w[1]);
}

// The sum (MAX: the largest) of x over the n lanes (a power of two, aligned) that share a
// head, in each. Lanes trade within a row of 16 by DPP: after each step the lanes that a
// mirror trades between hold one value already.
template <bool MAX, int CTRL>
__device__ __forceinline__ float dpp_join(float x) {
  const float y = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
  return MAX ? fmaxf(x, y) : x + y;
}
template <bool MAX>
__device__ __forceinline__ float head_join(float x, int n) {
  if (n >= 2) x = dpp_join<MAX, 0xB1>(x);    // quad_perm 1 0 3 2
  if (n >= 4) x = dpp_join<MAX, 0x4E>(x);    // quad_perm 2 3 0 1
  if (n >= 8) x = dpp_join<MAX, 0x141>(x);   // the two quads of eight lanes
  if (n >= 16) x = dpp_join<MAX, 0x140>(x);  // the two eights of a row
  if (n >= 32) {
    const float y = __shfl_xor(x, 16, kWave);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  if (n >= 64) {
    const float y = __shfl_xor(x, 32, kWave);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  return x;
}

// The largest of m, |x| and |y| (numbers), in one instruction: fmaxf's would be told apart
// from signalling NaNs first.
__device__ __forceinline__ float max3_abs(float m, float x, float y) {
  float r;
  asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(m), "v"(x), "v"(y));
  return r;
}

// Sine and cosine of r turns, |r| <= 1/2: of the nearest quarter turn's remainder t (in
// quarters, taken in fp64: its fp32 value is within 2^-28 of a turn), by their series in
// (pi t / 2)^2 up to the powers 9 and 10 (at an eighth of a turn the next terms are 2^-29
// and 2^-33), then by the quarter.
__device__ __forceinline__ void turn(double r, float& s, float& c) {
  const double k = __builtin_rint(4.0 * r);
  const float t = (float)__builtin_fma(4.0, r, -k), u = t * t;
  // (pi / 2)^n / n!
  float sine = fmaf(u, 1.60441185e-4f, -4.68175414e-3f);
  sine = fmaf(u, sine, 7.96926262e-2f);
  sine = fmaf(u, sine, -6.45964098e-1f);
  sine = fmaf(u, sine, 1.57079633f) * t;
  float cosine = fmaf(u, -2.52020424e-5f, 9.19260274e-4f);
  cosine = fmaf(u, cosine, -2.08634808e-2f);
  cosine = fmaf(u, cosine, 2.53669508e-1f);
  cosine = fmaf(u, cosine, -1.23370055f);
  cosine = fmaf(u, cosine, 1.0f);
  const int q = (int)k;
  const float x = q & 1 ? cosine : sine, y = q & 1 ? sine : cosine;
  s = __uint_as_float(__float_as_uint(x) ^ ((uint32_t)q << 30 & 0x80000000u));
  c = __uint_as_float(__float_as_uint(y) ^ ((uint32_t)(q + 1) << 30 & 0x80000000u));
}

// A head's piece over the head's root mean square: p / sqrt(sum of squares / D + eps),
// the sum over the head's n lanes in fp32. Squares that pass fp32's range (a value
// above 1.8e19) are summed again of values times 2^-72. With CODES only the power of two
// of 1 / sqrt is multiplied in, which rounds nothing; the rest, of [1, 2), is returned.
template <bool CODES>
__device__ __forceinline__ float normalise(Piece& p, int n, float inv_d, float eps, bool codes) {
  auto squares = [&] {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(p.hi[i], p.hi[i], fmaf(p.lo[i], p.lo[i], s));
    return head_join<false>(s, n);
  };
  auto times = [&](float f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p.lo[i] *= f;
      p.hi[i] *= f;
    }
  };
  float s = squares();
  if (s > 0x1.fffffep+127f) {
    times(0x1p-72f);
    s = squares();
    eps = eps * 0x1p-72f * 0x1p-72f;
  }
  const float f = __builtin_amdgcn_rsqf(fmaf(s, inv_d, eps));
  const uint32_t bits = __float_as_uint(f);
  const bool both = !CODES || !codes;
  times(both ? f : __uint_as_float(bits & 0x7F800000u));
  return both ? 1.0f : __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
}

// APPEND: keys and values go to the cache; FP8: as E4M3 codes with a scale. NORM:
// heads are normalised first. PH: pieces of a head, for those sizes that every cache has,
// 0: any number of them. With NORM five waves a SIMD, so that the calls which fill the
// device once do it with room: 2250 tokens of 16 + 8 heads of 256 into E4M3, normalised, are
// 4500 waves. Repeated in a graph they take 16.4 us (15.3 among calls on other inputs), with
// four waves a SIMD 18.3 (and no register spilled; five spill seven, outside the loop over
// heads).
template <int PH, bool APPEND, bool FP8, bool NORM>
__global__ __launch_bounds__(kRopeThreads, NORM ? 5 : 1) void rope_kernel(const RopeArgs a) {
  const int D = PH ? 16 * PH : a.D, per_head = D / 16;
  const int c = threadIdx.x % per_head;       // this thread's piece of a head
  const int g = threadIdx.x / per_head;
  const int slot = g % a.slots;
  const int64_t t0 = (int64_t)blockIdx.x * a.toks;
  const int64_t t = t0 + g / a.slots;
  const bool live = g / a.slots < a.toks && t < a.T;

  // What needs no other load is on its way before the token's place is looked up: the
  // first head and the position.
  const bool turning = c < a.rot16;
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
    const uint16_t* src = a.x[part] + t * a.ld[part] + head_of(h, part) * D;
    n0 = ldg16(src + o0);
    n1 = ldg16(src + o1);
  };
  const int step = gridDim.y * a.slots;
  int h = blockIdx.y * a.slots + slot;
  if (live) next(h);
  int32_t given = 0;
  if (live && turning && a.positions) given = a.positions[t];
  // every lane takes part in the sequence search before any leaves
  int64_t b = APPEND ? sequence_of(a.q_start, a.B, t0) : 0;
  if (!live) return;

  int64_t index = 0;      // the token's place in its sequence
  int32_t page = -1;      // its page; -1: not stored
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
  float cs[8], sn[8];
  if (turning) {
    const double pos = (double)(a.positions ? (int64_t)given : index);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double w = pos * a.turns[8 * c + i];
      const double r = w - __builtin_rint(w);
      float s, co;
      if (NORM)
        turn(r, s, co);
      else
        sincospif(2.0f * (float)r, &s, &co);
      cs[i] = co * a.magnitude;
      sn[i] = s * a.magnitude * a.sign;
      if (NORM && i % 2) __builtin_amdgcn_sched_barrier(0);  // (two at a time: registers)
    }
  }
  for (; h < h_all; h += step) {
    const int part = part_of(h), hh = head_of(h, part);
    uint4 r0 = n0, r1 = n1;
    // (this head's weights, which all heads of a part share, arrive while it is summed)
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    const uint16_t* weight = !NORM ? nullptr : part == 0 ? a.w[0] : part == 1 ? a.w[1] : a.w[2];
    if (NORM && weight) {
      w0 = ldg16(weight + o0);
      w1 = ldg16(weight + o1);
    }
    next(h + step);
    if (part > 0 && page < 0) continue;
    Piece p;
    unpack_bf16x8(r0, p.lo);
    unpack_bf16x8(r1, p.hi);
    const bool normed = NORM && ((a.normed >> part) & 1);
    float factor = 1.0f;  // of the whole row, not multiplied in: a row's scale takes it
    if (normed) {
      factor = normalise<FP8>(p, per_head, a.inv_d, a.eps, part > 0);
      // times (offset + weight), in fp32 as all up to the one rounding at the end
      const float offset = weight ? a.offset : 1.0f;
      Piece w;
      unpack_bf16x8(w0, w.lo);
      unpack_bf16x8(w1, w.hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p.lo[i] *= w.lo[i] + offset;
        p.hi[i] *= w.hi[i] + offset;
      }
    }
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
    }
    if (normed || (turning && part < 2)) {
      r0 = pack8(p.lo);
      r1 = pack8(p.hi);
    }
    if (part == 0) {
      uint16_t* dst = a.y + t * a.ldy + hh * D;
      *reinterpret_cast<uint4*>(dst + o0) = r0;
      *reinterpret_cast<uint4*>(dst + o1) = r1;
      continue;
    }
    const int in_page = (int)(index & ((1 << a.page_shift) - 1));
    const int64_t row = (((int64_t)page * a.page_heads + hh) << a.page_shift) + in_page;
    uint8_t* pool = part == 1 ? a.kc : a.vc;
    if (!FP8) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + row * D;
      *reinterpret_cast<uint4*>(dst + o0) = r0;
      *reinterpret_cast<uint4*>(dst + o1) = r1;
      continue;
    }
    // the row's threads (4, 8 or 16 neighbours of one wave) share its absmax
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max3_abs(m, p.lo[i], p.hi[i]);
    m = head_join<true>(m, per_head);
    const float sc = m > 0.0f ? m / 448.0f : 0.0f;
    // Rows that are stored as they came have the per-token quantiser's codes, of the
    // quotient by the rounded scale; of normalised ones nothing is rounded but the
    // weight's and rotation's products and the quotient by the largest / 448.
    const float rest = normed ? fmaf(-sc, 448.0f, m) * (1.0f / 448.0f) : 0.0f;
    uint2 q0 = make_uint2(0, 0), q1 = make_uint2(0, 0);
    if (sc > 0.0f) {
      if (divide<NORM>(p, sc, rest)) {
        q0 = codes8(p.lo);
        q1 = codes8(p.hi);
      } else {
        q0 = encode8<QLIN_E4M3>(p.lo);
        q1 = encode8<QLIN_E4M3>(p.hi);
      }
    }
    uint8_t* dst = pool + row * D;
    *reinterpret_cast<uint2*>(dst + o0) = q0;
    *reinterpret_cast<uint2*>(dst + o1) = q1;
    if (c == 0) (part == 1 ? a.ks : a.vs)[row] = sc * factor;
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
  // (24 heads in groups of 6 would leave a fourth of the threads without a head)
  if (groups / slots * slots < groups * 7 / 8)
    while (slots & (slots - 1)) ++slots;
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

template <bool APPEND, bool FP8, bool NORM>
static void launch_sizes(RopeArgs& a, hipStream_t st) {
  dim3 grid;
  rope_shape(a, grid);
  if (a.D == 64)
    rope_kernel<4, APPEND, FP8, NORM><<<grid, kRopeThreads, 0, st>>>(a);
  else if (a.D == 128)
    rope_kernel<8, APPEND, FP8, NORM><<<grid, kRopeThreads, 0, st>>>(a);
  else if (a.D == 256)
    rope_kernel<16, APPEND, FP8, NORM><<<grid, kRopeThreads, 0, st>>>(a);
  else if constexpr (!APPEND)  // (caches have these three)
    rope_kernel<0, APPEND, FP8, NORM><<<grid, kRopeThreads, 0, st>>>(a);
}

static void norm_args(RopeArgs& a, const qlin_head_norm& n) {
  a.w[0] = n.q_weight;
  a.w[1] = n.k_weight;
  a.w[2] = n.v_weight;
  a.eps = n.eps;
  a.offset = n.offset;
  a.inv_d = 1.0f / (float)a.D;
  a.normed = n.values ? 7 : 3;
}
static void rope_args(RopeArgs& a, const qlin_rope_plan* rope) {
  a.sign = 1.0f;
  if (!rope) return;
  a.rot16 = (int)(rope->rot / 16);
  a.interleaved = rope->interleaved;
  a.magnitude = rope->magnitude;
  a.turns = rope->turns;
}

int launch_rope(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, int64_t D, const qlin_head_norm* norm,
                const int32_t* positions, const qlin_rope_plan* rope, int inverse, uint16_t* y,
                int64_t ldy, hipStream_t st) {
  RopeArgs a = {};
  a.x[0] = x;
  a.ld[0] = ldx;
  a.heads[0] = (int)H;
  a.y = y;
  a.ldy = ldy;
  a.T = T;
  a.D = (int)D;
  rope_args(a, rope);
  if (inverse) a.sign = -1.0f;
  a.positions = positions;
  if (norm) {
    norm_args(a, *norm);
    launch_sizes<false, false, true>(a, st);
  } else {
    launch_sizes<false, false, false>(a, st);
  }
  return launch_status();
}

int launch_kv_append(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T,
                     const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, const qlin_head_norm* norm,
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
  rope_args(a, rope);
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
  const bool f8 = cache.fmt == QLIN_KV_E4M3;
  if (norm) {
    norm_args(a, *norm);
    f8 ? launch_sizes<true, true, true>(a, st) : launch_sizes<true, false, true>(a, st);
  } else {
    f8 ? launch_sizes<true, true, false>(a, st) : launch_sizes<true, false, false>(a, st);
  }
  return launch_status();
}

}  // namespace qlin
