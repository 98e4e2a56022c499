// Attention of new tokens over a paged key/value cache.
//
// Mathematics. For one sequence and one key/value head, the new tokens and the
// query heads that share that head are packed into rows (row = token * group +
// head of the group). Over tiles of 32 keys a wave computes
//   S^T = K Q^T          (32 keys x 32 rows, v_mfma_f32_32x32x16_bf16)
//   P^T = exp2(c S^T - m) with the running maximum m and sum l of each row
//   O^T = O^T 2^(m_old - m) + V^T P^T
// with the scores transposed: a lane then owns one row (lane & 31) and 16 of
// the 32 keys, so maximum and sum are taken inside the lane and once across the
// wave's halves, and P^T leaves the first product in the lanes where the
// second needs it. Lane half h holds keys 8b + 4h + r (b, r = 0..3) of a block,
// while the MFMA's B operand wants 8 consecutive keys a half: the products sum
// over keys in any order, so V^T is simply read in P's order
// (ds_read_b64_tr_b16 gives 4 keys of one column from 4 rows of V, two of them
// an operand; E4M3: ds_read_b64_tr_b8, 8 keys).
//
// The maximum is kept in the exponent's units (log2). It is raised only when a
// row's new maximum passes it by more than 8: until then the weights stay
// below 2^8, where bf16 and fp32 keep the same relative precision, and O
// needs no rescaling pass.
//
// K and V tiles arrive by buffer_load_dwordx4 ... lds (16 bytes a lane, 1 KB an
// instruction, no registers). A resource covers 16 rows of one page at most (a step's
// whole tile of 32 where the pages have as many), so the memory system itself zeroes
// rows behind the last visible key and before the first one, and pages that do not
// exist: stale values there, NaN too, never reach a product. LDS rows are stored with their 16-byte chunks
// exclusive-or-ed by row bits (k_swz, v_swz), so that both the row reads of K and
// the transposing reads of V touch every bank once.
//
// Two kernels share this: attn_step_kernel (16 or 32 rows a workgroup: a decode step, a
// small chunk, trees), where each wave takes its own key tiles and the waves merge at the
// end, and attn_chunk_kernel (128 rows; E4M3 attn_chunk_e4m3_kernel, 256), where each
// wave has its own rows and the workgroup shares the tiles. All split the key axis
// over workgroups when the rows alone do not fill the device; the parts are joined by
// the last workgroup to arrive (step) or by attn_join_kernel (chunk, whose parts are
// many rows). Both have a form (TREE) that takes a token's mask of the new keys in place
// of their order: only tiles that reach into the new tokens read the bits.
#include "qlin_internal.h"
#include "qlin_device.h"

#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

namespace qlin {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

#define QLIN_LDS __attribute__((address_space(3)))
#define QLIN_CONST __attribute__((address_space(4)))

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

struct AttnArgs {
  const uint8_t *k, *v;
  const float *ks, *vs;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t *q_start, *kv_len, *table;
  int64_t ldq, ldo, T, window;
  int B, cols, pages, page_shift, kv_heads, group, causal, splits;
  int tiles;   // row tiles over all sequences, at most (chunk)
  int negate;  // a negative scale: the queries change sign
  float c;     // |scale| * log2(e)
  // with splits > 1, parts of the key axis: unnormalised O rows and their running
  // maximum (log2) and sum. Chunk: [splits][T][q_heads][D] and [..][2]; step:
  // [batch * kv_heads * row_tiles][splits][part_rows][D] and [..][2], and arrival counters
  float *po, *pml;
  uint32_t* arrived;  // [batch * kv_heads * row_tiles], 0 between calls
  int part_rows, row_tiles;  // step: rows of a workgroup, workgroups for a sequence's rows
  // a tree: masks [T][words] of the new tokens that each one sees, 32 bits a word, and
  // positions [T] (with a window)
  const uint32_t* mask;
  const int32_t* positions;
  int words;
  int ordered;  // step: sequences with the most keys first (at most 256 sequences)
};

__device__ __forceinline__ v16f mfma32(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// 8 E4M3 codes to bf16 (exact).
__device__ __forceinline__ v8bf cvt_fp8x8(uint32_t lo, uint32_t hi) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Geometry of K and V rows in LDS. NARROW: read by the 16-row products of the
// step kernel, else by the 32-row ones of the chunk kernel (bf16 there).
template <int D, bool FP8, bool NARROW = false>
struct Geo {
  static constexpr int kRow = FP8 ? D : 2 * D;       // bytes of a row
  static constexpr int kChunks = kRow / 16;          // 16-byte chunks of a row
  static constexpr int kRowsPerLoad = 64 / kChunks;  // rows of one 1 KB load
  // Exclusive-or of a row's chunk index. K is read 16 bytes a lane, one chunk of
  // 32 (16) rows at a time; V by half a wave 64 bytes of 4 rows, narrow: 32 bytes
  // of 8 rows, or 16 of 16 rows in E4M3.
  static __device__ __forceinline__ int k_swz(int row) {
    return kChunks >= 16 ? row & 15 : kChunks == 8 ? row & 7 : (row >> 1) & 3;
  }
  static __device__ __forceinline__ int v_swz(int row) {
    if (NARROW) {
      if (FP8) {
        if (kChunks >= 16) return (row & 7) | ((row >> 1) & 8);
        if (kChunks == 8) return ((row >> 1) & 3) | ((row >> 2) & 4);
        return ((row >> 2) & 1) | ((row >> 3) & 2);
      }
      return kChunks >= 16 ? (row & 7) << 1 : ((row >> 1) & 3) << 1;
    }
    return kChunks >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
  }
};

// (token, head) rows of one sequence and key/value head, and its keys.
struct Item {
  int b, h;     // sequence, key/value head
  int64_t q0;   // its first row in q
  int n;        // new tokens
  int first;    // the first one's place in the sequence (below 0: before it)
  int len;      // keys: the sequence's, at most what its page table reaches
  int rows;     // packed rows
};

// One group of MOST (16) rows (first key `key`) of a page: its first row in the pool and
// how many of its rows lie before `hi` (0 if the page does not exist).
struct Rows16 {
  uint64_t row;
  int rows;
};
__device__ __forceinline__ bool no_page(const AttnArgs& a, int page) { return (uint32_t)page >= (uint32_t)a.pages; }
template <int MOST = 16>
__device__ __forceinline__ Rows16 rows_of(const AttnArgs& a, const Item& it, int key, int page, int hi) {
  const bool none = no_page(a, page);
  const uint32_t block = (uint32_t)(none ? 0 : page) * (uint32_t)a.kv_heads + (uint32_t)it.h;
  Rows16 w;
  w.row = ((uint64_t)block << a.page_shift) + (uint32_t)(key & ((1 << a.page_shift) - 1));
  w.rows = none ? 0 : max(min(hi - key, MOST), 0);
  return w;
}
template <int BYTES>
__device__ __forceinline__ v4i resource(const void* pool, const Rows16& w) {
  const uint64_t p = (uint64_t)(uintptr_t)pool + w.row * BYTES;
  return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)p), __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)),
             __builtin_amdgcn_readfirstlane(w.rows * BYTES), 0x00020000};
}

// Direct-to-LDS loads of N * 1 KB: lane i's 16 bytes at off[n] + 1024 n of the
// resource go to lds + 1024 n + 16 i (an instruction's offset adds to both
// sides). Inline assembly for the same reason as in the prefill GEMMs: the
// compiler would wait for every load in flight before the next LDS read. The
// kernels wait themselves (dma_wait) before they read what a load wrote and
// before they end. What the compiler would see to is written out: the wait
// state between a write of m0 and the load that uses it, and (settled) the five
// between a vector instruction's write of a scalar register and a load's use.
// No "memory" clobber: the phase and stage borders have one.
template <int N>
__device__ __forceinline__ void dma16(uint32_t lds, const uint32_t (&off)[N], const v4i& rs) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "");
  const int m = __builtin_amdgcn_readfirstlane((int)lds);
  if constexpr (N == 1)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(m), "v"(off[0]), "s"(rs)
                 : "m0");
  if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
                 "buffer_load_dwordx4 %2, %3, 0 offen offset:1024 lds" ::"s"(m), "v"(off[0]), "v"(off[1]), "s"(rs)
                 : "m0");
  if constexpr (N >= 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %5, 0 offen lds\n\t"
                 "buffer_load_dwordx4 %2, %5, 0 offen offset:1*1024 lds\n\t"
                 "buffer_load_dwordx4 %3, %5, 0 offen offset:2*1024 lds\n\t"
                 "buffer_load_dwordx4 %4, %5, 0 offen offset:3*1024 lds" ::"s"(m), "v"(off[0]), "v"(off[1]),
                 "v"(off[2]), "v"(off[3]), "s"(rs)
                 : "m0");
  if constexpr (N == 8) {
    const uint32_t hi[4] = {off[4] + 4096, off[5] + 4096, off[6] + 4096, off[7] + 4096};
    dma16<4>(lds + 4096, hi, rs);
  }
}
__device__ __forceinline__ void dma4(uint32_t lds, uint32_t off, const v4i& rs) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane((int)lds)),
               "v"(off), "s"(rs)
               : "m0");
}
__device__ __forceinline__ void settled(v4i& a) { asm volatile("s_nop 4" : "+s"(a)); }
__device__ __forceinline__ void settled(v4i& a, v4i& b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }
template <int N>
__device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void lds_reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const QLIN_LDS uint8_t*)p;
}

// Loads of a tile of TK keys into LDS: ROWS of its rows (8 or 16 rows of one
// 16-row group) from row r0 by one wave. Scales (E4M3): the first 16 of every 64
// floats of a group, because a load writes all 64 lanes. With EDGE, rows of the
// group before `skip` read as zero too (an offset far beyond the resource); only
// the first tile of a window has such rows.
template <int D, bool FP8, int TK, int ROWS, bool NARROW = false>
struct Stage {
  using G = Geo<D, FP8, NARROW>;
  static constexpr int kTile = TK * G::kRow;
  static constexpr int kScale = FP8 ? TK / 16 * 256 : 0;  // bytes of one scale area
  static constexpr int kLoads = ROWS / G::kRowsPerLoad;
  static_assert(kLoads >= 1, "a load must not pass the wave's rows");

  template <bool V, bool EDGE>
  static __device__ __forceinline__ void rows(const v4i& rs, int skip, int r0, uint32_t lds) {
    const int lane = threadIdx.x & 63;
    uint32_t off[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = r0 + i * G::kRowsPerLoad + lane / G::kChunks;
      const int slot = lane % G::kChunks;
      off[i] = (uint32_t)(((r0 & 15) + lane / G::kChunks) * G::kRow + 16 * (slot ^ (V ? G::v_swz(row) : G::k_swz(row))));
      if (EDGE && (row & 15) < skip) off[i] = 0x80000000u;
    }
    dma16<kLoads>(lds + r0 * G::kRow, off, rs);
  }
  // the same of 32 rows that lie together (a tile within a page), by one resource
  template <bool V, bool EDGE>
  static __device__ __forceinline__ void rows32(const v4i& rs, int skip, uint32_t lds) {
    constexpr int kAll = 32 / G::kRowsPerLoad, kOnce = kAll < 8 ? kAll : 8;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kAll; j += kOnce) {
      uint32_t off[kOnce];
#pragma unroll
      for (int i = 0; i < kOnce; ++i) {
        const int row = (j + i) * G::kRowsPerLoad + lane / G::kChunks;
        off[i] = (uint32_t)(j * 1024 + lane / G::kChunks * G::kRow +
                            16 * (lane % G::kChunks ^ (V ? G::v_swz(row) : G::k_swz(row))));
        if (EDGE && row < skip) off[i] = 0x80000000u;
      }
      dma16<kOnce>(lds + j * 1024, off, rs);
    }
  }
  template <bool EDGE>
  static __device__ __forceinline__ void scale_row(const v4i& rs, int skip, int r0, uint32_t lds) {
    const int lane = threadIdx.x & 63;
    const uint32_t at = lane >= 16 || (EDGE && lane < skip) ? 0x80000000u : (uint32_t)(lane * 4);
    dma4(lds + (r0 / 16) * 256, at, rs);
  }
  template <bool EDGE>
  static __device__ __forceinline__ void scale_rows32(const v4i& rs, int skip, uint32_t lds) {
    const int lane = threadIdx.x & 63;
    dma4(lds, lane >= 32 || (EDGE && lane < skip) ? 0x80000000u : (uint32_t)(lane * 4), rs);
  }
};

// The larger of the wave's halves' values, in both.
__device__ __forceinline__ float halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Running softmax state of a wave's 32 rows and their output.
template <int D>
struct State {
  v16f o[D / 32];
  float m, l;  // of row (lane & 31); l sums this lane's keys only
  __device__ __forceinline__ void clear() {
    m = -kInf;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = v16f{};
  }
};

// Operand fragments from LDS (bf16). K: 32 keys of block kb, step u; V^T: 16 keys
// of step t, columns 32 d.
template <int D>
__device__ __forceinline__ v8bf k_frag(const uint8_t* lds_k, int kb, int u, int lane) {
  using G = Geo<D, false>;
  const int row = 32 * kb + (lane & 31);
  return *reinterpret_cast<const v8bf*>(lds_k + row * G::kRow + 16 * ((2 * u + (lane >> 5)) ^ G::k_swz(row)));
}
template <int D>
__device__ __forceinline__ v8bf v_frag(const uint8_t* lds_v, int t, int d, int lane) {
  using G = Geo<D, false>;
  const int row = 16 * t + 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int chunk = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (QLIN_LDS v4s*)(lds_v + row * G::kRow + 16 * (chunk ^ G::v_swz(row)) + 8 * (lane & 1)));
  const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (QLIN_LDS v4s*)(lds_v + (row + 8) * G::kRow + 16 * (chunk ^ G::v_swz(row + 8)) + 8 * (lane & 1)));
  return __builtin_bit_cast(v8bf, (v8s){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
}
__device__ __forceinline__ v8bf as_bf16(const v4i& x) { return __builtin_bit_cast(v8bf, x); }

// Fragment n of the products of KB * 32 keys: first the values', then the keys'.
template <int D, int KB>
__device__ __forceinline__ v8bf frag(const uint8_t* lds_v, const uint8_t* lds_k, int n, int lane) {
  constexpr int nv = 2 * KB * (D / 32);
  return n < nv ? v_frag<D>(lds_v, n / (D / 32), n % (D / 32), lane)
                : k_frag<D>(lds_k, (n - nv) % KB, (n - nv) / KB, lane);
}
// The lane number, with heads of 256 in a form that keeps the fragments' addresses
// from being held in registers over the loop (12 of them, which would not fit).
template <int D>
__device__ __forceinline__ int frag_lane() {
  int lane = threadIdx.x & 63;
  if (D == 256) asm volatile("" : "+v"(lane));
  return lane;
}

// The products of KB * 32 keys with a wave's 32 rows: O^T += V^T P^T of the weights p
// over lds_v, then (QK) the scores S^T of lds_k. fr holds the first N fragments on
// entry; each product is followed by the read of the fragment N products on (an LDS
// read takes about as long as 4), and nothing moves past a product: left alone,
// the scheduler reads two ahead where registers are short.
// between(i) is called after every second product, for other work to be spread
// over them.
template <int D, int KB, int N, bool QK, class F>
__device__ __forceinline__ void multiply(const v8bf (&q)[D / 16], State<D>& st, v16f (&s)[KB], const v4i (&p)[2 * KB],
                                         v8bf (&fr)[N], const uint8_t* lds_v, const uint8_t* lds_k, F between) {
  constexpr int nv = 2 * KB * (D / 32), all = nv + (QK ? KB * (D / 16) : 0);
  const int lane = frag_lane<D>();
  if (QK) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) s[kb] = v16f{};
  }
#pragma unroll
  for (int n = 0; n < all; ++n) {
    const v8bf x = fr[n % N];
    if (n < nv)
      st.o[n % (D / 32)] = mfma32(x, as_bf16(p[n / (D / 32)]), st.o[n % (D / 32)]);
    else
      s[(n - nv) % KB] = mfma32(x, q[(n - nv) / KB], s[(n - nv) % KB]);
    if (n + N < all) fr[n % N] = frag<D, KB>(lds_v, lds_k, n + N, lane);
    if (n % 2) {
      between(n / 2);
      __builtin_amdgcn_sched_barrier(0x4);  // (scalar instructions may move)
    }
  }
}

// A tile's E4M3 scales of keys 8 n + 4 h + 0..3, h the lane's half.
__device__ __forceinline__ v4f scales(const uint8_t* lds_s, int n) {
  return *reinterpret_cast<const v4f*>(lds_s + n / 2 * 256 + (8 * (n & 1) + 4 * ((threadIdx.x & 63) >> 5)) * 4);
}

// The weights of a score block, rounded to bf16, and the running maximum and
// sum (and with a raised maximum O) that go with them.
//   vis_lo, vis_hi: keys that this lane's row sees, relative to the first
//   masked: whether some row sees only part of them; bad: bit g = the 16-row
//   group g lies in no page
//   TREE: tree[kb], the keys of block kb that the row's mask lets it see (if masked)
//   E4M3: lds_s, lds_s + SCALE: the keys' and values' scales; with HOLD the keys' are in
//   ks already, and the values' are read ahead of the work
template <int D, bool FP8, bool TREE, int KB, int SCALE, bool HOLD>
__device__ __forceinline__ void weight_block(const AttnArgs& a, State<D>& st, v16f (&s)[KB], v4i (&p)[2 * KB],
                                             const v4f (&ks)[4 * KB], const uint8_t* lds_s, bool masked, int vis_lo,
                                             int vis_hi, uint32_t bad, const uint32_t (&tree)[KB]) {
  const int h = (threadIdx.x & 63) >> 5;
  v4f vs[4 * KB];
  if (FP8) {
    if (HOLD) {
#pragma unroll
      for (int n = 0; n < 4 * KB; ++n) vs[n] = scales(lds_s + SCALE, n);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = 0; n < 4 * KB; ++n) {
      const v4f k = HOLD ? ks[n] : scales(lds_s, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n / 4][n % 4 * 4 + i] *= k[i];
    }
  }
  if (masked) {
    const int lo = vis_lo - 4 * h, hi = vis_hi - 4 * h;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const uint32_t mine = TREE ? tree[kb] >> (4 * h) : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = 32 * kb + 8 * (i / 4) + i % 4;
        bool see = lo <= key && hi > key && !((bad >> (2 * kb + i / 8)) & 1);
        if (TREE) see = see && ((mine >> (8 * (i / 4) + i % 4)) & 1);
        s[kb][i] = see ? s[kb][i] : -kInf;
      }
    }
  }
  float mx = s[0][0];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][i]);
  mx = halves_max(mx) * a.c;
  if (__any(mx > st.m + 8.0f)) {
    const float m = fmaxf(st.m, mx);
    const float f = m == -kInf ? 0.0f : exp2_hw(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) st.o[i][j] *= f;
  }
  const float m = st.m == -kInf ? 0.0f : st.m;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[kb][i] = exp2_hw(fmaf(s[kb][i], a.c, -m));
      st.l += s[kb][i];
    }
  if (FP8) {
#pragma unroll
    for (int n = 0; n < 4 * KB; ++n) {
      const v4f v = HOLD ? vs[n] : scales(lds_s + SCALE, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n / 4][n % 4 * 4 + i] *= v[i];
    }
  }
  // P rounded to bf16 for the product (at most 2^-8 of a weight; the sum l
  // keeps the unrounded weights)
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 8; ++i) p[2 * kb + i / 4][i % 4] = (int)pack_bf16x2(s[kb][2 * i], s[kb][2 * i + 1]);
}

// Eight values of a query row (negated for a negative scale).
__device__ __forceinline__ v8bf load_q8(const AttnArgs& a, const uint16_t* src) {
  uint4 x = ldg16(src);
  if (a.negate) {
    x.x ^= 0x80008000u;
    x.y ^= 0x80008000u;
    x.z ^= 0x80008000u;
    x.w ^= 0x80008000u;
  }
  return __builtin_bit_cast(v8bf, x);
}
// A packed row of queries; rows past the end repeat the last: never stored.
template <int D>
__device__ __forceinline__ const uint16_t* q_row(const AttnArgs& a, const Item& it, int row) {
  const int r = min(row, it.rows - 1);
  return a.q + (it.q0 + r / a.group) * a.ldq + (int64_t)(it.h * a.group + r % a.group) * D;
}
template <int D>
__device__ __forceinline__ void load_q(const AttnArgs& a, const Item& it, int row, v8bf (&q)[D / 16]) {
  const uint16_t* src = q_row<D>(a, it, row) + 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int u = 0; u < D / 16; ++u) q[u] = load_q8(a, src + 16 * u);
}

// Keys [row_lo, row_hi) that a packed row sees (none: row_hi <= row_lo). Of a TREE the
// keys from the first new token on are seen by the row's mask (tree_bits) beside, and
// the window ends at the token's position, which is that of one of the new tokens.
template <bool TREE>
__device__ __forceinline__ int row_hi(const AttnArgs& a, const Item& it, int row) {
  if (row >= it.rows) return 0;
  return !TREE && a.causal ? min(it.first + row / a.group + 1, it.len) : it.len;
}
template <bool TREE>
__device__ __forceinline__ int row_lo(const AttnArgs& a, const Item& it, int row) {
  if (a.window <= 0) return 0;
  int64_t p = (int64_t)it.first + row / a.group;
  if (TREE) {
    const int64_t own = a.positions[it.q0 + min(row, it.rows - 1) / a.group];
    p = min(max(own, (int64_t)it.first), (int64_t)it.first + it.n - 1);
  }
  const int64_t lo = p + 1 - a.window;
  return lo > 0 ? (int)lo : 0;
}
// Of rows [row0, row1): keys [lo, hi) that some row sees, and [all_lo, all_hi)
// that every row sees (of a tree: at least these, at most those).
struct Range {
  int lo, hi, all_lo, all_hi;
};
template <bool TREE>
__device__ __forceinline__ Range range_of(const AttnArgs& a, const Item& it, int row0, int row1) {
  Range r;
  r.hi = max(row_hi<TREE>(a, it, row1 - 1), 0);
  if (TREE) {
    const int64_t lo = a.window > 0 ? (int64_t)it.first + 1 - a.window : 0;
    r.lo = lo > 0 ? min((int)lo, r.hi) : 0;
    r.all_lo = a.window > 0 ? (int)max(lo + it.n - 1, (int64_t)0) : 0;
    r.all_hi = row0 < it.rows ? min(it.first, it.len) : 0;
  } else {
    r.lo = min(row_lo<TREE>(a, it, row0), r.hi);
    r.all_lo = row_lo<TREE>(a, it, row1 - 1);
    r.all_hi = row_hi<TREE>(a, it, row0);
  }
  r.lo = __builtin_amdgcn_readfirstlane(r.lo);
  r.hi = __builtin_amdgcn_readfirstlane(r.hi);
  r.all_lo = __builtin_amdgcn_readfirstlane(r.all_lo);
  r.all_hi = __builtin_amdgcn_readfirstlane(r.all_hi);
  return r;
}

// A packed row's mask (rows past the end: the last one's).
__device__ __forceinline__ const uint32_t* mask_row(const AttnArgs& a, const Item& it, int row) {
  return a.mask + (it.q0 + min(row, it.rows - 1) / a.group) * a.words;
}
// Of the 32 keys from `key` on, those that the mask lets the row see: all before the
// first new token, none behind the mask's end.
__device__ __forceinline__ uint32_t tree_bits(const AttnArgs& a, const Item& it, const uint32_t* mask, int key) {
  const int64_t u = (int64_t)key - it.first;
  if (u <= -32) return ~0u;
  if (u < 0) return mask[0] << (int)-u | ((1u << (int)-u) - 1);
  const int64_t w = u >> 5;
  const uint32_t lo = w < a.words ? mask[w] : 0, hi = w + 1 < a.words ? mask[w + 1] : 0;
  return (uint32_t)(((uint64_t)hi << 32 | lo) >> (u & 31));
}

// The page of a key, read through the scalar cache (keys outside the table:
// some entry, whose rows are then outside the visible range).
__device__ __forceinline__ int32_t page_of(const AttnArgs& a, const Item& it, int key) {
  const int col = min(max(key, 0) >> a.page_shift, a.cols - 1);
  return ((const QLIN_CONST int32_t*)(uintptr_t)a.table)[(int64_t)it.b * a.cols + col];
}

// A sequence's rows and keys from the batch's device data; false: no rows.
__device__ __forceinline__ bool item_from(const AttnArgs& a, int b, int h, int64_t s0, int64_t s1, int64_t len,
                                          Item& it) {
  if (s0 < 0 || s1 > a.T || s1 <= s0) return false;
  it.b = b;
  it.h = h;
  it.q0 = s0;
  it.n = (int)(s1 - s0);
  len = max(len, (int64_t)0);
  it.first = (int)(len - it.n);
  it.len = (int)min(len, (int64_t)a.cols << a.page_shift);
  it.rows = it.n * a.group;
  return true;
}
__device__ __forceinline__ bool item_of(const AttnArgs& a, int b, int h, Item& it) {
  return item_from(a, b, h, a.q_start[b], a.q_start[b + 1], a.kv_len[b], it);
}

// One row's part for attn_join_kernel. This lane holds the head's values 32 d +
// 8 (i / 4) + 4 h + i % 4 in o[d][i].
template <int D>
__device__ __forceinline__ void store_part(const AttnArgs& a, const Item& it, int split, int row, const State<D>& st) {
  const int h = (threadIdx.x & 63) >> 5;
  const float l = st.l + __shfl_xor(st.l, 32, kWave);
  if (row >= it.rows) return;
  const int64_t t = it.q0 + row / a.group;
  const int qh = it.h * a.group + row % a.group;
  const int64_t at = (split * a.T + t) * ((int64_t)a.kv_heads * a.group) + qh;
  if (h == 0) {
    a.pml[2 * at] = st.m;
    a.pml[2 * at + 1] = l;
  }
  if (st.m == -kInf && l == 0.0f) return;  // no key: the join does not read it
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<v4f*>(a.po + at * D + 32 * d + 8 * b + 4 * h) =
          v4f{st.o[d][4 * b], st.o[d][4 * b + 1], st.o[d][4 * b + 2], st.o[d][4 * b + 3]};
}

// A wave's 32 rows, in whole lines: through 64 D bytes of LDS of its own (128
// columns at a time), 16-byte chunks exclusive-or-ed by the row.
template <int D>
__device__ __forceinline__ void store_rows(const AttnArgs& a, const Item& it, int w0, const State<D>& st,
                                           uint8_t* lds) {
  constexpr int kCols = D < 128 ? D : 128, kChunks = kCols / 8, kLine = 2 * kCols;
  const int lane = threadIdx.x & 63;
  const int r = lane & 31, h = lane >> 5;
  const int64_t heads = (int64_t)a.kv_heads * a.group;
  const float l = st.l + __shfl_xor(st.l, 32, kWave);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += kCols) {
    if (c0) lds_reads_done();
#pragma unroll
    for (int d = 0; d < kCols / 32; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const v16f& o = st.o[c0 / 32 + d];
        *reinterpret_cast<uint2*>(lds + r * kLine + 16 * ((4 * d + b) ^ (r & (kChunks - 1))) + 8 * h) =
            make_uint2(pack_bf16x2(o[4 * b] * inv, o[4 * b + 1] * inv),
                       pack_bf16x2(o[4 * b + 2] * inv, o[4 * b + 3] * inv));
      }
    lds_reads_done();  // (and writes; one wave's LDS)
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i) {
      const int row = i * (64 / kChunks) + lane / kChunks, c = lane % kChunks;
      const uint4 x = *reinterpret_cast<const uint4*>(lds + row * kLine + 16 * (c ^ (row & (kChunks - 1))));
      const int gr = w0 + row;
      if (gr < it.rows)
        *reinterpret_cast<uint4*>(a.out + (it.q0 + gr / a.group) * a.ldo +
                                  (int64_t)(it.h * a.group + gr % a.group) * D + c0 + 8 * c) = x;
    }
  }
  const int gr = w0 + r;
  if (a.lse && h == 0 && gr < it.rows)
    a.lse[(it.q0 + gr / a.group) * heads + it.h * a.group + gr % a.group] =
        l == 0.0f ? -kInf : (st.m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- chunk
// A workgroup's BM rows: its sequence and head, its first row and its part of the
// keys; false: none.
template <int BM>
__device__ __forceinline__ bool chunk_item(const AttnArgs& a, Item& it, int& row0, int& split) {
  const int lane = threadIdx.x & 63;
  // Work order: consecutive workgroups go to the 8 XCDs in turn; each XCD gets a
  // contiguous run of (head, tile) items, so the tiles of one head share its L2.
  const int items = a.tiles * a.kv_heads * a.splits;
  const int per = (items + 7) / 8;
  const int item = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if ((int)(blockIdx.x / 8) >= per || item >= items) return false;
  split = item % a.splits;
  const int h = item / a.splits / a.tiles;
  int tile = item / a.splits % a.tiles;
  // the tile's sequence: 64 sequences a pass, a lane each, the ones with the most
  // keys first (of a batch of many lengths the longest work must not come last)
  int b = -1;
  for (int b0 = 0; b0 < a.B && b < 0; b0 += 64) {
    int mine = 0, keys = 0, from = 0, to = 0;
    if (b0 + lane < a.B) {
      from = a.q_start[b0 + lane];
      to = a.q_start[b0 + lane + 1];
      keys = a.kv_len[b0 + lane];
      const int64_t n = (int64_t)to - from;
      mine = n > 0 && n <= a.T ? (int)((n * a.group + BM - 1) / BM) : 0;
    }
    int before = 0, all = 0;  // tiles of the pass that come before this lane's; all
    for (int j = 0; j < min(a.B - b0, 64); ++j) {
      const int n = __builtin_amdgcn_readlane(mine, j), k = __builtin_amdgcn_readlane(keys, j);
      before += k > keys || (k == keys && j > lane) ? n : 0;
      all += n;
    }
    const unsigned long long here = __ballot(tile >= before && tile < before + mine);
    if (here) {
      const int j = __ffsll(here) - 1;
      b = b0 + j;
      tile -= __builtin_amdgcn_readlane(before, j);
      // its last tiles first: with a causal mask they have the most keys
      tile = __builtin_amdgcn_readlane(mine, j) - 1 - tile;
      if (!item_from(a, b, h, __builtin_amdgcn_readlane(from, j), __builtin_amdgcn_readlane(to, j),
                     __builtin_amdgcn_readlane(keys, j), it))
        return false;
    } else {
      tile -= all;
    }
  }
  if (b < 0) return false;
  row0 = __builtin_amdgcn_readfirstlane(tile) * BM;
  return true;
}

// What a wave of a workgroup of BM rows has to do: its first row w0, its lane's row, the
// keys that the workgroup's and the wave's rows see, those of the lane's row, and the
// tiles of TK keys of this part.
struct ChunkJob {
  Item it;
  int split, w0, row;
  Range wg, own;
  int vlo, vhi, t0, t1;
};
template <bool TREE, int BM, int TK>
__device__ __forceinline__ bool chunk_job(const AttnArgs& a, int wave, ChunkJob& j) {
  int row0;
  if (!chunk_item<BM>(a, j.it, row0, j.split)) return false;
  j.w0 = row0 + 32 * wave;
  j.row = j.w0 + ((int)threadIdx.x & 31);
  j.wg = range_of<TREE>(a, j.it, row0, min(row0 + BM, j.it.rows));
  j.own = range_of<TREE>(a, j.it, j.w0, max(min(j.w0 + 32, j.it.rows), j.w0 + 1));
  j.vlo = row_lo<TREE>(a, j.it, j.row);
  j.vhi = row_hi<TREE>(a, j.it, j.row);
  int t0 = j.wg.lo / TK, t1 = (j.wg.hi + TK - 1) / TK;
  if (a.splits > 1) {
    const int n = max((t1 - t0 + a.splits - 1) / a.splits, 1);
    t0 = min(t0 + j.split * n, t1);
    t1 = min(t0 + n, t1);
  }
  j.t0 = __builtin_amdgcn_readfirstlane(t0);
  j.t1 = __builtin_amdgcn_readfirstlane(t1);
  return true;
}

// bf16: a workgroup of 4 waves has 128 rows of one (sequence, key/value head), 32 a
// wave, and walks their keys in tiles of TK that its waves share. A wave multiplies
// (values of tile t - 1, scores of tile t), then takes the weights of tile t; a tile
// costs it about as many matrix cycles as vector cycles. Two workgroups share a CU
// (heads of 64: four), one wave of each a SIMD, so that while one multiplies another
// takes weights, and one's start and end hide behind the other's tiles.
// K and V have two places each. After the barrier that ends the products of tile t,
// K(t) and V(t-1) are free: the loads of K(t+2) and V(t+1) go there, and have until the
// end of the products of tile t+1, where the wave waits for them before the barrier.
// (One workgroup of 256 rows a CU, its wave pairs held in opposite phases by barriers,
// as below, on one machine: 234 us for 218 with heads of 256 and a window, 80 for 75 for
// eight prompts of up to 1024 with heads of 128, but 523 for 536 for a prompt of 8192 and
// 965 for 995 for 2048 tokens of 32768.)
//
// Measured, 32 + 8 heads of 128: a prompt of 8192 534 us (1029 TFLOP/s, 79 % of a large
// library matrix product's 1298); 2048 tokens of 32768 994 us (1072). 16 + 8 heads of 256,
// window 1024, four prompts of up to 4096: 219 us (750). (Another machine, with the same
// matrix product: 507, 943 and 205.) Bound by the issue of vector instructions, with heads
// of 128 about as many cycles as the products' (27 a tile beside the 32 products, about 140
// for the weights), and by what the two waves of a SIMD take from each other. With heads of
// 256 a tile has half the scores, but 102 vector instructions beside its 32 products: the
// fragments' LDS addresses, which there are computed anew for each (frag_lane).
template <int D, int TK, bool TREE>
__global__ __launch_bounds__(256, D == 64 ? 4 : 2) void attn_chunk_kernel(const AttnArgs a) {
  using St = Stage<D, false, TK, TK / 4>;
  using G = Geo<D, false>;
  constexpr int BM = 128, KB = TK / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_k[2][St::kTile], lds_v[2][St::kTile];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ChunkJob job;
  if (!chunk_job<TREE, BM, TK>(a, wave, job)) return;
  const Item it = job.it;
  const Range wg = job.wg, own = job.own;
  const int w0 = job.w0, row = job.row, vlo = job.vlo, vhi = job.vhi, t0 = job.t0, t1 = job.t1;
  // the rows of a tile that this wave loads, of one 16-row group
  constexpr int kRows = TK / 4;
  const int r0 = wave * kRows;
  const int g0 = r0 & ~15;
  auto page_at = [&](int t) { return page_of(a, it, t * TK + g0); };
  constexpr std::integral_constant<bool, true> kEdge;
  constexpr std::integral_constant<bool, false> kInner;
  auto load = [&](int t, int page, uint8_t* to, auto is_v, auto edge) {
    const Rows16 w = rows_of(a, it, t * TK + g0, page, wg.hi);
    v4i rs = resource<G::kRow>(is_v ? a.v : a.k, w);
    settled(rs);
    St::template rows<is_v, edge>(rs, wg.lo - t * TK - g0, r0, lds_addr(to));
  };
  constexpr int kAhead = 4;  // fragments ahead of the products (6, 8 and 12 with heads of 128: the same time)
  // the end of the products: this wave's loads have arrived, its LDS reads are done, and
  // nothing moves across
  auto products_end = [&] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // (tiles from t1 on load nothing: no row of theirs is visible)
  int p1 = page_at(t0 + 1), p2 = page_at(t0 + 2);  // pages of the next loads
  if (t0 < t1) {
    const int p0 = page_at(t0);
    load(t0, p0, lds_k[0], kInner, kEdge);
    load(t0, p0, lds_v[0], kEdge, kEdge);
    load(t0 + 1, p1, lds_k[1], kInner, kInner);
  }
  // whether some page of these keys does not exist
  bool hole = false;
  const int c1 = t0 < t1 ? (t1 * TK - 1) >> a.page_shift : -1;
  for (int c = ((t0 * TK) >> a.page_shift) + (int)threadIdx.x; c <= min(c1, a.cols - 1); c += 256)
    hole |= no_page(a, a.table[(int64_t)it.b * a.cols + c]);
  v8bf q[D / 16];
  load_q<D>(a, it, row, q);
  State<D> st;
  st.clear();
  dma_wait<0>();
  lds_reads_done();
  const bool holes = __syncthreads_or(hole);
  v16f s[KB];
  v4i p[2 * KB];
  v8bf fr[kAhead];
  const v4f none[4 * KB] = {};
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i) p[i] = v4i{};
  // (the first tile adds zero weights times its own values)
  auto prefetch = [&](int place) {  // (all of the values')
    static_assert(kAhead <= 2 * KB * (D / 32), "");
    const int lane = frag_lane<D>();
#pragma unroll
    for (int n = 0; n < kAhead; ++n) fr[n] = frag<D, KB>(lds_v[place], lds_k[0], n, lane);
  };
  int at = 0;  // the place of K(t) and V(t)
  for (int t = t0; t < t1; ++t) {
    const int vat = t > t0 ? at ^ 1 : at;
    prefetch(vat);
    __builtin_amdgcn_s_setprio(1);
    multiply<D, KB, kAhead, true>(q, st, s, p, fr, lds_v[vat], lds_k[at], [](int) {});
    __builtin_amdgcn_s_setprio(0);
    products_end();
    load(t + 2, p2, lds_k[at], kInner, kInner);
    load(t + 1, p1, lds_v[at ^ 1], kEdge, kInner);
    p1 = p2;
    p2 = page_at(t + 3);
    const int key = t * TK;
    uint32_t bad = 0;
    if (holes)
      for (int g = 0; g < TK / 16; ++g) bad |= (uint32_t)no_page(a, page_of(a, it, key + 16 * g)) << g;
    const bool masked = holes || key + TK > own.all_hi || key < own.all_lo;
    uint32_t tree[KB] = {};
    if (TREE && masked) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) tree[kb] = tree_bits(a, it, mask_row(a, it, row), key + 32 * kb);
    }
    weight_block<D, false, TREE, KB, 0, false>(a, st, s, p, none, nullptr, masked, vlo - key, vhi - key, bad, tree);
    __builtin_amdgcn_sched_barrier(0);
    at ^= 1;
  }
  if (t0 < t1) {
    prefetch(at ^ 1);
    multiply<D, KB, kAhead, false>(q, st, s, p, fr, lds_v[at ^ 1], lds_k[at], [](int) {});
  }
  dma_wait<0>();
  if (a.splits > 1) {
    store_part<D>(a, it, job.split, row, st);
    return;
  }
  __syncthreads();  // V's places are free
  store_rows<D>(a, it, w0, st, &lds_v[0][0] + wave * (TK * D));
}

// E4M3: tiles become bf16 on the way into LDS, once a workgroup (converting fragments
// would cost every wave 8 instructions a product), so a workgroup has 8 waves and 256
// rows (with 128 and the kernel above, twice the conversions: 655 us for 600 for the chunks
// below, 1220 for 1015 for 2048 tokens of 32768). The two waves of a SIMD, w and w + 4, work in opposite phases: while one
// multiplies, the other takes the weights of its tile; a barrier ends each phase.
//   phase   waves 0-3           waves 4-7
//   2t      PV(t-1), QK(t)      weights(t-1)
//   2t+1    weights(t)          PV(t-1), QK(t)
// K(t) and V(t-1) are free after phase 2t+1; K has three places, V four. Tiles pass
// through registers: spread over the products of tile t, each wave writes its piece of
// K(t+2) (waves 0-3) or V(t+2), loaded one tile before, and loads that of tile t+3.
// Scales come along: places for 8 tiles.
//
// Heads of 64 leave room for two workgroups a CU (four waves a SIMD) at the price of 6
// spilled registers, written before and read after the tile loop: each workgroup fills the
// other's waits, so the priority of the multiplying wave, which is worth 2 to 4 % with
// wider heads, costs 3 % there. Heads of 256 spill 7, one of which is read back in every
// tile; heads of 128 none.
//
// Measured, eight chunks of up to 1024 tokens in prompts of up to 9001: 32 + 8 heads of
// 128 597 us (856 TFLOP/s; bf16 532), heads of 64 437 (585; bf16 326), 16 + 8 heads of 256
// 659 (776; bf16 560). (Another machine: 560 with heads of 128.) Bound by the phases: a tile
// takes the two waves of a SIMD about 4000 cycles, of which their products need 2048 and
// their 240 vector instructions each (bf16: 168) 2400 at 5 cycles, so the most of what is
// missing goes to the two barriers a tile that hold the phases.
template <int D, int TK, bool TREE>
__global__ __launch_bounds__(512, D == 64 ? 4 : 2) void attn_chunk_e4m3_kernel(const AttnArgs a) {
  using St = Stage<D, false, TK, TK / 4>;
  using G = Geo<D, false>;
  constexpr int BM = 256, KB = TK / 32;
  constexpr int kScale = TK / 16 * 256;  // bytes of one scale area
  __shared__ __attribute__((aligned(1024))) uint8_t lds_k[3][St::kTile], lds_v[4][St::kTile];
  __shared__ __attribute__((aligned(1024))) uint8_t lds_s[8][2 * kScale];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  ChunkJob job;
  if (!chunk_job<TREE, BM, TK>(a, wave, job)) return;
  const Item it = job.it;
  const Range wg = job.wg, own = job.own;
  const int w0 = job.w0, row = job.row, vlo = job.vlo, vhi = job.vhi, t0 = job.t0, t1 = job.t1;
  const bool first = wave < 4;
  // the rows of a tile that this wave loads, of one 16-row group (waves 0-3 of K, 4-7 of V)
  constexpr int kRows = TK / 4;
  const int r0 = (wave & 3) * kRows;
  const int g0 = r0 & ~15;
  auto page_at = [&](int t) { return page_of(a, it, t * TK + g0); };
  constexpr std::integral_constant<bool, true> kEdge;
  constexpr std::integral_constant<bool, false> kInner;
  // Read the key scales over the last products and the values' ahead of the
  // weights, where registers allow; else where they are used, an LDS read's time
  // exposed eight times a tile (eight chunks of up to 1024 tokens, 32 heads of
  // 128, in prompts of up to 9001: 610 us and 663; heads of 256 would spill: four such
  // chunks 1600 us and 790).
  constexpr bool kHold = D == 128;
  constexpr int kProducts = 2 * KB * (D / 32) + KB * (D / 16);  // of a tile
  // This lane's codes of K (waves 0-3) or V, kMine * 16 of them, where they go as
  // bf16, and the scales of the wave's group
  constexpr int kMine = kRows * D / 1024;
  const uint8_t* pool = first ? a.k : a.v;
  const float* pool_s = first ? a.ks : a.vs;
  int from[kMine], to[kMine][2];
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int n = c * 64 + lane, r = r0 + n / (D / 16), chunk = n % (D / 16);
    const int sw = first ? G::k_swz(r) : G::v_swz(r);
    from[c] = (r & 15) * D + 16 * chunk;
    to[c][0] = r * G::kRow + 16 * ((2 * chunk) ^ sw);
    to[c][1] = r * G::kRow + 16 * ((2 * chunk + 1) ^ sw);
  }
  auto fetch = [&](int t, int page, v4i (&x)[kMine], auto edge) {
    const Rows16 w = rows_of(a, it, t * TK + g0, page, wg.hi);
    const int skip = wg.lo - t * TK - g0;
    if ((r0 & 15) == 0) {
      v4i rs = resource<4>(pool_s, w);
      settled(rs);
      St::template scale_row<edge>(rs, skip, g0, lds_addr(lds_s[t & 7]) + (first ? 0 : kScale));
    }
    // (uniform, which the compiler cannot see: without readfirstlane it loops over
    // the lanes' resources)
    const uint64_t base = (uint64_t)(uintptr_t)pool + w.row * D;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(uintptr_t)((uint64_t)hi << 32 | lo), (short)0, __builtin_amdgcn_readfirstlane(w.rows * D), 0x00020000);
#pragma unroll
    for (int c = 0; c < kMine; ++c)
      x[c] = __builtin_amdgcn_raw_buffer_load_b128(rs, edge && from[c] / D < skip ? (int)0x80000000 : from[c], 0, 0);
  };
  auto put = [&](const v4i (&x)[kMine], int t, int k_place, int i) {  // half i % 2 of piece i / 2
    uint8_t* base = first ? lds_k[k_place] : lds_v[t & 3];
    *reinterpret_cast<v8bf*>(base + to[i / 2][i % 2]) = cvt_fp8x8(x[i / 2][2 * (i % 2)], x[i / 2][2 * (i % 2) + 1]);
  };
  // Fragments that a wave holds ahead of its products (heads of 64 and 256: as many
  // as the registers allow). With heads of 256, where the multiply phases are the
  // longer ones, the first of them (values that arrived a tile before) are read at
  // the end of the weight phase.
  constexpr int kAhead = D == 128 ? 8 : 4;
  // the end of a phase; no instruction moves from one into another, and all but the
  // last `reads` LDS instructions have completed
  auto phase_end = [&](auto reads) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"((int)reads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  constexpr std::integral_constant<int, 0> kAll;
  constexpr std::integral_constant<int, 15> kNone;

  // (tiles from t1 on load nothing: no row of theirs is visible)
  int p1 = page_at(t0 + 1), p2 = page_at(t0 + 2);  // pages of the next loads
  v4i fx[kMine];                                   // tile t + 2 on its way
  if (t0 < t1) {
    const int p0 = page_at(t0);
    v4i x0[kMine], x1[kMine];
    fetch(t0, p0, x0, kEdge);
    fetch(t0 + 1, p1, x1, kInner);
    fetch(t0 + 2, p2, fx, kInner);
#pragma unroll
    for (int i = 0; i < 2 * kMine; ++i) {
      put(x0, t0, 0, i);
      put(x1, t0 + 1, 1, i);
    }
    p2 = page_at(t0 + 3);
  }
  // whether some page of these keys does not exist
  bool hole = false;
  const int c1 = t0 < t1 ? (t1 * TK - 1) >> a.page_shift : -1;
  for (int c = ((t0 * TK) >> a.page_shift) + (int)threadIdx.x; c <= min(c1, a.cols - 1); c += 512)
    hole |= no_page(a, a.table[(int64_t)it.b * a.cols + c]);
  v8bf q[D / 16];
  load_q<D>(a, it, row, q);
  State<D> st;
  st.clear();
  int at = 0, next = 1, last = 2;  // K's places of tiles t, t + 1 and t + 2 (t - 1)
  lds_reads_done();  // (and writes)
  const bool holes = __syncthreads_or(hole);
  v16f s[KB];
  v4i p[2 * KB];
  v8bf fr[kAhead];
  v4f ks[4 * KB];  // the tile's key scales, read over the last products
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i) p[i] = v4i{};
  // (the first tile adds zero weights times its own values)
  auto prefetch = [&](int t) {
    const int lane = frag_lane<D>();
#pragma unroll
    for (int n = 0; n < kAhead; ++n) fr[n] = frag<D, KB>(lds_v[t & 3], lds_k[0], n, lane);
  };
  if (D == 256 && t0 < t1) prefetch(t0);
  if (!first) phase_end(kAll);
  // Every wave takes every tile, also one that its rows do not see (past their
  // diagonal, before their windows, rows past the end): the phases keep the
  // waves in step, so leaving one out would save nothing.
  for (int t = t0; t < t1; ++t) {
    // multiply
    if (D > 64) __builtin_amdgcn_s_setprio(1);
    if (D < 256) prefetch(t > t0 ? t - 1 : t);
    multiply<D, KB, kAhead, true>(q, st, s, p, fr, lds_v[(t > t0 ? t - 1 : t) & 3], lds_k[at], [&](int i) {
      if (i < 2 * kMine) put(fx, t + 2, last, i);
      if (i == 2 * kMine) fetch(t + 3, p2, fx, kInner);
      if (kHold && i >= kProducts / 2 - 4 * KB)
        ks[i - (kProducts / 2 - 4 * KB)] = scales(lds_s[t & 7], i - (kProducts / 2 - 4 * KB));
    });
    if (D > 64) __builtin_amdgcn_s_setprio(0);
    phase_end(kAll);
    // weights
    p2 = page_at(t + 4);
    const int key = t * TK;
    uint32_t bad = 0;
    if (holes)
      for (int g = 0; g < TK / 16; ++g) bad |= (uint32_t)no_page(a, page_of(a, it, key + 16 * g)) << g;
    const bool masked = holes || key + TK > own.all_hi || key < own.all_lo;
    uint32_t tree[KB] = {};
    if (TREE && masked) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) tree[kb] = tree_bits(a, it, mask_row(a, it, row), key + 32 * kb);
    }
    weight_block<D, true, TREE, KB, kScale, kHold>(a, st, s, p, ks, lds_s[t & 7], masked, vlo - key, vhi - key, bad,
                                                   tree);
    if (D == 256) prefetch(t);
    phase_end(kNone);  // (no LDS writes in this phase)
    const int x = last;
    last = at;
    at = next;
    next = x;
  }
  if (t0 < t1) {
    if (D < 256) prefetch(t1 - 1);
    multiply<D, KB, kAhead, false>(q, st, s, p, fr, lds_v[(t1 - 1) & 3], lds_k[at], [](int) {});
  }
  dma_wait<0>();
  if (first) phase_end(kAll);
  if (a.splits > 1) {
    store_part<D>(a, it, job.split, row, st);
    return;
  }
  __syncthreads();  // V's places are free
  store_rows<D>(a, it, w0, st, &lds_v[0][0] + wave * (TK * D));
}

// ---------------------------------------------------------------- step
// A workgroup has up to 32 rows of a (sequence, key/value head), in RB blocks of 16:
// with so few rows the 16-row products (v_mfma_f32_16x16x32_bf16) do half the work of the
// 32-row ones, and their small state lets four waves share a SIMD. Lane group g =
// lane >> 4 holds keys 16 b + 4 g + i of the tile's score block b: P's order for
// the value product (slot j of group g: key 4 g + j, or 16 + 4 g + j - 4).
// NW waves have the same rows and take key tiles of 32 in turn (wave, wave + NW,
// ...), each with a K and a V place of its own in LDS, so the loop has no
// barrier: the next K tile is loaded as soon as the scores have read this one, the
// next V tile as soon as the values have, and each load has the other half of a
// tile's work, and the other waves, to hide behind. The waves' results are merged
// in LDS.
// With splits, every workgroup takes the same number of tiles, so a batch of many
// lengths is cut into equal pieces: about kPieces in all, more if the longest
// sequence would need more splits than there are (the lengths are device data, so
// the grid holds the most splits and the ones without tiles leave). The last
// workgroup of a (sequence, head) to arrive joins its parts, in their order.
//
// Bound by memory: eight bf16 sequences of 65536, 32 + 8 heads of 128, 362 us (5.93 TB/s
// read); 64 E4M3 ones of up to 1536 30.7 us (4.57 TB/s). One of 1025: 9.4 us, of which the
// launch, three loads that each need the one before (lengths, page, keys and values) and
// the join are all but 1.
constexpr int kPieces = 512;
// (one instruction; fmaxf's operands would be told apart from signalling NaNs first)
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
  return r;
}
__device__ __forceinline__ float groups_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float groups_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

// The place-th sequence in an order of sixteen classes of lengths, the longest first, and
// its rows and keys: of a grid that does not fit the device at once the long sequences
// must not come last (64 trees of 16 over up to 4096 E4M3 keys: 103 us for 112 in the batch's
// order). At most 256 sequences, a lane has four.
__device__ __forceinline__ bool item_by_length(const AttnArgs& a, int place, int h, Item& it) {
  const int lane = threadIdx.x & 63;
  int from[4], to[4], len[4], longest = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = 64 * i + lane;
    from[i] = to[i] = len[i] = 0;
    if (b < a.B) {
      from[i] = a.q_start[b];
      to[i] = a.q_start[b + 1];
      len[i] = a.kv_len[b];
    }
    longest = max(longest, len[i]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) longest = max(longest, __shfl_xor(longest, o, kWave));
  const float per = 16.0f / ((float)longest + 1.0f);
  int key[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) key[i] = 64 * i + lane < a.B ? min((int)((float)max(len[i], 0) * per), 15) : -1;
  for (int c = 15; c >= 0; --c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned long long these = __ballot(key[i] == c);
      const int n = __popcll(these);
      if (place < n) {
        const bool mine = key[i] == c && __popcll(these & ((1ull << lane) - 1)) == place;
        const int j = __ffsll(__ballot(mine)) - 1;
        return item_from(a, 64 * i + j, h, __builtin_amdgcn_readlane(from[i], j), __builtin_amdgcn_readlane(to[i], j),
                         __builtin_amdgcn_readlane(len[i], j), it);
      }
      place -= n;
    }
  }
  return false;
}

// Waves a SIMD that the LDS places (4 waves a workgroup) leave room for.
constexpr int step_waves(int D, bool fp8, int rb, int nw) {
  if (nw == 8) return D == 64 ? 4 : 2;
  return D == 64 ? 4 : D == 128 ? (fp8 ? (rb == 1 ? 4 : 2) : 2) : (fp8 && rb == 1 ? 2 : 1);
}

// Columns of the merge at a time: all, or as few (32 at least) as fit the places' room.
constexpr int merge_turns(int D, int rows, int ring) {
  int turns = 1;
  while (D / turns >= 64 && rows * (D / turns + 4) * 4 > ring) turns *= 2;
  return turns;
}

// Places for K and for V a wave. With one, a load is issued as soon as its place is free and
// only if there is such a tile; with two always (of tiles behind the part nothing is
// read), so that as many are on their way at every wait. Two where LDS has room for
// them beside as many workgroups: E4M3 tiles of 32 rows (with the one resource a tile
// below, 64 trees of 16 over up to 4096 keys: 97 us for 103).
constexpr int step_places(int D, bool fp8, int rb, bool tree) { return tree && fp8 && rb == 2 && D >= 128 ? 2 : 1; }

// WHOLE (E4M3): a page holds a tile, which then takes one resource: 64 times 8 tokens of 4096,
// 8 heads of 64 and 32: 51 us for 58. (In bf16, of twice the loads, it makes no difference.)
template <int D, bool FP8, int RB, int NW, bool TREE, bool WHOLE>
__global__ __launch_bounds__(NW * 64, step_waves(D, FP8, RB, NW)) void attn_step_kernel(const AttnArgs a) {
  using St = Stage<D, FP8, 32, 16, true>;
  using G = Geo<D, FP8, true>;
  constexpr int kStage = 2 * St::kTile + 2 * St::kScale;     // K, V, their scales
  constexpr int kOps = 2 * St::kLoads + (FP8 ? WHOLE ? 1 : 2 : 0);  // loads of a K or V tile
  constexpr int R = step_places(D, FP8, RB, TREE);
  // the merge, of all columns or of half of them at a time, where that keeps it in the
  // room of the places (E4M3, heads of 128, 32 rows: 37 KB for 68, three workgroups a CU
  // for two)
  constexpr int kRows = 16 * RB, kRing = NW * kStage * R;
  constexpr int kTurns = D >= 128 ? merge_turns(D, NW * kRows, kRing) : 1;
  constexpr int kCols = D / kTurns, kOut = kCols + 4;  // columns at a time, floats of a row
  constexpr int kMerge = NW * kRows * kOut * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing > kMerge ? kRing : kMerge];
  __shared__ float wm[NW][kRows], wl[NW][kRows];
  __shared__ int last_flag;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int split = blockIdx.z;  // slowest: the splits without tiles come last
  Item it;
  // (heads fastest: with eight or sixteen the row tiles of one share an XCD's L2)
  const int h = blockIdx.x % a.kv_heads, row0 = blockIdx.x / a.kv_heads * a.part_rows;
  if (!(TREE && a.ordered ? item_by_length(a, blockIdx.y, h, it) : item_of(a, blockIdx.y, h, it)) || row0 >= it.rows)
    return;
  const int rows = min(it.rows - row0, a.part_rows);  // this workgroup's
  const Range rg = range_of<TREE>(a, it, row0, row0 + rows);
  int t0 = rg.lo / 32, t1 = (rg.hi + 31) / 32;
  int parts = 1;
  if (a.splits > 1) {
    int longest = 0;  // the batch's ranges of keys, in tiles
    float sum = 0.0f;
    for (int b = lane; b < a.B; b += 64) {
      const int n = a.q_start[b + 1] - a.q_start[b];
      int len = (int)min((int64_t)a.kv_len[b], (int64_t)a.cols << a.page_shift);
      if (a.window > 0) len = (int)min((int64_t)len, a.window + n);
      const int tiles = n > 0 && len > 0 ? len / 32 + 2 : 0;
      longest = max(longest, tiles);
      sum += (float)tiles * (float)max((n * a.group + a.part_rows - 1) / a.part_rows, 0);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      longest = max(longest, __shfl_xor(longest, o, kWave));
      sum += __shfl_xor(sum, o, kWave);
    }
    // (at least 1: a batch without any key has rows to write too)
    const int share =
        max(max((longest + a.splits - 1) / a.splits, 1), (int)(sum * (float)a.kv_heads * (1.0f / kPieces)));
    const int n = __builtin_amdgcn_readfirstlane((share + NW - 1) / NW * NW);
    parts = max((t1 - t0 + n - 1) / n, 1);
    if (split >= parts) return;
    t0 = t0 + split * n;
    t1 = min(t0 + n, t1);
  }
  uint8_t* mine = lds + wave * kStage * R;
  const uint32_t lk0 = lds_addr(mine);
  uint32_t place = 0;  // of the tile that is worked on, in bytes
  auto next_place = [&] { place = R == 1 || place == (R - 1) * kStage ? 0 : place + kStage; };
  const int hi = R > 1 ? min(rg.hi, 32 * t1) : rg.hi;
  constexpr int kScaleStep = WHOLE ? 64 : 256;  // from the scales of a tile's first 16 keys to the others'
  // Where tile t lies, and K (or V) rows of it with their scales. (By value: an array of
  // these would lie in memory. The rows of two pages are found for K and for V: kept, they
  // cost scalar registers, E4M3, heads of 128, pages of 16, four times 16 tokens of 512: 11.9
  // us for 11.4.)
  struct Tile {
    Rows16 rows;      // WHOLE
    int page0, page1;
  };
  auto rows_at = [&](int t, int page0, int page1) {
    Tile w;
    if (WHOLE) w.rows = rows_of<32>(a, it, t * 32, page0, hi);
    w.page0 = page0;
    w.page1 = page1;
    return w;
  };
  auto load = [&](int t, const Tile w, auto is_v, auto edge) {
    const uint32_t to = lk0 + place + (is_v ? St::kTile : 0);
    const uint32_t scales = lk0 + place + 2 * St::kTile + (is_v ? St::kScale : 0);
    const int skip = rg.lo - t * 32;
    if constexpr (WHOLE) {
      v4i rs = resource<G::kRow>(is_v ? a.v : a.k, w.rows), sc = resource<4>(is_v ? a.vs : a.ks, w.rows);
      settled(rs, sc);
      St::template rows32<is_v, edge>(rs, skip, to);
      St::template scale_rows32<edge>(sc, skip, scales);
    } else {
      auto half = [&](int page, int n) {
        const Rows16 x = rows_of(a, it, t * 32 + 16 * n, page, hi);
        v4i rs = resource<G::kRow>(is_v ? a.v : a.k, x);
        settled(rs);
        St::template rows<is_v, edge>(rs, skip - 16 * n, 16 * n, to);
        if constexpr (FP8) {
          v4i sc = resource<4>(is_v ? a.vs : a.ks, x);
          settled(sc);
          St::template scale_row<edge>(sc, skip - 16 * n, 16 * n, scales);
        }
      };
      half(w.page0, 0);
      half(w.page1, 1);
    }
  };
  constexpr std::integral_constant<bool, true> kYes;
  constexpr std::integral_constant<bool, false> kNo;
  auto pages = [&](int t, int (&page)[2]) {
    page[0] = page_of(a, it, t * 32);
    page[1] = WHOLE ? page[0] : page_of(a, it, t * 32 + 16);
  };
  int t = t0 + wave;
  int page[R][2], next[2];  // of the tiles in the places; of the next one to be loaded
  Tile w = {};  // the rows of the tile that is loaded next
#pragma unroll
  for (int i = 0; i < R; ++i) pages(t + i * NW, page[i]);
  if (t < t1) {
    w = rows_at(t, page[0][0], page[0][1]);
    load(t, w, kNo, kYes);
    load(t, w, kYes, kYes);
#pragma unroll
    for (int i = 1; i < R; ++i) {
      next_place();
      w = rows_at(t + i * NW, page[i][0], page[i][1]);
      load(t + i * NW, w, kNo, kNo);
      load(t + i * NW, w, kYes, kNo);
    }
    next_place();
  }
  pages(t + R * NW, next);
  v8bf q[RB][D / 32];
  int vlo[RB], vhi[RB];
  float m[RB], l[RB];
  v4f o[RB][D / 16];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = 16 * rb + r;
    vlo[rb] = row_lo<TREE>(a, it, row0 + row);
    vhi[rb] = row_hi<TREE>(a, it, row0 + row);
    m[rb] = -kInf;
    l[rb] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[rb][d] = v4f{};
    const uint16_t* src = q_row<D>(a, it, row0 + row);
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
      q[rb][u] = load_q8(a, src + (FP8 ? 64 * (u / 2) + 16 * g + 8 * (u % 2) : 32 * u + 8 * g));
  }
  for (; t < t1; t += NW) {
    const bool more = R > 1 || t + NW < t1;
    const uint32_t bad = (no_page(a, page[0][0]) ? 1u : 0u) | (no_page(a, page[0][1]) ? 2u : 0u);
    const int key = t * 32;
    const uint8_t* at = mine + place;
    dma_wait<(2 * R - 1) * kOps>();  // K has arrived, V and the other place may be under way
    v4f s[RB][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint8_t* base = at + (16 * b + r) * G::kRow;
      const int sw = G::k_swz(16 * b + r);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) s[rb][b] = v4f{};
#pragma unroll
      for (int u = 0; u < (FP8 ? D / 64 : D / 32); ++u) {
        const v4i x = *reinterpret_cast<const v4i*>(base + 16 * ((4 * u + g) ^ sw));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          if (FP8) {
            s[rb][b] = mfma_bf16(cvt_fp8x8(x[0], x[1]), q[rb][2 * u], s[rb][b]);
            s[rb][b] = mfma_bf16(cvt_fp8x8(x[2], x[3]), q[rb][2 * u + 1], s[rb][b]);
          } else {
            s[rb][b] = mfma_bf16(as_bf16(x), q[rb][u], s[rb][b]);
          }
        }
      }
    }
    if (FP8) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4f k = *reinterpret_cast<const v4f*>(at + 2 * St::kTile + kScaleStep * b + 16 * g);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[rb][b][i] *= k[i];
      }
    }
    lds_reads_done();
    if (more) {
      w = rows_at(t + R * NW, next[0], next[1]);
      load(t + R * NW, w, kNo, kNo);
    }
    if (bad != 0 || key + 32 > rg.all_hi || key < rg.all_lo) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const uint32_t tree = TREE ? tree_bits(a, it, mask_row(a, it, row0 + 16 * rb + r), key) >> (4 * g) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = key + 16 * (i / 4) + 4 * g + i % 4;
          bool see = vlo[rb] <= j && vhi[rb] > j && !((bad >> (i / 4)) & 1);
          if (TREE) see = see && ((tree >> (16 * (i / 4) + i % 4)) & 1);
          s[rb][i / 4][i % 4] = see ? s[rb][i / 4][i % 4] : -kInf;
        }
      }
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      // (each lane's own keys first: the row's maximum is needed only where it is raised.
      // The first maximum, of both score blocks, is the compiler's, which waits for their
      // products; max3's, which it would not wait for, all follow from it.)
      float mx = fmaxf(s[rb][0][0], s[rb][1][0]);
#pragma unroll
      for (int b = 0; b < 2; ++b) mx = max3(mx, s[rb][b][1], s[rb][b][2]);
      mx = max3(mx, s[rb][0][3], s[rb][1][3]);
      if (__any(mx * a.c > m[rb] + 8.0f)) {
        const float top = fmaxf(m[rb], groups_max(mx) * a.c);
        const float f = top == -kInf ? 0.0f : exp2_hw(m[rb] - top);
        m[rb] = top;
        l[rb] *= f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[rb][d][i] *= f;
      }
      const float base = m[rb] == -kInf ? 0.0f : m[rb];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = exp2_hw(fmaf(s[rb][i / 4][i % 4], a.c, -base));
        s[rb][i / 4][i % 4] = w;
        l[rb] += w;
      }
    }
    if (more)
      dma_wait<(2 * R - 1) * kOps>();  // V has arrived, the next K may be under way
    else
      dma_wait<0>();
    v8bf p[RB];
    v4f sv[2];
    if (FP8) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        sv[b] = *reinterpret_cast<const v4f*>(at + 2 * St::kTile + St::kScale + kScaleStep * b + 16 * g);
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      v4i w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = s[rb][i / 2][2 * (i % 2)], y = s[rb][i / 2][2 * (i % 2) + 1];
        if (FP8) {
          x *= sv[i / 2][2 * (i % 2)];
          y *= sv[i / 2][2 * (i % 2) + 1];
        }
        w[i] = (int)pack_bf16x2(x, y);  // one rounding of the weight, as in the chunk kernel
      }
      p[rb] = as_bf16(w);
    }
    const uint8_t* vt = at + St::kTile;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      v8bf v;
      if (FP8) {
        const int n = r >> 1;
        const int row = 4 * g + (n & 3) + 16 * (n >> 2);
        const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (QLIN_LDS v2i*)(vt + row * G::kRow + 16 * (d ^ G::v_swz(row)) + 8 * (lane & 1)));
        v = cvt_fp8x8(x[0], x[1]);
      } else {
        const int row = 4 * g + (r >> 2);
        const int chunk = 2 * d + ((lane & 3) >> 1);
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (QLIN_LDS v4s*)(vt + row * G::kRow + 16 * (chunk ^ G::v_swz(row)) + 8 * (lane & 1)));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (QLIN_LDS v4s*)(vt + (row + 16) * G::kRow + 16 * (chunk ^ G::v_swz(row + 16)) + 8 * (lane & 1)));
        v = __builtin_bit_cast(v8bf, (v8s){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) o[rb][d] = mfma_bf16(v, p[rb], o[rb][d]);
    }
    lds_reads_done();
    if (more) load(t + R * NW, w, kYes, kNo);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      page[i][0] = i + 1 < R ? page[(i + 1) % R][0] : next[0];
      page[i][1] = i + 1 < R ? page[(i + 1) % R][1] : next[1];
    }
    pages(t + (R + 1) * NW, next);
    next_place();
  }
  if (R > 1) dma_wait<0>();  // the merge takes the places
  // merge: every wave's rows on the common maximum, then summed over the waves
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    l[rb] = groups_sum(l[rb]);
    if (g == 0) wm[wave][16 * rb + r] = m[rb];
  }
  __syncthreads();
  float* all = reinterpret_cast<float*>(lds);
  float factor[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = 16 * rb + r;
    float top = -kInf;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, wm[w][row]);
    factor[rb] = m[rb] == -kInf ? (l[rb] == 0.0f ? 0.0f : 1.0f) : exp2_hw(m[rb] - top);
    if (row < rows && g == 0) wl[wave][row] = l[rb] * factor[rb];
  }
  auto put = [&](int turn) {  // this wave's rows, the turn's columns
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = 16 * rb + r;
      const float f = factor[rb];
      if (row < rows) {
        float* dst = all + (wave * kRows + row) * kOut + 4 * g;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
          if (d / (kCols / 16) == turn)
            *reinterpret_cast<v4f*>(dst + 16 * d - kCols * turn) =
                v4f{o[rb][d][0] * f, o[rb][d][1] * f, o[rb][d][2] * f, o[rb][d][3] * f};
      }
    }
  };
  const int64_t heads = (int64_t)a.kv_heads * a.group;
  auto finish = [&](int row, int c4, const v4f& x, float mm, float ll) {
    const int64_t tok = it.q0 + (row0 + row) / a.group;
    const int qh = it.h * a.group + (row0 + row) % a.group;
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    *reinterpret_cast<uint2*>(a.out + tok * a.ldo + (int64_t)qh * D + c4) =
        make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
    if (a.lse && c4 == 0) a.lse[tok * heads + qh] = ll == 0.0f ? -kInf : (mm + log2f(ll)) * kLn2;
  };
  // Parts and counter move past the XCDs' own L2 caches (sc1, device scope): a
  // part is visible everywhere once its store has completed, so the wait before
  // the counter orders them without flushing a cache.
  constexpr int kSc1 = 16;
  const int wg = it.b * gridDim.x + blockIdx.x;
  const __amdgpu_buffer_rsrc_t ro = __builtin_amdgcn_make_buffer_rsrc(
      a.po + (int64_t)wg * a.splits * a.part_rows * D, (short)0, a.splits * a.part_rows * D * 4, 0x00020000);
  const __amdgpu_buffer_rsrc_t rm = __builtin_amdgcn_make_buffer_rsrc(
      a.pml + (int64_t)wg * a.splits * a.part_rows * 2, (short)0, a.splits * a.part_rows * 8, 0x00020000);
#pragma unroll
  for (int turn = 0; turn < kTurns; ++turn) {
    if (turn) __syncthreads();  // the last turn's columns have been read
    put(turn);
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (kCols / 4); i += NW * 64) {
      const int row = i / (kCols / 4), c = i % (kCols / 4) * 4, c4 = c + kCols * turn;
      float mm = -kInf, ll = 0.0f;
      v4f x = {};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        mm = fmaxf(mm, wm[w][row]);
        ll += wl[w][row];
        const v4f y = *reinterpret_cast<const v4f*>(all + (w * kRows + row) * kOut + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += y[j];
      }
      if (parts == 1) {
        finish(row, c4, x, mm, ll);
      } else {
        const int at = split * a.part_rows + row;
        if (c4 == 0) {
          const v2i y = {(int)__float_as_uint(mm), (int)__float_as_uint(ll)};
          __builtin_amdgcn_raw_buffer_store_b64(y, rm, at * 8, 0, kSc1);
        }
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, x), ro, (at * D + c4) * 4, 0, kSc1);
      }
    }
  }
  if (parts == 1) return;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0)
    last_flag = __hip_atomic_fetch_add(&a.arrived[wg], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (uint32_t)(parts - 1);
  __syncthreads();
  if (!last_flag) return;
  // join: the parts' maxima and sums by all threads at once, then the rows, eight
  // parts' loads at a time
  v2i* ml = reinterpret_cast<v2i*>(lds);
  for (int i = threadIdx.x; i < parts * a.part_rows; i += NW * 64)
    ml[i] = __builtin_amdgcn_raw_buffer_load_b64(rm, i * 8, 0, kSc1);
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += NW * 64) {
    const int row = i / (D / 4), c4 = i % (D / 4) * 4;
    float mm = -kInf, ll = 0.0f;
    for (int s = 0; s < parts; ++s) mm = fmaxf(mm, __uint_as_float((uint32_t)ml[s * a.part_rows + row][0]));
    v4f x = {};
    for (int s0 = 0; s0 < parts; s0 += 8) {
      v4i y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b)
        y[b] = __builtin_amdgcn_raw_buffer_load_b128(
            ro, ((min(s0 + b, parts - 1) * a.part_rows + row) * D + c4) * 4, 0, kSc1);
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (s0 + b < parts) {
          const v2i z = ml[(s0 + b) * a.part_rows + row];
          const float ms = __uint_as_float((uint32_t)z[0]);
          const float w = ms == -kInf ? 1.0f : exp2_hw(ms - mm);
          ll = fmaf(w, __uint_as_float((uint32_t)z[1]), ll);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = fmaf(w, __builtin_bit_cast(v4f, y[b])[j], x[j]);
        }
      }
    }
    finish(row, c4, x, mm, ll);
  }
  if (threadIdx.x == 0) __hip_atomic_store(&a.arrived[wg], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- join
// The parts of the key axis to one result: four values of a (token, query head) a
// thread. Everything that a row needs is loaded at once, before it is known which
// parts have a key (what a part without one holds is not used): bound by that
// one round trip, then by the parts' bytes.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  constexpr int kRow = D / 4, kRows = 64 / kRow;  // threads of a row, rows of a wave
  const int lane = threadIdx.x & 63;
  const int64_t heads = (int64_t)a.kv_heads * a.group, all = a.T * heads;
  const int64_t at0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kRows;  // the wave's first row
  if (at0 >= all) return;
  const int64_t mine = at0 + lane / kRow, at = min(mine, all - 1);
  const int c = 4 * (lane % kRow);
  // rows of no sequence have no parts (and are left as they are)
  bool in = false;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = min(b0 + lane, a.B - 1);
    const int from = a.q_start[b], to = a.q_start[b + 1];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t t = (at0 + i) / heads;
      const bool here = __any(from >= 0 && from <= t && t < to && to <= a.T);
      in |= here && lane / kRow == i;
    }
  }
  float m = -kInf, l = 0.0f;
  v4f o = {};
  for (int s0 = 0; s0 < a.splits; s0 += 4) {
    float ms[4], ls[4];
    v4f x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t p = min(s0 + i, a.splits - 1) * all + at;
      const float2 z = *reinterpret_cast<const float2*>(a.pml + 2 * p);
      ms[i] = z.x;
      ls[i] = z.y;
      x[i] = *reinterpret_cast<const v4f*>(a.po + p * D + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s0 + i >= a.splits || (ms[i] == -kInf && ls[i] == 0.0f)) continue;  // no such part, or one without a key
      const float top = fmaxf(m, ms[i]);
      const float f = m == -kInf ? 1.0f : exp2_hw(m - top), w = ms[i] == -kInf ? 1.0f : exp2_hw(ms[i] - top);
      m = top;
      l = l * f + ls[i] * w;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = o[j] * f + x[i][j] * w;
    }
  }
  if (!in || mine >= all) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + at / heads * a.ldo + at % heads * D + c) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && c == 0) a.lse[at] = l == 0.0f ? -kInf : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- host
struct Plan {
  bool step;
  int splits;
  int64_t tiles;             // chunk: workgroups for the rows, at most
  int part_rows, row_tiles;  // step
  bool wide;                 // step: eight waves
  size_t parts;              // rows of parts in the workspace
};

// Arrival counters at the start of the workspace, as the GEMMs' split-K.
constexpr size_t kAttnCounterBytes = kGemmCounterBytes;
// Rows of a chunk's workgroup, and its workgroups a CU.
int64_t chunk_rows(const qlin_kv_cache& c) { return c.fmt == QLIN_KV_E4M3 ? 256 : 128; }
int64_t chunk_room(const qlin_kv_cache& c) { return (c.head_dim == 64 ? 2 : 1) * (c.fmt == QLIN_KV_E4M3 ? 1 : 2); }
constexpr int kCus = 256;

Plan step_plan(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t rows, int64_t keys) {
  Plan p = {};
  p.step = true;
  p.part_rows = (int)std::min<int64_t>(32, rows);
  p.row_tiles = (int)((rows + 31) / 32);
  const int64_t wgs = batch.batch * cache.kv_heads * p.row_tiles;
  // A joined part costs about 6 us (its store has to be visible, then counted,
  // then read). With 64 E4M3 sequences of up to 1536 tokens (512 workgroups,
  // heads of 128) two parts took 37 us and none 30.5; with eight of 65536
  // bf16 (64 workgroups) 8 parts took 352 us, 4 357, 16 379. So: one workgroup a
  // CU; where sequences may be long enough not to notice the join, up to the
  // most that a ragged batch needs. (`keys` is what the page table reaches: the same
  // 64 sequences cost 30.7 us with a table of 1536 tokens and 34.6, with the longer ones
  // in two parts, with any of 4096 or more.)
  const int64_t most = keys >= 4096 ? 2048 : kCus;
  const int64_t piece = p.row_tiles > 1 ? 512 : 128;  // keys of a part, at least (more rows, a dearer join)
  // (64 parts at most: one workgroup reads them all)
  p.splits = (int)std::max<int64_t>(1, std::min({(most + wgs - 1) / wgs, (keys + piece - 1) / piece, (int64_t)64}));
  // The last workgroup reads all parts, a part's keys and its rows cost about the same
  // time at keys * 32 = parts^2 * rows * head_dim: 2 sequences of 50 rows, heads of 128,
  // 28454 keys: 36 us, 54 with 64 parts; 16 tokens of 32 heads, 32768 keys: 38 and 47.
  const int even = (int)std::sqrt(32.0 * (double)keys / (double)(p.part_rows * cache.head_dim));
  p.splits = std::max(1, std::min(p.splits, even));
  if (wgs >= most) p.splits = 1;
  p.parts = p.splits <= 1 ? 0 : (size_t)p.splits * wgs * p.part_rows;
  return p;
}

// Parts of a tree's key axis: of 256 keys or more, as many as fill the device; of long
// tables, whose sequences differ most, more. (More keys never mean fewer parts.)
int tree_splits(bool e4m3, int64_t keys, int64_t wgs) {
  if (keys < 2048) return 1;
  int64_t n = (keys >= 8192 && e4m3 ? 512 : 256) / wgs;
  if (keys >= 8192 && wgs <= 512) n = std::max<int64_t>(n, e4m3 ? keys / 4096 : 2);
  return (int)std::max<int64_t>(1, std::min({(int64_t)16, keys / 256, n}));
}

// The same for trees, whose calls have some 16 to 256 rows a sequence and head: workgroups
// of 16 or 32 rows, of four waves or (the tiles of a part taken by twice as many at once)
// eight. A workgroup of eight costs less than a second part, whose join takes as long as a
// thousand keys. us, 32 + 8 heads of 128, all in one run, calls behind each other in a graph:
//   16 rows and eight waves while all run at once and few bytes are read twice: a tree of 8,
//     1024 keys: 10.0 (four waves 11.6, 32 rows 13.6); 4096 keys in 16 parts 14.4 (17.6,
//     17.9). E4M3, eight trees of 32, 4096 keys: 32.5 (34.6; 32 rows 32.3);
//   32 rows beyond: a tree of 32, 16384 keys 29.5 (16 rows 33.8); eight trees of 32, 4096
//     keys 32.9 (16 rows 36.2, four waves 42.1); 64 trees of 16, four waves: 139 (eight 152,
//     16 rows 189). E4M3 beyond 2^30 bytes: three trees of 64, 65536 keys 187 (16 rows 227),
//     16 of 16, 16384 keys 106 (124), but eight of 32, 16384 keys 89 (75): such shapes
//     are the few that the limit on bytes decides wrong;
//   short tables: 16 rows, four waves: eight trees of 32, 256 keys: 9.0 (32 rows 9.9); E4M3,
//     64 of them, 1024 keys: 59.5 (64.3).
Plan tree_step_plan(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t rows, int64_t keys) {
  Plan p = {};
  p.step = true;
  const bool e4m3 = cache.fmt == QLIN_KV_E4M3;
  const int64_t D = cache.head_dim, heads = batch.batch * cache.kv_heads;
  const int64_t few = heads * ((rows + 15) / 16), many = heads * ((rows + 31) / 32);  // workgroups of 16, 32 rows
  const int64_t at_once = e4m3 && D < 256 ? 512 : 256;                                // of eight waves
  const double reread = (double)few * keys * D * (e4m3 ? 2 : 4);                      // bytes, by 16 rows each
  bool narrow = rows <= 16 || (e4m3 && D == 256);
  if (few <= at_once && reread < (e4m3 ? 0x1p30 : 0x1p29)) {
    narrow = p.wide = true;
  } else if (keys <= 1024 && (e4m3 ? D > 64 : D == 128 && few <= 512)) {
    narrow = true;
  } else {
    const int64_t wgs = narrow ? few : many;
    p.wide = wgs <= (keys >= 4096 ? 512 : 256);
  }
  if (D == 256 && !(e4m3 && narrow)) p.wide = false;  // (their places would not fit LDS)
  const int64_t tile = narrow ? 16 : 32, wgs = narrow ? few : many;
  p.part_rows = (int)std::min(tile, rows);
  p.row_tiles = (int)((rows + tile - 1) / tile);
  p.splits = tree_splits(e4m3, keys, wgs);
  p.parts = p.splits <= 1 ? 0 : (size_t)p.splits * wgs * p.part_rows;
  return p;
}

Plan chunk_plan(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t rows, int64_t group,
                int64_t keys) {
  Plan p = {};
  const int64_t bm = chunk_rows(cache), room = chunk_room(cache) * kCus;
  p.tiles = std::min(T * group / bm + batch.batch, (rows + bm - 1) / bm * batch.batch);
  const int64_t wgs = p.tiles * cache.kv_heads;
  // As many equal parts as fill the device once. bf16, 32 + 8 heads of 128: 512 tokens of
  // 4096 with 4 parts 49 us, 2 55, 8 (more workgroups than fit) 63; 1024 of 1024: 2 parts 34,
  // none 26. (Parts by each sequence's length instead: no gain over ragged batches, and
  // 1024 of 4096 90 us for 77.)
  p.splits = keys <= 2048 ? 1 : (int)std::max<int64_t>(1, std::min(room / wgs, keys / 512));
  p.parts = p.splits <= 1 ? 0 : (size_t)p.splits * T * cache.kv_heads * group;
  return p;
}

// Workgroups of 32 rows (a step's kernel) or of 128 (E4M3: 256; a chunk's). The chunk's
// do about twice the work a second once they fill the device, but a call of few rows
// leaves most of their rows or most CUs idle. 32 + 8 heads of 128, us of 32 rows and of
// 128 in bf16:
//   up to 64 rows a sequence: 200 of 16 tokens (16 + 4 heads) of up to 1024: 79 and 91;
//   more, at most 1024 workgroups of 32 rows and these times the keys below 2^20: 512
//     tokens of 512: 13 and 17; four chunks of 64 of 4000: 27 and 28;
//   the others: 1024 of 1024: 29 and 26; 512 of 4096: 52 and 49; 256 of 8192: 57 and 50;
//     8 of 32 of 4096: 41 and 31; 2048 of 2048: 74 and 51.
// Heads of 64 have four workgroups of 32 rows on a CU, twice as many: 1024 of 1024: 17 and
// 20, 2048 of 2048: 41 and 35. E4M3, 32 and 256 rows, up to 128 rows or below 2^21: 14 of 33
// of up to 3203 (16 + 4 heads): 38 and 46; 1024 of 1024: 31 and 36; 1024 of 4096: 105 and 84.
// Here: the most keys for which 32 rows are taken (0: never).
int64_t few_rows_keys(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t rows,
                      int64_t group) {
  const bool e4m3 = cache.fmt == QLIN_KV_E4M3;
  if (rows <= (e4m3 ? 128 : 64)) return INT64_MAX;
  const int64_t room = cache.head_dim == 64 ? 2 : 1;
  const int64_t tiles = (rows + 31) / 32 * batch.batch;  // (the grid: also those that a ragged batch leaves empty)
  const int64_t wgs = std::min(tiles, T * group / 32 + batch.batch) * cache.kv_heads;
  if (wgs > 1024 * room || tiles * cache.kv_heads > 8192) return 0;
  return ((room << (e4m3 ? 21 : 20)) - 1) / wgs;
}

// Whether a tree's call takes these workgroups: where the others do, and up to 256 rows
// also, in E4M3, over long tables (64 trees of 64, 4096 keys: 263 us, in workgroups of 256
// rows 301; eight, 16384 keys: 113 and 154), in bf16 with few of them (a tree of 32, 65536
// keys: 69 and 97; of 64, 16384 keys: 38 and 44). bf16 heads of 256 leave them sooner (64
// trees of 32, 1024 keys: 95 and 66; 16, 4096 keys: 201 and 180).
bool tree_steps(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t rows, int64_t group,
                int64_t keys) {
  const int64_t many = batch.batch * cache.kv_heads * ((rows + 31) / 32);
  const bool e4m3 = cache.fmt == QLIN_KV_E4M3;
  if (!e4m3 && cache.head_dim == 256 && rows > 32 && (many > 256 || many * keys > 1 << 18)) return false;
  if (keys <= few_rows_keys(cache, batch, T, rows, group)) return true;
  if (rows > 256) return false;
  if (e4m3) return keys > 1024 && (batch.batch > 1 || keys <= 32768 || cache.head_dim == 64);
  return many <= 32 || (many <= 64 && keys <= 16384);
}

Plan plan_of(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t q_heads, int64_t window,
             bool tree) {
  const int64_t group = q_heads / cache.kv_heads, rows = std::min(batch.max_q, T) * group;
  int64_t keys = batch.table_cols * cache.page_size;
  if (window > 0) keys = std::min(keys, std::min(window, keys) + batch.max_q);
  if (tree)
    return tree_steps(cache, batch, T, rows, group, keys) ? tree_step_plan(cache, batch, rows, keys)
                                                          : chunk_plan(cache, batch, T, rows, group, keys);
  return keys <= few_rows_keys(cache, batch, T, rows, group) ? step_plan(cache, batch, rows, keys)
                                                             : chunk_plan(cache, batch, T, rows, group, keys);
}

template <int D, bool FP8, bool TREE, bool WHOLE>
void launch_step(const AttnArgs& a, const Plan& p, hipStream_t st) {
  const dim3 grid(a.kv_heads * p.row_tiles, a.B, p.splits);
  if constexpr (TREE && (D < 256 || FP8)) {
    if (p.part_rows <= 16 && p.wide) {
      attn_step_kernel<D, FP8, 1, 8, TREE, WHOLE><<<grid, 512, 0, st>>>(a);
      return;
    }
  }
  if constexpr (TREE && D < 256) {
    if (p.part_rows > 16 && p.wide) {
      attn_step_kernel<D, FP8, 2, 8, TREE, WHOLE><<<grid, 512, 0, st>>>(a);
      return;
    }
  }
  if constexpr (!(TREE && FP8 && D == 256)) {  // (its trees have 16 rows a workgroup)
    if (p.part_rows > 16) {
      attn_step_kernel<D, FP8, 2, 4, TREE, WHOLE><<<grid, 256, 0, st>>>(a);
      return;
    }
  }
  attn_step_kernel<D, FP8, 1, 4, TREE, WHOLE><<<grid, 256, 0, st>>>(a);
}

template <int D, bool FP8, bool TREE>
void launch_parts(const AttnArgs& a, const Plan& p, hipStream_t st) {
  if (p.step) {
    FP8 && a.page_shift >= 5 ? launch_step<D, FP8, TREE, FP8>(a, p, st) : launch_step<D, FP8, TREE, false>(a, p, st);
  } else {
    const int64_t items = p.tiles * a.kv_heads * p.splits;
    const unsigned grid = (unsigned)((items + 7) / 8 * 8);
    constexpr int TK = D == 256 ? 32 : 64;
    if constexpr (FP8)
      attn_chunk_e4m3_kernel<D, TK, TREE><<<grid, 512, 0, st>>>(a);
    else
      attn_chunk_kernel<D, TK, TREE><<<grid, 256, 0, st>>>(a);
    if (p.splits > 1) {
      const int64_t rows = a.T * a.kv_heads * a.group, wg = 1024 / D;  // rows of a workgroup
      attn_join_kernel<D><<<(unsigned)((rows + wg - 1) / wg), 256, 0, st>>>(a);
    }
  }
}

template <int D, bool FP8>
void launch_heads(const AttnArgs& a, const Plan& p, hipStream_t st) {
  a.mask ? launch_parts<D, FP8, true>(a, p, st) : launch_parts<D, FP8, false>(a, p, st);
}

}  // namespace

bool attn_grid_ok(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t q_heads) {
  // (with one part: calls of more have at most chunk_room * 256 workgroups)
  if (std::min(batch.max_q, T) * (q_heads / cache.kv_heads) <= 64) return true;
  const int64_t wgs = T * q_heads / chunk_rows(cache) + batch.batch * cache.kv_heads;
  return (wgs + 7) / 8 * 8 * (cache.fmt == QLIN_KV_E4M3 ? 512 : 256) <= 0xFFFFFFFF;
}

static size_t parts_bytes(size_t parts, int64_t head_dim) {
  return parts == 0 ? 0 : kAttnCounterBytes + round_up(parts * head_dim * 4, 256) + round_up(parts * 8, 256);
}

size_t attn_workspace_bytes(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t q_heads) {
  // Enough for a call with any window: a window lowers the keys, which may also turn
  // a chunk into workgroups of 32 rows (either plan's parts only fall with the keys).
  Plan p = plan_of(cache, batch, T, q_heads, 0, false);
  if (!p.step) {
    const int64_t group = q_heads / cache.kv_heads, rows = std::min(batch.max_q, T) * group;
    p.parts = std::max(p.parts, step_plan(cache, batch, rows, few_rows_keys(cache, batch, T, rows, group)).parts);
  }
  return parts_bytes(p.parts, cache.head_dim);
}

size_t attn_tree_workspace_bytes(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t q_heads) {
  // For any window, as above: of fewer keys each kind of workgroup has as many parts or
  // fewer, but another kind may be taken, so the largest of all.
  const int64_t group = q_heads / cache.kv_heads, rows = std::min(batch.max_q, T) * group;
  const int64_t keys = batch.table_cols * cache.page_size, heads = batch.batch * cache.kv_heads;
  size_t parts = chunk_plan(cache, batch, T, rows, group, keys).parts;
  for (const int64_t tile : {16, 32}) {
    const int64_t wgs = heads * ((rows + tile - 1) / tile);
    const int64_t splits = tree_splits(cache.fmt == QLIN_KV_E4M3, keys, wgs);
    if (splits > 1) parts = std::max(parts, (size_t)(splits * wgs * std::min(tile, rows)));
  }
  return parts_bytes(parts, cache.head_dim);
}

void attn_plan(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, int64_t q_heads, int64_t window,
               bool tree, int64_t out[3]) {
  const Plan p = plan_of(cache, batch, T, q_heads, window, tree);
  out[0] = p.step ? (tree && p.part_rows <= 16 ? 16 : 32) : chunk_rows(cache);
  out[1] = p.splits;
  out[2] = (int64_t)parts_bytes(p.parts, cache.head_dim);
}

int launch_attn(const qlin_kv_cache& cache, const qlin_kv_batch& batch, int64_t T, const uint16_t* q, int64_t ldq,
                int64_t q_heads, float scale, int causal, int64_t window, const qlin_tree* tree, uint16_t* out,
                int64_t ldo, float* lse, void* ws, size_t ws_bytes, hipStream_t st) {
  const Plan p = plan_of(cache, batch, T, q_heads, window, tree != nullptr);
  const size_t used = parts_bytes(p.parts, cache.head_dim);
  if (used > ws_bytes || (used && !ws)) return QLIN_ERR_WORKSPACE;
  AttnArgs a = {};
  a.k = (const uint8_t*)cache.k;
  a.v = (const uint8_t*)cache.v;
  a.ks = cache.k_scale;
  a.vs = cache.v_scale;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_start = batch.q_start;
  a.kv_len = batch.kv_len;
  a.table = batch.page_table;
  a.ldq = ldq;
  a.ldo = ldo;
  a.pages = (int)cache.pages;
  a.T = T;
  a.window = std::min<int64_t>(window, (int64_t)1 << 32);  // (more is all keys; sums of it must not overflow)
  a.B = (int)batch.batch;
  a.cols = (int)batch.table_cols;
  a.page_shift = __builtin_ctzll((unsigned long long)cache.page_size);
  a.kv_heads = (int)cache.kv_heads;
  a.group = (int)(q_heads / cache.kv_heads);
  a.causal = causal;
  a.splits = p.splits;
  a.part_rows = p.part_rows;
  a.row_tiles = p.row_tiles;
  a.tiles = (int)p.tiles;
  a.ordered = p.step && a.B <= 256 && (int64_t)a.kv_heads * p.row_tiles * a.B > 512;
  a.negate = scale < 0.0f;
  // a scale of 0 must keep masked scores at -inf (0 * -inf is NaN): the smallest factor,
  // 2^-149, gives every finite score a weight within 2^-21 of 1. (Factors below fp32's
  // normal range are off by at most 2^-150, which moves no exponent by more than 2^-22.)
  a.c = std::max(attn_factor(scale), std::numeric_limits<float>::denorm_min());
  if (p.splits > 1) {
    a.arrived = (uint32_t*)ws;
    a.po = (float*)((uint8_t*)ws + kAttnCounterBytes);
    a.pml = (float*)((uint8_t*)a.po + round_up(p.parts * cache.head_dim * 4, 256));
  }
  if (tree) {
    a.mask = (const uint32_t*)tree->mask;
    a.positions = tree->positions;
    a.words = (int)(2 * tree->words);
  }
  const bool f8 = cache.fmt == QLIN_KV_E4M3;
  switch (cache.head_dim) {
    case 64: f8 ? launch_heads<64, true>(a, p, st) : launch_heads<64, false>(a, p, st); break;
    case 128: f8 ? launch_heads<128, true>(a, p, st) : launch_heads<128, false>(a, p, st); break;
    default: f8 ? launch_heads<256, true>(a, p, st) : launch_heads<256, false>(a, p, st); break;
  }
  return launch_status();
}

}  // namespace qlin
