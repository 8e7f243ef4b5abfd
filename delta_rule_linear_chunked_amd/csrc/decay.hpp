// Decayed linear attention (a scalar decay for each head): parameter block, launch plan and the
// device building blocks that its forward and backward kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace dr {

constexpr int DCH = 64;  // tokens per chunk

// Pieces of `unit` tokens that n tokens take, n + unit past 32 bits included.
__host__ __device__ constexpr int pieces(int n, int unit) { return n > 0 ? (n - 1) / unit + 1 : 0; }
static_assert(pieces(INT32_MAX, 1 << 21) == 1024 && pieces(INT32_MAX, INT32_MAX) == 1 && pieces(64, 64) == 1 &&
              pieces(65, 64) == 2 && pieces(0, 64) == 0, "whole and ragged lengths");

// Sequences are cut into segments of `seg` tokens (a multiple of 64; one segment when that fills the
// chip): a slot is one segment of one sequence. Fixed length: slot n * nseg + j. Packed: the plan pass
// writes the table.
struct DecayParams {
  const void* q;         // [B, T, Hk, d_k]
  const void* k;
  const void* v;         // [B, T, H, d_v]
  const float* alpha;    // [B, T, H], or [H] when !a_tok
  const float* S0;       // initial states (may be null)
  const int32_t* cu;     // packed offsets; past the plan pass its clamped copy
  float* o;              // may be null
  float* S;              // final states (may be null); step: states in and out
  int64_t T;             // tokens per batch row
  int64_t q_ts, q_bs, k_ts, k_bs, v_ts, v_bs;  // element strides (token, batch row)
  int32_t H, Hk, DK, DV;
  int32_t a_tok;
  int32_t nseq;
  int32_t seg;           // tokens per segment
  int32_t nseg;          // fixed length: segments per sequence
  int32_t slots;         // slots (packed: an upper bound)
  int32_t grid;          // logical workgroups of the launch
  int32_t ncb;           // value-column blocks of the launch
  const int32_t* sidx;   // slot of each sequence in the state buffers (null: row n)
  int64_t nslots;
  float* snap;           // states after every snap_chunks chunks (may be null)
  int32_t snap_chunks;
  // packed: written by the plan pass
  int32_t* cu_ok;        // [nseq + 1] offsets clamped to [0, T] and non-decreasing
  int32_t* slot_seq;     // [slots] sequence of the slot (-1: unused)
  int32_t* slot_first;   // [nseq + 1] first slot of each sequence
  int32_t* snap_first;   // [nseq] first snapshot row of each sequence
  // segments: each slot's own contribution to the state behind it, then the state at its start
  float* part;           // [slots, H, d_k, d_v]
  double* gpart;         // [slots, H] product of the slot's decays
  // backward
  const float* dO;       // [B, T, H, d_v]
  const float* dST;      // may be null
  float* cs;             // [chunk slots, H, d_k, d_v] state at each chunk's start
  float* ds;             // [chunk slots, H, d_k, d_v] state gradient at each chunk's end
  float* rpart;          // segments of the reverse pass, as part / gpart
  double* rgpart;
  int32_t* chunk_seq;    // packed: [cslots] sequence of the chunk slot (-1: unused)
  int32_t* chunk_first;  // packed: [nseq + 1]
  int32_t cslots;
  int32_t bwd_chunk;     // tokens per chunk slot
  float* dq;             // [B, T, Hk, d_k] or, with shared heads, per-head partial sums [B, T, H, d_k]
  float* dk;
  float* dv;
  float* dalpha;         // [B, T, H]
  float* dS0;
  float* pq;             // shared heads: partial sums [B, T, H, d_k]
  float* pk;
  float* head_da;        // one decay per head: its gradient [H] (dalpha is then a workspace)
  int32_t dq_heads;      // heads of dq and dk as the gradient kernel writes them
  int32_t nbatch;        // batch rows
};

// What the host decides for a call.
struct DecayPlan {
  int ct;              // column tiles of 16 per workgroup of the main pass (1, 2, 4 or 8)
  int64_t seg;         // tokens per segment
  int64_t nseg;        // fixed length: segments per sequence; packed: more than 1 if any may have more
  int64_t slots;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// The fp32 values x as three bf16 terms, each the remainder rounded to nearest: the sum is x to 2^-26, so an
// MFMA over the three terms against a bf16 operand is an fp32-grade product at three bf16 rates (the fp32
// MFMA runs at a sixteenth of one). Magnitudes from about 3.39e38 up round to infinity.
struct Tri {
  bf16x8 t[3];
};
__device__ __forceinline__ Tri split3(const float (&x)[8]) {
  uint32_t w[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      w[t][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
      if (t < 2) {
        a -= __builtin_bit_cast(float, w[t][j] << 16);
        b -= __builtin_bit_cast(float, w[t][j] & 0xffff0000u);
      }
    }
  }
  Tri r;
#pragma unroll
  for (int t = 0; t < 3; ++t) r.t[t] = __builtin_bit_cast(bf16x8, w[t]);
  return r;
}
// Four values' terms to LDS, `plane` bytes apart.
__device__ __forceinline__ void split_store4(unsigned char* at, int plane, const f32x4& v) {
  float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint2 w;
    w.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2));
    w.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2], x[3]}, bf16x2));
    *reinterpret_cast<uint2*>(at + t * plane) = w;
    if (t < 2) {
      x[0] -= __builtin_bit_cast(float, w.x << 16);
      x[1] -= __builtin_bit_cast(float, w.x & 0xffff0000u);
      x[2] -= __builtin_bit_cast(float, w.y << 16);
      x[3] -= __builtin_bit_cast(float, w.y & 0xffff0000u);
    }
  }
}

// Operand of one 32-deep slice: NP bf16 terms (1: bf16 data as they are, 3: fp32 data).
template <int NP>
struct Op {
  bf16x8 t[NP];
};
// acc += A B over the term pairs that reach fp32's significand (p + q <= 2), smallest first.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const bf16x8 (&a)[NA], const bf16x8 (&b)[NB]) {
#pragma unroll
  for (int sum = NA + NB - 2 < 2 ? NA + NB - 2 : 2; sum >= 0; --sum)
#pragma unroll
    for (int p = 0; p < NA; ++p)
#pragma unroll
      for (int q = 0; q < NB; ++q)
        if (p + q == sum) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], b[q], acc, 0, 0, 0);
}

// acc[i] += A B[i] for several i, the terms outermost: an accumulator's next MFMA then follows the others' instead
// of waiting for its own result (32 cycles, twice an MFMA's issue time).
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_rows(f32x4 (&acc)[N], const bf16x8 (&a)[NA], const bf16x8 (&b)[N][NB]) {
#pragma unroll
  for (int sum = NA + NB - 2 < 2 ? NA + NB - 2 : 2; sum >= 0; --sum)
#pragma unroll
    for (int p = 0; p < NA; ++p)
#pragma unroll
      for (int q = 0; q < NB; ++q)
        if (p + q == sum) {
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], b[i][q], acc[i], 0, 0, 0);
        }
}

// Nothing moves across (the scheduler otherwise sinks every LDS read to its use, and each then waits in full)
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// LDS tile of token rows x W bf16 channels (W 32, 64 or 128), 16-byte pieces permuted within a row so that both
// kinds of read are free of bank conflicts: a fragment along the channels (16 rows, one piece each; the
// hardware serves rows 0-3 and 12-15 of one piece together with rows 4-11 of its neighbour) and a
// transposing read (4 consecutive rows, 4 pieces of 8 bytes each). Measured per read and CU: 4.9 and 4.2 cycles, as
// for linear addresses; with the row number as the permutation 4.9 and 8.1, with no regard to the pairing 8.2 and 4.2.
template <int W>
__device__ __forceinline__ int swz(int row, int piece) {
  constexpr int CPR = W / 8;
  const int x = (row >> 2) & 3, h = ((x ^ (x >> 1)) & 1) << 1 | x >> 1;  // 0, 2, 3, 1
  if constexpr (CPR == 16) return row * 16 + (piece ^ (((row & 3) << 2) | h));
  if constexpr (CPR == 8) return row * 8 + (piece ^ ((((row >> 1) & 1) << 2) | h));
  return row * 4 + (piece ^ h);
}

// Fragment with token rows on the lanes: row row0 + l % 16 (row0 a multiple of 16), channels 32 u + 8 (l / 16) .. + 7.
// (The address is one lane term, an exclusive or with 64 u and constants: spelled out because the compiler
// otherwise keeps an address register for every fragment of a loop, and spills.)
template <int W>
__device__ __forceinline__ bf16x8 frag_rows(const unsigned char* tile, int row0, int u, int lane) {
  const int at = (16 * swz<W>(lane & 15, lane >> 4)) ^ (64 * u);
  return *reinterpret_cast<const bf16x8*>(tile + at + row0 * W * 2);
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
  union {
    s16x4 h[2];
    bf16x8 v;
  } x;
  x.h[0] = a;
  x.h[1] = b;
  return x.v;
}
// Fragment with channels on the lanes and tokens along the product: tokens 32 u + 16 a + 4 (l / 16) + b
// at item 4 a + b. ds_read_b64_tr_b16 transposes a 4 x 16 block per 16 lanes: lane p names 4 consecutive
// elements of row p / 4, columns 4 (p % 4) ..; it receives column l of the four rows. Lane l's channel of
// channel tile 2 w + e is 32 w + 8 ((l % 16) / 4) + 4 e + l % 4: the accumulators of a product with such
// rows hold, in a lane, channels 32 w + 8 (l / 16) + 4 e + i, and the two tiles e = 0, 1 together are the
// eight consecutive channels of a fragment along the channels.
template <int W>
__device__ __forceinline__ bf16x8 frag_chan(const unsigned char* tile, int w, int e, int u, int lane) {
  const int at = (16 * swz<W>(4 * (lane >> 4) + ((lane >> 2) & 3), lane & 3)) ^ (64 * w);
  const unsigned char* p = tile + at + 32 * u * W * 2 + 8 * e;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * W * 2));
  return join(a, b);
}
// The same for a tile with rows of CW elements in order, no swizzle: lane l's column is n0 + l % 16.
template <int CW>
__device__ __forceinline__ bf16x8 frag_cols(const unsigned char* tile, int n0, int u, int lane) {
  const int g = lane >> 4, p = lane & 15;
  const unsigned char* at = tile + ((32 * u + 4 * g + (p >> 2)) * CW + n0 + 4 * (p & 3)) * 2;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * CW * 2));
  return join(a, b);
}

// ---------------------------------------------------------------------------
// Products of a chunk's decays. ratio(r, s) = a_{s+1} ... a_r is formed as a product of products, never
// as a quotient or from logarithms: zero and negative decays are exact and nothing overflows that the
// recurrence itself would not. Per tile of 16 tokens: the inclusive products from the tile's start (pre),
// the products behind a token up to the tile's end (suf), the tile's whole product, and the 16 x 16
// products within the tile. Across tiles ratio(r, s) = pre_r * (tiles between) * suf_s.
// ---------------------------------------------------------------------------
// Decays close to 1, one for each head, leave the same roundings in every chunk, and a state sums them over its
// whole memory: the products are formed in 64 bits and rounded once, and a chunk's whole product, which the state is
// multiplied by, is kept as two floats. (One decay of 0.99 .. 1 per head, 1333 tokens, fp32: the final state's error
// 1.2e-6 of its norm with products in 32 bits, 2.8e-7 so.)
constexpr int LDP = 20;  // row pitch of the 16 x 16 products (floats; 16-byte reads of a row's 4 columns)
struct DecayTab {
  float pre[DCH];
  float suf[DCH];
  float tile[4];
  double whole[4];         // the tiles' products before rounding
  float in[4][16 * LDP];  // [r][s], s <= r (the rest is not written)
};
// Lane l takes x of lane l + D (CTRL 0x100 + D) or l - D (0x110 + D) of its 16, 1 past the end.
template <int CTRL>
__device__ __forceinline__ double dpp_or1(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0x3ff00000, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int D>
__device__ __forceinline__ double row_shl(double x) {
  return dpp_or1<0x100 + D>(x);
}
// Products over the lanes 0 .. l of a row of 16, and over those behind lane l.
__device__ __forceinline__ double row_prefix(double x) {
  x *= dpp_or1<0x111>(x);
  x *= dpp_or1<0x112>(x);
  x *= dpp_or1<0x114>(x);
  return x * dpp_or1<0x118>(x);
}
__device__ __forceinline__ double row_suffix_excl(double x) {
  x *= row_shl<1>(x);
  x *= row_shl<2>(x);
  x *= row_shl<4>(x);
  x *= row_shl<8>(x);
  return row_shl<1>(x);
}
// A factor of the state as two floats, and the state's four values times it.
struct Factor {
  float hi, lo;
  __device__ __forceinline__ explicit Factor(double x) {
    hi = (float)x;
    lo = __builtin_isfinite(hi) ? (float)(x - (double)hi) : 0.f;
  }
  __device__ __forceinline__ void scale(f32x4& v) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaf(v[e], lo, v[e] * hi);
  }
};
// Wave w fills tile w; a: the decay of token 16 w + l % 16 in every lane.
__device__ __forceinline__ void decay_table(DecayTab& t, int w, double a, int lane) {
  const int s = lane & 15, g = lane >> 4;
  const double pre = row_prefix(a), suf = row_suffix_excl(a);
  if (g == 0) {
    t.pre[16 * w + s] = (float)pre;
    t.suf[16 * w + s] = (float)suf;
    if (s == 15) {
      t.tile[w] = (float)pre;
      t.whole[w] = pre;
    }
  }
  // lane group g: rows r = s + 4 g .. + 3 of column s, from the products over 4, 8 and 12 tokens
  const double p1 = row_shl<1>(a);
  const double p2 = p1 * row_shl<1>(p1);
  const double p4 = p2 * row_shl<2>(p2);
  const double p8 = p4 * row_shl<4>(p4);
  const double p12 = p8 * row_shl<8>(p4);
  const double x0 = p1, x1 = row_shl<4>(p1), x2 = row_shl<8>(p1), x3 = row_shl<12>(p1);
  double v = g == 0 ? 1. : g == 1 ? p4 : g == 2 ? p8 : p12;
  double nx = g == 0 ? x0 : g == 1 ? x1 : g == 2 ? x2 : x3;  // a_{s + 4 g + 1}
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = s + 4 * g + i;
    if (r < 16) t.in[w][r * LDP + s] = (float)v;
    v *= nx;
    nx = row_shl<1>(nx);
  }
}

// Workgroups of a launch over slots, heads and column blocks. Those of one (slot, query/key head) read the same keys and
// queries: they take consecutive places on one XCD (workgroups go round-robin over the eight), and the
// (slot, query/key head) pairs are dealt over the XCDs in turn, so that unused slots, the last ones, leave none idle.
__host__ __device__ __forceinline__ int64_t work_grid(const DecayParams& p) {
  return ((int64_t)p.slots * p.Hk + 7) / 8 * 8 * (p.H / p.Hk * p.ncb);
}
__device__ __forceinline__ bool work_of(const DecayParams& p, int& cb, int& h, int& slot) {
  const int per = p.H / p.Hk * p.ncb, b = blockIdx.x / 8;
  const int unit = b / per * 8 + blockIdx.x % 8, in = b % per;
  slot = unit / p.Hk;
  cb = in % p.ncb;
  h = (unit - slot * p.Hk) * (p.H / p.Hk) + in / p.ncb;
  return slot < p.slots;
}

// One slot's sequence and token span.
struct Span {
  int n;         // sequence (-1: unused slot)
  int64_t b;     // batch row
  int64_t row0;  // first token of the segment within the batch row
  int len;       // tokens of the segment
  int t0;        // first token of the segment within the sequence
  int total;     // tokens of the sequence
};
__device__ __forceinline__ Span slot_span(const DecayParams& p, int slot) {
  Span x;
  if (p.cu) {
    x.n = p.slot_seq[slot];
    if (x.n < 0) return x;
    const int j = slot - p.slot_first[x.n];
    const int c0 = p.cu[x.n];
    x.total = p.cu[x.n + 1] - c0;
    x.t0 = j * p.seg;
    x.b = 0;
    x.row0 = (int64_t)c0 + x.t0;
  } else {
    x.n = slot / p.nseg;
    x.t0 = (slot - x.n * p.nseg) * p.seg;
    x.total = (int)p.T;
    x.b = x.n;
    x.row0 = x.t0;
  }
  x.len = x.total - x.t0 < p.seg ? x.total - x.t0 : p.seg;
  return x;
}

// 8 channels of one token row: raw bits as loaded (zeroed only when they are put away, so that nothing
// waits for the load before), then the bf16 terms in LDS (fp32 data: three tiles `plane` bytes apart).
template <typename InT>
struct Piece;
template <>
struct Piece<__bf16> {
  u32x4 v;
  __device__ __forceinline__ void load(const __bf16* p) { v = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void store(unsigned char* at, int) const { *reinterpret_cast<u32x4*>(at) = v; }
};
template <>
struct Piece<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void store(unsigned char* at, int plane) const {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    const Tri t = split3(x);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x8*>(at + i * plane) = t.t[i];
  }
};
template <typename InT>
struct Terms {
  static constexpr int N = 3;
};
template <>
struct Terms<__bf16> {
  static constexpr int N = 1;
};

// DC x W tile of an input: each thread's pieces of a chunk, loaded (rows past the end from the last one) and
// then put into LDS (those rows, and channels past d, as zeros). A thread's pieces lie NTH / (W / 8) rows apart, a
// multiple of 16, which the swizzle does not see. Offsets within a chunk are 32 bits (token strides are limited
// to 2^24 elements), the chunk's base is uniform.
template <int W, typename InT, int DC = DCH, bool SWZ = true, int NTH = 256>
struct Stage {
  static constexpr int CPR = W / 8, NPC = (DC * CPR + NTH - 1) / NTH, STEP = NTH / CPR;
  static_assert(!SWZ || STEP % 16 == 0, "the swizzle repeats every 16 rows");
  Piece<InT> x[NPC];
  uint32_t off, step, col;  // bytes: the first piece's offset, between pieces, the piece's column
  int row, at;
  __device__ __forceinline__ void init(int64_t ts, int d, int tid) {
    const int pc = tid % CPR;
    row = (tid / CPR) % DC;
    col = pc * 8 < d ? (uint32_t)(pc * 8 * sizeof(InT)) : 0u;
    step = (uint32_t)(STEP * ts * sizeof(InT));
    off = (uint32_t)(row * ts * sizeof(InT)) + col;
    at = 16 * (SWZ ? swz<W>(row, pc) : row * CPR + pc);
  }
  // base: the chunk's first row
  __device__ __forceinline__ void load(const InT* base, int64_t ts, int rows) {
    const char* b = reinterpret_cast<const char*>(base);
    if (rows >= DC) {
#pragma unroll
      for (int i = 0; i < NPC; ++i) x[i].load(reinterpret_cast<const InT*>(b + (off + i * step)));
    } else {
#pragma unroll
      for (int i = 0; i < NPC; ++i) {
        const int r = row + i * STEP;
        x[i].load(reinterpret_cast<const InT*>(b + ((uint32_t)((r < rows ? r : rows - 1) * ts * sizeof(InT)) + col)));
      }
    }
  }
  __device__ __forceinline__ void mask(int rows, int d, int tid) {
    if (rows < DC || d < W) {
#pragma unroll
      for (int i = 0; i < NPC; ++i)
        if (row + i * STEP >= rows || (tid % CPR) * 8 >= d) x[i].zero();
    }
  }
  __device__ __forceinline__ bool mine(int i, int tid) const { return DC * CPR >= NTH || tid < DC * CPR; }
  __device__ __forceinline__ void store(unsigned char* tile, int plane, int rows, int d, int tid) {
    mask(rows, d, tid);
#pragma unroll
    for (int i = 0; i < NPC; ++i)
      if (mine(i, tid)) x[i].store(tile + at + i * STEP * W * 2, plane);
  }
};

// Sizes of the launches, checked before the first of a call: the work items along an axis are a 32-bit number.
inline bool launch_fits(int64_t blocks, int threads) { return blocks <= INT32_MAX && blocks * threads <= (int64_t)UINT32_MAX; }
constexpr int MAIN_WAVES = 8, FILL_WAVES = 4;  // of the main pass (see decay.hip)
inline int64_t join_grid(const DecayParams& p) { return (int64_t)p.nseq * p.H * (((int64_t)p.DK * p.DV / 4 + 255) / 256); }
inline int64_t grad_grid(const DecayParams& p) { return ((int64_t)p.cslots * p.H + 7) / 8 * 8; }
inline int64_t shared_grid(const DecayParams& p) { return ((int64_t)p.nbatch * p.T * p.Hk * p.DK / 4 + 255) / 256; }
constexpr int state_tiles(int dv) { return dv >= 32 ? 2 : 1; }  // column tiles per workgroup of the state passes
inline bool decay_fwd_fits(DecayParams p, const DecayPlan& pl) {
  p.ncb = p.DV / (16 * pl.ct);
  return launch_fits(work_grid(p), 64 * (MAIN_WAVES + FILL_WAVES)) && (pl.nseg <= 1 || launch_fits(join_grid(p), 256));
}
inline bool decay_bwd_fits(DecayParams p, const DecayPlan& pl) {
  p.ncb = p.DV / (16 * state_tiles(p.DV));
  return launch_fits(work_grid(p), 256) && (pl.nseg <= 1 || launch_fits(join_grid(p), 256)) &&
         launch_fits(grad_grid(p), 512) && (p.H == p.Hk || launch_fits(shared_grid(p), 256));
}
// Value columns per workgroup of the step: whole rows once the heads alone give every CU a few workgroups, slices of 32
// columns for fewer (d = 128, us: 64 heads 3.9 in slices and 4.3 whole, 256 heads 6.4 and 7.5, 1024 heads 26.0 and
// 23.5; slices of 16 columns, 64 heads, 6.1).
inline int step_columns(const DecayParams& p) {
  int dvs = p.DV;
  const int64_t heads = (int64_t)p.nseq * p.H;
  while (dvs > 32 && heads * (p.DV / dvs) < 1024) dvs /= 2;
  return dvs;
}
constexpr int step_threads(int dk, int dvs) { return dk * (dvs / 4) < 256 ? dk * (dvs / 4) : 256; }
inline bool decay_step_fits(const DecayParams& p) {
  const int dvs = step_columns(p);
  return launch_fits((int64_t)p.nseq * p.H * (p.DV / dvs), step_threads(p.DK, dvs));
}

hipError_t launch_decay_plan(const DecayParams& p, hipStream_t s);
hipError_t launch_decay_fwd(DecayParams p, const DecayPlan& pl, bool bf16, hipStream_t s);
hipError_t launch_decay_step(const DecayParams& p, bool bf16, hipStream_t s);
hipError_t launch_decay_bwd(DecayParams p, const DecayPlan& pl, bool bf16, hipStream_t s);
// Tokens per chunk of the backward: its chunk holds q, k, v and dO in LDS, fp32 data three times as large.
constexpr int decay_bwd_chunk(bool bf16) { return bf16 ? 64 : 32; }
// The backward's state passes, forward and reverse together, and the joining of segments (forward alone, or both).
hipError_t launch_decay_states(const DecayParams& p, bool bf16, int local, hipStream_t s);
hipError_t launch_decay_join(const DecayParams& p, bool both, hipStream_t s);

}  // namespace dr
