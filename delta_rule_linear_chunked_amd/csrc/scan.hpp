// Selective scan, short convolution and norm: parameter blocks, what host and kernels agree on, launches.
#pragma once

#include <type_traits>

#include "decay.hpp"

namespace dr {

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------
// p + off bytes: with a uniform p the memory instruction adds the lane's 32 bits by itself.
template <typename T>
__device__ __forceinline__ T* byte_at(T* p, uint32_t off) {
  using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(p) + off);
}

// VEC consecutive elements as one load or store (bf16: 8 in 16 bytes, fp32: 4), or one element.
template <typename T, int VEC>
struct Vec {
  typedef T type __attribute__((ext_vector_type(VEC)));
};
template <typename T>
struct Vec<T, 1> {
  typedef T type;
};
template <int VEC, typename T>
__device__ __forceinline__ void unpack(const typename Vec<T, VEC>::type& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = (float)r;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = (float)r[j];
  }
}
// (a bf16 value is the float rounded to nearest, ties to even)
template <int VEC, typename T>
__device__ __forceinline__ typename Vec<T, VEC>::type pack(const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    return (T)f[0];
  } else {
    typename Vec<T, VEC>::type r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = (T)f[j];
    return r;
  }
}

constexpr float LN2 = 0.6931471805599453f;
__device__ __forceinline__ float sigmoid_f(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * LOG2E));
}
// A step d: softplus(v), or v itself. softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1].
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3: a small step (1e-3 and less is usual) keeps its relative precision, which log of
// the rounded 1 + e would lose. 2 atanh(s) / s as a polynomial of s^2 in [0, 1/9], a Chebyshev fit of degree 4, off by 8e-9 of it.
// The rounding of the exponent p alone is |v| / 2 ULP of a small step (8 at -16): what -|v| differs from p LN2 by is put back. (For
// infinities that is no number, and the smaller one of it and 1 is taken; e is 0.)
// `least` is 0, or -infinity for v itself: it takes e to 0 and the maximum to v.
__device__ __forceinline__ float step_least(bool softplus) { return softplus ? 0.f : -__builtin_inff(); }
__device__ __forceinline__ float step_f(float v, float least) {
  const float p = fmaf(-fabsf(v), LOG2E, least), left = fmaf(-p, LN2, -fabsf(v));
  float e = __builtin_amdgcn_exp2f(p);
  e = fmaf(e, fminf(left, 1.f), e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), z = s * s;
  float q = 0.28174657f;
  q = fmaf(q, z, 0.27961419f);
  q = fmaf(q, z, 0.40024854f);
  q = fmaf(q, z, 0.66666316f);
  q = fmaf(q, z, 2.00000001f);
  return fmaf(s, q, fmaxf(v, least));
}

// Waits for what is in flight. Loads and stores are counted together: where paths with different numbers of stores meet, a wait for the loads
// in front of them waits for the stores as well; with nothing in flight on one of the paths the number is the other's.
__device__ __forceinline__ void arrived() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // (vmcnt 0)

// Row of a state pool that sequence n has; -1: none.
__device__ __forceinline__ int64_t state_row(const int32_t* idx, int64_t slots, int64_t n) {
  if (!idx) return n;
  const int64_t r = idx[n];
  return r >= 0 && r < slots ? r : -1;
}
// Packed rows: the sequence that holds token t (the last one that starts at or before it; offsets out of order give some
// sequence), in [0, nseq).
__device__ __forceinline__ int seq_of(const int32_t* cu, int nseq, int t) {
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Convolution
// ---------------------------------------------------------------------------
struct ConvParams {
  const void* x;
  const float* w;          // [C, W]
  const float* bias;       // [C], may be null
  const void* state;       // [N, W - 1, C], may be null
  const int32_t* cu;
  void* y;
  void* state_T;           // may be null
  const int32_t* sidx;
  int64_t nslots;
  int64_t T, x_ts, x_bs;
  int32_t C, nbatch, nseq;
  int32_t silu;
  int32_t streamed;        // outputs larger than the L2 caches: stored around them
  int32_t run;             // tokens of a wave; step: sequences
  int32_t cblocks;         // channel blocks of 64 vectors
  int32_t runs;            // runs of one batch row
  int32_t block0, nblocks, nmain;  // logical blocks of this launch: the first, their number; those below nmain walk tokens, the others states
  // backward
  const void* dy;
  const void* dstate_T;    // may be null
  void* dx;
  void* dstate;            // may be null
  float* part;             // [run blocks, W + 1, C]
  float* dw;
  float* db;
};
constexpr int CONV_WAVES = 4;
hipError_t launch_conv_fwd(ConvParams p, int width, bool bf16, bool vec, hipStream_t s);
hipError_t launch_conv_step(const ConvParams& p, int width, bool bf16, bool vec, hipStream_t s);
hipError_t launch_conv_bwd(ConvParams p, int width, bool bf16, bool vec, hipStream_t s);
constexpr int conv_vec(bool bf16, bool vec, bool backward) { return !vec ? 1 : bf16 && !backward ? 8 : 4; }

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------
struct NormParams {
  const void* x;      // backward: h
  const void* r;      // residual, may be null
  const float* w;
  void* y;
  float* scales;
  void* h;            // may be null
  int64_t rows, x_rs, r_rs;
  int32_t C;
  float eps;
  const void* dy;
  const void* dh;     // may be null
  void* dx;
  float* part;        // [workgroups, C]
  float* dw;
  int32_t nwg;        // workgroups (of the backward's first kernel)
  int32_t few;        // norm_few
};
constexpr int NORM_ELEMS = 32;  // of a row in a lane's registers
constexpr int NORM_FEW = 8;     // with few rows
constexpr int NORM_MOST = 32768;
// Few rows leave most of the GPU idle: then four times as many waves take a row, with a quarter of it in each lane. Measured, in
// us, one (four) waves a row: 1 x 2048 3.8 (2.9), 1333 x 1531 e4m3 12.8 (8.3), 8192 x 2048 int8 26.4 (21.0); above 2048 channels
// four (sixteen): 256 x 4096 int8 5.6 (5.1), 4096 x 4096 26.6 (40.0). The backward's workgroups each leave a row of sums:
// 64 x 2048 7.1 (5.8), 512 x 2048 8.1 (10.9).
constexpr bool norm_few(int64_t rows, int64_t C, bool backward) {
  return C > 64 * NORM_FEW && C <= 1024 * NORM_FEW && rows <= (C <= 256 * NORM_FEW && !backward ? 8192 : 256);
}
// Waves of a row.
constexpr int norm_waves(int64_t C, bool few) {
  return (C <= 64 * NORM_ELEMS ? 1 : C <= 256 * NORM_ELEMS ? 4 : 16) * (few ? 4 : 1);
}
// Workgroups: rows are dealt to at most so many, each of which keeps the weights (backward: its sums) in registers.
constexpr int64_t norm_groups(int64_t rows, int64_t C, bool few, int64_t most) {
  const int64_t per = norm_waves(C, few) == 1 ? 4 : 1, n = (rows + per - 1) / per;
  return n < most ? n : most;
}
hipError_t launch_norm_fwd(const NormParams& p, int out, bool bf16, bool vec, hipStream_t s);
hipError_t launch_norm_bwd(const NormParams& p, bool bf16, bool vec, hipStream_t s);

// ---------------------------------------------------------------------------
// Scan
// ---------------------------------------------------------------------------
struct ScanParams {
  const void* x;
  const void* dt;
  const void* B;
  const void* Cm;
  const void* z;           // may be null
  const float* A;          // [C, N]
  const float* D;          // may be null
  const float* bias;       // may be null
  const float* S0;         // may be null
  const int32_t* cu;
  void* y;
  float* S;                // final states, may be null; step: states in and out
  const int32_t* sidx;
  int64_t nslots;
  int64_t T;
  int64_t x_ts, x_bs, dt_ts, dt_bs, b_ts, b_bs, c_ts, c_bs, z_ts, z_bs;
  int32_t C, G, Cg;        // channels, groups, channels of a group
  int32_t tiles;           // channel tiles of a group
  int32_t nseq, nbatch;
  int32_t run;         // sequences of a workgroup in a step
  int32_t softplus;
  int32_t seg;             // tokens of a segment
  int32_t nseg;            // fixed length: segments of a sequence; packed: more than 1 if any may have more
  int32_t slots;           // (sequence, segment) pairs; packed: an upper bound
  // packed: written by the plan pass
  int32_t* cu_ok;
  int32_t* slot_seq;
  int32_t* slot_first;
  // segments: each slot's own contribution to the state behind it, then the state at its start
  float* part;             // [slots, C, N]
  float* sumd;             // [slots, C] sum of the slot's steps d
  // backward
  const void* dy;
  const float* dST;        // may be null
  void* dx;
  void* ddt;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dD;
  float* dbias;
  float* dS0;              // may be null
  float* rpart;            // [slots, C, N] as part, of the reverse pass
  float* ck;               // [chunks, C, N] local states at chunk starts (slot_chunk)
  float* ckd;              // [chunks, C] sums of the slot's steps before them
  float* pA;               // [slots, C, N] partial sums of dA
  float* pD;               // [slots, 2, C] of dD and of ddt_bias
  float* pBC;              // [channel blocks of a group, tokens, G, 2, N] partial sums of dB and dC
  int32_t cblocks;         // channel blocks of a group in the gradient pass
};
struct ScanPlan {
  bool block;  // the main pass with a workgroup's waves along the tokens
  int64_t seg, nseg, slots;
};
// What a slot is: sequence n (-1: none) in batch row b, tokens t0 .. t0 + len, the first / last of its sequence.
struct SlotSpan {
  int n, b, len;
  int64_t t0;
  bool first, last;
  // (only then may a slot read the states that its call starts from: they may be the final ones, which a sequence's last slot writes)
  __device__ __forceinline__ bool whole() const { return first && last; }
};
__device__ __forceinline__ SlotSpan slot_span(const ScanParams& p, int slot) {
  SlotSpan s;
  int i, start = 0, end = (int)p.T;
  if (p.cu) {
    s.n = p.slot_seq[slot];
    s.b = 0;
    if (s.n < 0) return s;
    i = slot - p.slot_first[s.n];
    start = p.cu[s.n];
    end = p.cu[s.n + 1];
  } else {
    s.n = s.b = slot / p.nseg;
    i = slot - s.n * p.nseg;
  }
  s.t0 = start + (int64_t)i * p.seg;
  s.len = max(0, min(p.seg, end - (int)s.t0));
  s.first = i == 0;
  s.last = s.t0 + s.len >= end;
  return s;
}
constexpr int SCAN_CHUNK = 8;        // tokens whose states the gradient pass holds at once
// Chunks of 8 tokens: the first one of a slot, and the number that all slots take. Packed slots lie one behind the other in the row: one
// of L tokens from t0 takes (L + 7) / 8 chunks, at most one more than lie between t0 / 8 and (t0 + L) / 8, so each
// slot in front adds one, however short it is (a whole segment's room for each would be sequences x T where they are not cut).
__device__ __forceinline__ int64_t slot_chunk(const ScanParams& p, int slot, const SlotSpan& s) {
  return p.cu ? s.t0 / SCAN_CHUNK + slot : (int64_t)slot * (p.seg / SCAN_CHUNK);
}
constexpr int64_t scan_chunks(int64_t T, int64_t slots, int64_t seg, bool packed) {
  return packed ? T / SCAN_CHUNK + slots : slots * (seg / SCAN_CHUNK);
}
constexpr int SCAN_TILE = 32;        // channels of a wave
constexpr int SCAN_BLOCK_WAVES = 8;  // waves of a workgroup of scan_block.hip
hipError_t launch_scan_block(const ScanParams& p, int n, bool bf16, hipStream_t s);
constexpr int SCAN_STEP_RUN = 4;  // most sequences of a workgroup in a step
constexpr int scan_step_channels(int n) { return 1024 / n; }  // channels of a workgroup of the step (4 states a lane)
hipError_t launch_scan_plan(const ScanParams& p, hipStream_t s);
hipError_t launch_scan_fwd(ScanParams p, const ScanPlan& pl, int n, bool bf16, hipStream_t s);
hipError_t launch_scan_step(const ScanParams& p, int n, bool bf16, hipStream_t s);
hipError_t launch_scan_bwd(ScanParams p, int n, bool bf16, hipStream_t s);
constexpr int scan_grad_channels(int n) { return 2048 / n; }  // channels of a workgroup of the gradient pass

}  // namespace dr
