// Prefill of the decayed linear attention S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t on gfx950.
//
// Per chunk of 64 tokens with start state S0 (ratio(r, s) = a_{s+1} ... a_r, Gamma_r the product from the
// chunk's start):
//
//   O = Gamma . (Q S0) + ((Q K^T) . ratio) V,     S <- Gamma_C S0 + K^T (ratio(C, .) . V)
//
// One workgroup of 8 waves, with 4 more to fill the LDS, carries 16 CT value columns of one head through one
// segment of a sequence; the waves of a column tile hold its d_k x 16 state in their accumulators for the whole
// segment. The accumulators of K^T V are, lane for lane, the S^T operand of Q S0 (common index orders of the 32-deep
// products, see decay.hpp), so the state never leaves the registers and O^T comes out with 4 consecutive columns per
// lane. Through LDS go the inputs, with one or two column tiles V scaled for the state as well, P as three bf16 planes
// (the filling waves form it once for all columns), and with fewer column tiles than waves the parts of Q S0: 8 / CT
// waves then share a tile and split the state's channels, then the chunk's 16-token row tiles.
//
// What bounds it: a chunk's two phases (Q S0 and the scores; P V and the state) follow one another through
// barriers, with LDS reads and the cutting of the state and of scaled V into bf16 terms beside the MFMA. 4 x 4096
// tokens, 16 heads, d = 128, bf16: main pass 89 us (4.2 TB/s; MFMA busy a third of the time), states of the segments of
// 1024 tokens 37, join 7; all told 132 to 141, where the inputs and outputs alone take 66 at the copy rate.
#include <type_traits>

#include "decay.hpp"
#include "launch.hpp"

namespace dr {

// Packed sequences: clamped offsets, slots of `seg` tokens, chunk slots and snapshot rows. One workgroup.
__device__ __forceinline__ void scan_table(int nseq, int* s_scan, int* s_carry, int tid, int32_t* first,
                                           const int32_t* cu, int unit, bool ceil_one) {
  if (tid == 0) *s_carry = 0;
  __syncthreads();
  for (int base = 0; base < nseq; base += 256) {
    const int n = base + tid;
    int c = 0;
    if (n < nseq) {
      const int len = cu[n + 1] - cu[n];
      c = ceil_one ? max(pieces(len, unit), 1) : len / unit;
    }
    s_scan[tid] = c;
    __syncthreads();
    for (int d = 1; d < 256; d <<= 1) {
      const int x = tid >= d ? s_scan[tid - d] : 0;
      __syncthreads();
      s_scan[tid] += x;
      __syncthreads();
    }
    if (n < nseq) first[n] = *s_carry + s_scan[tid] - c;
    __syncthreads();
    if (tid == 255) *s_carry += s_scan[255];
    __syncthreads();
  }
}
__device__ __forceinline__ void fill_slots(int nseq, int tid, int32_t* first, int32_t* seq, int slots, int total) {
  if (tid == 0) first[nseq] = total;
  __syncthreads();  // (the workgroup-scope fence covers global memory)
  for (int s = tid; s < slots; s += 256) {
    int n = -1;
    if (s < total) {
      int lo = 0, hi = nseq;  // the last sequence whose first slot is <= s
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= s) lo = mid; else hi = mid;
      }
      n = lo;
    }
    seq[s] = n;
  }
}
__global__ __launch_bounds__(256) void decay_plan_kernel(DecayParams p) {
  __shared__ int s_scan[256];
  __shared__ int s_carry;
  const int tid = threadIdx.x;
  if (tid == 0) s_carry = 0;
  __syncthreads();
  for (int base = 0; base <= p.nseq; base += 256) {  // a running maximum of the clamped offsets
    const int n = base + tid;
    s_scan[tid] = n <= p.nseq ? min(max(p.cu[n], 0), (int32_t)p.T) : 0;
    __syncthreads();
    for (int d = 1; d < 256; d <<= 1) {
      const int y = tid >= d ? s_scan[tid - d] : 0;
      __syncthreads();
      s_scan[tid] = max(s_scan[tid], y);
      __syncthreads();
    }
    if (n <= p.nseq) p.cu_ok[n] = max(s_scan[tid], s_carry);
    __syncthreads();
    if (tid == 255) s_carry = max(s_carry, s_scan[255]);
    __syncthreads();
  }
  scan_table(p.nseq, s_scan, &s_carry, tid, const_cast<int32_t*>(p.slot_first), p.cu_ok, p.seg, true);
  fill_slots(p.nseq, tid, p.slot_first, p.slot_seq, p.slots, s_carry);
  __syncthreads();
  if (p.cslots > 0) {
    scan_table(p.nseq, s_scan, &s_carry, tid, p.chunk_first, p.cu_ok, p.bwd_chunk, true);
    fill_slots(p.nseq, tid, p.chunk_first, p.chunk_seq, p.cslots, s_carry);
    __syncthreads();
  }
  if (p.snap) scan_table(p.nseq, s_scan, &s_carry, tid, p.snap_first, p.cu_ok, p.snap_chunks * DCH, false);
}

// ---------------------------------------------------------------------------
// Main pass
// ---------------------------------------------------------------------------
// Eight waves work on the state, as CT column tiles x G = 8 / CT waves each; four more fill the LDS and form P. The G waves of a column split its channels in
// IS parts (whole 32-channel slices) and repeat them D times: a wave forms its channels' part of Q S0 for the row
// tiles of its repeat, hands the parts of row tiles that it does not finish to their owner, and updates its channels
// of the state.
template <int W, int CT>
struct Split {
  static constexpr int G = MAIN_WAVES / CT, IS = G < W / 32 ? G : W / 32, D = G / IS < 4 ? G / IS : 4;
  static constexpr int U = W / 32 / IS;           // 32-channel slices of a wave
  static constexpr int RT = 4 / D;                // row tiles of a repeat
  static constexpr int RO = (RT + IS - 1) / IS;   // of them finished by each part (the first RT / RO parts)
  // i-th row tile of repeat d; pairs are 0 with 3 and 1 with 2, which have equal work
  static constexpr int tile(int d, int i) {
    if (RT == 4) return RO == 2 ? (i == 0 ? 0 : i == 1 ? 3 : i == 2 ? 1 : 2) : i;
    if (RT == 2) return d == 0 ? (i == 0 ? 0 : 3) : (i == 0 ? 1 : 2);
    return d;
  }
};
template <int W, int CT, typename InT>
struct MainShape {
  static constexpr int NP = Terms<InT>::N;
  static constexpr int NB = NP == 1 ? 2 : 1;  // fp32 data is held as three bf16 terms: one buffer fits
  static constexpr int QK = DCH * W * 2;      // bytes of one plane
  static constexpr int VB = DCH * CT * 32;
  // Q has one buffer: it is read in the first half of a chunk and filled in the second
  // Up to two column tiles share each of the scaled rows of V among four waves or more: scaled and cut into terms
  // once, through LDS. With more tiles a row has one or two readers, which form their terms in registers.
  static constexpr bool VT = CT <= 2;
  static constexpr int QB = NP * QK, OFF_V = NP * QK, OFF_T = OFF_V + NP * VB, BUF = OFF_T + (VT ? 3 * VB : 0);
  static constexpr int PP = DCH + 8, PB = DCH * PP * 2;  // P: row pitch free of bank conflicts, bytes of one plane
  using Sp = Split<W, CT>;
  static constexpr int XCH = Sp::IS > 1 ? CT * 4 * (Sp::IS - 1) * 1024 : 0;  // parts of Q S0 on their way
};

// Column tile n of V, tokens along the product (see frag_cols). Rows of 16 or 32 columns lie in order, wider ones are
// swizzled as K is (four rows' 32 bytes of a tile are then in different banks as well).
template <int CT>
__device__ __forceinline__ bf16x8 frag_v(const unsigned char* tile, int n, int u, int lane) {
  if constexpr (CT <= 2) return frag_cols<16 * CT>(tile, 16 * n, u, lane);
  const int at = (16 * swz<16 * CT>(4 * (lane >> 4) + ((lane >> 2) & 3), (lane >> 1) & 1)) ^ (32 * n);
  const unsigned char* p = tile + at + 8 * (lane & 1) + 32 * u * CT * 32;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * CT * 32));
  return join(a, b);
}

// P = (Q K^T) . ratio of tile (R, S) as bf16 terms into LDS, rows r. Q's rows are kept for the tiles of a row, but
// for the widest fp32 heads, whose three terms do not fit the registers beside the loads on their way: there
// every tile reads them again.
template <int W, typename InT>
constexpr bool keep_rows() {
  return Terms<InT>::N * W <= 256;
}
template <int W, int CT, typename InT, int R, int S>
__device__ __forceinline__ void score_tile(const unsigned char* qbuf, const unsigned char* buf, const DecayTab& tb, const Op<Terms<InT>::N> (&qf)[W / 32],
                                           unsigned char* Pt, int lane) {
  using Sh = MainShape<W, CT, InT>;
  constexpr int NP = Sh::NP;
  const int g = lane >> 4, r16 = lane & 15;
  f32x4 sc = {0, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < W / 32; ++u) {
    Op<NP> kf;
#pragma unroll
    for (int i = 0; i < NP; ++i) kf.t[i] = frag_rows<W>(buf + i * Sh::QK, 16 * S, u, lane);
    if constexpr (keep_rows<W, InT>()) {
      mma(sc, kf.t, qf[u].t);
    } else {
      Op<NP> qr;
#pragma unroll
      for (int i = 0; i < NP; ++i) qr.t[i] = frag_rows<W>(qbuf + i * Sh::QK, 16 * R, u, lane);
      mma(sc, kf.t, qr.t);
      fence();
    }
  }
  if constexpr (S == R) {
    const f32x4 in = *reinterpret_cast<const f32x4*>(&tb.in[S][r16 * LDP + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = r16 >= 4 * g + i ? sc[i] * in[i] : 0.f;
  } else {
    float f = tb.pre[16 * R + r16];
#pragma unroll
    for (int j = S + 1; j < R; ++j) f *= tb.tile[j];
    const f32x4 suf = *reinterpret_cast<const f32x4*>(&tb.suf[16 * S + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] *= f * suf[i];
  }
  split_store4(Pt + ((16 * R + r16) * Sh::PP + 16 * S + 4 * g) * 2, Sh::PB, sc);
}
template <int W, typename InT, int R>
__device__ __forceinline__ void score_rows(const unsigned char* buf, Op<Terms<InT>::N> (&qf)[W / 32], int lane) {
  constexpr int NP = Terms<InT>::N;
  if constexpr (!keep_rows<W, InT>()) return;
#pragma unroll
  for (int u = 0; u < W / 32; ++u)
#pragma unroll
    for (int i = 0; i < NP; ++i) qf[u].t[i] = frag_rows<W>(buf + i * DCH * W * 2, 16 * R, u, lane);
}

// First half of a chunk, wave M of column tile ct: its part of Q S0, kept for the row tiles that it finishes, handed on for the others.
template <int W, int CT, typename InT, int M>
__device__ __forceinline__ void chunk_first(const unsigned char* buf, const f32x4* st, f32x4 (&oa)[Split<W, CT>::RO],
                                            unsigned char* xch, int ct, int lane) {
  using Sh = MainShape<W, CT, InT>;
  using Sp = Split<W, CT>;
  constexpr int NP = Sh::NP, IS = Sp::IS, PART = M % IS, REP = M / IS;
  if constexpr (REP < Sp::D) {
    f32x4 acc[Sp::RT];
    bf16x8 qf[2][Sp::RT][NP];
    Tri sf[2];
    auto load = [&](int u) {
#pragma unroll
      for (int i = 0; i < Sp::RT; ++i)
#pragma unroll
        for (int e = 0; e < NP; ++e)
          qf[u & 1][i][e] = frag_rows<W>(buf + e * Sh::QK, 16 * Sp::tile(REP, i), PART * Sp::U + u, lane);
    };
    auto split = [&](int u) {
      const float x[8] = {st[2 * u][0],     st[2 * u][1],     st[2 * u][2],     st[2 * u][3],
                          st[2 * u + 1][0], st[2 * u + 1][1], st[2 * u + 1][2], st[2 * u + 1][3]};
      sf[u & 1] = split3(x);
    };
    load(0);
    fence();
    split(0);
#pragma unroll
    for (int i = 0; i < Sp::RT; ++i) acc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < Sp::U; ++u) {
      if (u + 1 < Sp::U) load(u + 1);
      fence();
      if (u + 1 < Sp::U) split(u + 1);
      mma_rows(acc, sf[u & 1].t, qf[u & 1]);
      fence();
    }
#pragma unroll
    for (int i = 0; i < Sp::RT; ++i) {
      const int R = Sp::tile(REP, i), owner = i / Sp::RO;
      if (owner == PART)
        oa[i % Sp::RO] = acc[i];
      else  // slot of this part among the owner's IS - 1 others
        *reinterpret_cast<f32x4*>(xch + (((ct * 4 + R) * (IS - 1) + (PART < owner ? PART : PART - 1)) * 64 + lane) * 16) = acc[i];
    }
  }
}

// P by the filling waves, the ten tiles split 3, 2, 3, 2.
template <int W, int CT, typename InT, int WV>
__device__ __forceinline__ void scores(const unsigned char* qbuf, const unsigned char* buf, const DecayTab& tb,
                                       unsigned char* Pt, int lane) {
  Op<Terms<InT>::N> qf[W / 32];
  constexpr int R = WV < 2 ? 3 : WV == 2 ? 2 : 1, S0 = WV == 1 ? 2 : 0;
  score_rows<W, InT, R>(qbuf, qf, lane);
  score_tile<W, CT, InT, R, S0>(qbuf, buf, tb, qf, Pt, lane);
  score_tile<W, CT, InT, R, S0 + 1>(qbuf, buf, tb, qf, Pt, lane);
  if constexpr (WV == 2) score_tile<W, CT, InT, R, 2>(qbuf, buf, tb, qf, Pt, lane);
  if constexpr (WV == 0) {
    score_rows<W, InT, 0>(qbuf, qf, lane);
    score_tile<W, CT, InT, 0, 0>(qbuf, buf, tb, qf, Pt, lane);
  }
}

// The row tile of index j among those that a part finishes (-1: none)
template <int W, int CT>
constexpr int own_row(int rep, int part, int j) {
  using Sp = Split<W, CT>;
  return j < Sp::RO && part * Sp::RO + j < Sp::RT ? Sp::tile(rep, part * Sp::RO + j) : -1;
}
// Steps of P V: two row tiles j, j + 1 and one half of the tokens each, as 2 j + half
template <int W, int CT>
constexpr int pv_step(int rep, int part, int s, bool count) {
  int n = 0;
  for (int j = 0; j < 4; j += 2)
    for (int u = 0; u < 2; ++u)
      if (own_row<W, CT>(rep, part, j) >= 2 * u || own_row<W, CT>(rep, part, j + 1) >= 2 * u) {
        if (!count && n == s) return 2 * j + u;
        ++n;
      }
  return count ? n : 0;
}

// Second half: the row tiles that wave M of column tile ct finishes, and its channels of the state:
// S <- Gamma_C S + K^T (tail . V).
template <int W, int CT, typename InT, bool OUT, int M>
__device__ __forceinline__ void chunk_second(const unsigned char* buf, const DecayTab& tb, f32x4 (&st)[2 * Split<W, CT>::U],
                                             f32x4 (&oa)[Split<W, CT>::RO], const unsigned char* Pt,
                                             const unsigned char* xch, float* o, int o_ts, int rows, int ct, int lane) {
  using Sh = MainShape<W, CT, InT>;
  using Sp = Split<W, CT>;
  constexpr int NP = Sh::NP, IS = Sp::IS, PART = M % IS, REP = M / IS;
  const int g = lane >> 4, r16 = lane & 15;
  constexpr bool OWN = OUT && REP < Sp::D && PART * Sp::RO < Sp::RT;  // the wave finishes row tiles
  constexpr int NPV = OWN ? pv_step<W, CT>(REP, PART, 0, true) : 0, STEPS = NPV + Sp::U;
  // Steps: of P V (12 reads each), then the state's tiles in pairs (8 reads each); a step's reads are issued
  // before the products of the step before it.
  bf16x8 fr[2][4 * NP > 6 ? 4 * NP : 6];  // P: [row tile][term]; K: [tile][half][term]
  auto load = [&](int s) {
    if (s < NPV) {
      const int ju = pv_step<W, CT>(REP, PART, s, false), u = ju & 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int R = own_row<W, CT>(REP, PART, (ju >> 1) + i);
        if (R < 2 * u) continue;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const unsigned char* at = Pt + e * Sh::PB + ((16 * R + r16) * Sh::PP + 32 * u + 4 * g) * 2;
          fr[s & 1][3 * i + e] = join(*reinterpret_cast<const s16x4*>(at), *reinterpret_cast<const s16x4*>(at + 32));
        }
      }
    } else if (s < STEPS) {
      const int w = s - NPV;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < NP; ++e)
            fr[s & 1][(2 * i + u) * NP + e] = frag_chan<W>(buf + e * Sh::QK, PART * Sp::U + w, i, u, lane);
    }
  };
  // reads that the first steps need
  Op<NP> vf[2];
  bf16x8 vt[2][3];
  f32x4 suf[4], part[Sp::RO][IS > 1 ? IS - 1 : 1];
  float pre[Sp::RO], P[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) P[j] = tb.tile[j];
  double W4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) W4[j] = tb.whole[j];
  if constexpr (OWN || !Sh::VT) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < NP; ++i) vf[u].t[i] = frag_v<CT>(buf + Sh::OFF_V + i * Sh::VB, ct, u, lane);
  }
  if constexpr (OWN) {
#pragma unroll
    for (int j = 0; j < Sp::RO; ++j) {
      const int R = Sp::tile(REP, PART * Sp::RO + j);
      pre[j] = tb.pre[16 * R + r16];
#pragma unroll
      for (int e = 0; e < IS - 1; ++e)
        part[j][e] = *reinterpret_cast<const f32x4*>(xch + (((ct * 4 + R) * (IS - 1) + e) * 64 + lane) * 16);
    }
  }
  load(0);
  if constexpr (Sh::VT) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 3; ++e) vt[u][e] = frag_v<CT>(buf + Sh::OFF_T + e * Sh::VB, ct, u, lane);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) suf[j] = *reinterpret_cast<const f32x4*>(&tb.suf[16 * j + 4 * g]);
  }
  fence();
  // Gamma . (Q S0)
  if constexpr (OWN) {
#pragma unroll
    for (int j = 0; j < Sp::RO; ++j) {
      float gam = pre[j];
#pragma unroll
      for (int t = 0; t < Sp::tile(REP, PART * Sp::RO + j); ++t) gam *= P[t];
#pragma unroll
      for (int e = 0; e < IS - 1; ++e) oa[j] += part[j][e];
#pragma unroll
      for (int i = 0; i < 4; ++i) oa[j][i] *= gam;
    }
  }
  auto scale = [&](int u) {  // the scaled rows of V, in registers
    if constexpr (!Sh::VT) {
      float x[8];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float f = 1.f;
#pragma unroll
        for (int j = 2 * u + a + 1; j < 4; ++j) f *= P[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y = 0.f;
#pragma unroll
          for (int e = NP - 1; e >= 0; --e) y += (float)vf[u].t[e][4 * a + i];
          x[4 * a + i] = y * (suf[2 * u + a][i] * f);
        }
      }
      const Tri tr = split3(x);
#pragma unroll
      for (int e = 0; e < 3; ++e) vt[u][e] = tr.t[e];
    }
  };
  const Factor G(W4[0] * W4[1] * W4[2] * W4[3]);
  // rows past the end fall outside the descriptor and are dropped
  // (32-bit offsets: at most 64 rows of 2^16 heads of 128 columns of 4 bytes, 2^31)
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(o, 0, (int)((uint32_t)(rows < DCH ? rows : DCH) * (uint32_t)o_ts * 4u), 0x00020000);
  if constexpr (NPV == 0) {
    scale(0);
    scale(1);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    load(s + 1);
    fence();
    if (s < NPV) {
      const int ju = pv_step<W, CT>(REP, PART, s, false), j = ju >> 1, u = ju & 1;
      const int R0 = own_row<W, CT>(REP, PART, j), R1 = own_row<W, CT>(REP, PART, j + 1);
#pragma unroll
      for (int sum = NP + 1 < 2 ? NP + 1 : 2; sum >= 0; --sum)
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          if (sum - q < 0 || sum - q > 2) continue;
          if (R0 >= 2 * u)
            oa[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[u].t[q], fr[s & 1][sum - q], oa[j], 0, 0, 0);
          if (R1 >= 2 * u)
            oa[j + 1 < Sp::RO ? j + 1 : 0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                vf[u].t[q], fr[s & 1][3 + sum - q], oa[j + 1 < Sp::RO ? j + 1 : 0], 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int R = i ? R1 : R0;
        if (R >= 0 && u == R / 2)  // the row tile is complete
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, oa[j + i < Sp::RO ? j + i : 0]), rsrc,
                                                 (int)(((uint32_t)(16 * R + r16) * (uint32_t)o_ts + 16 * ct + 4 * g) * 4u), 0, 0);
      }
      if (s == 0) scale(0);
      if (s == (NPV > 1 ? 1 : 0)) scale(1);
    } else {
      const int w = s - NPV;
#pragma unroll
      for (int i = 0; i < 2; ++i) G.scale(st[2 * w + i]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int sum = NP + 1 < 2 ? NP + 1 : 2; sum >= 0; --sum)
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            if (sum - q < 0 || sum - q > 2) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              st[2 * w + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[s & 1][(2 * i + u) * NP + q], vt[u][sum - q], st[2 * w + i], 0, 0, 0);
          }
    }
    fence();
  }
}

// Column `col` of a d_k x d_v state in a lane's accumulators of NT channel tiles, the first of them t0 (see
// frag_chan). Only d_k = 16 has fewer channels than its accumulators (W = 32).
template <int W>
__device__ __forceinline__ int chan_of(int t, int i, int lane) {
  return 32 * (t >> 1) + 8 * (lane >> 4) + 4 * (t & 1) + i;
}
template <int W, int NT>
__device__ __forceinline__ void state_load(f32x4 (&st)[NT], const float* src, int t0, int DK, int DV, int col, int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t) st[t] = f32x4{0, 0, 0, 0};
  if (src == nullptr) return;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = chan_of<W>(t0 + t, i, lane);
      st[t][i] = src[(W == 32 && ch >= DK ? 0 : ch) * DV + col];
    }
  if (W == 32) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (chan_of<W>(t0 + t, i, lane) >= DK) st[t][i] = 0.f;
  }
}
template <int W, int NT>
__device__ __forceinline__ void state_store(const f32x4 (&st)[NT], float* dst, int t0, int DK, int DV, int col, int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = chan_of<W>(t0 + t, i, lane);
      if (W > 32 || ch < DK) dst[ch * DV + col] = st[t][i];
    }
}

// A chunk's token weights from its decays a (lane t: token t): the product of the decays behind the token (or, REV,
// from the chunk's start through it) and of the whole chunk.
template <bool REV>
__device__ __forceinline__ float chunk_weight(double a, int lane, double& all) {
  const double pre = row_prefix(a);
  double P[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t b = __builtin_bit_cast(uint64_t, pre);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 16 * j + 15);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 16 * j + 15);
    P[j] = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
  double wt = REV ? pre : row_suffix_excl(a);
#pragma unroll
  for (int j = 0; j < 4; ++j) wt *= (REV ? j < (lane >> 4) : j > (lane >> 4)) ? P[j] : 1.;
  all = P[0] * P[1] * P[2] * P[3];
  return (float)wt;
}
// One piece of V or dO, its row scaled by f, as three bf16 terms into LDS
template <typename T>
__device__ __forceinline__ void scaled_store(const Piece<T>& x, float f, unsigned char* at, int plane) {
  float z[8];
  if constexpr (sizeof(T) == 2) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, x.v);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = (float)b[e] * f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = (e < 4 ? x.a[e] : x.b[e - 4]) * f;
  }
  const Tri t = split3(z);
#pragma unroll
  for (int e = 0; e < 3; ++e) *reinterpret_cast<bf16x8*>(at + e * plane) = t.t[e];
}

// f with the (uniform) index m < N as a compile-time constant: what a wave does is then straight code
template <int N, class F, int I = 0>
__device__ __forceinline__ void by_wave(int m, const F& f) {
  if constexpr (I == N - 1) {
    f(std::integral_constant<int, I>{});
  } else {
    if (m == I)
      f(std::integral_constant<int, I>{});
    else
      by_wave<N, F, I + 1>(m, f);
  }
}

// The filling waves of a chunk step: P of the chunk in its first half; in its second half the next chunk's data from
// registers to LDS, and the loads of the one after it. Their latency and that of P's short chains then
// pass beside the state's work instead of in line with it.
template <int W, int CT, typename InT, bool OUT>
struct Filler {
  using Sh = MainShape<W, CT, InT>;
  Stage<W, InT> sq, sk;
  Stage<16 * CT, InT, DCH, (CT > 2)> sv;
  const InT *q, *k, *v;
  const float* al;
  int64_t a_ts, q_ts, k_ts, v_ts;
  int len, nc, d, tid, lane, wave;
  float a_next;  // decays of chunk 4 g + wave
  __device__ __forceinline__ void fetch(int c) {
    const int64_t c0 = (int64_t)(c < nc ? c : nc - 1) * DCH;  // (past the end the last chunk again: no branch, see below)
    const int rows = len - (int)c0;
    if constexpr (OUT) sq.load(q + c0 * q_ts, q_ts, rows);
    sk.load(k + c0 * k_ts, k_ts, rows);
    sv.load(v + c0 * v_ts, v_ts, rows);
  }
  // Decays lie H apart: each of the four waves takes one chunk of every four.
  __device__ __forceinline__ void fetch_decays(int g) {
    const int64_t t = (int64_t)(4 * g + wave) * DCH + lane;
    a_next = al[(t < len ? t : len - 1) * a_ts];
  }
  __device__ __forceinline__ void put_decays(int g, float (&ring)[2][4][DCH]) const { ring[g & 1][wave][lane] = a_next; }
  __device__ __forceinline__ void put(int c, unsigned char* qbuf, unsigned char* buf, DecayTab& tab, const float (&ring)[2][4][DCH]) {
    const int rows = len - c * DCH;
    const float* ac = ring[(c >> 2) & 1][c & 3];
    const int t16 = 16 * wave + (lane & 15);
    const float a16 = t16 < rows ? ac[t16] : 1.f;
    if constexpr (OUT) sq.store(qbuf, Sh::QK, rows, d, tid);
    sk.store(buf, Sh::QK, rows, d, tid);
    if constexpr (!Sh::VT) {
      sv.store(buf + Sh::OFF_V, Sh::VB, rows, 16 * CT, tid);
    } else {
      sv.mask(rows, 16 * CT, tid);
      double all;
      const float wt = chunk_weight<false>(lane < rows ? ac[lane] : 1.f, lane, all);
#pragma unroll
      for (int i = 0; i < sv.NPC; ++i) {
        const float f = __shfl(wt, sv.row + i * sv.STEP);
        if (sv.mine(i, tid)) {
          if constexpr (OUT) sv.x[i].store(buf + Sh::OFF_V + sv.at + i * sv.STEP * CT * 32, Sh::VB);
          scaled_store(sv.x[i], f, buf + Sh::OFF_T + sv.at + i * sv.STEP * CT * 32, Sh::VB);
        }
      }
    }
    decay_table(tab, wave, a16, lane);
  }
};

template <int W, int CT, typename InT, bool OUT>
__global__ __launch_bounds__(64 * (MAIN_WAVES + FILL_WAVES)) void decay_main_kernel(const DecayParams p, int local) {
  using Sh = MainShape<W, CT, InT>;
  using Sp = Split<W, CT>;
  constexpr int NB = Sh::NB, NT = 2 * Sp::U, NTH = 64 * (MAIN_WAVES + FILL_WAVES);
  __shared__ __align__(16) unsigned char qbuf[OUT ? Sh::QB : 16];
  __shared__ __align__(16) unsigned char smem[NB * Sh::BUF];
  __shared__ __align__(16) unsigned char Pt[OUT ? 3 * Sh::PB : 16];
  __shared__ __align__(16) unsigned char xch[OUT && Sh::XCH ? Sh::XCH : 16];
  __shared__ __align__(16) DecayTab tabs[NB];
  __shared__ float ring[2][4][DCH];
  int cb, h, slot;
  if (!work_of(p, cb, h, slot)) return;
  const Span sp = slot_span(p, slot);
  if (sp.n < 0) return;
  // local: a segment's own contribution; nothing comes behind a sequence's last segment
  if (local && sp.t0 + sp.len >= sp.total) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t trow = sp.b * p.T + sp.row0;  // row in the dense per-token arrays
  const int nc = pieces(sp.len, DCH);
  if constexpr (OUT) {
    // the two tiles of P above the diagonal that the 32-token products meet
    for (int i = tid; i < 3 * 2 * 16 * 2; i += NTH) {
      const int e = i / 64, w = i % 64, R = (w / 32) * 2, r = (w % 32) / 2, hf = w & 1;
      *reinterpret_cast<u32x4*>(Pt + e * Sh::PB + ((16 * R + r) * Sh::PP + 16 * (R + 1)) * 2 + 16 * hf) = u32x4{0, 0, 0, 0};
    }
  }
  // (both kinds of wave meet the same barriers: one in the prologue, then two or three a chunk)
  if (wave >= MAIN_WAVES) {
    const int hk = h / (p.H / p.Hk);
    Filler<W, CT, InT, OUT> f;
    f.q = static_cast<const InT*>(p.q) + sp.b * p.q_bs + sp.row0 * p.q_ts + (int64_t)hk * p.DK;
    f.k = static_cast<const InT*>(p.k) + sp.b * p.k_bs + sp.row0 * p.k_ts + (int64_t)hk * p.DK;
    f.v = static_cast<const InT*>(p.v) + sp.b * p.v_bs + sp.row0 * p.v_ts + (int64_t)h * p.DV + cb * 16 * CT;
    f.al = p.alpha + (p.a_tok ? trow * p.H : 0) + h;
    f.a_ts = p.a_tok ? p.H : 0;
    f.q_ts = p.q_ts;
    f.k_ts = p.k_ts;
    f.v_ts = p.v_ts;
    f.len = sp.len;
    f.nc = nc;
    f.d = p.DK;
    f.tid = tid - 64 * MAIN_WAVES;
    f.lane = lane;
    f.wave = wave - MAIN_WAVES;
    if constexpr (OUT) f.sq.init(p.q_ts, p.DK, f.tid);
    f.sk.init(p.k_ts, p.DK, f.tid);
    f.sv.init(p.v_ts, 16 * CT, f.tid);
    if (nc > 0) {
      f.fetch(0);
      f.fetch_decays(0);
      f.put_decays(0, ring);
      f.fetch_decays(1);
    }
    __syncthreads();
    if (nc > 0) {
      f.put(0, qbuf, smem, tabs[0], ring);
      f.fetch(1);
    }
    for (int c = 0; c < nc; ++c) {
      const int nb = (c + 1) % NB;
      __syncthreads();
      if constexpr (OUT) {
        const unsigned char* buf = smem + (c % NB) * Sh::BUF;
        const DecayTab& tb = tabs[c % NB];
        by_wave<4>(f.wave, [&](auto M) { scores<W, CT, InT, M.value>(qbuf, buf, tb, Pt, lane); });
      }
      __syncthreads();
      if constexpr (NB == 1) __syncthreads();
      if (c + 1 < nc) f.put(c + 1, qbuf, smem + nb * Sh::BUF, tabs[nb], ring);
      f.fetch(c + 2);
      if ((c & 3) == 0) {  // the next four chunks' decays; those two groups back are done with
        f.put_decays((c >> 2) + 1, ring);
        f.fetch_decays((c >> 2) + 2);
      }
    }
    return;
  }

  const int ct = wave % CT, m = wave / CT, part = m % Sp::IS;
  const int64_t o_ts = (int64_t)p.H * p.DV;
  float* o = OUT ? p.o + trow * o_ts + (int64_t)h * p.DV + cb * 16 * CT : nullptr;
  // the state at the segment's start: lane's column l % 16, channels 32 u + 8 (l / 16) + 4 e + i of the wave's slices
  const int col = cb * 16 * CT + 16 * ct + (lane & 15), tile0 = part * NT;
  const int64_t hsz = (int64_t)p.DK * p.DV;
  int64_t srow = sp.n;  // row of the state buffers
  if (p.sidx) {
    srow = p.sidx[sp.n];
    if (srow < 0 || srow >= p.nslots) srow = -1;
  }
  const float* src = nullptr;
  if (!local) src = p.part ? p.part + ((int64_t)slot * p.H + h) * hsz
                           : (p.S0 && srow >= 0 ? p.S0 + (srow * p.H + h) * hsz : nullptr);
  f32x4 st[NT];
  state_load<W>(st, src, tile0, p.DK, p.DV, col, lane);
  const int first_chunk = sp.t0 / DCH;
  double gall = 1.;
  __syncthreads();
  for (int c = 0; c < nc; ++c) {
    __syncthreads();
    const unsigned char* buf = smem + (c % NB) * Sh::BUF;
    const DecayTab& tb = tabs[c % NB];
    const int rows = sp.len - c * DCH;
    f32x4 oa[Sp::RO];
    float* oc = OUT ? o + (int64_t)c * DCH * o_ts : nullptr;
    // (addresses are formed anew in every chunk: kept over the loop, those of all eight waves' code would not fit
    // the registers)
    int ln = lane;
    asm volatile("" : "+v"(ln));
    if constexpr (OUT) {
      by_wave<Sp::G>(m, [&](auto M) { chunk_first<W, CT, InT, M.value>(qbuf, st, oa, xch, ct, ln); });
    }
    __syncthreads();
    by_wave<Sp::G>(m, [&](auto M) {
      chunk_second<W, CT, InT, OUT, M.value>(buf, tb, st, oa, Pt, xch, oc, (int)o_ts, rows, ct, ln);
    });
    if (local) gall *= tb.whole[0] * tb.whole[1] * tb.whole[2] * tb.whole[3];
    if (!local && p.snap && m < Sp::IS && rows >= DCH && (first_chunk + c + 1) % p.snap_chunks == 0) {
      const int64_t per = p.T / DCH / p.snap_chunks;  // fixed length: snapshots per sequence
      const int64_t row = (p.cu ? p.snap_first[sp.n] : sp.n * per) + (first_chunk + c + 1) / p.snap_chunks - 1;
      int cl = col, dv = p.DV;  // (formed here, not kept over the loop: see above)
      asm volatile("" : "+v"(cl), "+s"(dv));
      state_store<W>(st, p.snap + (row * p.H + h) * hsz, tile0, p.DK, dv, cl, ln);
    }
    if constexpr (NB == 1) __syncthreads();
  }
  if (local) {
    if (m < Sp::IS) state_store<W>(st, p.part + ((int64_t)slot * p.H + h) * hsz, tile0, p.DK, p.DV, col, lane);
    if (tid == 0 && cb == 0) p.gpart[(int64_t)slot * p.H + h] = gall;
  } else if (p.S && m < Sp::IS && srow >= 0 && sp.t0 + sp.len >= sp.total)
    state_store<W>(st, p.S + (srow * p.H + h) * hsz, tile0, p.DK, p.DV, col, lane);
}

template <int W, int CT, typename InT>
static hipError_t launch_main_t(DecayParams p, int local, hipStream_t s) {
  p.ncb = p.DV / (16 * CT);
  const int64_t grid = work_grid(p);
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const dim3 blocks((unsigned)grid);
  if (p.o && !local)
    hipLaunchKernelGGL((decay_main_kernel<W, CT, InT, true>), blocks, dim3(64 * (MAIN_WAVES + FILL_WAVES)), 0, s, p, local);
  else
    hipLaunchKernelGGL((decay_main_kernel<W, CT, InT, false>), blocks, dim3(64 * (MAIN_WAVES + FILL_WAVES)), 0, s, p, local);
  return hipGetLastError();
}
template <int W, typename InT>
static hipError_t launch_main_w(const DecayParams& p, const DecayPlan& pl, int local, hipStream_t s) {
  switch (pl.ct) {
    case 8: if constexpr (sizeof(InT) == 2) return launch_main_t<W, 8, InT>(p, local, s);
    case 4: if constexpr (sizeof(InT) == 2) return launch_main_t<W, 4, InT>(p, local, s);
    case 2: if constexpr (sizeof(InT) == 2 || W < 128) return launch_main_t<W, 2, InT>(p, local, s);
    default: return launch_main_t<W, 1, InT>(p, local, s);
  }
}
template <typename InT>
static hipError_t launch_main(const DecayParams& p, const DecayPlan& pl, int local, hipStream_t s) {
  if (p.DK == 128) return launch_main_w<128, InT>(p, pl, local, s);
  if (p.DK == 64) return launch_main_w<64, InT>(p, pl, local, s);
  return launch_main_w<32, InT>(p, pl, local, s);
}

// ---------------------------------------------------------------------------
// State pass: the states at chunk boundaries without the outputs. Forward: S <- Gamma_C S + K^T (tail . V).
// Reverse (state gradients): dS <- Gamma_C dS + Q^T (Gamma . dO), chunks from the last to the first. The rows
// of V or dO are scaled and cut into three bf16 terms once, as they go into LDS; the waves split the key
// channels, so what remains is LDS reads and MFMA.
//   LOCAL:  every segment's own contribution (from zero) into part, its decay into gpart
//   CHUNKS: the state at each chunk's start (reverse: the gradient at its end) into cs / ds, from the
//           segment's start state
// ---------------------------------------------------------------------------
// The state pass's accumulators hold the state's transpose (columns 4 (l / 16) + i of a column tile, channel by frag_chan
// in lane l % 16), so that a lane loads and stores 16 bytes of a row.
template <int W, bool STORE, class P>
__device__ __forceinline__ void state_rows(f32x4& st, P* at, int t, int DK, int DV, int col0, int lane) {
  const int r16 = lane & 15, ch = 32 * (t >> 1) + 8 * (r16 >> 2) + 4 * (t & 1) + (r16 & 3);
  if (W == 32 && ch >= DK) return;
  if constexpr (STORE)
    *reinterpret_cast<f32x4*>(at + ch * DV + col0 + 4 * (lane >> 4)) = st;
  else
    st = *reinterpret_cast<const f32x4*>(at + ch * DV + col0 + 4 * (lane >> 4));
}

template <int W, int CT, int DC, typename XT>
constexpr int state_buf() {
  return Terms<XT>::N * DC * W * 2 + 3 * DC * CT * 32;
}
template <int W, int CT, int DC, typename XT, typename YT, bool REV>
__device__ __forceinline__ void state_body(const DecayParams& p, int local, unsigned char* smem, double* s_gam) {
  constexpr int NPX = Terms<XT>::N;
  constexpr int IW = W / 16 < 4 ? W / 16 : 4, TI = W / 16 / IW, CW = 4 / IW, TC = CT / CW > 0 ? CT / CW : 1;
  constexpr int XB = DC * W * 2, YB = DC * CT * 32, BUF = NPX * XB + 3 * YB;
  constexpr int NB = NPX == 1 ? 2 : 1;
  int cb, h, slot;
  if (!work_of(p, cb, h, slot)) return;
  const Span sp = slot_span(p, slot);
  if (sp.n < 0) return;
  // nothing comes behind the last segment (before the first, in reverse)
  if (local && (REV ? sp.t0 == 0 : sp.t0 + sp.len >= sp.total)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % IW, wc = wave / IW;
  const bool active = wc * TC < CT;
  const int hk = h / (p.H / p.Hk);
  const int64_t trow = sp.b * p.T + sp.row0;
  const int64_t x_ts = REV ? p.q_ts : p.k_ts, y_ts = REV ? (int64_t)p.H * p.DV : p.v_ts;
  const XT* x = static_cast<const XT*>(REV ? p.q : p.k) + sp.b * (REV ? p.q_bs : p.k_bs) + sp.row0 * x_ts + (int64_t)hk * p.DK;
  const YT* y = (REV ? reinterpret_cast<const YT*>(p.dO) + trow * y_ts
                     : static_cast<const YT*>(p.v) + sp.b * p.v_bs + sp.row0 * y_ts) + (int64_t)h * p.DV + cb * 16 * CT;
  const float* al = p.alpha + (p.a_tok ? trow * p.H : 0) + h;
  const int64_t a_ts = p.a_tok ? p.H : 0;
  const int64_t hsz = (int64_t)p.DK * p.DV;
  float* part = REV ? p.rpart : p.part;
  const float* src = nullptr;
  if (!local) {
    if (part)
      src = part + ((int64_t)slot * p.H + h) * hsz;
    else if (REV ? p.dST != nullptr : p.S0 != nullptr)
      src = (REV ? p.dST : p.S0) + ((int64_t)sp.n * p.H + h) * hsz;
  }
  f32x4 st[TC][TI];
  const int t0 = wi * TI, col0 = cb * 16 * CT + 16 * wc * TC;
#pragma unroll
  for (int tc = 0; tc < TC; ++tc)
#pragma unroll
    for (int ti = 0; ti < TI; ++ti) {
      st[tc][ti] = f32x4{0, 0, 0, 0};
      if (active && src) state_rows<W, false>(st[tc][ti], src, t0 + ti, p.DK, p.DV, col0 + 16 * tc, lane);
    }
  auto save = [&](float* dst) {
    if (!active) return;
#pragma unroll
    for (int tc = 0; tc < TC; ++tc)
#pragma unroll
      for (int ti = 0; ti < TI; ++ti) state_rows<W, true>(st[tc][ti], dst, t0 + ti, p.DK, p.DV, col0 + 16 * tc, lane);
  };

  // two chunks on their way: with one, the loads' latency is the chunk's time (229 us on 4 x 4096 tokens,
  // 16 heads, d = 128; 218 so)
  Stage<W, XT, DC> sx[2];
  Stage<16 * CT, YT, DC, false> sy[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sx[e].init(x_ts, p.DK, tid);
    sy[e].init(y_ts, 16 * CT, tid);
  }
  float a_next[2] = {1.f, 1.f};
  const int nc = pieces(sp.len, DC);
  auto chunk_of = [&](int i) { return REV ? nc - 1 - i : i; };
  auto fetch = [&](int i, auto E) {  // chunk i (past the end the last one: no branch, see the main pass)
    constexpr int e = E.value;
    const int64_t c0 = (int64_t)chunk_of(i < nc ? i : nc - 1) * DC;
    const int rows = sp.len - (int)c0, t = lane & (DC - 1);
    sx[e].load(x + c0 * x_ts, x_ts, rows);
    sy[e].load(y + c0 * y_ts, y_ts, rows);
    a_next[e] = al[(c0 + (t < rows ? t : rows - 1)) * a_ts];
  };
  auto put = [&](int i, auto E) {
    constexpr int e = E.value;
    const int rows = sp.len - chunk_of(i) * DC;
    unsigned char* buf = smem + (i % NB) * BUF;
    sx[e].store(buf, XB, rows, p.DK, tid);
    sy[e].mask(rows, 16 * CT, tid);
    if (lane >= DC || lane >= rows) a_next[e] = 1.f;
    double all;
    const float wt = chunk_weight<REV>(a_next[e], lane, all);
    if (tid == 0) s_gam[i % NB] = all;
#pragma unroll
    for (int j = 0; j < sy[e].NPC; ++j) {
      const float f = __shfl(wt, sy[e].row + j * sy[e].STEP);
      if (sy[e].mine(j, tid)) scaled_store(sy[e].x[j], f, buf + NPX * XB + sy[e].at + j * sy[e].STEP * CT * 32, YB);
    }
  };
  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  if (nc > 0) {
    fetch(0, Even{});
    fetch(1, Odd{});
    // (the initial states' loads end here: else every chunk of the loop waits as if they were still on their way, for
    // the loads behind them as well)
#pragma unroll
    for (int tc = 0; tc < TC; ++tc)
#pragma unroll
      for (int ti = 0; ti < TI; ++ti) asm volatile("" : "+v"(st[tc][ti]));
    put(0, Even{});
    fetch(2, Even{});
  }
  const int64_t cslot0 = (p.cu ? (local ? 0 : p.chunk_first[sp.n]) : (int64_t)sp.n * ((p.T + DC - 1) / DC)) + sp.t0 / DC;
  double gall = 1.;
  auto step = [&](int i, auto E) {  // E: where chunk i + 1 is
    __syncthreads();
    if constexpr (NB == 2) {
      if (i + 1 < nc) put(i + 1, E);
      fetch(i + 3, E);
    }
    if (!local) save((REV ? p.ds : p.cs) + ((cslot0 + chunk_of(i)) * p.H + h) * hsz);
    const unsigned char* buf = smem + (i % NB) * BUF;
    const double all = s_gam[i % NB];
    const Factor G(all);
    gall *= all;
    if (active) {
      bf16x8 yf[TC][DC / 32][3];
#pragma unroll
      for (int tc = 0; tc < TC; ++tc)
#pragma unroll
        for (int u = 0; u < DC / 32; ++u)
#pragma unroll
          for (int e = 0; e < 3; ++e)
            yf[tc][u][e] = frag_cols<16 * CT>(buf + NPX * XB + e * YB, 16 * (wc * TC + tc), u, lane);
#pragma unroll
      for (int ti = 0; ti < TI; ++ti) {
        const int t = wi * TI + ti;
#pragma unroll
        for (int tc = 0; tc < TC; ++tc) G.scale(st[tc][ti]);
#pragma unroll
        for (int u = 0; u < DC / 32; ++u) {
          bf16x8 xf[NPX];
#pragma unroll
          for (int e = 0; e < NPX; ++e) xf[e] = frag_chan<W>(buf + e * XB, t >> 1, t & 1, u, lane);
#pragma unroll
          for (int tc = 0; tc < TC; ++tc) mma(st[tc][ti], yf[tc][u], xf);
        }
      }
    }
    if constexpr (NB == 1) {
      __syncthreads();
      if (i + 1 < nc) put(i + 1, E);
      fetch(i + 3, E);
    }
  };
  int i = 0;
  for (; i + 1 < nc; i += 2) {
    step(i, Odd{});
    step(i + 1, Even{});
  }
  if (i < nc) step(i, Odd{});
  if (local) {
    save(part + ((int64_t)slot * p.H + h) * hsz);
    if (tid == 0 && cb == 0) (REV ? p.rgpart : p.gpart)[(int64_t)slot * p.H + h] = gall;
  } else if (REV && p.dS0 && sp.t0 == 0) {
    save(p.dS0 + ((int64_t)sp.n * p.H + h) * hsz);
  }
}

// Both directions in one launch (blockIdx.y): each alone leaves half of the CUs' places empty.
template <int W, int CT, int DC, typename XT>
__global__ __launch_bounds__(256) void decay_state_kernel(const DecayParams p, int local) {
  constexpr int NB = Terms<XT>::N == 1 ? 2 : 1;
  __shared__ __align__(16) unsigned char smem[NB * state_buf<W, CT, DC, XT>()];
  __shared__ double s_gam[NB];
  if (blockIdx.y == 0)
    state_body<W, CT, DC, XT, XT, false>(p, local, smem, s_gam);
  else
    state_body<W, CT, DC, XT, float, true>(p, local, smem, s_gam);
}

// Segments joined: the state at each segment's start (reverse: the gradient at its end) from the
// segments' own contributions, in their place. One thread per 4 elements walks the sequence's segments.
__global__ __launch_bounds__(256) void decay_join_kernel(const DecayParams p) {
  const int rev = blockIdx.y;
  const int64_t hsz = (int64_t)p.DK * p.DV;
  const int per = (int)((hsz / 4 + 255) / 256);  // workgroups per (sequence, head)
  const int nh = blockIdx.x / per, n = nh / p.H, h = nh - n * p.H;
  const int64_t e = ((int64_t)(blockIdx.x - nh * per) * 256 + threadIdx.x) * 4;
  if (e >= hsz) return;
  int first, ns;
  if (p.cu) {
    first = p.slot_first[n];
    ns = p.slot_first[n + 1] - first;
  } else {
    first = n * p.nseg;
    ns = p.nseg;
  }
  int64_t srow = n;
  if (!rev && p.sidx) {
    srow = p.sidx[n];
    if (srow < 0 || srow >= p.nslots) srow = -1;
  }
  const float* init = rev ? p.dST : p.S0;
  f32x4 x = {0, 0, 0, 0};
  if (init && srow >= 0) x = *reinterpret_cast<const f32x4*>(init + (srow * p.H + h) * hsz + e);
  float* part = rev ? p.rpart : p.part;
  for (int j = 0; j < ns; ++j) {
    const int64_t sl = (int64_t)(first + (rev ? ns - 1 - j : j)) * p.H + h;
    f32x4* at = reinterpret_cast<f32x4*>(part + sl * hsz + e);
    if (j + 1 < ns) {
      const f32x4 own = *at;
      const double G = (rev ? p.rgpart : p.gpart)[sl];
      *at = x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (float)__builtin_fma(G, (double)x[i], (double)own[i]);
    } else {
      *at = x;
    }
  }
}

template <int W, int CT, int DC, typename XT>
static hipError_t launch_state_t(DecayParams p, int local, hipStream_t s) {
  p.ncb = p.DV / (16 * CT);
  const int64_t grid = work_grid(p);
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((decay_state_kernel<W, CT, DC, XT>), dim3((unsigned)grid, 2), dim3(256), 0, s, p, local);
  return hipGetLastError();
}
template <int W, int DC, typename XT>
static hipError_t launch_state_w(const DecayParams& p, int local, hipStream_t s) {
  return state_tiles(p.DV) == 2 ? launch_state_t<W, 2, DC, XT>(p, local, s) : launch_state_t<W, 1, DC, XT>(p, local, s);
}
template <int DC, typename XT>
static hipError_t launch_state(const DecayParams& p, int local, hipStream_t s) {
  if (p.DK == 128) return launch_state_w<128, DC, XT>(p, local, s);
  if (p.DK == 64) return launch_state_w<64, DC, XT>(p, local, s);
  return launch_state_w<32, DC, XT>(p, local, s);
}
hipError_t launch_decay_states(const DecayParams& p, bool bf16, int local, hipStream_t s) {
  return bf16 ? launch_state<decay_bwd_chunk(true), __bf16>(p, local, s)
              : launch_state<decay_bwd_chunk(false), float>(p, local, s);
}
hipError_t launch_decay_join(const DecayParams& p, bool both, hipStream_t s) {
  const int64_t grid = join_grid(p);
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(decay_join_kernel, dim3((unsigned)grid, both ? 2 : 1), dim3(256), 0, s, p);
  return hipGetLastError();
}
hipError_t launch_decay_plan(const DecayParams& p, hipStream_t s) {
  hipLaunchKernelGGL(decay_plan_kernel, dim3(1), dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_decay_fwd(DecayParams p, const DecayPlan& pl, bool bf16, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.cu) {
    e = launch_decay_plan(p, s);
    if (e != hipSuccess) return e;
    p.cu = p.cu_ok;
  }
  if (pl.nseg > 1) {
    e = bf16 ? launch_main<__bf16>(p, pl, 1, s) : launch_main<float>(p, pl, 1, s);
    if (e == hipSuccess) e = launch_decay_join(p, false, s);
    if (e != hipSuccess) return e;
  } else {
    p.part = nullptr;
  }
  return bf16 ? launch_main<__bf16>(p, pl, 0, s) : launch_main<float>(p, pl, 0, s);
}

}  // namespace dr
