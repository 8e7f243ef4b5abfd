// Gradients of the decayed linear attention on gfx950.
//
// The state passes of decay.hip leave, for every chunk, the state S at its start and the state gradient G at
// its end (the gradient reaching the state after the chunk's last token). One workgroup per (chunk, head) then
// forms the chunk's gradients. With ratio(r, s) = a_{s+1} ... a_r, Gamma_r the product from the chunk's
// start, tail_s the product behind s, P = (Q K^T) . ratio and E = (dO V^T) . ratio:
//
//   dQ = E K + Gamma . (dO S^T),   dK = E^T Q + tail . (V G^T),   dV = P^T dO + tail . (K G)
//
// The decay's gradient is the sum over every path that passes its token, each without that token's own
// factor, so it needs no quotient and holds for zero and negative decays:
//
//   da_t = sum_{r>=t} ratio(r, t) y_t[r] + tail_t y_t[end],   y_t[r] = sum_{s<t} ratio(t-1, s) A[r, s] + Gamma_{t-1} X_r
//   A[r, s] = (q_r . k_s)(dO_r . v_s),  X_r = q_r^T S dO_r,  A[end, s] = Y_s = k_s^T G v_s,  X_end = <S, G>
//
// sum_s ratio(t, s) A[r, s] is one more 64-deep product; the X part is a scan over tokens, as is the end row.
// All products are fp32-grade: fp32 operands are cut into three bf16 terms (decay.hpp).
//
// What bounds it: S and G in fp32 for every chunk, read once each (131 KB a chunk of 64 tokens at d = 128, beside
// 180 KB of inputs and gradients), and one workgroup a CU (162 KB of LDS), whose loads and products do not
// overlap those of another. 4 x 4096 tokens, 16 heads, d = 128, bf16: 350 us, 3.8 TB/s (a copy 5.2; four waves that took
// the two halves of the work in turn 489, with 13 registers spilled 376), after 217 us of the state passes (4.2 TB/s).
#include "decay.hpp"
#include "launch.hpp"

namespace dr {

template <int W, int V, typename InT, int DC>
struct GradShape {
  static constexpr int NP = Terms<InT>::N;
  static constexpr int QK = DC * W * 2, VO = DC * V * 2;  // bytes of one plane
  static constexpr int EP = DC + 8;                       // row pitch of P and E (bf16): no bank conflicts
  static constexpr int EB = DC * EP * 2;
  static constexpr int OFF_K = NP * QK, OFF_V = 2 * NP * QK, OFF_O = OFF_V + NP * VO, OFF_P = OFF_O + 3 * VO,
                       OFF_E = OFF_P + 3 * EB, BYTES = OFF_E + 3 * EB;
};

// ratio(r, s) of row tile R and column tile S <= R: lane r = 16 R + r16, values s = 16 S + 4 g + i
__device__ __forceinline__ f32x4 ratio_row(const DecayTab& tb, const float (&P)[4], int R, int S, int r16, int g) {
  f32x4 x;
  if (S == R) {
    const f32x4 in = *reinterpret_cast<const f32x4*>(&tb.in[S][r16 * LDP + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = r16 >= 4 * g + i ? in[i] : 0.f;
  } else {
    float f = tb.pre[16 * R + r16];
    for (int j = S + 1; j < R; ++j) f *= P[j];
    const f32x4 suf = *reinterpret_cast<const f32x4*>(&tb.suf[16 * S + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f * suf[i];
  }
  return x;
}
// lane s = 16 S + c16, values r = 16 R + 4 g + i
__device__ __forceinline__ f32x4 ratio_col(const DecayTab& tb, const float (&P)[4], int R, int S, int c16, int g) {
  f32x4 x;
  if (S == R) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 4 * g + i >= c16 ? tb.in[S][(4 * g + i) * LDP + c16] : 0.f;
  } else {
    float f = tb.suf[16 * S + c16];
    for (int j = S + 1; j < R; ++j) f *= P[j];
    const f32x4 pre = *reinterpret_cast<const f32x4*>(&tb.pre[16 * R + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f * pre[i];
  }
  return x;
}

// Rows of tile R: P = (Q K^T) . ratio and E = (dO V^T) . ratio as bf16 terms into LDS, and their path sums
// sum_r ratio(r, t) sum_{s<t} ratio(t-1, s) A[r, s] for the tile's rows r. R is a template argument: the tiles
// of A are then registers that no index selects at run time, and the loops over them straight code.
template <int W, int V, typename InT, int DC, int R>
__device__ __forceinline__ void grad_rows(unsigned char* sm, const DecayTab& tb, const float (&PT)[4], float* s_da, int lane) {
  using Sh = GradShape<W, V, InT, DC>;
  constexpr int NP = Sh::NP, NS = R + 2 - (R & 1), UW = W / 32, UV = V / 32;  // NS: tiles of the 32 tokens halves
  const int g = lane >> 4, r16 = lane & 15;
  const unsigned char *Qt = sm, *Kt = sm + Sh::OFF_K, *Vt = sm + Sh::OFF_V, *Ot = sm + Sh::OFF_O;
  Op<NP> qf[UW];
  bf16x8 of[UV][3];
#pragma unroll
  for (int u = 0; u < UW; ++u)
#pragma unroll
    for (int i = 0; i < NP; ++i) qf[u].t[i] = frag_rows<W>(Qt + i * Sh::QK, 16 * R, u, lane);
#pragma unroll
  for (int u = 0; u < UV; ++u)
#pragma unroll
    for (int i = 0; i < 3; ++i) of[u][i] = frag_rows<V>(Ot + i * Sh::VO, 16 * R, u, lane);
  f32x4 A[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    f32x4 qk = {0, 0, 0, 0}, ov = {0, 0, 0, 0};
    A[s] = f32x4{0, 0, 0, 0};
    if (s <= R) {
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        Op<NP> kf;
#pragma unroll
        for (int i = 0; i < NP; ++i) kf.t[i] = frag_rows<W>(Kt + i * Sh::QK, 16 * s, u, lane);
        mma(qk, kf.t, qf[u].t);
      }
#pragma unroll
      for (int u = 0; u < UV; ++u) {
        Op<NP> vf;
#pragma unroll
        for (int i = 0; i < NP; ++i) vf.t[i] = frag_rows<V>(Vt + i * Sh::VO, 16 * s, u, lane);
        mma(ov, vf.t, of[u]);
      }
      const f32x4 L = ratio_row(tb, PT, R, s, r16, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        A[s][i] = qk[i] * ov[i];
        qk[i] *= L[i];
        ov[i] *= L[i];
      }
    }
    const int at = ((16 * R + r16) * Sh::EP + 16 * s + 4 * g) * 2;
    split_store4(sm + Sh::OFF_P + at, Sh::EB, qk);
    split_store4(sm + Sh::OFF_E + at, Sh::EB, ov);
  }
  // M[r, t] = sum_{s <= t} ratio(t, s) A[r, s];  y_t = M[., t - 1]
  f32x4 prev = {0, 0, 0, 0};  // the previous tile of M
#pragma unroll
  for (int t = 0; t <= R; ++t) {
    f32x4 M = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < t / 2 + 1; ++u) {
      const f32x4 l0 = ratio_row(tb, PT, t, 2 * u, r16, g);
      f32x4 l1 = {0, 0, 0, 0};
      if (2 * u + 1 <= t) l1 = ratio_row(tb, PT, t, 2 * u + 1, r16, g);
      const f32x4 a0 = A[2 * u], a1 = A[2 * u + 1];
      const float lx[8] = {l0[0], l0[1], l0[2], l0[3], l1[0], l1[1], l1[2], l1[3]};
      const float ax[8] = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
      const Tri lf = split3(lx), af = split3(ax);
      mma(M, af.t, lf.t);  // rows r, columns t
    }
    const f32x4 rc = ratio_col(tb, PT, R, t, r16, g);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // column t - 1: the lane to the left, or the previous tile's last column
      const float left = dpp_or<ROW_SHR1>(0.f, M[i]);
      const float edge = __shfl(prev[i], (lane & 48) + 15);
      sum += rc[i] * (r16 == 0 ? edge : left);
    }
    prev = M;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0) s_da[16 * t + r16] = sum;
  }
}

template <int W, int V, typename InT, int DC>
__global__ __launch_bounds__(512) void decay_grad_kernel(const DecayParams p) {
  using Sh = GradShape<W, V, InT, DC>;
  constexpr int NP = Sh::NP, NT = DC / 16, NU = DC / 32, UW = W / 32, UV = V / 32, NTH = 512;
  constexpr int NIT = W / 16, TI = NIT >= 4 ? NIT / 4 : 1, NVT = V / 16, TV = NVT >= 4 ? NVT / 4 : 1;
  __shared__ __align__(16) unsigned char sm[Sh::BYTES];
  __shared__ __align__(16) DecayTab tb;
  __shared__ float s_x[4][DC], s_y[4][DC], s_da[4][DC], s_z[4];
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  if (id >= p.grid) return;
  const int h = id % p.H, cslot = id / p.H;
  // the chunk's sequence and rows
  int n, c0, len;
  int64_t b, row0;
  if (p.cu) {
    n = p.chunk_seq[cslot];
    if (n < 0) return;
    c0 = (cslot - p.chunk_first[n]) * DC;
    len = p.cu[n + 1] - p.cu[n] - c0;
    b = 0;
    row0 = (int64_t)p.cu[n] + c0;
  } else {
    const int per = (int)((p.T + DC - 1) / DC);
    n = cslot / per;
    c0 = (cslot - n * per) * DC;
    len = (int)(p.T - c0);
    b = n;
    row0 = c0;
  }
  if (len <= 0) return;  // an empty sequence's slot
  if (len > DC) len = DC;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hk = h / (p.H / p.Hk);
  const int64_t trow = b * p.T + row0;
  const int64_t hsz = (int64_t)p.DK * p.DV;
  const float* S = p.cs + ((int64_t)cslot * p.H + h) * hsz;
  const float* G = p.ds + ((int64_t)cslot * p.H + h) * hsz;
  const int64_t o_ts = (int64_t)p.H * p.DV;
  const bool second = wave >= 4;  // waves 0-3: P, E and the path sums, then dV; waves 4-7: dQ and dK
  const int rw = wave & 3;

  // rows of S and G as operands along the value columns (dQ, dK): channel as frag_chan has it
  auto load_sg = [&](int ti, int u, float (&sx)[8], float (&gx)[8]) {
    const int it = rw * TI + ti, ch = 32 * (it >> 1) + 8 * (r16 >> 2) + 4 * (it & 1) + (r16 & 3), nn = 32 * u + 8 * g;
    const bool ok = (W > 32 || ch < p.DK) && (V > 32 || nn < p.DV);
    const int at = ok ? ch * p.DV + nn : 0;
    load8(S + at, sx);
    load8(G + at, gx);
    if (W == 32 || V == 32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sx[j] = ok ? sx[j] : 0.f;
        gx[j] = ok ? gx[j] : 0.f;
      }
    }
  };
  // columns of G as operands along the channels (dV)
  auto load_g = [&](int tv, int u, float (&gx)[8]) {
    const int vt = rw * TV + tv, col = 32 * (vt >> 1) + 8 * (r16 >> 2) + 4 * (vt & 1) + (r16 & 3);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ch = 32 * u + 8 * g + j;
      const bool ok = (W > 32 || ch < p.DK) && (V > 32 || col < p.DV);
      gx[j] = G[ok ? ch * p.DV + col : 0];
      if (W == 32 || V == 32) gx[j] = ok ? gx[j] : 0.f;
    }
  };
  // the first tile's rows of S and G are on their way while the inputs go to LDS
  float sx[UV][8], gx[UV][8];
  {
    Stage<W, InT, DC, true, NTH> sq, sk;
    Stage<V, InT, DC, true, NTH> sv;
    Stage<V, float, DC, true, NTH> so;
    sq.init(p.q_ts, p.DK, tid);
    sk.init(p.k_ts, p.DK, tid);
    sv.init(p.v_ts, p.DV, tid);
    so.init(o_ts, p.DV, tid);
    const int t = 16 * rw + r16;
    float a = p.alpha[(p.a_tok ? (trow + (t < len ? t : len - 1)) * p.H : 0) + h];
    sq.load(static_cast<const InT*>(p.q) + b * p.q_bs + row0 * p.q_ts + (int64_t)hk * p.DK, p.q_ts, len);
    sk.load(static_cast<const InT*>(p.k) + b * p.k_bs + row0 * p.k_ts + (int64_t)hk * p.DK, p.k_ts, len);
    sv.load(static_cast<const InT*>(p.v) + b * p.v_bs + row0 * p.v_ts + (int64_t)h * p.DV, p.v_ts, len);
    so.load(p.dO + trow * o_ts + (int64_t)h * p.DV, o_ts, len);
    fence();
    if (second && rw * TI < NIT) {
#pragma unroll
      for (int u = 0; u < UV; ++u) load_sg(0, u, sx[u], gx[u]);
    }
    fence();
    if (t >= len) a = 1.f;
    if (!second) decay_table(tb, rw, a, lane);
    sq.store(sm, Sh::QK, len, p.DK, tid);
    sk.store(sm + Sh::OFF_K, Sh::QK, len, p.DK, tid);
    sv.store(sm + Sh::OFF_V, Sh::VO, len, p.DV, tid);
    so.store(sm + Sh::OFF_O, Sh::VO, len, p.DV, tid);
  }
  if (tid < 4 * DC) {
    (&s_da[0][0])[tid] = 0.f;
    (&s_x[0][0])[tid] = 0.f;
    (&s_y[0][0])[tid] = 0.f;
  }
  if (tid < 4) s_z[tid] = 0.f;
  __syncthreads();
  float PT[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) PT[i] = tb.tile[i];
  const unsigned char *Qt = sm, *Kt = sm + Sh::OFF_K, *Vt = sm + Sh::OFF_V, *Ot = sm + Sh::OFF_O;

  if (!second) {
    // ---- P and E into LDS, the path sums of the decay's gradient: wave w, rows of tile w
    if (wave == 0)
      grad_rows<W, V, InT, DC, 0>(sm, tb, PT, s_da[0], lane);
    else if (wave == 1)
      grad_rows<W, V, InT, DC, 1>(sm, tb, PT, s_da[1], lane);
    if constexpr (NT == 4) {
      if (wave == 2)
        grad_rows<W, V, InT, DC, 2>(sm, tb, PT, s_da[2], lane);
      else if (wave == 3)
        grad_rows<W, V, InT, DC, 3>(sm, tb, PT, s_da[3], lane);
    }
    // ---- dV, the wave's value-column tiles: tail . (K G), then P^T dO
    f32x4 av[TV][NT];
    if (rw * TV < NVT) {
#pragma unroll
      for (int tv = 0; tv < TV; ++tv) {
#pragma unroll
        for (int r = 0; r < NT; ++r) av[tv][r] = f32x4{0, 0, 0, 0};
        float gc[UW][8];
#pragma unroll
        for (int u = 0; u < UW; ++u) load_g(tv, u, gc[u]);
        fence();
#pragma unroll
        for (int u = 0; u < UW; ++u) {
          const Tri gf = split3(gc[u]);
          bf16x8 kf[NT][NP];
#pragma unroll
          for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int i = 0; i < NP; ++i) kf[r][i] = frag_rows<W>(Kt + i * Sh::QK, 16 * r, u, lane);
          mma_rows(av[tv], gf.t, kf);
        }
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          float tail = tb.suf[16 * r + r16];
#pragma unroll
          for (int j = r + 1; j < NT; ++j) tail *= PT[j];
#pragma unroll
          for (int i = 0; i < 4; ++i) av[tv][r][i] *= tail;
        }
      }
    }
    __syncthreads();
    if (rw * TV < NVT) {
#pragma unroll
      for (int tv = 0; tv < TV; ++tv) {
        const int vt = rw * TV + tv, w2 = vt >> 1, e2 = vt & 1;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          bf16x8 of[3];
#pragma unroll
          for (int e = 0; e < 3; ++e) of[e] = frag_chan<V>(Ot + e * Sh::VO, w2, e2, u, lane);
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            if (r <= 2 * u + 1) {
              bf16x8 pf[3];
#pragma unroll
              for (int e = 0; e < 3; ++e) pf[e] = frag_cols<Sh::EP>(sm + Sh::OFF_P + e * Sh::EB, 16 * r, u, lane);
              mma(av[tv][r], of, pf);
            }
          }
        }
        const int oc = 32 * w2 + 8 * g + 4 * e2;
        if (V > 32 || oc < p.DV) {
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            const int row = 16 * r + r16;
            if (row < len) *reinterpret_cast<f32x4*>(p.dv + (trow + row) * o_ts + (int64_t)h * p.DV + oc) = av[tv][r];
          }
        }
      }
    }
  } else {
    // ---- dQ and dK, the wave's channel tiles: Gamma . (dO S^T) and tail . (V G^T), then E K and E^T Q
    float xs[NT], ys[NT], z = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) xs[i] = ys[i] = 0.f;
    f32x4 aq[TI][NT], ak[TI][NT];
    if (rw * TI < NIT) {
#pragma unroll
      for (int ti = 0; ti < TI; ++ti) {
        const int it = rw * TI + ti, w2 = it >> 1, e2 = it & 1;
        if (ti > 0) {
#pragma unroll
          for (int u = 0; u < UV; ++u) load_sg(ti, u, sx[u], gx[u]);
          fence();
        }
#pragma unroll
        for (int r = 0; r < NT; ++r) aq[ti][r] = ak[ti][r] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < UV; ++u) {
#pragma unroll
          for (int j = 0; j < 8; ++j) z = fmaf(sx[u][j], gx[u][j], z);
          const Tri sf = split3(sx[u]);
          bf16x8 of[NT][3], vf[NT][NP];
#pragma unroll
          for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int i = 0; i < 3; ++i) of[r][i] = frag_rows<V>(Ot + i * Sh::VO, 16 * r, u, lane);
          mma_rows(aq[ti], sf.t, of);
          fence();  // (both products' operands at once do not fit the registers)
          const Tri gf = split3(gx[u]);
#pragma unroll
          for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int i = 0; i < NP; ++i) vf[r][i] = frag_rows<V>(Vt + i * Sh::VO, 16 * r, u, lane);
          mma_rows(ak[ti], gf.t, vf);
        }
        // X_r, Y_s from these channels, then the chunk's ends
        const int oc = 32 * w2 + 8 * g + 4 * e2;  // the lane's 4 output channels
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          const int row = 16 * r + r16, at = 16 * swz<W>(row, oc >> 3) + 2 * (oc & 7);
          float gam = tb.pre[row], tail = tb.suf[row];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j < r) gam *= PT[j];
            if (j > r) tail *= PT[j];
          }
          float qv[4] = {0.f, 0.f, 0.f, 0.f}, kv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = NP - 1; e >= 0; --e) {
            const bf16x4 q4 = *reinterpret_cast<const bf16x4*>(Qt + e * Sh::QK + at);
            const bf16x4 k4 = *reinterpret_cast<const bf16x4*>(Kt + e * Sh::QK + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              qv[i] += (float)q4[i];
              kv[i] += (float)k4[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xs[r] = fmaf(qv[i], aq[ti][r][i], xs[r]);
            ys[r] = fmaf(kv[i], ak[ti][r][i], ys[r]);
            aq[ti][r][i] *= gam;
            ak[ti][r][i] *= tail;
          }
        }
      }
    }
    __syncthreads();
    if (rw * TI < NIT) {
#pragma unroll
      for (int ti = 0; ti < TI; ++ti) {
        const int it = rw * TI + ti, w2 = it >> 1, e2 = it & 1, oc = 32 * w2 + 8 * g + 4 * e2;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          Op<NP> kf, qf;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            kf.t[i] = frag_chan<W>(Kt + i * Sh::QK, w2, e2, u, lane);
            qf.t[i] = frag_chan<W>(Qt + i * Sh::QK, w2, e2, u, lane);
          }
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            if (r >= 2 * u) {  // tokens s of half u reach row tile r
              bf16x8 ef[3];
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                const unsigned char* at = sm + Sh::OFF_E + e * Sh::EB + ((16 * r + r16) * Sh::EP + 32 * u + 4 * g) * 2;
                ef[e] = join(*reinterpret_cast<const s16x4*>(at), *reinterpret_cast<const s16x4*>(at + 32));
              }
              mma(aq[ti][r], kf.t, ef);
            }
            if (r <= 2 * u + 1) {  // rows r' of half u reach token tile r
              bf16x8 ef[3];
#pragma unroll
              for (int e = 0; e < 3; ++e) ef[e] = frag_cols<Sh::EP>(sm + Sh::OFF_E + e * Sh::EB, 16 * r, u, lane);
              mma(ak[ti][r], qf.t, ef);
            }
          }
        }
        const int heads = p.dq_heads;  // heads of the buffers: Hk, or H for the partial sums of shared heads
        const int hq = heads == p.H ? h : hk;
        if (W > 32 || oc < p.DK) {
#pragma unroll
          for (int r = 0; r < NT; ++r) {
            const int row = 16 * r + r16;
            if (row < len) {
              const int64_t at = ((trow + row) * heads + hq) * p.DK + oc;
              *reinterpret_cast<f32x4*>(p.dq + at) = aq[ti][r];
              *reinterpret_cast<f32x4*>(p.dk + at) = ak[ti][r];
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        xs[r] += __shfl_xor(xs[r], 16);
        xs[r] += __shfl_xor(xs[r], 32);
        ys[r] += __shfl_xor(ys[r], 16);
        ys[r] += __shfl_xor(ys[r], 32);
        if (g == 0) {
          s_x[rw][16 * r + r16] = xs[r];
          s_y[rw][16 * r + r16] = ys[r];
        }
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) z += __shfl_xor(z, d);
      if (lane == 0) s_z[rw] = z;
    }
  }
  __syncthreads();

  // ---- D: the decay's gradient: path sums within the chunk, from its start and to its end
  if (wave == 0) {
    const int t = lane & (DC - 1);
    const int tile = t >> 4;
    float x = s_x[0][t] + s_x[1][t] + s_x[2][t] + s_x[3][t];
    float y = s_y[0][t] + s_y[1][t] + s_y[2][t] + s_y[3][t];
    const float da = s_da[0][t] + s_da[1][t] + s_da[2][t] + s_da[3][t];
    const float zz = s_z[0] + s_z[1] + s_z[2] + s_z[3];
    float a = p.alpha[(p.a_tok ? (trow + (t < len ? t : len - 1)) * p.H : 0) + h];
    if (t >= len) a = 1.f;
    float gam = tb.pre[t], tail = tb.suf[t];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j < tile) gam *= PT[j];
      if (j > tile) tail *= PT[j];
    }
    // forward scan of y_{t+1} = a_t y_t + Y_t: inclusive maps (m, c), y_{t+1} = m y_0 + c
    float m = a, c = y;
#pragma unroll
    for (int d = 1; d < DC; d <<= 1) {
      const float m0 = __shfl_up(m, d), c0_ = __shfl_up(c, d);
      if (t >= d) {
        c = fmaf(m, c0_, c);
        m *= m0;
      }
    }
    const float c_up = __shfl_up(c, 1), g_up = __shfl_up(gam, 1);  // (every lane takes part)
    const float c_before = t > 0 ? c_up : 0.f;
    const float g_before = t > 0 ? g_up : 1.f;
    const float y_end = fmaf(g_before, zz, c_before);
    // reverse scan of x_t = X_t + a_{t+1} x_{t+1}
    const float a_dn = __shfl_down(a, 1);
    m = t < DC - 1 ? a_dn : 0.f;
    c = x;
#pragma unroll
    for (int d = 1; d < DC; d <<= 1) {
      const float m0 = __shfl_down(m, d), c0_ = __shfl_down(c, d);
      if (t + d < DC) {
        c = fmaf(m, c0_, c);
        m *= m0;
      }
    }
    const float out = da + g_before * c + tail * y_end;
    if (lane < DC && t < len) p.dalpha[(trow + t) * p.H + h] = out;
  }
}

// Sums over the value heads of a query/key head: partial sums [rows, H, d_k] to [rows, Hk, d_k], rows of
// sequences only. One thread per 4 channels.
__global__ __launch_bounds__(256) void decay_shared_kernel(const DecayParams p, const float* pq, const float* pk) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t per = (int64_t)p.Hk * p.DK;
  const int64_t row = e / per;
  const int64_t rows = (int64_t)p.nbatch * p.T;
  if (row >= rows) return;
  if (p.cu && (row < p.cu[0] || row >= p.cu[p.nseq])) return;
  const int64_t in = e - row * per;
  const int hk = (int)(in / p.DK), ch = (int)(in - (int64_t)hk * p.DK), grp = p.H / p.Hk;
  f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  for (int j = 0; j < grp; ++j) {
    const int64_t at = (row * p.H + (int64_t)hk * grp + j) * p.DK + ch;
    a += *reinterpret_cast<const f32x4*>(pq + at);
    b += *reinterpret_cast<const f32x4*>(pk + at);
  }
  *reinterpret_cast<f32x4*>(p.dq + e) = a;
  *reinterpret_cast<f32x4*>(p.dk + e) = b;
}

// The gradient of one decay per head: the sum of the tokens' (rows of sequences only). One workgroup per head;
// every thread sums its rows in pairs of growing blocks' order, the same on every call.
__global__ __launch_bounds__(256) void decay_head_kernel(const DecayParams p, const float* da, float* out) {
  __shared__ float s_sum[256];
  const int h = blockIdx.x, tid = threadIdx.x;
  int64_t lo = 0, hi = (int64_t)p.nbatch * p.T;
  if (p.cu) {
    lo = p.cu[0];
    hi = p.cu[p.nseq];
  }
  float x = 0.f, low = 0.f;  // compensated: a long sum of one thread loses nothing
  for (int64_t r = lo + tid; r < hi; r += 256) {
    const float v = da[r * p.H + h], s = x + v, bb = s - x;
    low += (x - (s - bb)) + (v - bb);
    x = s;
  }
  s_sum[tid] = x + low;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (tid < d) s_sum[tid] += s_sum[tid + d];
    __syncthreads();
  }
  if (tid == 0) out[h] = s_sum[0];
}

template <int W, int V, typename InT>
static hipError_t launch_grad_t(const DecayParams& p, hipStream_t s) {
  constexpr int DC = decay_bwd_chunk(sizeof(InT) == 2);
  hipLaunchKernelGGL((decay_grad_kernel<W, V, InT, DC>), dim3((unsigned)grad_grid(p)), dim3(512), 0, s, p);
  return hipGetLastError();
}
template <int W, typename InT>
static hipError_t launch_grad_w(const DecayParams& p, hipStream_t s) {
  if (p.DV == 128) return launch_grad_t<W, 128, InT>(p, s);
  if (p.DV == 64) return launch_grad_t<W, 64, InT>(p, s);
  return launch_grad_t<W, 32, InT>(p, s);
}
template <typename InT>
static hipError_t launch_grad(const DecayParams& p, hipStream_t s) {
  if (p.DK == 128) return launch_grad_w<128, InT>(p, s);
  if (p.DK == 64) return launch_grad_w<64, InT>(p, s);
  return launch_grad_w<32, InT>(p, s);
}

hipError_t launch_decay_bwd(DecayParams p, const DecayPlan& pl, bool bf16, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.cu) {
    e = launch_decay_plan(p, s);
    if (e != hipSuccess) return e;
    p.cu = p.cu_ok;
  }
  if (pl.nseg > 1) {
    e = launch_decay_states(p, bf16, 1, s);
    if (e == hipSuccess) e = launch_decay_join(p, true, s);
  }
  if (e == hipSuccess) e = launch_decay_states(p, bf16, 0, s);
  if (e != hipSuccess || p.cslots == 0) {
    if (e == hipSuccess && p.head_da) {
      hipLaunchKernelGGL(decay_head_kernel, dim3((unsigned)p.H), dim3(256), 0, s, p, p.dalpha, p.head_da);
      e = hipGetLastError();
    }
    return e;
  }
  DecayParams g = p;
  g.dq_heads = p.Hk;
  if (p.H != p.Hk) {
    g.dq = p.pq;
    g.dk = p.pk;
    g.dq_heads = p.H;
  }
  g.grid = p.cslots * p.H;
  e = bf16 ? launch_grad<__bf16>(g, s) : launch_grad<float>(g, s);
  if (e == hipSuccess && p.H != p.Hk && p.T > 0) {
    hipLaunchKernelGGL(decay_shared_kernel, dim3((unsigned)shared_grid(p)), dim3(256), 0, s, p, p.pq, p.pk);
    e = hipGetLastError();
  }
  if (e == hipSuccess && p.head_da) {
    hipLaunchKernelGGL(decay_head_kernel, dim3((unsigned)p.H), dim3(256), 0, s, p, p.dalpha, p.head_da);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace dr
