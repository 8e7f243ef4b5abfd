// Prefill of the decayed linear attention S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t on gfx950.
//
// Per chunk of 64 tokens with start state S0 (ratio(r, s) = a_{s+1} ... a_r, Gamma_r the product from the
// chunk's start):
//
//   O = Gamma . (Q S0) + ((Q K^T) . ratio) V,     S <- Gamma_C S0 + K^T (ratio(C, .) . V)
//
// One workgroup of 4 waves carries 16 CT value columns of one head through one segment of a sequence;
// a wave holds the d_k x 16 state of one column tile in its accumulators for the whole segment. The
// layouts are chosen so that nothing but the inputs goes through LDS: the accumulators of K^T V are, lane
// for lane, the S^T operand of Q S0, and the accumulators of K Q^T are the P^T operand of P V (common
// index orders of the 32-deep products, see decay.hpp), so O^T comes out with 4 consecutive columns per
// lane and the state never leaves the registers. With fewer column tiles than waves, 4 / CT waves
// hold the same state columns and share the chunk's 16-token row tiles.
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
      c = ceil_one ? max((len + unit - 1) / unit, 1) : len / unit;
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
template <int W, int CT, typename InT>
struct MainShape {
  static constexpr int NP = Terms<InT>::N;
  static constexpr int NB = NP == 1 ? 2 : 1;  // fp32 data is held as three bf16 terms: one buffer fits
  static constexpr int QK = DCH * W * 2;      // bytes of one plane
  static constexpr int VB = DCH * CT * 32;
  static constexpr int BUF = NP * (2 * QK + VB);
};

// One chunk of a wave: row tiles R..., column tile at column n0 of the block.
template <int W, int CT, typename InT, bool OUT, int... R>
__device__ __forceinline__ void main_chunk(const unsigned char* buf, const DecayTab& tb, f32x4 (&st)[W / 16], int n0,
                                           float* o, int64_t o_ts, int rows, int lane) {
  using Sh = MainShape<W, CT, InT>;
  constexpr int NP = Sh::NP, U = W / 32;
  constexpr int RL[] = {R...};
  constexpr int NR = sizeof...(R);
  constexpr int RMAX = RL[NR - 1];
  const unsigned char* Qt = buf;
  const unsigned char* Kt = buf + NP * Sh::QK;
  const unsigned char* Vt = buf + 2 * NP * Sh::QK;
  const int g = lane >> 4, r16 = lane & 15;
  float P[4];
  f32x4 suf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    P[i] = tb.tile[i];
    suf[i] = *reinterpret_cast<const f32x4*>(&tb.suf[16 * i + 4 * g]);
  }
  Op<NP> vf[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < NP; ++i) vf[u].t[i] = frag_cols<16 * CT>(Vt + i * Sh::VB, n0, u, lane);

  if constexpr (OUT) {
    Op<NP> qf[NR][U];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NP; ++i) qf[n][u].t[i] = frag_rows<W>(Qt + i * Sh::QK, 16 * RL[n], u, lane);
    // Gamma . (Q S0), as its transpose
    f32x4 oa[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) oa[n] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float x[8] = {st[2 * u][0],     st[2 * u][1],     st[2 * u][2],     st[2 * u][3],
                          st[2 * u + 1][0], st[2 * u + 1][1], st[2 * u + 1][2], st[2 * u + 1][3]};
      const Tri sf = split3(x);
#pragma unroll
      for (int n = 0; n < NR; ++n) mma(oa[n], sf.t, qf[n][u].t);
    }
    float pre[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      pre[n] = tb.pre[16 * RL[n] + r16];
      float gam = pre[n];
#pragma unroll
      for (int j = 0; j < RL[n]; ++j) gam *= P[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) oa[n][i] *= gam;
    }
    // ((Q K^T) . ratio) V over the 32-token halves that reach the row tiles
#pragma unroll
    for (int u = 0; u < RMAX / 2 + 1; ++u) {
      f32x4 sc[NR][2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int S = 2 * u + a;
#pragma unroll
        for (int n = 0; n < NR; ++n) sc[n][a] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < (S <= RMAX ? U : 0); ++w) {
          Op<NP> kf;
#pragma unroll
          for (int i = 0; i < NP; ++i) kf.t[i] = frag_rows<W>(Kt + i * Sh::QK, 16 * S, w, lane);
#pragma unroll
          for (int n = 0; n < NR; ++n)
            if (RL[n] >= S) mma(sc[n][a], kf.t, qf[n][w].t);
        }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float x[8];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int S = 2 * u + a;
          if (S < RL[n]) {
            float f = pre[n];
#pragma unroll
            for (int j = S + 1; j < RL[n]; ++j) f *= P[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * a + i] = sc[n][a][i] * (f * suf[S][i]);
          } else if (S == RL[n]) {
            const f32x4 in = *reinterpret_cast<const f32x4*>(&tb.in[S][r16 * LDP + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * a + i] = r16 >= 4 * g + i ? sc[n][a][i] * in[i] : 0.f;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * a + i] = 0.f;
          }
        }
        if (RL[n] >= 2 * u) {
          const Tri pf = split3(x);
          mma(oa[n], vf[u].t, pf.t);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = 16 * RL[n] + r16;
      if (r < rows) *reinterpret_cast<f32x4*>(o + r * o_ts + n0 + 4 * g) = oa[n];
    }
  }

  // S <- Gamma_C S + K^T (ratio(C, .) . V)
  Tri vt[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
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
        for (int t = NP - 1; t >= 0; --t) y += (float)vf[u].t[t][4 * a + i];
        x[4 * a + i] = y * (suf[2 * u + a][i] * f);
      }
    }
    vt[u] = split3(x);
  }
  const float G = P[0] * P[1] * P[2] * P[3];
#pragma unroll
  for (int t = 0; t < W / 16; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) st[t][i] *= G;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Op<NP> kf;
#pragma unroll
      for (int i = 0; i < NP; ++i) kf.t[i] = frag_chan<W>(Kt + i * Sh::QK, t >> 1, t & 1, u, lane);
      mma(st[t], kf.t, vt[u].t);
    }
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

template <int W, int CT, typename InT, bool OUT>
__global__ __launch_bounds__(256) void decay_main_kernel(const DecayParams p) {
  using Sh = MainShape<W, CT, InT>;
  constexpr int NB = Sh::NB;
  __shared__ __align__(16) unsigned char smem[NB * Sh::BUF];
  __shared__ __align__(16) DecayTab tabs[NB];
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  if (id >= p.grid) return;
  const int cb = id % p.ncb, sh = id / p.ncb;
  const int h = sh % p.H, slot = sh / p.H;
  const Span sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ct = wave % CT, m = wave / CT;
  const int hk = h / (p.H / p.Hk);
  const InT* q = static_cast<const InT*>(p.q) + sp.b * p.q_bs + sp.row0 * p.q_ts + (int64_t)hk * p.DK;
  const InT* k = static_cast<const InT*>(p.k) + sp.b * p.k_bs + sp.row0 * p.k_ts + (int64_t)hk * p.DK;
  const InT* v = static_cast<const InT*>(p.v) + sp.b * p.v_bs + sp.row0 * p.v_ts + (int64_t)h * p.DV + cb * 16 * CT;
  const int64_t trow = sp.b * p.T + sp.row0;  // row in the dense per-token arrays
  const float* al = p.alpha + (p.a_tok ? trow * p.H : 0) + h;
  const int64_t a_ts = p.a_tok ? p.H : 0;
  const int64_t o_ts = (int64_t)p.H * p.DV;
  float* o = OUT ? p.o + trow * o_ts + (int64_t)h * p.DV + cb * 16 * CT : nullptr;

  // the state at the segment's start: lane's column l % 16, rows 32 u + 8 (l / 16) + 4 e + i
  const int col = cb * 16 * CT + 16 * ct + (lane & 15);
  const int64_t hsz = (int64_t)p.DK * p.DV;
  int64_t srow = sp.n;  // row of the state buffers
  if (p.sidx) {
    srow = p.sidx[sp.n];
    if (srow < 0 || srow >= p.nslots) srow = -1;
  }
  const float* src = p.part ? p.part + ((int64_t)slot * p.H + h) * hsz
                            : (p.S0 && srow >= 0 ? p.S0 + (srow * p.H + h) * hsz : nullptr);
  f32x4 st[W / 16];
  state_load<W>(st, src, 0, p.DK, p.DV, col, lane);

  Stage<W, InT> sq, sk;
  StageCols<16 * CT, InT> sv;
  float a_next = 1.f;
  const int nc = (sp.len + DCH - 1) / DCH;
  auto fetch = [&](int c) {
    const int c0 = c * DCH;
    if constexpr (OUT) sq.load(q, p.q_ts, c0, sp.len, p.DK, tid);
    sk.load(k, p.k_ts, c0, sp.len, p.DK, tid);
    sv.load(v, p.v_ts, c0, sp.len, tid);
    const int t = c0 + 16 * wave + (lane & 15);
    a_next = al[(int64_t)(t < sp.len ? t : sp.len - 1) * a_ts];
  };
  auto put = [&](int c) {
    const int c0 = c * DCH;
    unsigned char* buf = smem + (c % NB) * Sh::BUF;
    if constexpr (OUT) sq.store(buf, Sh::QK, c0, sp.len, p.DK, tid);
    sk.store(buf + Sh::NP * Sh::QK, Sh::QK, c0, sp.len, p.DK, tid);
    sv.store(buf + 2 * Sh::NP * Sh::QK, Sh::VB, c0, sp.len, tid);
    decay_table(tabs[c % NB], wave, c0 + 16 * wave + (lane & 15) < sp.len ? a_next : 1.f, lane);
  };
  if (nc > 0) {
    fetch(0);
    put(0);
  }
  const int first_chunk = sp.t0 / DCH;
  for (int c = 0; c < nc; ++c) {
    if (c + 1 < nc) fetch(c + 1);
    __syncthreads();
    const unsigned char* buf = smem + (c % NB) * Sh::BUF;
    const DecayTab& tb = tabs[c % NB];
    float* oc = OUT ? o + (int64_t)c * DCH * o_ts : nullptr;
    const int rows = sp.len - c * DCH;
    if constexpr (CT == 4) {
      main_chunk<W, CT, InT, OUT, 0, 1, 2, 3>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
    } else if constexpr (CT == 2) {
      if (m == 0)
        main_chunk<W, CT, InT, OUT, 0, 3>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
      else
        main_chunk<W, CT, InT, OUT, 1, 2>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
    } else {
      if (m == 0)
        main_chunk<W, CT, InT, OUT, 0>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
      else if (m == 1)
        main_chunk<W, CT, InT, OUT, 1>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
      else if (m == 2)
        main_chunk<W, CT, InT, OUT, 2>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
      else
        main_chunk<W, CT, InT, OUT, 3>(buf, tb, st, 16 * ct, oc, o_ts, rows, lane);
    }
    if (p.snap && m == 0 && rows >= DCH && (first_chunk + c + 1) % p.snap_chunks == 0) {
      const int64_t per = p.T / DCH / p.snap_chunks;  // fixed length: snapshots per sequence
      const int64_t row = (p.cu ? p.snap_first[sp.n] : sp.n * per) + (first_chunk + c + 1) / p.snap_chunks - 1;
      state_store<W>(st, p.snap + (row * p.H + h) * hsz, 0, p.DK, p.DV, col, lane);
    }
    if constexpr (NB == 1) __syncthreads();
    if (c + 1 < nc) put(c + 1);
  }
  if (p.S && m == 0 && srow >= 0 && sp.t0 + sp.len >= sp.total)
    state_store<W>(st, p.S + (srow * p.H + h) * hsz, 0, p.DK, p.DV, col, lane);
}

template <int W, int CT, typename InT>
static hipError_t launch_main_t(DecayParams p, hipStream_t s) {
  p.ncb = p.DV / (16 * CT);
  const int64_t grid = (int64_t)p.slots * p.H * p.ncb;
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX - 8) return hipErrorInvalidValue;
  p.grid = (int32_t)grid;
  const dim3 blocks((unsigned)((grid + 7) / 8 * 8));
  if (p.o)
    hipLaunchKernelGGL((decay_main_kernel<W, CT, InT, true>), blocks, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((decay_main_kernel<W, CT, InT, false>), blocks, dim3(256), 0, s, p);
  return hipGetLastError();
}
template <int W, typename InT>
static hipError_t launch_main_w(const DecayParams& p, const DecayPlan& pl, hipStream_t s) {
  if (pl.ct == 4) return launch_main_t<W, 4, InT>(p, s);
  if (pl.ct == 2) return launch_main_t<W, 2, InT>(p, s);
  return launch_main_t<W, 1, InT>(p, s);
}
template <typename InT>
static hipError_t launch_main(const DecayParams& p, const DecayPlan& pl, hipStream_t s) {
  if (p.DK == 128) return launch_main_w<128, InT>(p, pl, s);
  if (p.DK == 64) return launch_main_w<64, InT>(p, pl, s);
  return launch_main_w<32, InT>(p, pl, s);
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
template <int W, int CT, int DC, typename XT, typename YT, bool REV>
__global__ __launch_bounds__(256) void decay_state_kernel(const DecayParams p, int local) {
  constexpr int NPX = Terms<XT>::N;
  constexpr int IW = W / 16 < 4 ? W / 16 : 4, TI = W / 16 / IW, CW = 4 / IW, TC = CT / CW > 0 ? CT / CW : 1;
  constexpr int XB = DC * W * 2, YB = DC * CT * 32, BUF = NPX * XB + 3 * YB;
  constexpr int NB = NPX == 1 ? 2 : 1;
  __shared__ __align__(16) unsigned char smem[NB * BUF];
  __shared__ float s_gam[NB];
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  if (id >= p.grid) return;
  const int cb = id % p.ncb, sh = id / p.ncb;
  const int h = sh % p.H, slot = sh / p.H;
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
  const int t0 = wi * TI, col0 = cb * 16 * CT + 16 * wc * TC + (lane & 15);
#pragma unroll
  for (int tc = 0; tc < TC; ++tc) state_load<W>(st[tc], active ? src : nullptr, t0, p.DK, p.DV, col0 + 16 * tc, lane);
  auto save = [&](float* dst) {
    if (!active) return;
#pragma unroll
    for (int tc = 0; tc < TC; ++tc) state_store<W>(st[tc], dst, t0, p.DK, p.DV, col0 + 16 * tc, lane);
  };

  Stage<W, XT, DC> sx;
  StageCols<16 * CT, YT, DC> sy;
  float a_next = 1.f;
  const int nc = (sp.len + DC - 1) / DC;
  auto chunk_of = [&](int i) { return REV ? nc - 1 - i : i; };
  auto fetch = [&](int i) {
    const int c0 = chunk_of(i) * DC;
    sx.load(x, x_ts, c0, sp.len, p.DK, tid);
    sy.load(y, y_ts, c0, sp.len, tid);
    const int t = c0 + (lane & (DC - 1));
    a_next = al[(int64_t)(t < sp.len ? t : sp.len - 1) * a_ts];
  };
  auto put = [&](int i) {
    const int c0 = chunk_of(i) * DC;
    unsigned char* buf = smem + (i % NB) * BUF;
    sx.store(buf, XB, c0, sp.len, p.DK, tid);
    sy.mask(c0, sp.len, tid);
    if (lane >= DC || c0 + lane >= sp.len) a_next = 1.f;
    // lane t: the weight of token t, from its tile's products and the whole tiles before or behind it
    const float pre = row_prefix_prod(a_next), suf = row_suffix_prod_excl(a_next);
    float P[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      P[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, pre), 16 * j + 15));
    float wt = REV ? pre : suf;
#pragma unroll
    for (int j = 0; j < 4; ++j) wt *= (REV ? j < (lane >> 4) : j > (lane >> 4)) ? P[j] : 1.f;
    if (tid == 0) s_gam[i % NB] = P[0] * P[1] * P[2] * P[3];
    constexpr int CPR = StageCols<16 * CT, YT, DC>::CPR;
#pragma unroll
    for (int j = 0; j < StageCols<16 * CT, YT, DC>::NPC; ++j) {
      const int idx = tid + 256 * j;
      const float f = __shfl(wt, (idx / CPR) & (DC - 1));
      if (idx < DC * CPR) {
        float z[8];
        if constexpr (sizeof(YT) == 2) {
          const bf16x8 b = __builtin_bit_cast(bf16x8, sy.x[j].v);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = (float)b[e] * f;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = (e < 4 ? sy.x[j].a[e] : sy.x[j].b[e - 4]) * f;
        }
        const Tri t = split3(z);
#pragma unroll
        for (int e = 0; e < 3; ++e) *reinterpret_cast<bf16x8*>(buf + NPX * XB + e * YB + idx * 16) = t.t[e];
      }
    }
  };
  if (nc > 0) {
    fetch(0);
    put(0);
  }
  const int64_t cslot0 = (p.cu ? (local ? 0 : p.chunk_first[sp.n]) : (int64_t)sp.n * ((p.T + DC - 1) / DC)) + sp.t0 / DC;
  float gall = 1.f;
  for (int i = 0; i < nc; ++i) {
    if (i + 1 < nc) fetch(i + 1);
    __syncthreads();
    if (!local) save((REV ? p.ds : p.cs) + ((cslot0 + chunk_of(i)) * p.H + h) * hsz);
    const unsigned char* buf = smem + (i % NB) * BUF;
    const float G = s_gam[i % NB];
    gall *= G;
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
        for (int tc = 0; tc < TC; ++tc)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[tc][ti][e] *= G;
#pragma unroll
        for (int u = 0; u < DC / 32; ++u) {
          bf16x8 xf[NPX];
#pragma unroll
          for (int e = 0; e < NPX; ++e) xf[e] = frag_chan<W>(buf + e * XB, t >> 1, t & 1, u, lane);
#pragma unroll
          for (int tc = 0; tc < TC; ++tc) mma(st[tc][ti], xf, yf[tc][u]);
        }
      }
    }
    if constexpr (NB == 1) __syncthreads();
    if (i + 1 < nc) put(i + 1);
  }
  if (local) {
    save(part + ((int64_t)slot * p.H + h) * hsz);
    if (tid == 0 && cb == 0) p.gpart[(int64_t)slot * p.H + h] = gall;
  } else if (REV && p.dS0 && sp.t0 == 0) {
    save(p.dS0 + ((int64_t)sp.n * p.H + h) * hsz);
  }
}

// Segments joined: the state at each segment's start (reverse: the gradient at its end) from the
// segments' own contributions, in their place. One thread per 4 elements walks the sequence's segments.
__global__ __launch_bounds__(256) void decay_join_kernel(const DecayParams p, int rev) {
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
      const float G = p.gpart[sl];
      *at = x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(G, x[i], own[i]);
    } else {
      *at = x;
    }
  }
}

template <int W, int CT, int DC, typename XT, typename YT, bool REV>
static hipError_t launch_state_t(DecayParams p, int local, hipStream_t s) {
  p.ncb = p.DV / (16 * CT);
  const int64_t grid = (int64_t)p.slots * p.H * p.ncb;
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX - 8) return hipErrorInvalidValue;
  p.grid = (int32_t)grid;
  hipLaunchKernelGGL((decay_state_kernel<W, CT, DC, XT, YT, REV>), dim3((unsigned)((grid + 7) / 8 * 8)), dim3(256), 0, s, p,
                     local);
  return hipGetLastError();
}
template <int W, int DC, typename XT, typename YT, bool REV>
static hipError_t launch_state_w(const DecayParams& p, int local, hipStream_t s) {
  return p.DV >= 32 ? launch_state_t<W, 2, DC, XT, YT, REV>(p, local, s) : launch_state_t<W, 1, DC, XT, YT, REV>(p, local, s);
}
template <int DC, typename XT, typename YT, bool REV>
static hipError_t launch_state(const DecayParams& p, int local, hipStream_t s) {
  if (p.DK == 128) return launch_state_w<128, DC, XT, YT, REV>(p, local, s);
  if (p.DK == 64) return launch_state_w<64, DC, XT, YT, REV>(p, local, s);
  return launch_state_w<32, DC, XT, YT, REV>(p, local, s);
}

// (the contribution of whole segments does not depend on the chunk length)
hipError_t launch_decay_states(const DecayParams& p, bool bf16, bool rev, int local, hipStream_t s) {
  constexpr int CB = decay_bwd_chunk(true), CF = decay_bwd_chunk(false);
  if (rev) return bf16 ? launch_state<CB, __bf16, float, true>(p, local, s) : launch_state<CF, float, float, true>(p, local, s);
  return bf16 ? launch_state<CB, __bf16, __bf16, false>(p, local, s) : launch_state<CF, float, float, false>(p, local, s);
}
hipError_t launch_decay_join(const DecayParams& p, int rev, hipStream_t s) {
  const int64_t hsz = (int64_t)p.DK * p.DV;
  const int64_t grid = (int64_t)p.nseq * p.H * ((hsz / 4 + 255) / 256);
  if (grid == 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(decay_join_kernel, dim3((unsigned)grid), dim3(256), 0, s, p, rev);
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
    e = launch_decay_states(p, bf16, false, 1, s);
    if (e == hipSuccess) e = launch_decay_join(p, 0, s);
    if (e != hipSuccess) return e;
  } else {
    p.part = nullptr;
  }
  return bf16 ? launch_main<__bf16>(p, pl, s) : launch_main<float>(p, pl, s);
}

}  // namespace dr
