// Gradients of the selective scan on gfx950.
//
// With G_t the gradient that reaches h_t (from y_t, from h_{t+1} and from the final state) and a_t = exp(d_t A):
//   G_t = dy'_t C_t + a_{t+1} G_{t+1},  dy' = dy silu(z)
//   dB_t = sum_c G_t d_t x_t,  dC_t = sum_c dy'_t h_t,  u = sum_n G_t B_t,  e = sum_n G_t a_t h_{t-1} A
//   dx = u d + D dy',  d(d) = u x + e,  dA = sum_t d_t G_t a_t h_{t-1},  dz = dy (C h + D x) silu'(z)
// Three steps. scan_states_kernel walks every segment once (a lane has a channel, as in the forward pass) and leaves its
// state from zero at every 8th token, behind it, and the gradient that its outputs send to the state in front of it.
// scan_join2_kernel joins segments in both directions. scan_grad_kernel takes a segment's chunks of 8 tokens from the last to the first: states and
// decays of the chunk again from its checkpoint, held in registers (8 tokens x 4 channels x 2 states a lane), then
// the tokens in reverse. A lane's square of channels and states shares the two kinds of sums between lanes evenly: over states (dx,
// dd, y) across the lanes' rows, over channels (dB, dC) within eight lanes.
#include "scan_tile.hpp"

namespace dr {

// Local states at every 8th token and behind the segment, the sums of d there, and (BOTH) the reverse part: tiles as in the
// forward pass, dy C by the matrix units as d x B is.
template <int SL, typename InT, bool BOTH>
__global__ __launch_bounds__(64 * SL) void scan_states_kernel(const ScanParams p) {
  constexpr int N = 16 * SL, K = TILE_TOK, O = TILE_OWN;
  static_assert(K == 2 * SCAN_CHUNK, "two checkpoints to a tile");
  const int lane = threadIdx.x & 63, sl = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int ntiles = p.G * p.tiles;
  const int slot = blockIdx.x / ntiles, tile = blockIdx.x - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int g = tile / p.tiles, in_g = (tile - g * p.tiles) * SCAN_TILE + (lane & 31);
  const bool on = in_g < p.Cg;
  const int c = g * p.Cg + min(in_g, p.Cg - 1), n0 = sl * 16 + 4 * half;
  float A[8], h[8], P[8], R[8];
  load_states(p.A + (int64_t)c * N + n0, A);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    A[j] *= LOG2E;
    h[j] = R[j] = 0.f;
    P[j] = 1.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f;
  const int len = sp.len;
  const bool soft = p.softplus != 0, gate = BOTH && p.z != nullptr;
  Rows<InT> X, T, Z, B, Y, Cr;
  X.init(p.x, sp.b * p.x_bs + sp.t0 * p.x_ts, p.x_ts, half, c);
  T.init(p.dt, sp.b * p.dt_bs + sp.t0 * p.dt_ts, p.dt_ts, half, c);
  B.init(p.B, sp.b * p.b_bs + sp.t0 * p.b_ts, p.b_ts, half, g * N + sl * 16 + (lane & 15));
  if constexpr (BOTH) {
    if (gate)
      Z.init(p.z, sp.b * p.z_bs + sp.t0 * p.z_ts, p.z_ts, half, c);
    else
      Z = X;
    Cr.init(p.Cm, sp.b * p.c_bs + sp.t0 * p.c_ts, p.c_ts, half, g * N + sl * 16 + (lane & 15));
    Y.init(p.dy, (sp.b * p.T + sp.t0) * (int64_t)p.C, p.C, half, c);
  }
  const int64_t cps = p.seg / SCAN_CHUNK;
  float* ck = p.ck + ((int64_t)slot * cps * p.C + c) * N + n0;
  float* ckd = p.ckd + (int64_t)slot * cps * p.C + c;
  float sumd = 0.f;
  uint32_t xn[O], dn[O], zn[O], yn[O], bn[O], cn[O];
  auto fetch = [&](int left) {
    if (left >= K) {
      X.whole(xn);
      T.whole(dn);
      B.whole(bn);
      if constexpr (BOTH) {
        Z.whole(zn);
        Y.whole(yn);
        Cr.whole(cn);
      }
      whole_tile();
    } else {
      X.part(xn, left);
      T.part(dn, left);
      B.part(bn, left);
      if constexpr (BOTH) {
        Z.part(zn, left);
        Y.part(yn, left);
        Cr.part(cn, left);
      }
    }
    X.at += K * X.ts;
    T.at += K * T.ts;
    B.at += K * B.ts;
    if constexpr (BOTH) {
      Z.at += K * Z.ts;
      Y.at += K * Y.ts;
      Cr.at += K * Cr.ts;
    }
  };
  if (len > 0) fetch(len);
  for (int t = 0; t < len; t += K) {
    float dv[O], dx[O], gy[O], bo[O], co[O];
#pragma unroll
    for (int i = 0; i < O; ++i) {
      const float raw = raw_value<InT>(dn[i]) + bias, sf = softplus_f(raw);
      float own = soft ? sf : raw;
      here(own);
      // (tokens past the end: a decay of one, nothing in or out)
      const bool inside = t + K <= len || t + 2 * i + half < len;
      dv[i] = inside ? own : 0.f;
      dx[i] = inside ? dv[i] * raw_value<InT>(xn[i]) : 0.f;
      bo[i] = operand<InT>(bn[i], lane);
      if constexpr (BOTH) {
        const float zv = raw_value<InT>(zn[i]), sg = zv * sigmoid_f(zv);
        float out = raw_value<InT>(yn[i]) * (gate ? sg : 1.f);
        here(out);
        gy[i] = inside ? out : 0.f;
        co[i] = operand<InT>(cn[i], lane);
      }
    }
    if (t + K < len) fetch(len - t - K);
    f32x16 in = outer_pair(bo[0], dx[0]), out = BOTH ? outer_pair(co[0], gy[0]) : f32x16{};
#pragma unroll
    for (int i = 0; i < O; ++i) {
      tile_step();
      if (i % (O / 2) == 0 && (i == 0 || t + SCAN_CHUNK < len)) {
        if (on && (t > 0 || i > 0)) store_states(ck, h);  // (a segment begins at zero)
        float lo, hi;
        both_halves(sumd, lo, hi);
        if (on && sl == 0 && half == 0) *ckd = lo + hi;
        ck += (int64_t)p.C * N;
        ckd += p.C;
      }
      float d[2];
      both_halves(dv[i], d[0], d[1]);
      sumd += dv[i];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = __builtin_amdgcn_exp2f(d[k] * A[j]);
          h[j] = fmaf(a, h[j], in[8 * k + j]);
          if constexpr (BOTH) {
            P[j] *= a;
            R[j] = fmaf(P[j], out[8 * k + j], R[j]);
          }
        }
      if (i + 1 < O) {
        in = outer_pair(bo[i + 1], dx[i + 1]);
        if constexpr (BOTH) out = outer_pair(co[i + 1], gy[i + 1]);
      }
      if constexpr (BOTH) here(R);
    }
  }
  if constexpr (BOTH) {
    float lo, hi;
    both_halves(sumd, lo, hi);
    if (!on) return;
    const int64_t at = ((int64_t)slot * p.C + c) * N + n0;
    store_states(p.part + at, h);
    store_states(p.rpart + at, R);
    if (sl == 0 && half == 0) p.sumd[(int64_t)slot * p.C + c] = lo + hi;
  }
}

// Segments joined: forward (blockIdx.y 0) the state at each one's start in the place of its own, in reverse (1) the gradient that reaches
// the state behind each one in the place of what it sends forward.
template <int N>
__global__ __launch_bounds__(256) void scan_join2_kernel(const ScanParams p) {
  const int per = (p.C * (N / 4) + 255) / 256;
  const int n = blockIdx.x / per, e = (blockIdx.x - n * per) * 256 + threadIdx.x;
  if (e >= p.C * (N / 4)) return;
  const int c = e / (N / 4), j = e - c * (N / 4);
  const int first = p.cu ? p.slot_first[n] : n * p.nseg, past = p.cu ? p.slot_first[n + 1] : first + p.nseg;
  const bool back = blockIdx.y == 1;
  f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * N + 4 * j), v = {0, 0, 0, 0};
  const float* from = back ? p.dST : p.S0;
  float* part = back ? p.rpart : p.part;
  if (from) v = *reinterpret_cast<const f32x4*>(from + ((int64_t)n * p.C + c) * N + 4 * j);
  for (int k = first; k < past; ++k) {
    const int64_t s = back ? past - 1 - (k - first) : k;
    f32x4* at = reinterpret_cast<f32x4*>(part + (s * p.C + c) * N + 4 * j);
    const f32x4 own = *at;
    const float d = p.sumd[s * p.C + c] * LOG2E;
    *at = v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(__builtin_amdgcn_exp2f(d * A[i]), v[i], own[i]);
  }
}

// ---------------------------------------------------------------------------
// Sums across lanes
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// over 8 neighbouring lanes, in all of them: swapped in pairs, in quads' halves, mirrored in eight
__device__ __forceinline__ float sum8(float v) { return dpp_add<0x141>(dpp_add<0x4e>(dpp_add<0xb1>(v))); }
// a of lanes l and l ^ 32 (l ^ 16) in the lower lanes of the pair, b's sum in the upper ones
__device__ __forceinline__ float pair32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float pair16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// A workgroup: 4 waves, each 32 channels x 16 states (SL waves share channels), one segment.
template <int N>
struct GradShape {
  static constexpr int SL = N / 16;           // slices of states
  static constexpr int CB = 4 / SL;           // channel blocks
  static constexpr int CH = 32 * CB;          // channels
  static constexpr int ROWS = 256 / CH;       // token rows that the threads cover at once
  static constexpr int PP = SCAN_CHUNK / ROWS;  // (token, channel) pairs of a thread
};
template <int N, typename InT, bool GATE>
__global__ __launch_bounds__(256, 2) void scan_grad_kernel(const ScanParams p) {
  using Sh = GradShape<N>;
  constexpr int K = SCAN_CHUNK, CH = Sh::CH, SL = Sh::SL, PP = Sh::PP, ROWS = Sh::ROWS;
  __shared__ __align__(16) float s_d[K][CH], s_dx[K][CH], s_dy[K][CH];
  __shared__ __align__(16) float s_b[K][N], s_c[K][N];
  __shared__ float s_u[SL][K][CH], s_e[SL][K][CH], s_y[GATE ? SL : 1][GATE ? K : 1][GATE ? CH : 1];
  __shared__ __align__(16) float s_bc[4][K][32];
  // what a thread needs of its pairs again at the end of a chunk, and its starting state, wait here instead of in registers
  __shared__ __align__(16) float s_own[GATE ? 4 : 2][PP][256], s_hs[2][256][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sl = wave % SL, cb = wave / SL;
  const int per = p.G * p.cblocks;
  const int slot = blockIdx.x / per, blk = blockIdx.x - slot * per;
  const int g = blk / p.cblocks, in0 = (blk - g * p.cblocks) * CH;  // the group, the first channel within it
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int len = sp.len, cps = p.seg / K, C = p.C;
  // as the lane of states and gradients: 4 channels, 2 states
  const int ng = lane >> 3, cg = lane & 7;
  const int l_ch = cb * 32 + cg * 4, n0 = sl * 16 + ng * 2;
  int lc[4];  // (channels past the group's count as its last)
#pragma unroll
  for (int i = 0; i < 4; ++i) lc[i] = g * p.Cg + min(in0 + l_ch + i, p.Cg - 1);
  const int lim = max(p.Cg - 1 - in0 - l_ch, 0);
  float A[4][2], carry[4][2], dA[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t at = (int64_t)lc[i] * N + n0 + j;
      A[i][j] = p.A[at] * LOG2E;
      dA[i][j] = 0.f;
      const float* from = p.part ? p.part + (int64_t)slot * C * N : p.S0 ? p.S0 + (int64_t)sp.n * C * N : nullptr;
      s_hs[j][tid][i] = from ? from[at] : 0.f;
      const float* back = p.part ? p.rpart + (int64_t)slot * C * N : p.dST ? p.dST + (int64_t)sp.n * C * N : nullptr;
      carry[i][j] = back ? back[at] : 0.f;
    }
  // as the thread of (token, channel) pairs: one channel, PP tokens of a chunk
  const int pc = tid % CH, prow = tid / CH;
  const bool on = in0 + pc < p.Cg;
  const int c = g * p.Cg + min(in0 + pc, p.Cg - 1);
  const float bias = p.bias ? p.bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
  // Addresses: a uniform pointer for the chunk, moved back by a chunk after each, and 32-bit offsets of the lane that stay
  // (token strides are limited to 2^24 elements, groups to 2^16).
  const int last = len > 0 ? (len - 1) / K * K : 0;
  const int64_t row0 = sp.b * p.T + sp.t0, x_ts = p.x_ts, dt_ts = p.dt_ts, z_ts = p.z_ts;
  const InT* xb = static_cast<const InT*>(p.x) + sp.b * p.x_bs + (sp.t0 + last) * x_ts;
  const InT* db = static_cast<const InT*>(p.dt) + sp.b * p.dt_bs + (sp.t0 + last) * dt_ts;
  const InT* zb = GATE ? static_cast<const InT*>(p.z) + sp.b * p.z_bs + (sp.t0 + last) * z_ts : nullptr;
  int64_t row = row0 + last, next = row;  // of the outputs, of dy
  constexpr uint32_t E = sizeof(InT);
  const uint32_t xo = (uint32_t)(prow * x_ts + c) * E, dto = (uint32_t)(prow * dt_ts + c) * E, zo = GATE ? (uint32_t)(prow * z_ts + c) * E : 0u;
  const uint32_t oo = (uint32_t)(prow * C + c) * E, cko = ((uint32_t)lc[0] * N + n0) * 4;
  int64_t chunk = (int64_t)slot * cps + last / K;
  constexpr int BCN = 2 * K * N / 256;  // elements of B and C of a thread: B's first, then C's (a wave has one of them)
  static_assert(2 * K * N % 256 == 0 && K * N % 64 == 0, "whole waves");
  uint32_t bco[BCN];
#pragma unroll
  for (int i = 0; i < BCN; ++i) {
    const int e = (tid + i * 256) % (K * N);
    const bool isC = (wave * 64 + i * 256) / (K * N) == 1;
    bco[i] = (uint32_t)(e / N * (isC ? p.c_ts : p.b_ts) + g * N + e % N) * E;
  }
  const bool soft = p.softplus != 0;
  float accD = 0.f, accb = 0.f;
  InT xn[PP], dn[PP], zn[PP], yn[PP];
  float hn[4][2], dsum[4];
  InT bn[BCN];
  auto fetch = [&](int t) {  // (rows past the end are read from the last one and not used; those of B and C are zeros)
    const InT *xr = xb, *dr = db, *zr = zb, *yr = static_cast<const InT*>(p.dy) + next * C;
    if (t + K <= len) {
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        xn[i] = *byte_at(xr, xo);
        dn[i] = *byte_at(dr, dto);
        if constexpr (GATE) zn[i] = *byte_at(zr, zo);
        yn[i] = *byte_at(yr, oo);
        xr += ROWS * x_ts;
        dr += ROWS * dt_ts;
        if constexpr (GATE) zr += ROWS * z_ts;
        yr += ROWS * (int64_t)C;
      }
      whole_tile();
    } else {
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        const int64_t r = min(prow + i * ROWS, len - 1 - t);
        xn[i] = xr[r * x_ts + c];
        dn[i] = dr[r * dt_ts + c];
        if constexpr (GATE) zn[i] = zr[r * z_ts + c];
        yn[i] = yr[r * C + c];
      }
    }
    xb -= K * x_ts;
    db -= K * dt_ts;
    if constexpr (GATE) zb -= K * z_ts;
    next -= K;
#pragma unroll
    for (int i = 0; i < BCN; ++i) {
      const bool isC = (wave * 64 + i * 256) / (K * N) == 1;
      const InT* from = isC ? static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + (sp.t0 + t) * p.c_ts : static_cast<const InT*>(p.B) + sp.b * p.b_bs + (sp.t0 + t) * p.b_ts;
      bn[i] = InT(0);
      if (t + K <= len || t + (tid + i * 256) % (K * N) / N < len) bn[i] = *byte_at(from, bco[i]);
    }
    const float *ck = p.ck + chunk * C * N, *ckd = p.ckd + chunk * C;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dsum[i] = 0.f;
      hn[i][0] = hn[i][1] = 0.f;
      if (t > 0) {
        const uint32_t o = min(i, lim);
        dsum[i] = *byte_at(ckd, ((uint32_t)lc[0] + o) * 4);
        const f32x2 v = *reinterpret_cast<const f32x2*>(byte_at(ck, cko + o * (4 * N)));
        hn[i][0] = v[0];
        hn[i][1] = v[1];
      }
    }
    --chunk;
  };
  // this workgroup's part of dB and dC: 2 N values to a token
  float* pbc = p.pBC + (((int64_t)(blk - g * p.cblocks) * p.nbatch * p.T + row0 + last) * p.G + g) * (2 * N);
  const uint32_t pbo = ((uint32_t)(tid / (2 * N)) * p.G * (2 * N) + tid % (2 * N)) * 4;
  if (len > 0) fetch(last);
  for (int t = last; len > 0 && t >= 0; t -= K) {
    __syncthreads();  // (the chunk before has been written out)
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int r = prow + i * ROWS;
      const bool here = on && t + r < len;
      const float xv = (float)xn[i], raw = (float)dn[i] + bias, sf = softplus_f(raw), sr = sigmoid_f(raw);
      const float dv = soft ? sf : raw;
      float gv = (float)yn[i];
      s_own[0][i][tid] = xv;
      s_own[1][i][tid] = soft ? sr : 1.f;
      if constexpr (GATE) {
        const float zv = (float)zn[i];
        s_own[2][i][tid] = zv;
        s_own[3][i][tid] = gv;
        gv *= zv * sigmoid_f(zv);
      }
      // tokens past the end and channels past the group's: a decay of one, nothing in or out
      s_d[r][pc] = here ? dv : 0.f;
      s_dx[r][pc] = here ? dv * xv : 0.f;
      s_dy[r][pc] = here ? gv : 0.f;
    }
#pragma unroll
    for (int i = 0; i < BCN; ++i) {
      const int q = tid + i * 256;
      (q < K * N ? &s_b[0][0] : &s_c[0][0] - K * N)[q] = (float)bn[i];
    }
    // the state in front of the chunk
    float a[K][4][2], h[K + 1][4][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4 hs = *reinterpret_cast<const f32x4*>(&s_hs[j][tid][0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[0][i][j] = fmaf(__builtin_amdgcn_exp2f(dsum[i] * A[i][j]), hs[i], hn[i][j]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k % 2 == 0) __builtin_amdgcn_sched_barrier(0);
      const f32x4 d = *reinterpret_cast<const f32x4*>(&s_d[k][l_ch]), dx = *reinterpret_cast<const f32x4*>(&s_dx[k][l_ch]);
      const f32x2 b = *reinterpret_cast<const f32x2*>(&s_b[k][n0]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[k][i][j] = __builtin_amdgcn_exp2f(d[i] * A[i][j]);
          h[k + 1][i][j] = fmaf(a[k][i][j], h[k][i][j], dx[i] * b[j]);
        }
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      // the next chunk's loads start where half of this one's states and decays are no longer held
      if (k == K / 2 - 1 && t > 0) fetch(t - K);
      __builtin_amdgcn_sched_barrier(0);
      const f32x4 d = *reinterpret_cast<const f32x4*>(&s_d[k][l_ch]), dx = *reinterpret_cast<const f32x4*>(&s_dx[k][l_ch]);
      const f32x4 gy = *reinterpret_cast<const f32x4*>(&s_dy[k][l_ch]);
      const f32x2 b = *reinterpret_cast<const f32x2*>(&s_b[k][n0]), cc = *reinterpret_cast<const f32x2*>(&s_c[k][n0]);
      float u[4], e[4], yo[4], vb[2] = {0.f, 0.f}, vc[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = e[i] = yo[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          vc[j] = fmaf(gy[i], h[k + 1][i][j], vc[j]);
          if constexpr (GATE) yo[i] = fmaf(cc[j], h[k + 1][i][j], yo[i]);
          const float G = fmaf(gy[i], cc[j], carry[i][j]);
          vb[j] = fmaf(G, dx[i], vb[j]);
          u[i] = fmaf(G, b[j], u[i]);
          const float aG = a[k][i][j] * G;
          const float w = aG * h[k][i][j];
          e[i] = fmaf(w, A[i][j], e[i]);
          dA[i][j] = fmaf(w, d[i], dA[i][j]);
          carry[i][j] = aG;
        }
      }
      // sums over states: the lower 32 lanes end with u, the upper with e; of four channels, even rows of 16 lanes have
      // 0 and 1, odd rows 2 and 3; the last step is the same in both halves of a row, each of which writes one channel
      {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair32(u[i], e[i]);
        const float r0 = dpp_add<0x128>(pair16(v[0], v[2])), r1 = dpp_add<0x128>(pair16(v[1], v[3]));
        const int ch = l_ch + 2 * ((lane >> 4) & 1) + ((lane >> 3) & 1);
        float* to = lane < 32 ? &s_u[sl][k][ch] : &s_e[sl][k][ch];
        *to = lane & 8 ? r1 : r0;
      }
      if constexpr (GATE) {  // (one channel a row of 16 lanes: 0, 1, 2, 3)
        const float v = dpp_add<0x128>(pair16(pair32(yo[0], yo[2]), pair32(yo[1], yo[3])));
        if (!(lane & 8)) s_y[sl][k][l_ch + 2 * (lane >> 5) + ((lane >> 4) & 1)] = v;
      }
      // sums over channels
      const float b0 = sum8(vb[0]), b1 = sum8(vb[1]), c0 = sum8(vc[0]), c1 = sum8(vc[1]);
      if (cg == 0) *reinterpret_cast<f32x4*>(&s_bc[wave][k][ng * 4]) = f32x4{b0, b1, c0, c1};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int r = prow + i * ROWS;
      if (t + r >= len || !on) continue;
      float u = 0.f, e = 0.f, yo = 0.f;
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        u += s_u[s][r][pc];
        e += s_e[s][r][pc];
        if constexpr (GATE) yo += s_y[s][r][pc];
      }
      const float xv = s_own[0][i][tid], gv = s_dy[r][pc];
      const float draw = fmaf(u, xv, e * LN2) * s_own[1][i][tid];
      const int64_t base = (row + i * ROWS) * C;
      *byte_at(static_cast<InT*>(p.ddt) + base, oo) = (InT)draw;
      *byte_at(static_cast<InT*>(p.dx) + base, oo) = (InT)fmaf(u, s_d[r][pc], D * gv);
      if constexpr (GATE) {
        const float zv = s_own[2][i][tid], sz = sigmoid_f(zv);
        *byte_at(static_cast<InT*>(p.dz) + base, oo) = (InT)(s_own[3][i][tid] * fmaf(D, xv, yo) * (sz * fmaf(zv, 1.f - sz, 1.f)));
      }
      accD = fmaf(gv, xv, accD);
      accb += draw;
    }
#pragma unroll
    for (int i = 0; i < BCN; ++i) {
      const int q = tid + i * 256, r = q / (2 * N), m = q / N & 1, n = q % N;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < Sh::CB; ++w) v += s_bc[w * SL + n / 16][r][(n % 16) / 2 * 4 + 2 * m + (n & 1)];
      if (t + r < len) *byte_at(pbc + i * (256 / (2 * N)) * (int64_t)p.G * (2 * N), pbo) = v;
    }
    row -= K;
    pbc -= K * (int64_t)p.G * (2 * N);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (in0 + l_ch + i >= p.Cg) continue;
      const int64_t at = (int64_t)lc[i] * N + n0 + j;
      p.pA[(int64_t)slot * C * N + at] = dA[i][j];
      if (sp.first && p.dS0) p.dS0[(int64_t)sp.n * C * N + at] = carry[i][j];
    }
  // D and the bias: the token rows of a channel
  __syncthreads();
  float* red = &s_u[0][0][0];
  red[tid] = accD;
  red[256 + tid] = accb;
  __syncthreads();
  if (prow == 0 && on) {
    float vD = 0.f, vb = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      vD += red[r * CH + pc];
      vb += red[256 + r * CH + pc];
    }
    p.pD[(int64_t)slot * 2 * C + c] = vD;
    p.pD[(int64_t)slot * 2 * C + C + c] = vb;
  }
}

// dA [C, N], dD and ddt_bias from the slots' parts (blocks below nA: dA), 64 columns x 16 groups of slots a workgroup.
template <int N>
__global__ __launch_bounds__(1024) void scan_dparam_kernel(const ScanParams p, int nA) {
  __shared__ float s[16][64];
  const bool isA = (int)blockIdx.x < nA;
  const int cols = isA ? p.C * N : 2 * p.C, col = ((int)blockIdx.x - (isA ? 0 : nA)) * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  const float* part = isA ? p.pA : p.pD;
  const int slots = p.cu ? p.slot_first[p.nseq] : p.slots;
  float v = 0.f;
  if (col < cols)
    for (int r = g; r < slots; r += 16) v += part[(int64_t)r * cols + col];
  s[g][threadIdx.x & 63] = v;
  __syncthreads();
  if (g == 0 && col < cols) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) a += s[k][threadIdx.x];
    if (isA)
      p.dA[col] = a;
    else if (col < p.C && p.dD)
      p.dD[col] = a;
    else if (col >= p.C && p.dbias)
      p.dbias[col - p.C] = a;
  }
}

// dB and dC from the channel blocks' parts, a value a thread.
template <int N, typename InT>
__global__ __launch_bounds__(256) void scan_dbc_kernel(const ScanParams p) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (int64_t)p.nbatch * p.T * p.G * (2 * N);
  if (q >= per) return;
  const int64_t row = q / (2 * N), tok = row / p.G;
  if (p.cu && (tok < p.cu[0] || tok >= p.cu[p.nseq])) return;  // no sequence holds it
  const int m = (int)(q / N & 1), n = (int)(q % N);
  float v = 0.f;
  for (int k = 0; k < p.cblocks; ++k) v += p.pBC[k * per + q];
  static_cast<InT*>(m ? p.dC : p.dB)[row * N + n] = (InT)v;
}

template <int SL, typename InT>
static void launch_states(const ScanParams& p, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.tiles)), block(64 * SL);
  if (p.part)
    hipLaunchKernelGGL((scan_states_kernel<SL, InT, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((scan_states_kernel<SL, InT, false>), grid, block, 0, s, p);
}
template <int N, typename InT>
static hipError_t launch_bwd_t(const ScanParams& p, hipStream_t s) {
  if (p.slots > 0 && p.nseq > 0) {
    launch_states<N / 16, InT>(p, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.part) {
      hipLaunchKernelGGL((scan_join2_kernel<N>), dim3((unsigned)((int64_t)p.nseq * ((p.C * (N / 4) + 255) / 256)), 2), dim3(256), 0, s, p);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.cblocks));
    if (p.z)
      hipLaunchKernelGGL((scan_grad_kernel<N, InT, true>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((scan_grad_kernel<N, InT, false>), grid, dim3(256), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int nA = (int)(((int64_t)p.C * N + 63) / 64);
  hipLaunchKernelGGL((scan_dparam_kernel<N>), dim3(nA + (2 * p.C + 63) / 64), dim3(1024), 0, s, p, nA);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t vals = (int64_t)p.nbatch * p.T * p.G * (2 * N);
  if (vals > 0 && p.nseq > 0)
    hipLaunchKernelGGL((scan_dbc_kernel<N, InT>), dim3((unsigned)((vals + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename InT>
static hipError_t launch_bwd_n(const ScanParams& p, int n, hipStream_t s) {
  return n == 16 ? launch_bwd_t<16, InT>(p, s) : n == 32 ? launch_bwd_t<32, InT>(p, s) : launch_bwd_t<64, InT>(p, s);
}
hipError_t launch_scan_bwd(ScanParams p, int n, bool bf16, hipStream_t s) {
  if (p.cu) {
    const hipError_t e = launch_scan_plan(p, s);
    if (e != hipSuccess) return e;
    p.cu = p.cu_ok;
  }
  return bf16 ? launch_bwd_n<__bf16>(p, n, s) : launch_bwd_n<float>(p, n, s);
}

}  // namespace dr
