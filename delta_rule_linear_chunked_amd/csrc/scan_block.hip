// Selective scan with a workgroup's waves along the tokens (gfx950): whole sequences, where a wave for each would leave the GPU idle.
//
// The exponentials are the scan's largest part, and cutting sequences into segments forms each of them twice. Here a workgroup has 32
// channels and walks 128 tokens at a time (64 or 32 with more states), a tile of 16 tokens a wave (scan_tile.hpp): a wave forms its decays
// once and holds them in registers (16 tokens x 8 states a lane), runs them from zero for its own end state, hands that and the
// decays' product on through LDS, and behind one barrier runs them again from the state that the waves before it leave.
// A workgroup fills a CU (230 registers, 78 KB of LDS): two waves a SIMD, whose vector units issue 75% of the time. 4 x 4096 x 2048, 16 states, bf16:
// 196 us a call; in segments of 256 tokens 257. The tensors alone would take 52 at the copy rate, an exponential (two issues), a
// product and two sums for each state 68, softplus and gate about 30 more.
#include "scan_tile.hpp"

namespace dr {

template <int SL, typename InT>
__global__ __launch_bounds__(64 * SCAN_BLOCK_WAVES, 1) void scan_block_kernel(const ScanParams p) {
  constexpr int N = 16 * SL, K = TILE_TOK, O = TILE_OWN, TS = SCAN_BLOCK_WAVES / SL, IT = TS * K;
  __shared__ f32x4 s_end[2][SCAN_BLOCK_WAVES][4][64];  // products of decays (2 pieces of 4 states), then end states
  __shared__ f32x4 s_carry[2][SL][2][64];
  __shared__ __align__(16) float s_c[SCAN_BLOCK_WAVES][K][16];  // a wave's own rows of C
  __shared__ float s_y[SL > 1 ? SCAN_BLOCK_WAVES : 1][SL > 1 ? O : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, sl = wave % SL, ts = wave / SL;
  // neighbouring channel tiles share cache lines: they go to the same XCD (workgroups are dealt over eight)
  const int ntiles = p.G * p.tiles, total = p.slots * ntiles, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (id >= total) return;
  const int slot = id / ntiles, tile = id - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int g = tile / p.tiles, in_g = (tile - g * p.tiles) * SCAN_TILE + (lane & 31);
  const bool on = in_g < p.Cg;  // (channels past the group's count as its last and store nothing)
  const int c = g * p.Cg + min(in_g, p.Cg - 1), n0 = sl * 16 + 4 * half;
  float A[8], h[8];
  load_states(p.A + (int64_t)c * N + n0, A);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    A[j] *= LOG2E;
    h[j] = 0.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
  if (p.S0) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) load_states(p.S0 + (r * p.C + c) * N + n0, h);
  }
  if (ts == TS - 1) {
    s_carry[0][sl][0][lane] = f32x4{h[0], h[1], h[2], h[3]};
    s_carry[0][sl][1][lane] = f32x4{h[4], h[5], h[6], h[7]};
  }
  const int len = sp.len;
  const float least = step_least(p.softplus != 0);
  const bool gate = p.z != nullptr;
  const int64_t mine = sp.t0 + ts * K;  // the wave's tile; IT tokens further on after each
  Rows<InT> X, T, Z, B;
  X.init(p.x, sp.b * p.x_bs + mine * p.x_ts, p.x_ts, half, c);
  T.init(p.dt, sp.b * p.dt_bs + mine * p.dt_ts, p.dt_ts, half, c);
  if (gate)
    Z.init(p.z, sp.b * p.z_bs + mine * p.z_ts, p.z_ts, half, c);
  else
    Z = X;
  B.init(p.B, sp.b * p.b_bs + mine * p.b_ts, p.b_ts, half, g * N + sl * 16 + (lane & 15));
  // C: lane l brings states 4 (l % 4) .. + 3 of token l / 4
  typedef typename Vec<InT, 4>::type V4;
  auto c_at = [&](uint32_t l) { return ((l >> 2) * (uint32_t)p.c_ts + (uint32_t)(g * N + sl * 16) + 4 * (l & 3)) * (uint32_t)sizeof(InT); };
  const InT* Ca = static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + mine * p.c_ts;
  InT* y = static_cast<InT*>(p.y) + (sp.b * p.T + mine) * (int64_t)p.C;
  uint32_t xn[O], dn[O], bn[O];
  V4 cn;
  auto fetch = [&](int step) {  // (as for a wave on its own)
    X.at += step * X.ts;
    T.at += step * T.ts;
    B.at += step * B.ts;
    Ca += step * p.c_ts;
    X.whole(xn);
    T.whole(dn);
    B.whole(bn);
    cn = *reinterpret_cast<const V4*>(byte_at(Ca, c_at(fresh(lane))));
  };
  int par = 0;
  auto tokens = [&](int t0, auto cut) {
    constexpr bool CUT = decltype(cut)::value;
    const int t = t0 + ts * K;
    float xv[O], dv[O], dx[O], bo[O];
    {
      float f[4];
      unpack<4, InT>(cn, f);
      *reinterpret_cast<f32x4*>(&s_c[wave][lane >> 2][4 * (lane & 3)]) = f32x4{f[0], f[1], f[2], f[3]};
    }
    float sumd = 0.f;
#pragma unroll
    for (int i = 0; i < O; ++i) {
      xv[i] = raw_value<InT>(xn[i]);
      float own = step_f(raw_value<InT>(dn[i]) + bias, least);
      here(own);
      // (tokens past the end: a decay of one and nothing added)
      const bool inside = !CUT || t + 2 * i + half < len;
      dv[i] = inside ? own : 0.f;
      dx[i] = inside ? dv[i] * xv[i] : 0.f;
      own_token(dv[i], dx[i]);
      bo[i] = inside ? operand<InT>(bn[i], lane) : 0.f;
      sumd += dv[i];
    }
    // from zero
    float a[K][8], e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    {
      f32x16 in = outer_pair(bo[0], dx[0]);
#pragma unroll
      for (int i = 0; i < O; ++i) {
        tile_step();
        float d[2];
        both_halves(dv[i], d[0], d[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[2 * i + k][j] = __builtin_amdgcn_exp2f(d[k] * A[j]);
            e[j] = fmaf(a[2 * i + k][j], e[j], in[8 * k + j]);
          }
        if (i + 1 < O) in = outer_pair(bo[i + 1], dx[i + 1]);  // (the next decays hide it)
      }
    }
    float lo, hi, P[8];
    both_halves(sumd, lo, hi);
#pragma unroll
    for (int j = 0; j < 8; ++j) P[j] = __builtin_amdgcn_exp2f((lo + hi) * A[j]);
    s_end[par][wave][0][lane] = f32x4{P[0], P[1], P[2], P[3]};
    s_end[par][wave][1][lane] = f32x4{P[4], P[5], P[6], P[7]};
    s_end[par][wave][2][lane] = f32x4{e[0], e[1], e[2], e[3]};
    s_end[par][wave][3][lane] = f32x4{e[4], e[5], e[6], e[7]};
    __syncthreads();
    // the state in front of the wave's tokens
    {
      const f32x4 c0 = s_carry[par][sl][0][lane], c1 = s_carry[par][sl][1][lane];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = j < 4 ? c0[j & 3] : c1[j & 3];
      for (int w = 0; w < ts; ++w) {
        f32x4 q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = s_end[par][w * SL + sl][k][lane];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = fmaf(q[j >> 2][j & 3], h[j], q[2 + (j >> 2)][j & 3]);
      }
    }
    uint32_t zn[O];
    if constexpr (CUT)
      Z.part(zn, len - t);
    else
      Z.whole(zn);
    Z.at += IT * Z.ts;
    float v[O];
    f32x16 in = outer_pair(bo[0], dx[0]);
#pragma unroll
    for (int i = 0; i < O; ++i) {
      tile_step();
      if (!CUT && i == O / 2) fetch(t0 + 2 * IT <= len ? IT : 0);  // (half of the decays are no longer held)
      float s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 c0 = *reinterpret_cast<const f32x4*>(&s_c[wave][2 * i + k][4 * half]), c1 = *reinterpret_cast<const f32x4*>(&s_c[wave][2 * i + k][8 + 4 * half]);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = fmaf(a[2 * i + k][j], h[j], in[8 * k + j]);
        if (k == 1 && i + 1 < O) in = outer_pair(bo[i + 1], dx[i + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < 4)
            s0 = fmaf(c0[j & 3], h[j], s0);
          else
            s1 = fmaf(c1[j & 3], h[j], s1);
        s[k] = s0 + s1;
      }
      v[i] = sum_halves(s[0], s[1]);
      here(v[i]);  // (the states of all tokens would be held otherwise)
    }
    __builtin_amdgcn_wave_barrier();
    if (ts == TS - 1) {
      s_carry[par ^ 1][sl][0][lane] = f32x4{h[0], h[1], h[2], h[3]};
      s_carry[par ^ 1][sl][1][lane] = f32x4{h[4], h[5], h[6], h[7]};
    }
    if constexpr (SL > 1) {
#pragma unroll
      for (int i = 0; i < O; ++i) s_y[wave][i][lane] = v[i];
      __syncthreads();
    }
    InT* row = y;
    if constexpr (SL > 1) row += 2 * sl * (int64_t)p.C;
#pragma unroll
    for (int q = 0; q < O / SL; ++q, row += 2 * SL * (int64_t)p.C) {  // (as for a wave on its own)
      float o = v[q], x = xv[q];
      uint32_t raw = zn[q];
      if constexpr (SL > 1) {
        o = 0.f;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          o += s_y[ts * SL + s][q * SL + sl][lane];
          x = s == 0 || sl == s ? xv[q * SL + s] : x;
          raw = s == 0 || sl == s ? zn[q * SL + s] : raw;
        }
      }
      o = fmaf(D, x, o);
      const float zv = raw_value<InT>(raw), sg = zv * sigmoid_f(zv);
      if (!CUT || (on && t + 2 * (q * SL + sl) + half < len)) *byte_at(row, (fresh(c) + (fresh(half) ? (uint32_t)p.C : 0u)) * (uint32_t)sizeof(InT)) = (InT)(o * (gate ? sg : 1.f));
    }
    y += IT * (int64_t)p.C;
    par ^= 1;
  };
  const int whole = len / IT * IT;
  if (whole > 0) {
    fetch(0);
    arrived();
    for (int t0 = 0; t0 < whole; t0 += IT) tokens(t0, std::false_type{});
  }
  if (whole < len) {  // (waves whose tile lies past the end read the last token)
    const int step = whole > 0 ? IT : 0, left = len - whole - ts * K;
    X.at += step * X.ts;
    T.at += step * T.ts;
    B.at += step * B.ts;
    Ca += step * p.c_ts;
    X.part(xn, left);
    T.part(dn, left);
    B.part(bn, left);
    cn = *reinterpret_cast<const V4*>(Ca + ((int64_t)min(lane >> 2, left - 1) * p.c_ts + g * N + sl * 16 + 4 * (lane & 3)));
    tokens(whole, std::true_type{});
  }
  if (ts == TS - 1 && p.S && on) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) store_states(p.S + (r * p.C + c) * N + n0, h);
  }
}

template <typename InT>
static hipError_t launch_t(const ScanParams& p, int n, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)p.slots * p.G * p.tiles + 7) / 8 * 8)), block(64 * SCAN_BLOCK_WAVES);
  if (n == 16)
    hipLaunchKernelGGL((scan_block_kernel<1, InT>), grid, block, 0, s, p);
  else if (n == 32)
    hipLaunchKernelGGL((scan_block_kernel<2, InT>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((scan_block_kernel<4, InT>), grid, block, 0, s, p);
  return hipGetLastError();
}
hipError_t launch_scan_block(const ScanParams& p, int n, bool bf16, hipStream_t s) {
  return bf16 ? launch_t<__bf16>(p, n, s) : launch_t<float>(p, n, s);
}

}  // namespace dr
