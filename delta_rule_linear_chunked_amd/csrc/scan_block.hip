// Selective scan with a workgroup's waves along the tokens (gfx950): few channels and sequences, or few tokens.
//
// The exponentials bound the scan (one at a quarter of the vector rate beside four products and sums), and cutting sequences into
// segments forms each of them twice. Here a workgroup has 32 channels and walks 128 tokens at a time (64 or 32 with more states), 16 tokens a wave:
// a wave forms its decays once and holds them in registers (16 tokens x 8 states a lane), runs them from zero for its own
// end state, hands that and the decays' product on through LDS, and behind one barrier runs them again from the state that the
// waves before it leave. Two halves of a wave have the same channels and eight states each; the halves share what belongs to a (token,
// channel) pair, eight tokens each.
#include "scan.hpp"

namespace dr {

__device__ __forceinline__ void both_halves(float v, float& low, float& high) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  low = __builtin_bit_cast(float, (uint32_t)r[0]);
  high = __builtin_bit_cast(float, (uint32_t)r[1]);
}
// a of lanes l and l ^ 32 in the lower half, b's sum in the upper
__device__ __forceinline__ float sum_halves(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

template <int SL, typename InT>
__global__ __launch_bounds__(512, 1) void scan_block_kernel(const ScanParams p) {
  constexpr int N = 16 * SL, K = 16, TS = SCAN_BLOCK_WAVES / SL, IT = TS * K;
  __shared__ f32x4 s_end[2][SCAN_BLOCK_WAVES][4][64];  // products of decays (2 pieces of 4 states), then end states
  __shared__ f32x4 s_carry[2][SL][2][64];
  __shared__ __align__(16) float s_bc[SCAN_BLOCK_WAVES][K][32];  // a wave's own: 16 states of B, then of C
  __shared__ float s_y[SL > 1 ? SCAN_BLOCK_WAVES : 1][SL > 1 ? 8 : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, sl = wave % SL, ts = wave / SL;
  // neighbouring channel tiles share cache lines: they go to the same XCD (workgroups are dealt over eight)
  const int ntiles = p.G * p.btiles, total = p.slots * ntiles, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (id >= total) return;
  const int slot = id / ntiles, tile = id - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int g = tile / p.btiles, in_g = (tile - g * p.btiles) * SCAN_BLOCK_CH + (lane & 31);
  const bool on = in_g < p.Cg;
  const int c = g * p.Cg + min(in_g, p.Cg - 1), n0 = sl * 16 + half * 8;
  float A[8], h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    A[j] = p.A[(int64_t)c * N + n0 + j] * LOG2E;
    h[j] = 0.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
  const float* from = nullptr;
  if (p.part) {
    from = p.part + ((int64_t)slot * p.C + c) * N;
  } else if (p.S0) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) from = p.S0 + (r * p.C + c) * N;
  }
  if (from)
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(from + n0 + j);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[j + k] = v[k];
    }
  if (ts == TS - 1) {
    s_carry[0][sl][0][lane] = f32x4{h[0], h[1], h[2], h[3]};
    s_carry[0][sl][1][lane] = f32x4{h[4], h[5], h[6], h[7]};
  }
  const int len = sp.len;
  const bool soft = p.softplus != 0, gate = p.z != nullptr;
  // the lane's rows of the wave's first tokens; a tile further on after each
  const int64_t x_ts = p.x_ts, dt_ts = p.dt_ts, z_ts = gate ? p.z_ts : p.x_ts, C = p.C, mine = sp.t0 + ts * K + half * 8;
  const InT* xp = static_cast<const InT*>(p.x) + sp.b * p.x_bs + mine * x_ts + c;
  const InT* dp = static_cast<const InT*>(p.dt) + sp.b * p.dt_bs + mine * dt_ts + c;
  const InT* zp = gate ? static_cast<const InT*>(p.z) + sp.b * p.z_bs + mine * z_ts + c : xp;
  InT* yp = static_cast<InT*>(p.y) + (sp.b * p.T + mine) * C + c;
  // B and C: lane l brings 8 states of token (l % 32) / 2 of one of them
  const InT* bc = lane < 32 ? static_cast<const InT*>(p.B) + sp.b * p.b_bs + sp.t0 * p.b_ts : static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + sp.t0 * p.c_ts;
  bc += g * N + sl * 16 + (lane & 1) * 8;
  const int64_t bc_ts = lane < 32 ? p.b_ts : p.c_ts;
  typedef typename Vec<InT, 8>::type V8;
  InT xn[8], dn[8];
  V8 bcn;
  bc += (int64_t)(ts * K + (lane & 31) / 2) * bc_ts;
  // (rows past the end are read from the last one and not used)
  auto back = [&](int t, int i) { return (int64_t)min(len - 1 - (t + half * 8), i); };
  auto fetch = [&](int t) {
    if (t + K <= len) {
      const InT *xr = xp, *dr = dp;
#pragma unroll
      for (int i = 0; i < 8; ++i, xr += x_ts, dr += dt_ts) {
        xn[i] = *xr;
        dn[i] = *dr;
      }
      bcn = *reinterpret_cast<const V8*>(bc);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = back(t, i);
        xn[i] = xp[r * x_ts];
        dn[i] = dp[r * dt_ts];
      }
      bcn = *reinterpret_cast<const V8*>(bc + min(len - 1 - (t + (lane & 31) / 2), 0) * bc_ts);
    }
    xp += IT * x_ts;
    dp += IT * dt_ts;
    bc += IT * bc_ts;
  };
  if (len > 0) fetch(ts * K);
  int par = 0;
  for (int t0 = 0; t0 < len; t0 += IT, par ^= 1) {
    const int t = t0 + ts * K;  // the wave's tokens t .. t + 16, the lane's t + 8 half .. + 8
    float d[K], dx[K], xv[8];
    {
      float f[8];
      unpack<8, InT>(bcn, f);
      f32x4* to = reinterpret_cast<f32x4*>(&s_bc[wave][(lane & 31) / 2][(lane >> 5) * 16 + (lane & 1) * 8]);
      to[0] = f32x4{f[0], f[1], f[2], f[3]};
      to[1] = f32x4{f[4], f[5], f[6], f[7]};
    }
    float sumd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      xv[i] = (float)xn[i];
      const float raw = (float)dn[i] + bias, sf = softplus_f(raw);
      // (tokens past the end: a decay of one and nothing added)
      const bool inside = t + half * 8 + i < len;
      const float own = soft ? sf : raw;
      both_halves(inside ? own : 0.f, d[i], d[8 + i]);
      both_halves(inside ? own * xv[i] : 0.f, dx[i], dx[8 + i]);
      sumd += d[i] + d[8 + i];
    }
    __builtin_amdgcn_wave_barrier();
    // from zero
    float a[K][8], e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k % 2 == 0) asm volatile("" ::: "memory");  // (B and C are read when their tokens come, not all at once)
      const f32x4 b0 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][half * 8]), b1 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][half * 8 + 4]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[k][j] = __builtin_amdgcn_exp2f(d[k] * A[j]);
        e[j] = fmaf(a[k][j], e[j], dx[k] * (j < 4 ? b0[j & 3] : b1[j & 3]));
      }
    }
    float P[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) P[j] = __builtin_amdgcn_exp2f(sumd * A[j]);
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
    InT zn[8];
    if (t + K <= len) {
      const InT* zr = zp;
#pragma unroll
      for (int i = 0; i < 8; ++i, zr += z_ts) zn[i] = *zr;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) zn[i] = zp[back(t, i) * z_ts];
    }
    zp += IT * z_ts;
    float yv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k % 2 == 0) asm volatile("" ::: "memory");  // (B and C are read when their tokens come, not all at once)
      if (k == K / 2) {  // (half of the decays are no longer held)
        if (t0 + IT < len) fetch(t + IT);
        __builtin_amdgcn_sched_barrier(0);
      }
      const f32x4 b0 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][half * 8]), b1 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][half * 8 + 4]);
      const f32x4 c0 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][16 + half * 8]), c1 = *reinterpret_cast<const f32x4*>(&s_bc[wave][k][20 + half * 8]);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] = fmaf(a[k][j], h[j], dx[k] * (j < 4 ? b0[j & 3] : b1[j & 3]));
        if (j < 4)
          s0 = fmaf(c0[j & 3], h[j], s0);
        else
          s1 = fmaf(c1[j & 3], h[j], s1);
      }
      yv[k] = s0 + s1;
      asm volatile("" : "+v"(yv[k]));  // (formed here: the states of all tokens would be held otherwise)
    }
    __builtin_amdgcn_wave_barrier();
    if (ts == TS - 1) {
      s_carry[par ^ 1][sl][0][lane] = f32x4{h[0], h[1], h[2], h[3]};
      s_carry[par ^ 1][sl][1][lane] = f32x4{h[4], h[5], h[6], h[7]};
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sum_halves(yv[i], yv[8 + i]);
    if constexpr (SL > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_y[wave][i][lane] = v[i];
      __syncthreads();
    }
    InT* yr = yp;
#pragma unroll
    for (int i = 0; i < 8; ++i, yr += C) {
      if (SL > 1 && i % SL != sl) continue;
      float o = v[i];
      if constexpr (SL > 1) {
        o = 0.f;
#pragma unroll
        for (int s = 0; s < SL; ++s) o += s_y[ts * SL + s][i][lane];
      }
      o = fmaf(D, xv[i], o);
      const float zv = (float)zn[i], sg = zv * sigmoid_f(zv);
      if (on && t + half * 8 + i < len) *yr = (InT)(o * (gate ? sg : 1.f));
    }
    yp += IT * C;
  }
  if (ts == TS - 1 && sp.last && p.S && on) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) {
      float* to = p.S + (r * p.C + c) * N + n0;
      *reinterpret_cast<f32x4*>(to) = f32x4{h[0], h[1], h[2], h[3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{h[4], h[5], h[6], h[7]};
    }
  }
}

template <typename InT>
static hipError_t launch_t(const ScanParams& p, int n, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)p.slots * p.G * p.btiles + 7) / 8 * 8)), block(64 * SCAN_BLOCK_WAVES);
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
