// Selective scan over the tokens of every channel on gfx950: h <- exp(d A) h + d x B, y = (C h + D x) silu(z).
//
// A decay of its own for every (token, channel, state): per state one exponential (twice an ordinary operation), one product and
// two sums on the vector units, which bound the pass; what is added to the state comes from the matrix units (scan_tile.hpp). A wave
// walks the tokens of 32 channels x 16 states; with more states the waves of a workgroup share the channels and add their parts of y
// through LDS.
// Sequences that are too few to fill the GPU are cut into segments: their own states from zero first (one more pass without
// C and y), then each segment's start by a walk over the segments, whose decay is exp(A sum d); or a workgroup's waves
// go along the tokens (scan_block.hip).
//
// 64 x 256 tokens x 2048 channels, 16 states, bf16: 136 us, four waves a SIMD. Packed, fp32, 32 states (5.2 million token-channels): segments'
// states 54 us, main pass 60, join 10, plan 5; the vector units issue 73 and 77% of the time. Loads and stores of whole tiles stand under no
// condition (1 x 8192 x 2048: main pass 0.195 us a token with them under conditions, 0.17 without).
#include "scan_tile.hpp"

namespace dr {

// The main pass (LOCAL false: outputs and final states) or the segments' own states and sums of d. (16 states, bf16: the compiler would take 154 registers,
// three waves a SIMD; 64 x 256 x 2048 142 us so, 137 with four.)
template <int SL, typename InT, bool LOCAL>
__global__ __launch_bounds__(64 * SL, !LOCAL && SL == 1 && sizeof(InT) == 2 ? 4 : 1) void scan_kernel(const ScanParams p) {
  constexpr int N = 16 * SL, K = TILE_TOK, O = TILE_OWN;
  __shared__ __align__(16) float s_c[LOCAL ? 1 : SL][LOCAL ? 1 : K][16];          // a wave's own rows of C
  __shared__ float s_y[SL > 1 && !LOCAL ? 2 : 1][SL > 1 && !LOCAL ? SL : 1][SL > 1 && !LOCAL ? O : 1][64];
  const int lane = threadIdx.x & 63, sl = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int ntiles = p.G * p.tiles;
  const int slot = blockIdx.x / ntiles, tile = blockIdx.x - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0 || (LOCAL && sp.last)) return;
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
  const float bias = p.bias ? p.bias[c] : 0.f, D = !LOCAL && p.D ? p.D[c] : 0.f;
  if constexpr (!LOCAL) {
    if (p.part && !sp.whole()) {
      load_states(p.part + ((int64_t)slot * p.C + c) * N + n0, h);
    } else if (p.S0) {
      const int64_t r = state_row(p.sidx, p.nslots, sp.n);
      if (r >= 0) load_states(p.S0 + (r * p.C + c) * N + n0, h);
    }
  }
  const int len = sp.len;
  const float least = step_least(p.softplus != 0);
  const bool gate = !LOCAL && p.z != nullptr;
  Rows<InT> X, T, Z, B;
  X.init(p.x, sp.b * p.x_bs + sp.t0 * p.x_ts, p.x_ts, half, c);
  T.init(p.dt, sp.b * p.dt_bs + sp.t0 * p.dt_ts, p.dt_ts, half, c);
  if (gate)
    Z.init(p.z, sp.b * p.z_bs + sp.t0 * p.z_ts, p.z_ts, half, c);
  else
    Z = X;
  B.init(p.B, sp.b * p.b_bs + sp.t0 * p.b_ts, p.b_ts, half, g * N + sl * 16 + (lane & 15));
  // C: lane l brings states 4 (l % 4) .. + 3 of token l / 4
  typedef typename Vec<InT, 4>::type V4;
  auto c_at = [&](uint32_t l) { return ((l >> 2) * (uint32_t)p.c_ts + (uint32_t)(g * N + sl * 16) + 4 * (l & 3)) * (uint32_t)sizeof(InT); };
  const InT* Ca = static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + sp.t0 * p.c_ts;
  InT* y = LOCAL ? nullptr : static_cast<InT*>(p.y) + (sp.b * p.T + sp.t0) * (int64_t)p.C;
  float sumd = 0.f;
  uint32_t xn[O], dn[O], zn[O], bn[O];
  V4 cn{};
  // a whole tile, the next one if there is one, the same again if not (loads under a condition would be waited for where its branches meet)
  auto fetch = [&](int step) {
    X.at += step * X.ts;
    T.at += step * T.ts;
    B.at += step * B.ts;
    X.whole(xn);
    T.whole(dn);
    B.whole(bn);
    if constexpr (!LOCAL) {
      Z.at += step * Z.ts;
      Ca += step * p.c_ts;
      Z.whole(zn);
      cn = *reinterpret_cast<const V4*>(byte_at(Ca, c_at(fresh(lane))));
    }
  };
  int buf = 0;
  auto tokens = [&](int t, auto cut) {
    constexpr bool CUT = decltype(cut)::value;
    float xv[O], dv[O], zv[O], dx[O], bo[O], v[O];
#pragma unroll
    for (int i = 0; i < O; ++i) {
      xv[i] = raw_value<InT>(xn[i]);
      float own = step_f(raw_value<InT>(dn[i]) + bias, least);
      here(own);
      // (tokens past the end: a decay of one and nothing added)
      const bool inside = !CUT || t + 2 * i + half < len;
      dv[i] = inside ? own : 0.f;
      dx[i] = inside ? dv[i] * xv[i] : 0.f;
      if constexpr (!LOCAL) own_token(dv[i], dx[i]);  // (the segment's last state is not finite either way)
      bo[i] = inside ? operand<InT>(bn[i], lane) : 0.f;
      if constexpr (!LOCAL) zv[i] = raw_value<InT>(zn[i]);
      if constexpr (LOCAL) sumd += dv[i];
    }
    if constexpr (!LOCAL) {
      float f[4];
      unpack<4, InT>(cn, f);
      *reinterpret_cast<f32x4*>(&s_c[sl][lane >> 2][4 * (lane & 3)]) = f32x4{f[0], f[1], f[2], f[3]};
      __builtin_amdgcn_wave_barrier();
    }
    if constexpr (!CUT) fetch(t + 2 * K <= len ? K : 0);
    f32x16 in = outer_pair(bo[0], dx[0]);
#pragma unroll
    for (int i = 0; i < O; ++i) {
      tile_step();
      float d[2], s[2];
      both_halves(dv[i], d[0], d[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f32x4 c0{}, c1{};
        if constexpr (!LOCAL) {
          c0 = *reinterpret_cast<const f32x4*>(&s_c[sl][2 * i + k][4 * half]);
          c1 = *reinterpret_cast<const f32x4*>(&s_c[sl][2 * i + k][8 + 4 * half]);
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = fmaf(__builtin_amdgcn_exp2f(d[k] * A[j]), h[j], in[8 * k + j]);
        if (k == 1 && i + 1 < O) in = outer_pair(bo[i + 1], dx[i + 1]);  // (the decays hide it; two at once would hold 16 more registers)
        if constexpr (!LOCAL) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < 4)
              s0 = fmaf(c0[j & 3], h[j], s0);
            else
              s1 = fmaf(c1[j & 3], h[j], s1);
        }
        s[k] = s0 + s1;
      }
      if constexpr (!LOCAL) {
        v[i] = sum_halves(s[0], s[1]);
        here(v[i]);  // (the states of all tokens would be held otherwise)
      }
    }
    if constexpr (!LOCAL) {
      __builtin_amdgcn_wave_barrier();
      if constexpr (SL > 1) {
#pragma unroll
        for (int i = 0; i < O; ++i) s_y[buf][sl][i][lane] = v[i];
        __syncthreads();
      }
      InT* row = y;
      if constexpr (SL > 1) row += 2 * sl * (int64_t)p.C;
      // (of SL pairs a wave has one; in a whole tile lanes past the last channel write that one's outputs again: stores under a condition
      // would be waited for with the next tile's inputs)
#pragma unroll
      for (int q = 0; q < O / SL; ++q, row += 2 * SL * (int64_t)p.C) {
        float o = v[q], x = xv[q], z = zv[q];
        if constexpr (SL > 1) {
          o = 0.f;
#pragma unroll
          for (int w = 0; w < SL; ++w) {
            o += s_y[buf][w][q * SL + sl][lane];
            x = w == 0 || sl == w ? xv[q * SL + w] : x;
            z = w == 0 || sl == w ? zv[q * SL + w] : z;
          }
        }
        o = fmaf(D, x, o);
        const float sg = z * sigmoid_f(z);
        if (!CUT || (on && t + 2 * (q * SL + sl) + half < len)) *byte_at(row, (fresh(c) + (fresh(half) ? (uint32_t)p.C : 0u)) * (uint32_t)sizeof(InT)) = (InT)(o * (gate ? sg : 1.f));
      }
      y += K * (int64_t)p.C;
    }
    buf ^= 1;
  };
  const int whole = len / K * K;
  if (whole > 0) {
    fetch(0);
    arrived();
    for (int t = 0; t < whole; t += K) tokens(t, std::false_type{});
  }
  if (whole < len) {
    const int step = whole > 0 ? K : 0, left = len - whole;
    X.at += step * X.ts;
    T.at += step * T.ts;
    B.at += step * B.ts;
    X.part(xn, left);
    T.part(dn, left);
    B.part(bn, left);
    if constexpr (!LOCAL) {
      Z.at += step * Z.ts;
      Ca += step * p.c_ts;
      Z.part(zn, left);
      cn = *reinterpret_cast<const V4*>(Ca + ((int64_t)min(lane >> 2, left - 1) * p.c_ts + g * N + sl * 16 + 4 * (lane & 3)));
    }
    tokens(whole, std::true_type{});
  }
  if (!on) return;
  if constexpr (LOCAL) {
    store_states(p.part + ((int64_t)slot * p.C + c) * N + n0, h);
    float lo, hi;  // (the halves' tokens)
    both_halves(sumd, lo, hi);
    if (sl == 0 && half == 0) p.sumd[(int64_t)slot * p.C + c] = lo + hi;
  } else if (sp.last && p.S) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) store_states(p.S + (r * p.C + c) * N + n0, h);
  }
}

// Each segment's start state in the place of its own: a walk over a sequence's segments, four states a lane.
template <int N>
__global__ __launch_bounds__(256) void scan_join_kernel(const ScanParams p) {
  const int per = (p.C * (N / 4) + 255) / 256;
  const int n = blockIdx.x / per, e = (blockIdx.x - n * per) * 256 + threadIdx.x;
  if (e >= p.C * (N / 4)) return;
  const int c = e / (N / 4), j = e - c * (N / 4);
  const int first = p.cu ? p.slot_first[n] : n * p.nseg, past = p.cu ? p.slot_first[n + 1] : first + p.nseg;
  if (past - first == 1) return;  // (a sequence that is not cut starts from S0 itself)
  f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * N + 4 * j), h = {0, 0, 0, 0};
  const int64_t r = state_row(p.sidx, p.nslots, n);
  if (p.S0 && r >= 0) h = *reinterpret_cast<const f32x4*>(p.S0 + (r * p.C + c) * N + 4 * j);
  for (int s = first; s < past; ++s) {
    f32x4* at = reinterpret_cast<f32x4*>(p.part + ((int64_t)s * p.C + c) * N + 4 * j);
    f32x4 own = {0, 0, 0, 0};
    float d = 0.f;
    if (s + 1 < past) {  // (a sequence's last segment has no state of its own)
      own = *at;
      d = p.sumd[(int64_t)s * p.C + c];
    }
    *at = h;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = fmaf(__builtin_amdgcn_exp2f(d * LOG2E * A[k]), h[k], own[k]);
  }
}

template <int SL, typename InT>
static hipError_t launch_t(const ScanParams& p, bool local, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.tiles)), block(64 * SL);
  if (local)
    hipLaunchKernelGGL((scan_kernel<SL, InT, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((scan_kernel<SL, InT, false>), grid, block, 0, s, p);
  return hipGetLastError();
}
template <typename InT>
static hipError_t launch_any(const ScanParams& p, int n, bool local, hipStream_t s) {
  return n == 16 ? launch_t<1, InT>(p, local, s) : n == 32 ? launch_t<2, InT>(p, local, s) : launch_t<4, InT>(p, local, s);
}

// Offsets and slot tables of packed sequences: the plan pass of the decayed linear attention makes the same ones.
hipError_t launch_scan_plan(const ScanParams& p, hipStream_t s) {
  DecayParams q{};
  q.cu = p.cu;
  q.cu_ok = p.cu_ok;
  q.T = p.T;
  q.nseq = p.nseq;
  q.seg = p.seg;
  q.slots = p.slots;
  q.slot_seq = p.slot_seq;
  q.slot_first = p.slot_first;
  return launch_decay_plan(q, s);
}

hipError_t launch_scan_fwd(ScanParams p, const ScanPlan& pl, int n, bool bf16, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.cu) {
    e = launch_scan_plan(p, s);
    if (e != hipSuccess) return e;
    p.cu = p.cu_ok;
  }
  if (pl.nseg > 1) {
    e = bf16 ? launch_any<__bf16>(p, n, true, s) : launch_any<float>(p, n, true, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((int64_t)p.nseq * ((p.C * (n / 4) + 255) / 256)));
    if (n == 16)
      hipLaunchKernelGGL((scan_join_kernel<16>), grid, dim3(256), 0, s, p);
    else if (n == 32)
      hipLaunchKernelGGL((scan_join_kernel<32>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((scan_join_kernel<64>), grid, dim3(256), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    p.part = nullptr;
  }
  if (pl.block) return launch_scan_block(p, n, bf16, s);
  return bf16 ? launch_any<__bf16>(p, n, false, s) : launch_any<float>(p, n, false, s);
}

}  // namespace dr
