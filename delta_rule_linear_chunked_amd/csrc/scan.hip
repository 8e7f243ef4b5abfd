// Selective scan over the tokens of every channel on gfx950: h <- exp(d A) h + d x B, y = (C h + D x) silu(z).
//
// A decay of its own for every (token, channel, state) leaves nothing for a matrix product: per state one exponential and four more
// operations on the vector units, which is what bounds the pass. A lane has one channel and NS of its states in registers, so B and C are
// the same for a whole wave and come through the scalar unit; the sum over states needs no exchange between lanes. With
// more states than NS the waves of a workgroup share a channel tile and add their parts of y through LDS.
// Sequences that are too few to fill the GPU are cut into segments: their own states from zero first (one more pass without
// C and y), then each segment's start by a walk over the segments, whose decay is exp(A sum d).
#include "scan.hpp"

namespace dr {

// ---------------------------------------------------------------------------
// Scalar loads of NS elements of a token's B or C (uniform addresses, 4-byte aligned, nothing writes them meanwhile).
// ---------------------------------------------------------------------------
typedef const __attribute__((address_space(4))) uint32_t* const_u32;
template <typename InT, int NS>
struct Row {
  static constexpr int NW = NS * (int)sizeof(InT) / 4;
  uint32_t w[NW];
  __device__ __forceinline__ void load(const InT* at) {
    const const_u32 q = (const_u32)(uintptr_t)at;
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = q[i];
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(InT) == 4)
      return __builtin_bit_cast(float, w[i]);
    else
      return __builtin_bit_cast(float, i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// The main pass (LOCAL false: outputs and final states) or the segments' own states and sums of d.
template <int NS, int NW, typename InT, bool LOCAL>
__global__ __launch_bounds__(64 * NW) void scan_kernel(const ScanParams p) {
  constexpr int N = NS * NW, TT = 8;
  __shared__ float s_y[NW > 1 ? 2 : 1][NW > 1 ? NW : 1][NW > 1 ? TT : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ntiles = p.G * p.tiles;
  const int slot = blockIdx.x / ntiles, tile = blockIdx.x - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0 || (LOCAL && sp.last)) return;
  const int g = tile / p.tiles, in_g = (tile - g * p.tiles) * SCAN_TILE + lane;
  const bool on = in_g < p.Cg;
  const int c = g * p.Cg + min(in_g, p.Cg - 1);
  float A[NS], h[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    A[j] = p.A[(int64_t)c * N + wave * NS + j] * LOG2E;
    h[j] = 0.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f, D = !LOCAL && p.D ? p.D[c] : 0.f;
  if constexpr (!LOCAL) {
    const float* from = nullptr;
    if (p.part) {
      from = p.part + ((int64_t)slot * p.C + c) * N;
    } else if (p.S0) {
      const int64_t r = state_row(p.sidx, p.nslots, sp.n);
      if (r >= 0) from = p.S0 + (r * p.C + c) * N;
    }
    if (from)
#pragma unroll
      for (int j = 0; j < NS; j += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(from + wave * NS + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[j + k] = v[k];
      }
  }
  const int len = sp.len;
  const InT* x = static_cast<const InT*>(p.x) + sp.b * p.x_bs + sp.t0 * p.x_ts + c;
  const InT* dt = static_cast<const InT*>(p.dt) + sp.b * p.dt_bs + sp.t0 * p.dt_ts + c;
  const InT* z = !LOCAL && p.z ? static_cast<const InT*>(p.z) + sp.b * p.z_bs + sp.t0 * p.z_ts + c : nullptr;
  const InT* Bp = static_cast<const InT*>(p.B) + sp.b * p.b_bs + sp.t0 * p.b_ts + g * N + wave * NS;
  const InT* Cp = static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + sp.t0 * p.c_ts + g * N + wave * NS;
  InT* y = LOCAL ? nullptr : static_cast<InT*>(p.y) + (sp.b * p.T + sp.t0) * (int64_t)p.C + c;
  float sumd = 0.f;
  InT xn[TT], dn[TT], zn[TT];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t r = min(t + i, len - 1);
      xn[i] = x[r * p.x_ts];
      dn[i] = dt[r * p.dt_ts];
      zn[i] = z ? z[r * p.z_ts] : InT(0);
    }
  };
  if (len > 0) fetch(0);
  int buf = 0;
  for (int t = 0; t < len; t += TT, buf ^= 1) {
    float xv[TT], dv[TT], zv[TT], yv[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      xv[i] = (float)xn[i];
      const float raw = (float)dn[i] + bias;
      dv[i] = p.softplus ? softplus_f(raw) : raw;
      zv[i] = (float)zn[i];
    }
    if (t + TT < len) fetch(t + TT);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      yv[i] = 0.f;
      if (t + i < len) {
        Row<InT, NS> Bt, Ct;
        Bt.load(Bp + (t + i) * p.b_ts);
        if constexpr (!LOCAL) Ct.load(Cp + (t + i) * p.c_ts);
        const float d = dv[i], dx = d * xv[i];
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          h[j] = fmaf(__builtin_amdgcn_exp2f(d * A[j]), h[j], dx * Bt[j]);
          if constexpr (!LOCAL) acc[j & 3] = fmaf(Ct[j], h[j], acc[j & 3]);
        }
        yv[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        if constexpr (LOCAL) sumd += d;
      }
    }
    if constexpr (!LOCAL) {
      if constexpr (NW > 1) {
#pragma unroll
        for (int i = 0; i < TT; ++i) s_y[buf][wave][i][lane] = yv[i];
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        if (t + i >= len || (NW > 1 && i % NW != wave)) continue;  // (uniform over the wave)
        float v = yv[i];
        if constexpr (NW > 1) {
          v = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) v += s_y[buf][w][i][lane];
        }
        v = fmaf(D, xv[i], v);
        if (z) v *= zv[i] * sigmoid_f(zv[i]);
        if (on) y[(int64_t)(t + i) * p.C] = (InT)v;
      }
    }
  }
  if constexpr (LOCAL) {
    if (on) {
      float* to = p.part + ((int64_t)slot * p.C + c) * N + wave * NS;
#pragma unroll
      for (int j = 0; j < NS; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{h[j], h[j + 1], h[j + 2], h[j + 3]};
      if (wave == 0) p.sumd[(int64_t)slot * p.C + c] = sumd;
    }
  } else if (sp.last && p.S && on) {
    const int64_t r = state_row(p.sidx, p.nslots, sp.n);
    if (r >= 0) {
      float* to = p.S + (r * p.C + c) * N + wave * NS;
#pragma unroll
      for (int j = 0; j < NS; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{h[j], h[j + 1], h[j + 2], h[j + 3]};
    }
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

template <int NS, int NW, typename InT>
static hipError_t launch_t(const ScanParams& p, bool local, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.tiles)), block(64 * NW);
  if (local)
    hipLaunchKernelGGL((scan_kernel<NS, NW, InT, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((scan_kernel<NS, NW, InT, false>), grid, block, 0, s, p);
  return hipGetLastError();
}
template <typename InT>
static hipError_t launch_any(const ScanParams& p, int n, bool local, hipStream_t s) {
  return n == 16 ? launch_t<16, 1, InT>(p, local, s) : n == 32 ? launch_t<16, 2, InT>(p, local, s) : launch_t<16, 4, InT>(p, local, s);
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
  return bf16 ? launch_any<__bf16>(p, n, false, s) : launch_any<float>(p, n, false, s);
}

}  // namespace dr
