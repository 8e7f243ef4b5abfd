// Selective scan over the tokens of every channel on gfx950: h <- exp(d A) h + d x B, y = (C h + D x) silu(z).
//
// A decay of its own for every (token, channel, state) leaves nothing for a matrix product: per state one exponential and four more
// operations on the vector units, which is what bounds the pass. A lane has one channel and NS of its states in registers, so B and C are
// the same for a whole wave and come through the scalar unit; the sum over states needs no exchange between lanes. With
// more states than NS the waves of a workgroup share a channel tile and add their parts of y through LDS.
// Sequences that are too few to fill the GPU are cut into segments: their own states from zero first (one more pass without
// C and y), then each segment's start by a walk over the segments, whose decay is exp(A sum d).
#include <type_traits>

#include "scan.hpp"

namespace dr {

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
  if (in_g >= p.Cg) return;  // (the same lanes of every wave, and never all of a wave's: the barriers below still meet)
  const int c = g * p.Cg + in_g;
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
  const bool soft = p.softplus != 0, gate = !LOCAL && p.z != nullptr;
  const InT* xp = static_cast<const InT*>(p.x) + sp.b * p.x_bs + sp.t0 * p.x_ts + c;
  const InT* dp = static_cast<const InT*>(p.dt) + sp.b * p.dt_bs + sp.t0 * p.dt_ts + c;
  const InT* zp = gate ? static_cast<const InT*>(p.z) + sp.b * p.z_bs + sp.t0 * p.z_ts + c : xp;
  const InT* Bp = static_cast<const InT*>(p.B) + sp.b * p.b_bs + sp.t0 * p.b_ts + g * N + wave * NS;
  const InT* Cp = static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + sp.t0 * p.c_ts + g * N + wave * NS;
  InT* y = LOCAL ? nullptr : static_cast<InT*>(p.y) + (sp.b * p.T + sp.t0) * (int64_t)p.C + c;
  const int64_t x_ts = p.x_ts, dt_ts = p.dt_ts, z_ts = gate ? p.z_ts : p.x_ts, b_ts = p.b_ts, c_ts = p.c_ts, C = p.C;
  float sumd = 0.f;
  // A tile's inputs come a tile ahead, a token's rows of B and C a token ahead; nothing past the last token is read.
  InT xn[TT], dn[TT], zn[TT];
  auto fetch = [&](int n) {  // the next n tokens (TT of them but at the end)
    if (n >= TT) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        xn[i] = *xp;
        dn[i] = *dp;
        xp += x_ts;
        dp += dt_ts;
        if constexpr (!LOCAL) {
          zn[i] = *zp;
          zp += z_ts;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        xn[i] = dn[i] = zn[i] = InT(0);
        if (i < n) {
          xn[i] = *xp;
          dn[i] = *dp;
          xp += x_ts;
          dp += dt_ts;
          if constexpr (!LOCAL) {
            zn[i] = *zp;
            zp += z_ts;
          }
        }
      }
    }
  };
  Row<InT, NS> Bt[2], Ct[2];
  auto rows = [&](int to, bool more) {
    Bt[to].load(Bp);
    Bp += more ? b_ts : 0;
    if constexpr (!LOCAL) {
      Ct[to].load(Cp);
      Cp += more ? c_ts : 0;
    }
  };
  if (len > 0) {
    fetch(len);
    rows(0, len > 1);
  }
  int buf = 0;
  auto run = [&](int t, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    float xv[TT], dv[TT], zv[TT], yv[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      xv[i] = (float)xn[i];
      const float raw = (float)dn[i] + bias, sf = softplus_f(raw);
      dv[i] = soft ? sf : raw;
      // (tokens past the end: a decay of one and nothing added)
      if (!WHOLE && t + i >= len) dv[i] = 0.f;
      if constexpr (!LOCAL) {
        zv[i] = (float)zn[i];
        const float sg = zv[i] * sigmoid_f(zv[i]);
        zv[i] = gate ? sg : 1.f;
      }
    }
    if (WHOLE && t + TT < len) fetch(len - t - TT);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      rows((i + 1) & 1, t + i + 2 < len);
      __builtin_amdgcn_sched_barrier(0);
      const float d = dv[i], dx = d * xv[i];
      float a[NS], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NS; ++j) a[j] = __builtin_amdgcn_exp2f(d * A[j]);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        h[j] = fmaf(a[j], h[j], dx * Bt[i & 1][j]);
        if constexpr (!LOCAL) acc[j & 3] = fmaf(Ct[i & 1][j], h[j], acc[j & 3]);
      }
      yv[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      if constexpr (LOCAL) sumd += d;
      if constexpr (!LOCAL) asm volatile("" : "+v"(yv[i]));  // (here, not where it is stored: C's rows are held no longer)
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!LOCAL) {
      if constexpr (NW > 1) {
#pragma unroll
        for (int i = 0; i < TT; ++i) s_y[buf][wave][i][lane] = yv[i];
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        if ((WHOLE || t + i < len) && (NW == 1 || i % NW == wave)) {  // (uniform over the wave)
          float v = yv[i];
          if constexpr (NW > 1) {
            v = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v += s_y[buf][w][i][lane];
          }
          *y = (InT)(fmaf(D, xv[i], v) * zv[i]);
        }
        y += C;
      }
    }
  };
  int t = 0;
  for (; t + TT <= len; t += TT, buf ^= 1) run(t, std::true_type{});
  if (t < len) run(t, std::false_type{});
  if constexpr (LOCAL) {
    float* to = p.part + ((int64_t)slot * p.C + c) * N + wave * NS;
#pragma unroll
    for (int j = 0; j < NS; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{h[j], h[j + 1], h[j + 2], h[j + 3]};
    if (wave == 0) p.sumd[(int64_t)slot * p.C + c] = sumd;
  } else if (sp.last && p.S) {
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
  if (pl.block) return launch_scan_block(p, n, bf16, s);
  return bf16 ? launch_any<__bf16>(p, n, false, s) : launch_any<float>(p, n, false, s);
}

}  // namespace dr
