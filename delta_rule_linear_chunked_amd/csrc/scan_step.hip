// Single-token step of the selective scan on gfx950: h <- exp(d A) h + d x B in place, y = (C h + D x) silu(z).
//
// The fp32 state is the traffic, read and written once: a lane has four states of a channel (16 bytes), N / 4
// neighbouring lanes a channel, whose sum is a butterfly over them. A workgroup takes up to four sequences one after the other on its channels,
// whose A it holds, the next one's inputs in flight. Bound by memory: 512 sequences x 4096 channels x 16 states in bf16 51 us in a graph
// (285 MB, 5.6 TB/s; 55 at the rate of a large copy), 65 with one sequence a workgroup.
#include "scan_tile.hpp"

namespace dr {

template <int N, typename InT>
__global__ __launch_bounds__(256) void scan_step_kernel(const ScanParams p) {
  constexpr int LPC = N / 4, CH = scan_step_channels(N);
  using V4 = typename Vec<InT, 4>::type;
  const int per = (p.C + CH - 1) / CH;
  const int n0 = blockIdx.x / per * p.run, c = (blockIdx.x % per) * CH + threadIdx.x / LPC, j = (threadIdx.x % LPC) * 4;
  const int n1 = min(n0 + p.run, p.nseq);
  if (c >= p.C) return;  // (a channel's lanes leave together)
  const f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * N + j);
  const int g = c / p.Cg;
  const float bias = p.bias ? p.bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
  const float least = step_least(p.softplus != 0);
  const bool gate = p.z != nullptr;
  const InT* zs = static_cast<const InT*>(gate ? p.z : p.x);
  const int64_t zst = gate ? p.z_bs : p.x_bs;
  // lane i: of sequence n0 + i. Read from lanes by number: the first channel's, which are there wherever a wave has a channel at all.
  static_assert(LPC >= SCAN_STEP_RUN, "a sequence for each of them");
  const int lane = threadIdx.x & 63;
  int rows = -1;
  if (n0 + lane < n1) rows = (int)state_row(p.sidx, p.nslots, n0 + lane);
  // the next sequence's inputs are loaded ahead of their use; one without a stored state reads A in its place
  f32x4 hn;
  V4 Bn, Cn;
  uint32_t xn, dn, zn;
  auto fetch = [&](int64_t n) {
    const int r = __builtin_amdgcn_readlane(rows, (int)n - n0);
    const float* row = r >= 0 ? p.S + (int64_t)r * p.C * N : p.A;
    hn = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(row + (int64_t)c * N + j));
    xn = raw_bits(static_cast<const InT*>(p.x) + n * p.x_bs + c);
    dn = raw_bits(static_cast<const InT*>(p.dt) + n * p.dt_bs + c);
    zn = raw_bits(zs + n * zst + c);
    Bn = *reinterpret_cast<const V4*>(static_cast<const InT*>(p.B) + n * p.b_bs + g * N + j);
    Cn = *reinterpret_cast<const V4*>(static_cast<const InT*>(p.Cm) + n * p.c_bs + g * N + j);
  };
  auto token = [&](int n, auto more) {
    f32x4 h = hn;
    const float x = raw_value<InT>(xn), raw = raw_value<InT>(dn) + bias, z = raw_value<InT>(zn);
    float B[4], C[4];
    unpack<4, InT>(Bn, B);
    unpack<4, InT>(Cn, C);
    if constexpr (decltype(more)::value) fetch(n + 1);
    const float d = step_f(raw, least), dx = d * x;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[k] = fmaf(__builtin_amdgcn_exp2f(d * LOG2E * A[k]), h[k], dx * B[k]);
      v = fmaf(C[k], h[k], v);
    }
#pragma unroll
    for (int k = 1; k < LPC; k <<= 1) v += __shfl_xor(v, k);
    v = fmaf(D, x, v);
    v *= gate ? z * sigmoid_f(z) : 1.f;
    InT* y = static_cast<InT*>(p.y) + (int64_t)n * p.C + c;  // (a channel's lanes have the same sum and write it together)
    const int r = __builtin_amdgcn_readlane(rows, n - n0);
    if (r >= 0) {
      __builtin_nontemporal_store(h, reinterpret_cast<f32x4*>(p.S + ((int64_t)r * p.C + c) * N + j));
      *y = (InT)v;
    } else {
      *y = (InT)0.f;
      arrived();
    }
  };
  fetch(n0);
  arrived();
  for (int n = n0; n + 1 < n1; ++n) token(n, std::true_type{});
  token(n1 - 1, std::false_type{});
}

template <int N>
static hipError_t launch_t(const ScanParams& p, bool bf16, hipStream_t s) {
  const int64_t groups = ((int64_t)p.nseq + p.run - 1) / p.run;
  const dim3 grid((unsigned)(groups * ((p.C + scan_step_channels(N) - 1) / scan_step_channels(N))));
  if (bf16)
    hipLaunchKernelGGL((scan_step_kernel<N, __bf16>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((scan_step_kernel<N, float>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}
hipError_t launch_scan_step(const ScanParams& p, int n, bool bf16, hipStream_t s) {
  return n == 16 ? launch_t<16>(p, bf16, s) : n == 32 ? launch_t<32>(p, bf16, s) : launch_t<64>(p, bf16, s);
}

}  // namespace dr
