// Single-token step of the selective scan on gfx950: h <- exp(d A) h + d x B in place, y = (C h + D x) silu(z).
//
// The fp32 state is the traffic, read and written once: a lane has four states of a channel (16 bytes), N / 4
// neighbouring lanes a channel, whose sum is a butterfly over them. Bound by memory: 512 sequences x 4096 channels x 16
// states, 63 us (4.5 TB/s; 55 at the rate of a large copy).
#include "scan.hpp"

namespace dr {

template <int N, typename InT>
__global__ __launch_bounds__(256) void scan_step_kernel(const ScanParams p) {
  constexpr int LPC = N / 4, CH = scan_step_channels(N);
  const int per = (p.C + CH - 1) / CH;
  const int n = blockIdx.x / per, c = (blockIdx.x - n * per) * CH + threadIdx.x / LPC, j = (threadIdx.x % LPC) * 4;
  if (c >= p.C) return;  // (a channel's lanes leave together)
  InT* y = static_cast<InT*>(p.y) + (int64_t)n * p.C + c;
  const int64_t r = state_row(p.sidx, p.nslots, n);
  if (r < 0) {  // no stored state
    if (j == 0) *y = (InT)0.f;
    return;
  }
  f32x4* S = reinterpret_cast<f32x4*>(p.S + (r * p.C + c) * N + j);
  f32x4 h = __builtin_nontemporal_load(S);
  const f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * N + j);
  const int g = c / p.Cg;
  const float x = (float)static_cast<const InT*>(p.x)[n * p.x_bs + c];
  const float raw = (float)static_cast<const InT*>(p.dt)[n * p.dt_bs + c] + (p.bias ? p.bias[c] : 0.f);
  float B[4], C[4];
  unpack<4, InT>(*reinterpret_cast<const typename Vec<InT, 4>::type*>(static_cast<const InT*>(p.B) + n * p.b_bs + g * N + j), B);
  unpack<4, InT>(*reinterpret_cast<const typename Vec<InT, 4>::type*>(static_cast<const InT*>(p.Cm) + n * p.c_bs + g * N + j), C);
  const float d = p.softplus ? softplus_f(raw) : raw, dx = d * x;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = fmaf(__builtin_amdgcn_exp2f(d * LOG2E * A[k]), h[k], dx * B[k]);
    v = fmaf(C[k], h[k], v);
  }
  __builtin_nontemporal_store(h, S);
#pragma unroll
  for (int k = 1; k < LPC; k <<= 1) v += __shfl_xor(v, k);
  if (j == 0) {
    v = fmaf(p.D ? p.D[c] : 0.f, x, v);
    if (p.z) {
      const float z = (float)static_cast<const InT*>(p.z)[n * p.z_bs + c];
      v *= z * sigmoid_f(z);
    }
    *y = (InT)v;
  }
}

template <int N>
static hipError_t launch_t(const ScanParams& p, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.nseq * ((p.C + scan_step_channels(N) - 1) / scan_step_channels(N))));
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
