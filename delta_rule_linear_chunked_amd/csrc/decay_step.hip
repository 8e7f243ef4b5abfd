// Single-token step of the decayed linear attention on gfx950: S <- a S + k v^T in place, o = S^T q.
//
// The fp32 state is the traffic (read and written once); value columns are independent, so a head splits
// into slices of DVS columns with no exchange between workgroups. Every thread holds 4 columns of a few
// rows; o sums over the rows by a butterfly within the wave and one pass through LDS. Bound by the state's bytes:
// 512 sequences x 32 heads, d = 128, 392 us, 5530 GB/s; one sequence of 16 heads 3.5 us.
#include "decay.hpp"

namespace dr {

template <int DK, int DVS>
struct StepShape {
  static constexpr int COLS4 = DVS / 4;
  static constexpr int NT = step_threads(DK, DVS);
  static constexpr int RG = NT / COLS4;       // row groups
  static constexpr int RPT = DK / RG;         // rows per thread
  static constexpr int NW = NT / 64;
  static_assert(NT % 64 == 0 && COLS4 <= 64, "whole waves");
};

template <int DK, int DVS, typename InT>
__global__ __launch_bounds__((StepShape<DK, DVS>::NT)) void decay_step_kernel(const DecayParams p) {
  using Sh = StepShape<DK, DVS>;
  constexpr int COLS4 = Sh::COLS4, RG = Sh::RG, RPT = Sh::RPT, NW = Sh::NW, NT = Sh::NT;
  __shared__ float s_q[DK], s_k[DK];
  __shared__ __align__(16) float s_red[NW][DVS];
  const int tid = threadIdx.x, c4 = tid % COLS4, rg = tid / COLS4;
  const int ncb = p.DV / DVS;
  const int64_t nh = blockIdx.x / ncb;
  const int col0 = (int)(blockIdx.x - nh * ncb) * DVS;
  const int64_t n = nh / p.H;
  const int h = (int)(nh - n * p.H);
  float* o = p.o + nh * p.DV + col0;
  int64_t row = n;
  if (p.sidx) {
    row = p.sidx[n];
    if (row < 0 || row >= p.nslots) {  // no stored state
      for (int j = tid; j < DVS; j += NT) o[j] = 0.f;
      return;
    }
  }
  const int hk = h / (p.H / p.Hk);
  const InT* q = static_cast<const InT*>(p.q) + n * p.q_bs + (int64_t)hk * DK;
  const InT* k = static_cast<const InT*>(p.k) + n * p.k_bs + (int64_t)hk * DK;
  const InT* v = static_cast<const InT*>(p.v) + n * p.v_bs + (int64_t)h * p.DV + col0 + 4 * c4;
  float* S = p.S + (row * p.H + h) * (int64_t)DK * p.DV + col0 + 4 * c4;
  // small loads first (memory returns in order), then the state
  float qv[(DK + NT - 1) / NT], kv[(DK + NT - 1) / NT];
#pragma unroll
  for (int i = 0; i < (DK + NT - 1) / NT; ++i) {
    const int j = tid + i * NT;
    qv[i] = j < DK ? ld_f32(q + j) : 0.f;
    kv[i] = j < DK ? ld_f32(k + j) : 0.f;
  }
  f32x4 vv;
#pragma unroll
  for (int j = 0; j < 4; ++j) vv[j] = ld_f32(v + j);
  const float a = p.alpha[p.a_tok ? nh : h];
  f32x4 st[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    st[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + (int64_t)(rg + RG * i) * p.DV));
#pragma unroll
  for (int i = 0; i < (DK + NT - 1) / NT; ++i) {
    const int j = tid + i * NT;
    if (j < DK) {
      s_q[j] = qv[i];
      s_k[j] = kv[i];
    }
  }
  __syncthreads();
  f32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
    const float kr = s_k[r], qr = s_q[r];
    f32x4 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = fmaf(kr, vv[j], a * st[i][j]);
      acc[j] = fmaf(qr, x[j], acc[j]);
    }
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(S + (int64_t)r * p.DV));
  }
#pragma unroll
  for (int d = COLS4; d < 64; d <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d);
  const int wave = tid >> 6;
  if ((tid & 63) < COLS4) *reinterpret_cast<f32x4*>(&s_red[wave][4 * c4]) = acc;
  __syncthreads();
  for (int j = tid; j < DVS; j += NT) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) x += s_red[w][j];
    o[j] = x;
  }
}

template <int DK, int DVS>
static hipError_t launch_step_t(const DecayParams& p, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.nseq * p.H * (p.DV / DVS)));
  if (bf16)
    hipLaunchKernelGGL((decay_step_kernel<DK, DVS, __bf16>), grid, dim3(StepShape<DK, DVS>::NT), 0, s, p);
  else
    hipLaunchKernelGGL((decay_step_kernel<DK, DVS, float>), grid, dim3(StepShape<DK, DVS>::NT), 0, s, p);
  return hipGetLastError();
}
template <int DK>
static hipError_t launch_step_k(const DecayParams& p, int dvs, bool bf16, hipStream_t s) {
  if (dvs == 128) return launch_step_t<DK, 128>(p, bf16, s);
  if (dvs == 64) return launch_step_t<DK, 64>(p, bf16, s);
  if (dvs == 32) return launch_step_t<DK, 32>(p, bf16, s);
  return launch_step_t<DK, 16>(p, bf16, s);
}
hipError_t launch_decay_step(const DecayParams& p, bool bf16, hipStream_t s) {
  const int dvs = step_columns(p);
  if (p.DK == 128) return launch_step_k<128>(p, dvs, bf16, s);
  if (p.DK == 64) return launch_step_k<64>(p, dvs, bf16, s);
  if (p.DK == 32) return launch_step_k<32>(p, dvs, bf16, s);
  return launch_step_k<16>(p, dvs, bf16, s);
}

}  // namespace dr
