// Residual addition and root-mean-square norm on gfx950, with an output in the type of x or in 8 bits, and its
// gradients.
//
// A row stays in registers (32 elements a lane; one wave for up to 2048 channels, 4 or 16 above), so x and the residual are
// read once and every output is written once; the weights stay in registers over the rows of a workgroup. Above 8192 channels (few rows
// aside) 1024 threads leave each 128 registers, too few: 14 to 26 of them wait in scratch forward, 97 to 197 backward.
// 8 bits: p = h w does not contain the mean, so codes and the row's scale come from p exactly as the state cache's from
// a state, and the statistic only multiplies the scale.
//
// Bound by memory where there are rows enough: 16384 x 2048 bf16 with residual and codes 56 us (235 MB, 46 at the copy rate), backward 49 and 5 for the
// sums of dw (268 MB, 52); 1333 x 1531 fp32 with e4m3 codes 9.3 (27 MB, 5.2), one row 2.4. In a graph, bf16: values 16384 x 2048 54 (52), 4096 x 16384 102 (104), backward
// 4096 x 8192 62 (52), 4096 x 16384 416 (104: the registers above). Stores around the caches: between 10% less and
// 10% more time from 128 MiB on, without a rule, so they are ordinary.
#include <type_traits>

#include "scan.hpp"
#include "state_code.hpp"

namespace dr {

template <int WAVES>
struct NormShape {
  static constexpr int RPW = WAVES == 1 ? 4 : 1;  // rows of a workgroup at a time
  static constexpr int NT = 64 * WAVES * RPW;
  static constexpr int LANES = 64 * WAVES;        // of a row
};

// Sums of K values over the lanes of a row, the same in every lane and call.
template <int WAVES, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[K], int wave) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], d);
  if constexpr (WAVES > 1) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v[k] += red[w][k];
    }
  }
}
template <int WAVES>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, int wave) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v = max(v, red[w]);
    __syncthreads();
  }
  return v;
}

template <typename InT, int VEC, int WAVES, int ELEMS, int OUT>
__global__ __launch_bounds__(NormShape<WAVES>::NT) void norm_fwd_kernel(const NormParams p) {
  using Sh = NormShape<WAVES>;
  using V = typename Vec<InT, VEC>::type;
  constexpr int NV = ELEMS / VEC, LANES = Sh::LANES;
  __shared__ float s_sum[WAVES][1];
  __shared__ uint32_t s_max[WAVES];
  const int lane = threadIdx.x % LANES, wave = (threadIdx.x % LANES) >> 6, C = p.C;
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * LANES + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = 0.f;
    if (e < C) unpack<VEC, float>(*reinterpret_cast<const typename Vec<float, VEC>::type*>(p.w + e), w[i]);
  }
  const float mean = 1.f / (float)C;
  // (rows of a workgroup with several waves a row are uniform over it: its barriers meet)
  for (int64_t row = (int64_t)blockIdx.x * Sh::RPW + threadIdx.x / LANES; row < p.rows; row += (int64_t)gridDim.x * Sh::RPW) {
    const InT* x = static_cast<const InT*>(p.x) + row * p.x_rs;
    const InT* r = p.r ? static_cast<const InT*>(p.r) + row * p.r_rs : nullptr;
    V xv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * LANES + lane) * VEC;
      xv[i] = V{};
      rv[i] = V{};
      if (e < C) {
        xv[i] = *reinterpret_cast<const V*>(x + e);
        if (r) rv[i] = *reinterpret_cast<const V*>(r + e);
      }
    }
    float h[NV][VEC], sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<VEC, InT>(xv[i], h[i]);
      if (r) {
        float a[VEC];
        unpack<VEC, InT>(rv[i], a);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i][j] += a[j];
        // the sum is used as it is handed on: rounded to the type of x
        const V out = pack<VEC, InT>(h[i]);
        unpack<VEC, InT>(out, h[i]);
        const int e = (i * LANES + lane) * VEC;
        if (p.h && e < C) *reinterpret_cast<V*>(static_cast<InT*>(p.h) + row * (int64_t)C + e) = out;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[0] = fmaf(h[i][j], h[i][j], sum[0]);
    }
    row_sum<WAVES, 1>(sum, s_sum, wave);
    const float rs = rsqrtf(fmaf(sum[0], mean, p.eps));
    if constexpr (OUT == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * LANES + lane) * VEC;
        float y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[j] = h[i][j] * w[i][j] * rs;
        if (e < C) *reinterpret_cast<V*>(static_cast<InT*>(p.y) + row * (int64_t)C + e) = pack<VEC, InT>(y);
      }
    } else {
      constexpr bool E4M3 = OUT == 2;
      uint32_t top = 0;  // the largest magnitude as bits: NaN and infinity compare above every number
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[i][j] *= w[i][j];
          top = max(top, __builtin_bit_cast(uint32_t, h[i][j]) & 0x7fffffffu);
        }
      top = row_max<WAVES>(top, s_max, wave);
      const bool bad = top >= 0x7f800000u;
      float inv;
      const float scale = row_scale<E4M3>(top, &inv);
      uint8_t* y = static_cast<uint8_t*>(p.y) + row * (int64_t)C;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * LANES + lane) * VEC;
        if (e >= C) continue;
        if constexpr (VEC == 1) {
          y[e] = bad ? 0 : (uint8_t)codes4<E4M3>(h[i][0], 0.f, 0.f, 0.f, scale, inv);
        } else {
          uint32_t c[VEC / 4];
#pragma unroll
          for (int j = 0; j < VEC / 4; ++j)
            c[j] = bad ? 0u : codes4<E4M3>(h[i][4 * j], h[i][4 * j + 1], h[i][4 * j + 2], h[i][4 * j + 3], scale, inv);
          if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(y + e) = make_uint2(c[0], c[1]);
          else
            *reinterpret_cast<uint32_t*>(y + e) = c[0];
        }
      }
      if (lane == 0) p.scales[row] = bad ? __builtin_nanf("") : scale * rs;
    }
  }
}

// dx = dh + r (w dy - h r^2 mean(w dy h)); each workgroup's sum of dy h r over its rows for dw.
template <typename InT, int VEC, int WAVES, int ELEMS>
__global__ __launch_bounds__(NormShape<WAVES>::NT) void norm_bwd_kernel(const NormParams p) {
  using Sh = NormShape<WAVES>;
  using V = typename Vec<InT, VEC>::type;
  constexpr int NV = ELEMS / VEC, LANES = Sh::LANES;
  __shared__ float s_sum[WAVES][2];
  __shared__ float s_dw[WAVES == 1 ? 3 : 1][WAVES == 1 ? 64 * ELEMS : 1];
  const int lane = threadIdx.x % LANES, wave = (threadIdx.x % LANES) >> 6, C = p.C;
  float w[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * LANES + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = dw[i][j] = 0.f;
    if (e < C) unpack<VEC, float>(*reinterpret_cast<const typename Vec<float, VEC>::type*>(p.w + e), w[i]);
  }
  const float mean = 1.f / (float)C;
  for (int64_t row = (int64_t)blockIdx.x * Sh::RPW + threadIdx.x / LANES; row < p.rows; row += (int64_t)gridDim.x * Sh::RPW) {
    const InT* h = static_cast<const InT*>(p.x) + row * p.x_rs;
    const InT* dy = static_cast<const InT*>(p.dy) + row * (int64_t)C;
    V hv[NV], yv[NV], dv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * LANES + lane) * VEC;
      hv[i] = yv[i] = dv[i] = V{};
      if (e < C) {
        hv[i] = *reinterpret_cast<const V*>(h + e);
        yv[i] = *reinterpret_cast<const V*>(dy + e);
        if (p.dh) dv[i] = *reinterpret_cast<const V*>(static_cast<const InT*>(p.dh) + row * (int64_t)C + e);
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[VEC], b[VEC];
      unpack<VEC, InT>(hv[i], a);
      unpack<VEC, InT>(yv[i], b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        sum[0] = fmaf(a[j], a[j], sum[0]);
        sum[1] = fmaf(a[j] * w[i][j], b[j], sum[1]);
      }
    }
    row_sum<WAVES, 2>(sum, s_sum, wave);
    const float rs = rsqrtf(fmaf(sum[0], mean, p.eps)), k = rs * rs * (sum[1] * mean);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * LANES + lane) * VEC;
      float a[VEC], b[VEC], d[VEC];
      unpack<VEC, InT>(hv[i], a);
      unpack<VEC, InT>(yv[i], b);
      unpack<VEC, InT>(dv[i], d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        d[j] = fmaf(rs, fmaf(-a[j], k, w[i][j] * b[j]), d[j]);
        dw[i][j] = fmaf(b[j], a[j] * rs, dw[i][j]);
      }
      if (e < C) *reinterpret_cast<V*>(static_cast<InT*>(p.dx) + row * (int64_t)C + e) = pack<VEC, InT>(d);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * C;
  if constexpr (WAVES == 1) {  // the four rows' sums of a workgroup
    const int g = threadIdx.x >> 6;
    if (g > 0)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s_dw[g - 1][(i * VEC + j) * 64 + lane] = dw[i][j];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int k = 0; k < 3; ++k) dw[i][j] += s_dw[k][(i * VEC + j) * 64 + lane];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * LANES + lane) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (e < C) part[e + j] = dw[i][j];
  }
}

// out[c] = sum over the rows of part [rows, C]: 16 channels x 64 row groups a workgroup.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const NormParams p) {
  __shared__ float s[64][16];
  const int i = threadIdx.x & 15, c = blockIdx.x * 16 + i, g = threadIdx.x >> 4;
  float v = 0.f;
  if (c < p.C)
    for (int r = g; r < p.nwg; r += 64) v += p.part[(int64_t)r * p.C + c];
  s[g][i] = v;
  __syncthreads();
  if (g == 0 && c < p.C) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 64; ++k) a += s[k][i];
    p.dw[c] = a;
  }
}

// f(waves of a row, elements of a lane), as constants
template <typename F>
static void with_shape(const NormParams& p, F&& f) {
  using std::integral_constant;
  if (p.few)
    norm_waves(p.C, p.few) == 4 ? f(integral_constant<int, 4>{}, integral_constant<int, NORM_FEW>{})
                                 : f(integral_constant<int, 16>{}, integral_constant<int, NORM_FEW>{});
  else if (norm_waves(p.C, p.few) == 1)
    f(integral_constant<int, 1>{}, integral_constant<int, NORM_ELEMS>{});
  else if (norm_waves(p.C, p.few) == 4)
    f(integral_constant<int, 4>{}, integral_constant<int, NORM_ELEMS>{});
  else
    f(integral_constant<int, 16>{}, integral_constant<int, NORM_ELEMS>{});
}
template <typename InT, int VEC>
static void launch_fwd_v(const NormParams& p, int out, hipStream_t s) {
  with_shape(p, [&](auto waves, auto elems) {
    constexpr int W = decltype(waves)::value, E = decltype(elems)::value;
    const dim3 grid((unsigned)p.nwg), block(NormShape<W>::NT);
    if (out == 0)
      hipLaunchKernelGGL((norm_fwd_kernel<InT, VEC, W, E, 0>), grid, block, 0, s, p);
    else if (out == 1)
      hipLaunchKernelGGL((norm_fwd_kernel<InT, VEC, W, E, 1>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((norm_fwd_kernel<InT, VEC, W, E, 2>), grid, block, 0, s, p);
  });
}
hipError_t launch_norm_fwd(const NormParams& p, int out, bool bf16, bool vec, hipStream_t s) {
  if (bf16)
    vec ? launch_fwd_v<__bf16, 8>(p, out, s) : launch_fwd_v<__bf16, 1>(p, out, s);
  else
    vec ? launch_fwd_v<float, 4>(p, out, s) : launch_fwd_v<float, 1>(p, out, s);
  return hipGetLastError();
}

template <typename InT, int VEC>
static void launch_bwd_v(const NormParams& p, hipStream_t s) {
  with_shape(p, [&](auto waves, auto elems) {
    constexpr int W = decltype(waves)::value, E = decltype(elems)::value;
    hipLaunchKernelGGL((norm_bwd_kernel<InT, VEC, W, E>), dim3((unsigned)p.nwg), dim3(NormShape<W>::NT), 0, s, p);
  });
}
hipError_t launch_norm_bwd(const NormParams& p, bool bf16, bool vec, hipStream_t s) {
  if (p.nwg > 0) {
    if (bf16)
      vec ? launch_bwd_v<__bf16, 8>(p, s) : launch_bwd_v<__bf16, 1>(p, s);
    else
      vec ? launch_bwd_v<float, 4>(p, s) : launch_bwd_v<float, 1>(p, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((p.C + 15) / 16)), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace dr
