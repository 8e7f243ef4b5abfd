// 8-bit state cache on gfx950: fp32 states to codes with a scale for each key channel, and back.
//
// Both directions only move memory (5 bytes a value); a workgroup takes 16 KiB of one head's state, every
// thread 4 x 16 bytes of it, all loads issued before the first use. A row of d_v values lies in d_v / 4
// neighbouring lanes of one wave, so its largest magnitude is a butterfly over those lanes. 256 states of 32
// heads, d = 128, written in int8 and read back: 255 us, 5300 GB/s (a large copy on the card: 5175).
#include "state_cache.hpp"
#include "state_code.hpp"

namespace dr {

// Row of the state buffer and of the cache of item n; -1: outside.
__device__ __forceinline__ int64_t cache_row(const int32_t* idx, int64_t rows, int64_t n) {
  const int64_t r = idx ? (int64_t)idx[n] : n;
  return r >= 0 && r < rows ? r : -1;
}

template <int DV, bool E4M3>
__global__ __launch_bounds__(256) void state_pack_kernel(const CacheParams p) {
  constexpr int LPR = DV / 4;  // lanes per row
  const int hsz4 = p.DK * LPR;
  const int per = (hsz4 + CACHE_BLOCK - 1) / CACHE_BLOCK;
  const int64_t nh = blockIdx.x / per;
  const int part = (int)(blockIdx.x - nh * per);
  const int64_t n = nh / p.H;
  const int h = (int)(nh - n * p.H);
  const int64_t src = cache_row(p.state_idx, p.nstates, n), dst = cache_row(p.slot_idx, p.nslots, n);
  if (dst < 0) return;
  const f32x4* in = reinterpret_cast<const f32x4*>(p.S) + (src * p.H + h) * (int64_t)hsz4;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.codes) + (dst * p.H + h) * (int64_t)hsz4;
  float* sc = p.scales + (dst * p.H + h) * (int64_t)p.DK;
  f32x4 x[CACHE_VPT];
#pragma unroll
  for (int i = 0; i < CACHE_VPT; ++i) {
    const int e = part * CACHE_BLOCK + i * 256 + threadIdx.x;
    x[i] = f32x4{0, 0, 0, 0};
    if (src >= 0 && e < hsz4) x[i] = __builtin_nontemporal_load(in + e);
  }
#pragma unroll
  for (int i = 0; i < CACHE_VPT; ++i) {
    const int e = part * CACHE_BLOCK + i * 256 + threadIdx.x;
    // the largest magnitude as bits: NaN and infinity compare above every number
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = x[i][j];
      top = max(top, __builtin_bit_cast(uint32_t, y) & 0x7fffffffu);
    }
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const bool bad = top >= 0x7f800000u;
    float inv, scale = row_scale<E4M3>(top, &inv);
    const uint32_t code = bad ? 0u : codes4<E4M3>(x[i][0], x[i][1], x[i][2], x[i][3], scale, inv);
    if (bad) scale = __builtin_nanf("");
    if (e < hsz4) {
      __builtin_nontemporal_store(code, out + e);
      if (e % LPR == 0) sc[e / LPR] = scale;
    }
  }
}

template <int DV, bool E4M3>
__global__ __launch_bounds__(256) void state_unpack_kernel(const CacheParams p) {
  constexpr int LPR = DV / 4;
  const int hsz4 = p.DK * LPR;
  const int per = (hsz4 + CACHE_BLOCK - 1) / CACHE_BLOCK;
  const int64_t nh = blockIdx.x / per;
  const int part = (int)(blockIdx.x - nh * per);
  const int64_t n = nh / p.H;
  const int h = (int)(nh - n * p.H);
  const int64_t dst = cache_row(p.state_idx, p.nstates, n), src = cache_row(p.slot_idx, p.nslots, n);
  if (dst < 0) return;
  const uint32_t* in = reinterpret_cast<const uint32_t*>(p.codes) + (src * p.H + h) * (int64_t)hsz4;
  const float* sc = p.scales + (src * p.H + h) * (int64_t)p.DK;
  f32x4* out = reinterpret_cast<f32x4*>(p.S) + (dst * p.H + h) * (int64_t)hsz4;
  uint32_t w[CACHE_VPT];
  float s[CACHE_VPT];
#pragma unroll
  for (int i = 0; i < CACHE_VPT; ++i) {
    const int e = part * CACHE_BLOCK + i * 256 + threadIdx.x;
    w[i] = 0;
    s[i] = 0.f;
    if (src >= 0 && e < hsz4) {
      w[i] = __builtin_nontemporal_load(in + e);
      s[i] = sc[e / LPR];
    }
  }
#pragma unroll
  for (int i = 0; i < CACHE_VPT; ++i) {
    const int e = part * CACHE_BLOCK + i * 256 + threadIdx.x;
    f32x4 x;
    if constexpr (E4M3) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      x = f32x4{a[0], a[1], b[0], b[1]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = (float)(int8_t)(w[i] >> (8 * j));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= s[i];
    if (e < hsz4) __builtin_nontemporal_store(x, out + e);
  }
}

template <int DV>
static hipError_t launch_cache(const CacheParams& p, bool e4m3, bool pack, hipStream_t s) {
  const dim3 grid((unsigned)(p.count * p.H * cache_parts(p.DK * DV)));
  if (pack && e4m3)
    hipLaunchKernelGGL((state_pack_kernel<DV, true>), grid, dim3(256), 0, s, p);
  else if (pack)
    hipLaunchKernelGGL((state_pack_kernel<DV, false>), grid, dim3(256), 0, s, p);
  else if (e4m3)
    hipLaunchKernelGGL((state_unpack_kernel<DV, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((state_unpack_kernel<DV, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}
static hipError_t launch_cache_any(const CacheParams& p, bool e4m3, bool pack, hipStream_t s) {
  switch (p.DV) {
    case 16: return launch_cache<16>(p, e4m3, pack, s);
    case 32: return launch_cache<32>(p, e4m3, pack, s);
    case 64: return launch_cache<64>(p, e4m3, pack, s);
    default: return launch_cache<128>(p, e4m3, pack, s);
  }
}
hipError_t launch_state_pack(const CacheParams& p, bool e4m3, hipStream_t s) { return launch_cache_any(p, e4m3, true, s); }
hipError_t launch_state_unpack(const CacheParams& p, bool e4m3, hipStream_t s) { return launch_cache_any(p, e4m3, false, s); }

}  // namespace dr
