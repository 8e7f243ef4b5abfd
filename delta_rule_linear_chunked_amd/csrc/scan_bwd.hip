// Gradients of the selective scan on gfx950.
//
// With G_t the gradient that reaches h_t (from y_t, from h_{t+1} and from the final state) and a_t = exp(d_t A):
//   G_t = dy'_t C_t + a_{t+1} G_{t+1},  dy' = dy silu(z)
//   dB_t = sum_c G_t d_t x_t,  dC_t = sum_c dy'_t h_t,  u = sum_n G_t B_t,  e = sum_n G_t a_t h_{t-1} A
//   dx = u d + D dy',  d(d) = u x + e,  dA = sum_t d_t G_t a_t h_{t-1},  dz = dy (C h + D x) silu'(z)
// Three steps. scan_states_kernel walks every segment once (a lane has a channel, as in the forward pass) and leaves its
// state from zero at every 8th token, behind it, and the gradient that its outputs send to the state in front of it.
// scan_join2_kernel joins segments in both directions. scan_grad_kernel takes a segment's chunks of 8 tokens from the last to the first: states and
// decays of the chunk again from its checkpoint, held in registers (8 tokens x 4 channels x 2 states a lane), then
// the tokens in reverse. A lane's square of channels and states shares the two kinds of sums between lanes evenly: over states (dx,
// dd, y) across the lanes' rows, over channels (dB, dC) within eight lanes.
//
// 2 x 4096 x 2048, 16 states, bf16: 341 us, of them states 104, join 10, gradients 240 (the vector units issue 84% of the time, about
// 1480 instructions for a chunk of 32 channels x 16 states: 830 of the formulas, 250 sums across lanes, 400 inputs, outputs and
// addresses), dB and dC 9, dA and the rest 5. With a gate 9 to 11 registers wait in scratch over the loop of chunks; none are reloaded in it. Checkpoints are
// 134 MB, written and read (one for every 4th token would double that; not tried).
#include "scan_tile.hpp"

namespace dr {

// Local states at every 8th token and behind the segment, the sums of d there, and (BOTH) the reverse part: tiles as in the
// forward pass, dy C by the matrix units as d x B is. (A product that is not finite may reach the other token of its pair: both lie between the same
// checkpoints. In fp32 three waves a SIMD, 168 registers.)
template <int SL, typename InT, bool BOTH>
__global__ __launch_bounds__(64 * SL, BOTH && sizeof(InT) == 4 ? 3 : 1) void scan_states_kernel(const ScanParams p) {
  constexpr int N = 16 * SL, K = TILE_TOK, O = TILE_OWN;
  static_assert(K == 2 * SCAN_CHUNK, "two checkpoints to a tile");
  const int lane = threadIdx.x & 63, sl = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int ntiles = p.G * p.tiles;
  const int slot = blockIdx.x / ntiles, tile = blockIdx.x - slot * ntiles;
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int g = tile / p.tiles, in_g = (tile - g * p.tiles) * SCAN_TILE + (lane & 31);
  const bool on = in_g < p.Cg;
  const int c = g * p.Cg + min(in_g, p.Cg - 1), n0 = sl * 16 + 4 * half;
  float A[8], h[8], P[8], R[8];
  load_states(p.A + (int64_t)c * N + n0, A);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    A[j] *= LOG2E;
    h[j] = R[j] = 0.f;
    P[j] = 1.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f;
  const int len = sp.len;
  const float least = step_least(p.softplus != 0);
  const bool gate = BOTH && p.z != nullptr;
  Rows<InT> X, T, Z, B, Y, Cr;
  X.init(p.x, sp.b * p.x_bs + sp.t0 * p.x_ts, p.x_ts, half, c);
  T.init(p.dt, sp.b * p.dt_bs + sp.t0 * p.dt_ts, p.dt_ts, half, c);
  B.init(p.B, sp.b * p.b_bs + sp.t0 * p.b_ts, p.b_ts, half, g * N + sl * 16 + (lane & 15));
  if constexpr (BOTH) {
    if (gate)
      Z.init(p.z, sp.b * p.z_bs + sp.t0 * p.z_ts, p.z_ts, half, c);
    else
      Z = X;
    Cr.init(p.Cm, sp.b * p.c_bs + sp.t0 * p.c_ts, p.c_ts, half, g * N + sl * 16 + (lane & 15));
    Y.init(p.dy, (sp.b * p.T + sp.t0) * (int64_t)p.C, p.C, half, c);
  }
  const int64_t chunk0 = slot_chunk(p, slot, sp);
  float* ck = p.ck + (chunk0 * p.C + c) * N + n0;
  float* ckd = p.ckd + chunk0 * p.C + c;
  float sumd = 0.f;
  uint32_t xn[O], dn[O], zn[O], yn[O], bn[O], cn[O];
  auto fetch = [&](int step) {  // (as in the forward pass)
    X.at += step * X.ts;
    T.at += step * T.ts;
    B.at += step * B.ts;
    X.whole(xn);
    T.whole(dn);
    B.whole(bn);
    if constexpr (BOTH) {
      Z.at += step * Z.ts;
      Y.at += step * Y.ts;
      Cr.at += step * Cr.ts;
      Z.whole(zn);
      Y.whole(yn);
      Cr.whole(cn);
    }
  };
  auto tokens = [&](int t, auto cut) {
    constexpr bool CUT = decltype(cut)::value;
    float dv[O], dx[O], gy[O], bo[O], co[O];
#pragma unroll
    for (int i = 0; i < O; ++i) {
      float own = step_f(raw_value<InT>(dn[i]) + bias, least);
      here(own);
      // (tokens past the end: a decay of one, nothing in or out)
      const bool inside = !CUT || t + 2 * i + half < len;
      dv[i] = inside ? own : 0.f;
      dx[i] = inside ? dv[i] * raw_value<InT>(xn[i]) : 0.f;
      bo[i] = inside ? operand<InT>(bn[i], lane) : 0.f;
      if constexpr (BOTH) {
        const float zv = raw_value<InT>(zn[i]), sg = zv * sigmoid_f(zv);
        float out = raw_value<InT>(yn[i]) * (gate ? sg : 1.f);
        here(out);
        gy[i] = inside ? out : 0.f;
        co[i] = inside ? operand<InT>(cn[i], lane) : 0.f;
      }
    }
    if constexpr (!CUT) fetch(t + 2 * K <= len ? K : 0);
    f32x16 in = outer_pair(bo[0], dx[0]), out = BOTH ? outer_pair(co[0], gy[0]) : f32x16{};
#pragma unroll
    for (int i = 0; i < O; ++i) {
      tile_step();
      if (i % (O / 2) == 0 && (i == 0 || !CUT || t + SCAN_CHUNK < len)) {
        // (lanes and waves that share a channel write the same; stores under a condition would be waited for with the next tile's inputs)
        store_states(ck, h);
        float lo, hi;
        both_halves(sumd, lo, hi);
        *ckd = lo + hi;
        ck += (int64_t)p.C * N;
        ckd += p.C;
      }
      float d[2];
      both_halves(dv[i], d[0], d[1]);
      sumd += dv[i];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = __builtin_amdgcn_exp2f(d[k] * A[j]);
          h[j] = fmaf(a, h[j], in[8 * k + j]);
          if constexpr (BOTH) {
            P[j] *= a;
            R[j] = fmaf(P[j], out[8 * k + j], R[j]);
          }
        }
      if (i + 1 < O) {
        in = outer_pair(bo[i + 1], dx[i + 1]);
        if constexpr (BOTH) out = outer_pair(co[i + 1], gy[i + 1]);
      }
      if constexpr (BOTH) here(R);
    }
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
    if constexpr (BOTH) {
      Z.at += step * Z.ts;
      Y.at += step * Y.ts;
      Cr.at += step * Cr.ts;
      Z.part(zn, left);
      Y.part(yn, left);
      Cr.part(cn, left);
    }
    tokens(whole, std::true_type{});
  }
  if constexpr (BOTH) {
    float lo, hi;
    both_halves(sumd, lo, hi);
    if (!on || sp.whole()) return;
    const int64_t at = ((int64_t)slot * p.C + c) * N + n0;
    store_states(p.part + at, h);
    store_states(p.rpart + at, R);
    if (sl == 0 && half == 0) p.sumd[(int64_t)slot * p.C + c] = lo + hi;
  }
}

// Segments joined: forward (blockIdx.y 0) the state at each one's start in the place of its own, in reverse (1) the gradient that reaches
// the state behind each one in the place of what it sends forward.
template <int N>
__global__ __launch_bounds__(256) void scan_join2_kernel(const ScanParams p) {
  const int per = (p.C * (N / 4) + 255) / 256;
  const int n = blockIdx.x / per, e = (blockIdx.x - n * per) * 256 + threadIdx.x;
  if (e >= p.C * (N / 4)) return;
  const int c = e / (N / 4), j = e - c * (N / 4);
  const int first = p.cu ? p.slot_first[n] : n * p.nseg, past = p.cu ? p.slot_first[n + 1] : first + p.nseg;
  if (past - first == 1) return;  // (a sequence that is not cut has S0 and dS_T themselves)
  const bool back = blockIdx.y == 1;
  f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * N + 4 * j), v = {0, 0, 0, 0};
  const float* from = back ? p.dST : p.S0;
  float* part = back ? p.rpart : p.part;
  if (from) v = *reinterpret_cast<const f32x4*>(from + ((int64_t)n * p.C + c) * N + 4 * j);
  for (int k = first; k < past; ++k) {
    const int64_t s = back ? past - 1 - (k - first) : k;
    f32x4* at = reinterpret_cast<f32x4*>(part + (s * p.C + c) * N + 4 * j);
    const f32x4 own = *at;
    const float d = p.sumd[s * p.C + c] * LOG2E;
    *at = v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(__builtin_amdgcn_exp2f(d * A[i]), v[i], own[i]);
  }
}

// ---------------------------------------------------------------------------
// Sums across lanes
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// over 8 neighbouring lanes, in all of them: swapped in pairs, in quads' halves, mirrored in eight
__device__ __forceinline__ float sum8(float v) { return dpp_add<0x141>(dpp_add<0x4e>(dpp_add<0xb1>(v))); }
// a of lanes l and l ^ 32 (l ^ 16) in the lower lanes of the pair, b's sum in the upper ones
__device__ __forceinline__ float pair32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float pair16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// A workgroup: 4 waves, each 32 channels x 16 states, one segment. With 16 states nothing but the sums of dB and dC passes between
// waves, and they meet once for every two chunks; with more, SL waves share their channels' inputs and add their parts of
// the sums over states.
template <int N>
struct GradShape {
  static constexpr int SL = N / 16;                      // slices of states
  static constexpr int CB = 4 / SL;                      // channel blocks
  static constexpr int CH = 32 * CB;                     // channels
  static constexpr int ROWS = 2 * SL;                    // token rows of a chunk that the lanes of a channel cover at once
  static constexpr int PP = SCAN_CHUNK / ROWS;           // (token, channel) pairs of a lane
  static constexpr int F = 2;                            // chunks between two meetings of the workgroup
};
// What lanes of a channel block wrote to LDS is seen by its other lanes (one wave's LDS accesses are in order).
template <int SL>
__device__ __forceinline__ void block_sync() {
  if constexpr (SL == 1) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}
template <int N, typename InT, bool GATE>
__global__ __launch_bounds__(256, 2) void scan_grad_kernel(const ScanParams p) {
  using Sh = GradShape<N>;
  constexpr int K = SCAN_CHUNK, CH = Sh::CH, SL = Sh::SL, CB = Sh::CB, PP = Sh::PP, ROWS = Sh::ROWS, F = Sh::F;
  __shared__ __align__(16) float s_d[K][CH], s_dx[K][CH], s_dy[K][CH];
  __shared__ __align__(16) float s_in[4][K][32];  // a wave's 16 states of B and of C
  __shared__ float s_u[SL][K][CH], s_e[SL][K][CH], s_y[GATE ? SL : 1][GATE ? K : 1][GATE ? CH : 1];
  __shared__ __align__(16) float s_bc[2][F][4][K][32];
  // what a lane needs of its pairs again at the end of a chunk, and its starting state, wait here instead of in registers
  __shared__ __align__(16) float s_own[GATE ? 3 : 2][PP][256], s_hs[2][256][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sl = wave % SL, cb = wave / SL;
  const int per = p.G * p.cblocks;
  const int slot = blockIdx.x / per, blk = blockIdx.x - slot * per;
  const int g = blk / p.cblocks, in0 = (blk - g * p.cblocks) * CH;  // the group, the first channel within it
  const SlotSpan sp = slot_span(p, slot);
  if (sp.n < 0) return;
  const int len = sp.len, C = p.C;
  // as the lane of states and gradients: 4 channels, 2 states
  const int ng = lane >> 3, cg = lane & 7;
  const int l_ch = cb * 32 + cg * 4, n0 = sl * 16 + ng * 2;
  // channel i of lane l (those past the group's count as its last)
  auto chan = [&](uint32_t l, int i) { return g * p.Cg + min(in0 + cb * 32 + (int)(l & 7) * 4 + i, p.Cg - 1); };
  float A[4][2], carry[4][2], dA[4][2];
  const bool cut = p.part && !sp.whole();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t at = (int64_t)chan(lane, i) * N + n0 + j;
      A[i][j] = p.A[at] * LOG2E;
      dA[i][j] = 0.f;
      const float* from = cut ? p.part + (int64_t)slot * C * N : p.S0 ? p.S0 + (int64_t)sp.n * C * N : nullptr;
      s_hs[j][tid][i] = from ? from[at] : 0.f;
      const float* back = cut ? p.rpart + (int64_t)slot * C * N : p.dST ? p.dST + (int64_t)sp.n * C * N : nullptr;
      carry[i][j] = back ? back[at] : 0.f;
    }
  // as the lane of (token, channel) pairs: one channel, PP tokens of a chunk
  const int pc = cb * 32 + (lane & 31), prow = (lane >> 5) + 2 * sl;
  const bool on = in0 + pc < p.Cg;
  // Addresses: a uniform pointer for the chunk, moved back by a chunk after each, and 32-bit offsets of the lane that stay
  // (token strides are limited to 2^24 elements, groups to 2^16).
  const int last = len > 0 ? (len - 1) / K * K : 0;
  const int64_t row0 = sp.b * p.T + sp.t0, x_ts = p.x_ts, dt_ts = p.dt_ts, z_ts = p.z_ts;
  const InT* xb = static_cast<const InT*>(p.x) + sp.b * p.x_bs + (sp.t0 + last + 2 * sl) * x_ts;
  const InT* db = static_cast<const InT*>(p.dt) + sp.b * p.dt_bs + (sp.t0 + last + 2 * sl) * dt_ts;
  const InT* zb = GATE ? static_cast<const InT*>(p.z) + sp.b * p.z_bs + (sp.t0 + last + 2 * sl) * z_ts : nullptr;
  int64_t row = row0 + last + 2 * sl, next = row;  // of the outputs, of dy
  constexpr uint32_t E = sizeof(InT);
  // bytes to the channel of lane l's pairs, and one row on in the upper lanes
  auto pair_at = [&](uint32_t l, int64_t ts) { return (uint32_t)(g * p.Cg + min(in0 + cb * 32 + (int)(l & 31), p.Cg - 1)) * E + (l & 32 ? (uint32_t)ts * E : 0u); };
  const float bias = p.bias ? p.bias[pair_at(lane, 0) / E] : 0.f, D = p.D ? p.D[pair_at(lane, 0) / E] : 0.f;
  int64_t chunk = slot_chunk(p, slot, sp) + last / K;
  // B and C: lane l brings states 2 (l % 8), + 1 of token l / 8
  typedef uint32_t Raw2 __attribute__((ext_vector_type(2 * sizeof(InT) / 4)));
  const InT* Bb = static_cast<const InT*>(p.B) + sp.b * p.b_bs + (sp.t0 + last) * p.b_ts + g * N + sl * 16;
  const InT* Cb = static_cast<const InT*>(p.Cm) + sp.b * p.c_bs + (sp.t0 + last) * p.c_ts + g * N + sl * 16;
  const float least = step_least(p.softplus != 0);
  const bool soft = p.softplus != 0, full = in0 + CH <= p.Cg;
  float accD = 0.f, accb = 0.f;
  uint32_t xn[PP], dn[PP], zn[PP], yn[PP];
  f32x2 hn[4];
  float dsum[4];
  Raw2 bn, cn;
  // (first: the segment's last chunk, whose rows past the end are read from the last one and not used; those of B and C are zeros)
  auto fetch = [&](int t, auto first) {
    const InT *xr = xb, *dr = db, *zr = zb, *yr = static_cast<const InT*>(p.dy) + next * C;
    const uint32_t l = fresh(lane), brow = l >> 3;
    const uint32_t bo = (brow * (uint32_t)p.b_ts + 2 * (l & 7)) * E, co = (brow * (uint32_t)p.c_ts + 2 * (l & 7)) * E;
    if (!decltype(first)::value || t + K <= len) {
      const uint32_t xo = pair_at(l, x_ts), dto = pair_at(l, dt_ts), zo = GATE ? pair_at(l, z_ts) : 0u, oo = pair_at(l, C);
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        xn[i] = raw_bits(byte_at(xr, xo));
        dn[i] = raw_bits(byte_at(dr, dto));
        if constexpr (GATE) zn[i] = raw_bits(byte_at(zr, zo));
        yn[i] = raw_bits(byte_at(yr, oo));
        xr += ROWS * x_ts;
        dr += ROWS * dt_ts;
        if constexpr (GATE) zr += ROWS * z_ts;
        yr += ROWS * (int64_t)C;
      }
      bn = *reinterpret_cast<const Raw2*>(byte_at(Bb, bo));
      cn = *reinterpret_cast<const Raw2*>(byte_at(Cb, co));
      whole_tile();
    } else {
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        const int64_t r = min((int)(l >> 5) + 2 * sl + i * ROWS, len - 1 - t) - 2 * sl;
        const int c = (int)(pair_at(l, 0) / E);
        xn[i] = raw_bits(xr + (r * x_ts + c));
        dn[i] = raw_bits(dr + (r * dt_ts + c));
        if constexpr (GATE) zn[i] = raw_bits(zr + (r * z_ts + c));
        yn[i] = raw_bits(yr + (r * C + c));
      }
#pragma unroll
      for (int i = 0; i < (int)(sizeof(Raw2) / 4); ++i) bn[i] = cn[i] = 0;
      if (t + (int)brow < len) {
        bn = *reinterpret_cast<const Raw2*>(byte_at(Bb, bo));
        cn = *reinterpret_cast<const Raw2*>(byte_at(Cb, co));
      }
    }
    xb -= K * x_ts;
    db -= K * dt_ts;
    if constexpr (GATE) zb -= K * z_ts;
    next -= K;
    Bb -= K * p.b_ts;
    Cb -= K * p.c_ts;
    const float *ck = p.ck + chunk * C * N, *ckd = p.ckd + chunk * C;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (a segment's first chunk has none: not used there)
      const uint32_t ch = (uint32_t)chan(l, i) * 4;
      dsum[i] = *byte_at(ckd, ch);
      hn[i] = *reinterpret_cast<const f32x2*>(byte_at(ck, ch * N + (sl * 16 + (l >> 3) * 2) * 4));
    }
    --chunk;
  };
  // this workgroup's part of dB and dC: 2 N values to a token
  float* pbc = p.pBC + (((int64_t)(blk - g * p.cblocks) * p.nbatch * p.T + row0) * p.G + g) * (2 * N);
  if (len > 0) fetch(last, std::true_type{});
  arrived();
  int met = 0;  // chunks since the last meeting, and which half of s_bc they use
  int part = 0;
  for (int t = last; len > 0 && t >= 0; t -= K) {
    block_sync<SL>();  // (the chunk before has been written out)
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int r = prow + i * ROWS;
      const bool inside = on && t + r < len;
      const float xv = raw_value<InT>(xn[i]), raw = raw_value<InT>(dn[i]) + bias, sr = sigmoid_f(raw);
      float dv = step_f(raw, least), gv = raw_value<InT>(yn[i]);
      s_own[0][i][tid] = xv;
      s_own[1][i][tid] = soft ? sr : 1.f;
      if constexpr (GATE) {
        const float zv = raw_value<InT>(zn[i]);
        const float sz = sigmoid_f(zv);
        s_own[2][i][tid] = gv * (sz * fmaf(zv, 1.f - sz, 1.f));  // dy silu'(z)
        gv *= zv * sz;
      }
      here(dv);
      here(gv);
      // tokens past the end and channels past the group's: a decay of one, nothing in or out
      s_d[r][pc] = inside ? dv : 0.f;
      s_dx[r][pc] = inside ? dv * xv : 0.f;
      s_dy[r][pc] = inside ? gv : 0.f;
    }
    {
      f32x2 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if constexpr (sizeof(InT) == 4) {
          v[0][i] = __builtin_bit_cast(float, (uint32_t)bn[i]);
          v[1][i] = __builtin_bit_cast(float, (uint32_t)cn[i]);
        } else {
          v[0][i] = __builtin_bit_cast(float, i ? (uint32_t)bn[0] & 0xffff0000u : (uint32_t)bn[0] << 16);
          v[1][i] = __builtin_bit_cast(float, i ? (uint32_t)cn[0] & 0xffff0000u : (uint32_t)cn[0] << 16);
        }
      *reinterpret_cast<f32x2*>(&s_in[wave][ng][2 * cg]) = v[0];
      *reinterpret_cast<f32x2*>(&s_in[wave][ng][16 + 2 * cg]) = v[1];
    }
    // the state in front of the chunk
    float a[K][4][2], h[K + 1][4][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4 hs = *reinterpret_cast<const f32x4*>(&s_hs[j][tid][0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[0][i][j] = t > 0 ? fmaf(__builtin_amdgcn_exp2f(dsum[i] * A[i][j]), hs[i], hn[i][j]) : hs[i];
    }
    block_sync<SL>();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k % 2 == 0) tile_step();
      const f32x4 d = *reinterpret_cast<const f32x4*>(&s_d[k][l_ch]), dx = *reinterpret_cast<const f32x4*>(&s_dx[k][l_ch]);
      const f32x2 b = *reinterpret_cast<const f32x2*>(&s_in[wave][k][ng * 2]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[k][i][j] = __builtin_amdgcn_exp2f(d[i] * A[i][j]);
          h[k + 1][i][j] = fmaf(a[k][i][j], h[k][i][j], dx[i] * b[j]);
        }
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      // the next chunk's loads start where half of this one's states and decays are no longer held
      if (k == K / 2 - 1 && t > 0) fetch(t - K, std::false_type{});
      tile_step();
      const f32x4 d = *reinterpret_cast<const f32x4*>(&s_d[k][l_ch]), dx = *reinterpret_cast<const f32x4*>(&s_dx[k][l_ch]);
      const f32x4 gy = *reinterpret_cast<const f32x4*>(&s_dy[k][l_ch]);
      const f32x2 b = *reinterpret_cast<const f32x2*>(&s_in[wave][k][ng * 2]), cc = *reinterpret_cast<const f32x2*>(&s_in[wave][k][16 + ng * 2]);
      float u[4], e[4], yo[4], vb[2] = {0.f, 0.f}, vc[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = e[i] = yo[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          vc[j] = fmaf(gy[i], h[k + 1][i][j], vc[j]);
          if constexpr (GATE) yo[i] = fmaf(cc[j], h[k + 1][i][j], yo[i]);
          const float G = fmaf(gy[i], cc[j], carry[i][j]);
          vb[j] = fmaf(G, dx[i], vb[j]);
          u[i] = fmaf(G, b[j], u[i]);
          const float aG = a[k][i][j] * G;
          const float w = aG * h[k][i][j];
          e[i] = fmaf(w, A[i][j], e[i]);
          dA[i][j] = fmaf(w, d[i], dA[i][j]);
          carry[i][j] = aG;
        }
      }
      // sums over states: the lower 32 lanes end with u, the upper with e; of four channels, even rows of 16 lanes have
      // 0 and 1, odd rows 2 and 3; the last step is the same in both halves of a row, each of which writes one channel
      {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair32(u[i], e[i]);
        const float r0 = dpp_add<0x128>(pair16(v[0], v[2])), r1 = dpp_add<0x128>(pair16(v[1], v[3]));
        const int ch = l_ch + 2 * ((lane >> 4) & 1) + ((lane >> 3) & 1);
        float* to = lane < 32 ? &s_u[sl][k][ch] : &s_e[sl][k][ch];
        *to = lane & 8 ? r1 : r0;
      }
      if constexpr (GATE) {  // (one channel a row of 16 lanes: 0, 1, 2, 3)
        float v = dpp_add<0x128>(pair16(pair32(yo[0], yo[2]), pair32(yo[1], yo[3])));
        here(v);  // (in the branch below a sum across lanes is two instructions)
        if (!(lane & 8)) s_y[sl][k][l_ch + 2 * (lane >> 5) + ((lane >> 4) & 1)] = v;
      }
      // sums over channels
      float b0 = sum8(vb[0]), b1 = sum8(vb[1]), c0 = sum8(vc[0]), c1 = sum8(vc[1]);
      here(b0);
      here(b1);
      here(c0);
      here(c1);
      if (cg == 0) *reinterpret_cast<f32x4*>(&s_bc[part][met][wave][k][ng * 4]) = f32x4{b0, b1, c0, c1};
    }
    block_sync<SL>();
    auto outputs = [&](int i) {
      const int r = prow + i * ROWS;
      const uint32_t oo = pair_at(fresh(lane), C);
      float u = 0.f, e = 0.f, yo = 0.f;
#pragma unroll
      for (int s = 0; s < SL; ++s) {
        u += s_u[s][r][pc];
        e += s_e[s][r][pc];
        if constexpr (GATE) yo += s_y[s][r][pc];
      }
      const float xv = s_own[0][i][tid], gv = s_dy[r][pc];
      const float draw = fmaf(u, xv, e * LN2) * s_own[1][i][tid];
      const int64_t base = (row + i * ROWS) * C;
      *byte_at(static_cast<InT*>(p.ddt) + base, oo) = (InT)draw;
      *byte_at(static_cast<InT*>(p.dx) + base, oo) = (InT)fmaf(u, s_d[r][pc], D * gv);
      if constexpr (GATE) {
        *byte_at(static_cast<InT*>(p.dz) + base, oo) = (InT)(s_own[2][i][tid] * fmaf(D, xv, yo));
      }
      accD = fmaf(gv, xv, accD);
      accb += draw;
    };
    if (full && t + K <= len) {
#pragma unroll
      for (int i = 0; i < PP; ++i) outputs(i);
    } else {
#pragma unroll
      for (int i = 0; i < PP; ++i)
        if (t + prow + i * ROWS < len && on) outputs(i);
      arrived();
    }
    row -= K;
    // the channel blocks' sums of dB and dC for the chunks since the last meeting; the next ones go to the other half of s_bc, and
    // this one is used again only behind the next meeting
    if (++met == F || t == 0) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < F * K * 2 * N / 256; ++i) {
        const int q = tid + i * 256, f = q / (K * 2 * N), r = q / (2 * N) % K, m = q / N & 1, n = q % N;
        const int tok = t + (met - 1 - f) * K + r;
        if (f >= met || tok >= len) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < CB; ++w) v += s_bc[part][f][w * SL + n / 16][r][(n % 16) / 2 * 4 + 2 * m + (n & 1)];
        pbc[(int64_t)tok * p.G * (2 * N) + m * N + n] = v;
      }
      met = 0;
      part ^= 1;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (in0 + l_ch + i >= p.Cg) continue;
      const int64_t at = (int64_t)chan(lane, i) * N + n0 + j;
      p.pA[(int64_t)slot * C * N + at] = dA[i][j];
      if (sp.first && p.dS0) p.dS0[(int64_t)sp.n * C * N + at] = carry[i][j];
    }
  // D and the bias: the lanes of a channel
  __syncthreads();
  float* red = &s_u[0][0][0];
  red[prow * CH + pc] = accD;
  red[256 + prow * CH + pc] = accb;
  __syncthreads();
  if (prow == 0 && on) {
    float vD = 0.f, vb = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      vD += red[r * CH + pc];
      vb += red[256 + r * CH + pc];
    }
    const int c = g * p.Cg + in0 + pc;
    p.pD[(int64_t)slot * 2 * C + c] = vD;
    p.pD[(int64_t)slot * 2 * C + C + c] = vb;
  }
}

// dA [C, N], dD and ddt_bias from the slots' parts (blocks below nA: dA), 64 columns x 16 groups of slots a workgroup.
template <int N>
__global__ __launch_bounds__(1024) void scan_dparam_kernel(const ScanParams p, int nA) {
  __shared__ float s[16][64];
  const bool isA = (int)blockIdx.x < nA;
  const int cols = isA ? p.C * N : 2 * p.C, col = ((int)blockIdx.x - (isA ? 0 : nA)) * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  const float* part = isA ? p.pA : p.pD;
  const int slots = p.cu ? p.slot_first[p.nseq] : p.slots;
  float v = 0.f;
  if (col < cols)
    for (int r = g; r < slots; r += 16) v += part[(int64_t)r * cols + col];
  s[g][threadIdx.x & 63] = v;
  __syncthreads();
  if (g == 0 && col < cols) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) a += s[k][threadIdx.x];
    if (isA)
      p.dA[col] = a;
    else if (col < p.C && p.dD)
      p.dD[col] = a;
    else if (col >= p.C && p.dbias)
      p.dbias[col - p.C] = a;
  }
}

// dB and dC from the channel blocks' parts, a value a thread.
template <int N, typename InT>
__global__ __launch_bounds__(256) void scan_dbc_kernel(const ScanParams p) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x, per = (int64_t)p.nbatch * p.T * p.G * (2 * N);
  if (q >= per) return;
  const int64_t row = q / (2 * N), tok = row / p.G;
  if (p.cu && (tok < p.cu[0] || tok >= p.cu[p.nseq])) return;  // no sequence holds it
  const int m = (int)(q / N & 1), n = (int)(q % N);
  float v = 0.f;
  for (int k = 0; k < p.cblocks; ++k) v += p.pBC[k * per + q];
  static_cast<InT*>(m ? p.dC : p.dB)[row * N + n] = (InT)v;
}

template <int SL, typename InT>
static void launch_states(const ScanParams& p, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.tiles)), block(64 * SL);
  if (p.part)
    hipLaunchKernelGGL((scan_states_kernel<SL, InT, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((scan_states_kernel<SL, InT, false>), grid, block, 0, s, p);
}
template <int N, typename InT>
static hipError_t launch_bwd_t(const ScanParams& p, hipStream_t s) {
  if (p.slots > 0 && p.nseq > 0) {
    launch_states<N / 16, InT>(p, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.part) {
      hipLaunchKernelGGL((scan_join2_kernel<N>), dim3((unsigned)((int64_t)p.nseq * ((p.C * (N / 4) + 255) / 256)), 2), dim3(256), 0, s, p);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((int64_t)p.slots * p.G * p.cblocks));
    if (p.z)
      hipLaunchKernelGGL((scan_grad_kernel<N, InT, true>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((scan_grad_kernel<N, InT, false>), grid, dim3(256), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int nA = (int)(((int64_t)p.C * N + 63) / 64);
  hipLaunchKernelGGL((scan_dparam_kernel<N>), dim3(nA + (2 * p.C + 63) / 64), dim3(1024), 0, s, p, nA);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t vals = (int64_t)p.nbatch * p.T * p.G * (2 * N);
  if (vals > 0 && p.nseq > 0)
    hipLaunchKernelGGL((scan_dbc_kernel<N, InT>), dim3((unsigned)((vals + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename InT>
static hipError_t launch_bwd_n(const ScanParams& p, int n, hipStream_t s) {
  return n == 16 ? launch_bwd_t<16, InT>(p, s) : n == 32 ? launch_bwd_t<32, InT>(p, s) : launch_bwd_t<64, InT>(p, s);
}
hipError_t launch_scan_bwd(ScanParams p, int n, bool bf16, hipStream_t s) {
  if (p.cu) {
    const hipError_t e = launch_scan_plan(p, s);
    if (e != hipSuccess) return e;
    p.cu = p.cu_ok;
  }
  return bf16 ? launch_bwd_n<__bf16>(p, n, s) : launch_bwd_n<float>(p, n, s);
}

}  // namespace dr
