// Short causal convolution over the tokens of every channel on gfx950, its single-token step and its gradients.
//
// A few operations per value: bound by memory. A lane has one 16-byte piece of the channels (or one channel where rows are
// not aligned), a wave a run of consecutive tokens whose last inputs slide through registers, so an input is read once
// (and the width - 1 in front of a run again). A run that holds the ends of packed sequences is walked in
// pieces, one per sequence. Loads are issued a batch of tokens in front of their use.
//
// 4 x 4096 x 2048 bf16: 30 us (134 MB, 26 at the copy rate). Backward, packed, fp32, 1531 channels (rows not aligned: single channels): 32 us and
// 4 for the sums of dw (28). Step, 4096 channels, bf16, in a graph: 1 sequence 3.6 us, 64 5.1, 256 6.4, 512
// 8.7-9.5 (33 MB, 6.5), 2048 24.4 (26): some 4 us of a launch and its rounds of loads, then memory. Backward, bf16, 4 x 2048 x 2048 35.6 us
// (19.5 at the copy rate), 4 x 8192 x 2048 92.8 (78).
#include "scan.hpp"

namespace dr {

// The part of a run that lies in one sequence: tokens a .. b of row `row`, of sequence n with tokens start .. end.
struct RunPiece {
  int n, a, b, start, end;
};
__device__ __forceinline__ RunPiece piece_at(const ConvParams& p, int row, int t, int t1) {
  RunPiece q;
  q.a = t;
  if (p.cu) {
    q.n = seq_of(p.cu, p.nseq, t);
    // (offsets out of order or outside the row still give 0 <= start <= t < end <= T)
    q.start = min(max(p.cu[q.n], 0), t);
    q.end = p.cu[q.n + 1];
    if (q.end <= t || p.cu[q.n] > t) {  // no sequence holds token t
      q.n = -1;
      q.end = t1;
    }
    q.end = min(q.end, (int)p.T);
  } else {
    q.n = row;
    q.start = 0;
    q.end = (int)p.T;
  }
  q.b = min(t1, q.end);
  return q;
}

template <typename InT, int VEC, int W>
struct Conv {
  using V = typename Vec<InT, VEC>::type;
  const ConvParams& p;
  int c;          // the lane's first channel; lanes past the last channels have those again and store nothing
  bool in;
  uint32_t off;   // its bytes
  float w[W][VEC], bias[VEC];
  __device__ __forceinline__ Conv(const ConvParams& p_, int c_) : p(p_), c(min(c_, p_.C - VEC)), in(c_ < p_.C), off((uint32_t)c * sizeof(InT)) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      bias[v] = p.bias ? p.bias[c + v] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][v] = p.w[(int64_t)(c + v) * W + j];
    }
  }
  // the lane's channels of a row (uniform)
  __device__ __forceinline__ V load(const void* rows, int64_t row, int64_t stride) const {
    return *reinterpret_cast<const V*>(byte_at(static_cast<const InT*>(rows) + row * stride, off));
  }
  __device__ __forceinline__ void store(void* rows, int64_t row, int64_t stride, const V& v) const {
    if (in) *reinterpret_cast<V*>(byte_at(static_cast<InT*>(rows) + row * stride, off)) = v;
  }
  __device__ __forceinline__ void store_same(void* rows, int64_t row, int64_t stride, const V& v) const {
    *reinterpret_cast<V*>(byte_at(static_cast<InT*>(rows) + row * stride, off)) = v;
  }
  // a row of an output that no cache will hold until it is read (whole lines: stores of single channels got slower that way)
  template <bool STREAM>
  __device__ __forceinline__ void put(void* rows, int64_t row, int64_t stride, const V& v) const {
    if constexpr (STREAM) {
      if (in) __builtin_nontemporal_store(v, reinterpret_cast<V*>(byte_at(static_cast<InT*>(rows) + row * stride, off)));
    } else {
      store(rows, row, stride, v);
    }
  }
  // input number k (0: the oldest) of row `srow` of the states
  __device__ __forceinline__ V old(int64_t srow, int k) const {
    return p.state && srow >= 0 ? load(p.state, srow * (W - 1) + k, p.C) : V{};
  }
  // the W - 1 inputs in front of token a of a sequence that starts at `start`
  __device__ __forceinline__ void window(const InT* x, int a, int start, int64_t srow, float (&e)[W][VEC]) const {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int t = a - (W - 1) + j;
      unpack<VEC, InT>(t >= start ? load(x, t, p.x_ts) : old(srow, t - start + W - 1), e[j]);
    }
  }
  __device__ __forceinline__ void dot(const float (&e)[W][VEC], float (&u)[VEC]) const {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      u[v] = bias[v];
#pragma unroll
      for (int j = 0; j < W; ++j) u[v] = fmaf(w[j][v], e[j][v], u[v]);
    }
  }
  static __device__ __forceinline__ void slide(float (&e)[W][VEC]) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) e[j][v] = e[j + 1][v];
  }
};

// The last W - 1 inputs of sequence n, into its state (every row read before the first is written: they may be the same).
template <typename InT, int VEC, int W>
__device__ __forceinline__ void conv_tail(const ConvParams& p, int n, int c) {
  using V = typename Vec<InT, VEC>::type;
  const Conv<InT, VEC, W> k(p, c);
  int start = 0, end = (int)p.T;
  int64_t row = n;
  if (p.cu) {
    start = min(max(p.cu[n], 0), (int)p.T);
    end = min(max(p.cu[n + 1], start), (int)p.T);
    row = 0;
  }
  const int64_t s = state_row(p.sidx, p.nslots, n);
  const InT* x = static_cast<const InT*>(p.x) + row * p.x_bs;
  V v[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int t = end - (W - 1) + j;
    v[j] = t >= start ? k.load(x, t, p.x_ts) : k.old(s, t - start + W - 1);
  }
  if (s < 0) return;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) k.store(p.state_T, s * (W - 1) + j, p.C, v[j]);
}

// Neighbouring channel blocks share the cache lines of rows that are not aligned, neighbouring runs the inputs between them: consecutive
// logical blocks go to one XCD (workgroups are dealt over eight). Of `total` blocks; past them: nothing to do.
__device__ __forceinline__ int logical_block(int total) {
  const int per = (total + 7) / 8;
  return (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
}

template <typename InT, int VEC, int W, bool SILU, bool STREAM>
__global__ __launch_bounds__(64 * CONV_WAVES) void conv_fwd_kernel(const ConvParams p) {
  using V = typename Vec<InT, VEC>::type;
  constexpr int AHEAD = 8;  // tokens whose loads are issued together, a batch in front of their use
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = logical_block(p.nblocks), blk = p.block0 + at, cb = blk % p.cblocks;
  if (at >= p.nblocks) return;
  const int c = (cb * 64 + lane) * VEC;
  if (blk >= p.nmain) {
    const int n = (blk - p.nmain) / p.cblocks * CONV_WAVES + wave;
    if (n < p.nseq) conv_tail<InT, VEC, W>(p, n, c);
    return;
  }
  const int rid = blk / p.cblocks * CONV_WAVES + wave;
  const int row = rid / p.runs;
  if (row >= p.nbatch) return;
  const int t0 = (rid - row * p.runs) * p.run;
  const int t1 = (int)(p.T - t0 < p.run ? p.T : t0 + p.run);
  const Conv<InT, VEC, W> k(p, c);
  const InT* x = static_cast<const InT*>(p.x) + row * p.x_bs;
  InT* y = static_cast<InT*>(p.y) + (int64_t)row * p.T * p.C;
  for (int t = t0; t < t1;) {
    const RunPiece q = piece_at(p, row, t, t1);
    if (q.n >= 0) {
      float e[W][VEC];
      V next[AHEAD], raw[AHEAD];
      auto fetch = [&](int a) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) next[i] = k.load(x, min(a + i, q.b - 1), p.x_ts);
      };
      auto token = [&](int at_t, int i) {
        unpack<VEC, InT>(raw[i], e[W - 1]);
        float u[VEC];
        k.dot(e, u);
        if constexpr (SILU)
#pragma unroll
          for (int v = 0; v < VEC; ++v) u[v] *= sigmoid_f(u[v]);
        k.template put<STREAM>(y, at_t, p.C, pack<VEC, InT>(u));
        k.slide(e);
      };
      fetch(q.a);
      k.window(x, q.a, q.start, state_row(p.sidx, p.nslots, q.n), e);
      for (int a = q.a; a < q.b; a += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) raw[i] = next[i];
        if (a + AHEAD < q.b) fetch(a + AHEAD);
        if (a + AHEAD <= q.b) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) token(a + i, i);
        } else {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i)
            if (a + i < q.b) token(a + i, i);
        }
      }
    }
    t = q.b;
  }
}

// A wave takes `run` sequences one after the other on one block of channels (the weights are twice a token's inputs and outputs),
// the next one's inputs loaded ahead.
template <typename InT, int VEC, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvParams p) {
  using V = typename Vec<InT, VEC>::type;
  const int cb = blockIdx.x % p.cblocks;
  const int n0 = (blockIdx.x / p.cblocks * CONV_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * p.run;
  const int c = (cb * 64 + (threadIdx.x & 63)) * VEC, n1 = min(n0 + p.run, p.nseq);
  if (n0 >= n1) return;
  // (every lane stays: those past the last channels have the last ones again and store the same; `rows` is read from lanes by number)
  const Conv<InT, VEC, W> k(p, c);
  const int lane = threadIdx.x & 63;
  int rows = -1;  // lane i: of sequence n0 + i (at most 64 of them)
  if (n0 + lane < n1) rows = (int)state_row(p.sidx, p.nslots, n0 + lane);
  V next[W];
  auto fetch = [&](int n) {  // (one without a stored state reads its input in its place)
    const int s = __builtin_amdgcn_readlane(rows, n - n0);
    const InT* x = static_cast<const InT*>(p.x) + n * p.x_bs;
    const InT* old = s >= 0 ? static_cast<const InT*>(p.state_T) + (int64_t)s * (W - 1) * p.C : x;
    const int64_t stride = s >= 0 ? p.C : 0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) next[j] = k.load(old, j, stride);
    next[W - 1] = k.load(x, 0, 0);
  };
  auto token = [&](int n, auto more) {
    V r[W];
    float e[W][VEC], u[VEC];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      r[j] = next[j];
      unpack<VEC, InT>(r[j], e[j]);
    }
    if constexpr (decltype(more)::value) fetch(n + 1);
    k.dot(e, u);
    if (p.silu)
#pragma unroll
      for (int v = 0; v < VEC; ++v) u[v] *= sigmoid_f(u[v]);
    const int s = __builtin_amdgcn_readlane(rows, n - n0);
    if (s >= 0) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) k.store_same(p.state_T, (int64_t)s * (W - 1) + j, p.C, r[j + 1]);
      k.store_same(p.y, n, p.C, pack<VEC, InT>(u));
    } else {  // no stored state
      k.store_same(p.y, n, p.C, V{});
      arrived();
    }
  };
  fetch(n0);
  arrived();
  for (int n = n0; n + 1 < n1; ++n) token(n, std::true_type{});
  token(n1 - 1, std::false_type{});
}

// Gradient of a token's sum before the activation: dy, with silu times sigmoid(u) (1 + u sigmoid(-u)).
template <int VEC, bool SILU>
__device__ __forceinline__ void conv_du(const float (&u)[VEC], const float (&dy)[VEC], float (&du)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    du[v] = dy[v];
    if constexpr (SILU) {
      const float sg = sigmoid_f(u[v]);
      du[v] *= sg * fmaf(u[v], 1.f - sg, 1.f);
    }
  }
}

// An input reaches the outputs of its own and the next W - 1 tokens of its sequence: the gradients du of W consecutive
// tokens slide through registers behind the inputs, and token t completes the gradient of input t - W + 1. The
// gradients of the weights stay in registers over the run; a workgroup adds its four runs'.
template <typename InT, int VEC, int W, bool SILU, bool STREAM>
__global__ __launch_bounds__(64 * CONV_WAVES) void conv_bwd_kernel(const ConvParams p) {
  using V = typename Vec<InT, VEC>::type;
  constexpr int AHEAD = 4;
  __shared__ float s_part[CONV_WAVES - 1][W + 1][64 * VEC];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blk = logical_block(p.nblocks), cb = blk % p.cblocks;
  if (blk >= p.nblocks) return;
  const int c = (cb * 64 + lane) * VEC;
  if (blk >= p.nmain) {  // the gradient of sequence n's starting state
    const int n = (blk - p.nmain) / p.cblocks * CONV_WAVES + wave;
    if (n >= p.nseq) return;
    const Conv<InT, VEC, W> k(p, c);
    int start = 0, end = (int)p.T, row = n;
    if (p.cu) {
      start = min(max(p.cu[n], 0), (int)p.T);
      end = min(max(p.cu[n + 1], start), (int)p.T);
      row = 0;
    }
    const InT* x = static_cast<const InT*>(p.x) + row * p.x_bs;
    const InT* dy = static_cast<const InT*>(p.dy) + (int64_t)row * p.T * p.C;
    float e[W][VEC], ds[W - 1][VEC];
    k.window(x, start, start, n, e);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) ds[j][v] = 0.f;
      const int L = end - start;
      if (j >= L && p.dstate_T) unpack<VEC, InT>(k.load(p.dstate_T, (int64_t)n * (W - 1) + j - L, p.C), ds[j]);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      if (start + i < end) {
        float u[VEC], g[VEC], du[VEC];
        unpack<VEC, InT>(k.load(x, start + i, p.x_ts), e[W - 1]);
        k.dot(e, u);
        unpack<VEC, InT>(k.load(dy, start + i, p.C), g);
        conv_du<VEC, SILU>(u, g, du);
#pragma unroll
        for (int j = i; j < W - 1; ++j)
#pragma unroll
          for (int v = 0; v < VEC; ++v) ds[j][v] = fmaf(k.w[j - i][v], du[v], ds[j][v]);
        k.slide(e);
      }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) k.store(p.dstate, (int64_t)n * (W - 1) + j, p.C, pack<VEC, InT>(ds[j]));
    return;
  }
  const Conv<InT, VEC, W> k(p, c);
  float dw[W + 1][VEC];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) dw[j][v] = 0.f;
  const int rb = blk / p.cblocks, rid = rb * CONV_WAVES + wave;
  const int row = rid / p.runs;
  if (row < p.nbatch) {
    const int t0 = (rid - row * p.runs) * p.run;
    const int t1 = (int)(p.T - t0 < p.run ? p.T : t0 + p.run);
    const InT* x = static_cast<const InT*>(p.x) + row * p.x_bs;
    const InT* dy = static_cast<const InT*>(p.dy) + (int64_t)row * p.T * p.C;
    InT* dx = static_cast<InT*>(p.dx) + (int64_t)row * p.T * p.C;
    for (int t = t0; t < t1;) {
      const RunPiece q = piece_at(p, row, t, t1);
      if (q.n >= 0) {
        float e[W][VEC], du[W][VEC];  // du[j]: of token t - W + 1 + j
        V xn[AHEAD], gn[AHEAD], xr[AHEAD], gr[AHEAD];
        auto fetch = [&](int a) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            const int at_t = min(a + i, q.end - 1);
            xn[i] = k.load(x, at_t, p.x_ts);
            gn[i] = k.load(dy, at_t, p.C);
          }
        };
        // token tt, in the run and the sequence (USED), behind the run (its weights' gradients are another's), or behind the
        // sequence (no gradient); then the gradient of input tt - W + 1, which is complete
        auto token = [&](int tt, int i, auto used) {
          constexpr bool USED = decltype(used)::value;
          k.slide(du);
          if (USED || tt < q.end) {
            float u[VEC], g[VEC];
            unpack<VEC, InT>(xr[i], e[W - 1]);
            unpack<VEC, InT>(gr[i], g);
            k.dot(e, u);
            conv_du<VEC, SILU>(u, g, du[W - 1]);
            if (USED || tt < q.b)
#pragma unroll
              for (int v = 0; v < VEC; ++v) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j][v] = fmaf(du[W - 1][v], e[j][v], dw[j][v]);
                dw[W][v] += du[W - 1][v];
              }
            k.slide(e);
          } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) du[W - 1][v] = 0.f;
          }
          const int i0 = tt - (W - 1);
          if (i0 < q.a) return;
          float g[VEC];
#pragma unroll
          for (int v = 0; v < VEC; ++v) g[v] = 0.f;
          if (i0 >= q.end - (W - 1) && p.dstate_T)
            unpack<VEC, InT>(k.load(p.dstate_T, (int64_t)q.n * (W - 1) + i0 - (q.end - (W - 1)), p.C), g);
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) g[v] = fmaf(k.w[W - 1 - j][v], du[j][v], g[v]);
          k.template put<STREAM>(dx, i0, p.C, pack<VEC, InT>(g));
        };
        fetch(q.a);
        k.window(x, q.a, q.start, q.n, e);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int v = 0; v < VEC; ++v) du[j][v] = 0.f;
        const int stop = q.b + W - 1;
        for (int a = q.a; a < stop; a += AHEAD) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            xr[i] = xn[i];
            gr[i] = gn[i];
          }
          if (a + AHEAD < stop) fetch(a + AHEAD);
          if (a + AHEAD <= q.b) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) token(a + i, i, std::true_type{});
          } else {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
              if (a + i < stop) token(a + i, i, std::false_type{});
          }
        }
      }
      t = q.b;
    }
  }
  if (wave > 0)
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) s_part[wave - 1][j][v * 64 + lane] = dw[j][v];
  __syncthreads();
  if (wave > 0 || !k.in) return;
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float a = dw[j][v];
#pragma unroll
      for (int g = 0; g < CONV_WAVES - 1; ++g) a += s_part[g][j][v * 64 + lane];
      p.part[((int64_t)rb * (W + 1) + j) * p.C + c + v] = a;
    }
}

// dw [C, W] and db [C] from the workgroups' sums: 64 columns x 16 groups of run blocks a workgroup.
template <int W>
__global__ __launch_bounds__(1024) void conv_dw_kernel(const ConvParams p, int parts) {
  __shared__ float s[16][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  const int n = (W + 1) * p.C;
  float v = 0.f;
  if (col < n)
    for (int r = g; r < parts; r += 16) v += p.part[(int64_t)r * n + col];
  s[g][threadIdx.x & 63] = v;
  __syncthreads();
  if (g == 0 && col < n) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) a += s[k][threadIdx.x];
    const int j = col / p.C, c = col - j * p.C;
    if (j < W)
      p.dw[(int64_t)c * W + j] = a;
    else if (p.db)
      p.db[c] = a;
  }
}

static int64_t run_blocks(const ConvParams& p) { return ((int64_t)p.nbatch * p.runs + CONV_WAVES - 1) / CONV_WAVES; }
static dim3 eights(int64_t n) { return dim3((unsigned)((n + 7) / 8 * 8)); }
static int64_t seq_blocks(const ConvParams& p) { return ((int64_t)p.nseq + CONV_WAVES - 1) / CONV_WAVES; }

template <typename InT, int VEC, int W>
static hipError_t launch_fwd_t(ConvParams p, hipStream_t s) {
  const int64_t main = run_blocks(p) * p.cblocks, tail = p.state_T ? seq_blocks(p) * p.cblocks : 0;
  p.nmain = (int32_t)main;
  p.block0 = 0;
  // the states' own launch where the tokens' still read the states that it writes
  const bool apart = tail > 0 && p.state == p.state_T;
  p.nblocks = (int32_t)(apart ? main : main + tail);
  constexpr bool S = VEC > 1;
  const auto kernel = S && p.streamed ? (p.silu ? conv_fwd_kernel<InT, VEC, W, true, S> : conv_fwd_kernel<InT, VEC, W, false, S>)
                                      : (p.silu ? conv_fwd_kernel<InT, VEC, W, true, false> : conv_fwd_kernel<InT, VEC, W, false, false>);
  if (p.nblocks > 0) hipLaunchKernelGGL(kernel, eights(p.nblocks), dim3(64 * CONV_WAVES), 0, s, p);
  if (apart) {
    p.block0 = p.nmain;
    p.nblocks = (int32_t)tail;
    hipLaunchKernelGGL(kernel, eights(p.nblocks), dim3(64 * CONV_WAVES), 0, s, p);
  }
  return hipGetLastError();
}
template <typename InT, int VEC, int W>
static hipError_t launch_step_t(const ConvParams& p, hipStream_t s) {
  const int64_t waves = ((int64_t)p.nseq + p.run - 1) / p.run;
  hipLaunchKernelGGL((conv_step_kernel<InT, VEC, W>), dim3((unsigned)((waves + CONV_WAVES - 1) / CONV_WAVES * p.cblocks)), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename InT, int VEC, int W>
static hipError_t launch_bwd_t(ConvParams p, hipStream_t s) {
  const int64_t main = run_blocks(p) * p.cblocks, tail = p.dstate ? seq_blocks(p) * p.cblocks : 0;
  p.nmain = (int32_t)main;
  p.block0 = 0;
  p.nblocks = (int32_t)(main + tail);
  constexpr bool S = VEC > 1;
  const auto kernel = S && p.streamed ? (p.silu ? conv_bwd_kernel<InT, VEC, W, true, S> : conv_bwd_kernel<InT, VEC, W, false, S>)
                                      : (p.silu ? conv_bwd_kernel<InT, VEC, W, true, false> : conv_bwd_kernel<InT, VEC, W, false, false>);
  if (p.nblocks > 0) hipLaunchKernelGGL(kernel, eights(p.nblocks), dim3(64 * CONV_WAVES), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((conv_dw_kernel<W>), dim3((unsigned)(((W + 1) * (int64_t)p.C + 63) / 64)), dim3(1024), 0, s, p, (int)run_blocks(p));
  return hipGetLastError();
}

#define DR_CONV_LAUNCH(FN)                                                                      \
  template <typename InT, int VEC>                                                              \
  static hipError_t FN##_w(const ConvParams& p, int width, hipStream_t s) {                     \
    return width == 4 ? FN##_t<InT, VEC, 4>(p, s) : width == 3 ? FN##_t<InT, VEC, 3>(p, s) : FN##_t<InT, VEC, 2>(p, s); \
  }
DR_CONV_LAUNCH(launch_fwd)
DR_CONV_LAUNCH(launch_step)
DR_CONV_LAUNCH(launch_bwd)
#undef DR_CONV_LAUNCH

hipError_t launch_conv_fwd(ConvParams p, int width, bool bf16, bool vec, hipStream_t s) {
  if (bf16) return vec ? launch_fwd_w<__bf16, 8>(p, width, s) : launch_fwd_w<__bf16, 1>(p, width, s);
  return vec ? launch_fwd_w<float, 4>(p, width, s) : launch_fwd_w<float, 1>(p, width, s);
}
hipError_t launch_conv_step(const ConvParams& p, int width, bool bf16, bool vec, hipStream_t s) {
  if (bf16) return vec ? launch_step_w<__bf16, 8>(p, width, s) : launch_step_w<__bf16, 1>(p, width, s);
  return vec ? launch_step_w<float, 4>(p, width, s) : launch_step_w<float, 1>(p, width, s);
}
hipError_t launch_conv_bwd(ConvParams p, int width, bool bf16, bool vec, hipStream_t s) {
  if (bf16) return vec ? launch_bwd_w<__bf16, 4>(p, width, s) : launch_bwd_w<__bf16, 1>(p, width, s);
  return vec ? launch_bwd_w<float, 4>(p, width, s) : launch_bwd_w<float, 1>(p, width, s);
}

}  // namespace dr
