// What the scan's kernels share: a wave's tile of 16 tokens x 32 channels x 16 states.
//
// Lane l has channel l % 32 and of its 16 states those of its half (l / 32): 4 half .. + 3 and 8 + 4 half .. + 3, in this order. Of the tokens each
// half loads every other one (2 i + half), and what belongs to a (token, channel) pair is computed once.
// What a token adds to the state, d x B, is an outer product over channels and states. One fp32 matrix instruction
// (32 x 32 x 2) forms it for two tokens: rows 0 .. 15 are the first token's states, rows 16 .. 31 the second's, the first operand is B in the
// places of its token (zeros elsewhere), the second is d x as the lanes hold it; the result lies as the lanes hold states. So
// neither B nor d x is ever handed around, and a state costs the vector units its exponential, one product and two sums.
#pragma once

#include "scan.hpp"

namespace dr {

typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int TILE_TOK = 16, TILE_OWN = TILE_TOK / 2;

__device__ __forceinline__ f32x16 outer_pair(float states, float channels) {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return __builtin_amdgcn_mfma_f32_32x32x2f32(states, channels, z, 0, 0, 0);
}
// Two tokens share that instruction, and the zeros in the other one's places times a d x that is not finite would make the other's sum NaN, the
// earlier one's too. Such a d x goes in as a finite number, and its own token's decay is made NaN, so that the state is from there on.
__device__ __forceinline__ void own_token(float& d, float& dx) {
  d = fmaf(dx, 0.f, d);
  dx = __builtin_amdgcn_fmed3f(dx, -3.402823466e38f, 3.402823466e38f);
}
// Between the pairs of a tile: what a pair loads and forms is not moved in front of the pairs before it, where it would only hold registers.
__device__ __forceinline__ void tile_step() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// A value formed where it stands, not in the branch that would use it (or behind the stores that follow).
__device__ __forceinline__ void here(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void here(float (&v)[8]) {
  asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]));
}
// Ends the branch of a whole tile's loads: without it the compiler joins them with those of a cut tile, whose addresses are the lanes'
// own, and forms 64-bit addresses for both.
__device__ __forceinline__ void whole_tile() { asm volatile("; whole tile" ::: "memory"); }
// A lane's offset (or number) as a value of its own: what is computed from it is computed where it is used. Loads from a uniform pointer
// want 32-bit offsets beside them; those that a loop keeps are kept as 64 bits and added for each load, or spilled, and the reload of a
// spilled register waits for every load in front of it (gradients of 2 x 4096 x 2048: 340 us so, 240 without).
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
// A value of the lower half's token and of the upper half's, in both halves.
__device__ __forceinline__ void both_halves(float v, float& low, float& high) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  low = __builtin_bit_cast(float, (uint32_t)r[0]);
  high = __builtin_bit_cast(float, (uint32_t)r[1]);
}
// a of both halves summed, in the lower half; b's sum in the upper.
__device__ __forceinline__ float sum_halves(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
// The lane's eight states from and to a row of N of them.
__device__ __forceinline__ void load_states(const float* row, float (&h)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(row), b = *reinterpret_cast<const f32x4*>(row + 8);
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = j < 4 ? a[j & 3] : b[j & 3];
}
__device__ __forceinline__ void store_states(float* row, const float (&h)[8]) {
  *reinterpret_cast<f32x4*>(row) = f32x4{h[0], h[1], h[2], h[3]};
  *reinterpret_cast<f32x4*>(row + 8) = f32x4{h[4], h[5], h[6], h[7]};
}

// An element as it comes from memory, in a register of its own: 16-bit values would be paired up where the branches that load them
// meet, and that waits for them there.
__device__ __forceinline__ uint32_t raw_bits(const float* p) { return __builtin_bit_cast(uint32_t, *p); }
__device__ __forceinline__ uint32_t raw_bits(const __bf16* p) { return *reinterpret_cast<const uint16_t*>(p); }
template <typename InT>
__device__ __forceinline__ float raw_value(uint32_t v) {
  return __builtin_bit_cast(float, sizeof(InT) == 2 ? v << 16 : v);
}

// An input [tokens, channels] as a wave reads it: a uniform pointer to the tile's first token, moved on with the tile,
// and the lane's offset in it, 32 bits of bytes (token strides are at most 2^24 elements), which the loads add by themselves; formed for
// each tile (see fresh).
template <typename InT>
struct Rows {
  const InT* at;
  int64_t ts;
  int half, col;
  __device__ __forceinline__ void init(const void* base, int64_t first, int64_t ts_, int half_, int col_) {
    at = static_cast<const InT*>(base) + first;
    ts = ts_;
    half = half_;
    col = col_;
  }
  // own tokens 2 i + half; `left`: tokens from the tile's first to the end (those past it are read from the last and not used)
  __device__ __forceinline__ void whole(uint32_t (&v)[TILE_OWN]) const {
    const InT* q = at;
    const uint32_t o = fresh(col) * sizeof(InT) + (fresh(half) ? (uint32_t)ts * sizeof(InT) : 0u);
#pragma unroll
    for (int i = 0; i < TILE_OWN; ++i, q += 2 * ts) v[i] = raw_bits(byte_at(q, o));
  }
  __device__ __forceinline__ void part(uint32_t (&v)[TILE_OWN], int left) const {
    const int h = (int)fresh(half), c = (int)fresh(col);
#pragma unroll
    for (int i = 0; i < TILE_OWN; ++i) v[i] = raw_bits(at + ((int64_t)min(2 * i + h, left - 1) * ts + c));
  }
};

// The first operand of outer_pair: elements of B (or C) of the own tokens, zeros in the other token's places.
template <typename InT>
__device__ __forceinline__ float operand(uint32_t raw, int lane) {
  return ((lane >> 4) & 1) == (lane >> 5) ? raw_value<InT>(raw) : 0.f;
}

}  // namespace dr
