/*
 * deltarule_decay.h — C ABI of the decayed linear attention and of the 8-bit state cache (MI355X, gfx950).
 *
 * Decayed linear attention is the recurrence of deltarule.h without its erase term and with one scalar
 * decay for each head:
 *
 *     S_t = a_t S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t
 *
 * with a_t given for every token and head or once for every head (the state update of Mamba-2 and of
 * retention, which the course page "GDN, KDA và Mamba-2 · cập nhật state trong hybrid" sets beside the
 * gated delta rule). Query/key heads may be shared: q and k have num_k_heads heads, v, the decay and the
 * states num_heads, and value head h reads query/key head h / (num_heads / num_k_heads).
 *
 * Memory, layout, streams, errors, cu_seqlens and stored states are those of deltarule.h: device pointers
 * on the current device, 16-byte aligned, work enqueued on `stream`, argument errors found on the host before
 * anything is launched, no pointer kept. Products and sums are held to fp32 (bf16 inputs enter exactly, fp32
 * values as three bf16 terms that hold all 24 bits): results agree with a float64 evaluation to about 1e-6
 * of the output's size (2-norm; the gradient of one decay per head: of the sum of its tokens' magnitudes).
 * Zero and negative decays are exact: no quotient or logarithm of a decay is formed.
 * Decays are not range-checked; the accuracy statement covers |a| <= 1. A NaN or an infinity in a token's
 * inputs makes the outputs of its 64-token chunk (earlier tokens of the chunk included) and of every later
 * chunk of that head unspecified; other heads and sequences are not affected, and neither are tokens that
 * no sequence holds.
 */
#ifndef DELTARULE_DECAY_H
#define DELTARULE_DECAY_H

#include "deltarule.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Where the decay of (batch row b, token t, head h) is. */
typedef enum dr_decay_layout {
  DR_DECAY_TOKEN = 0, /* alpha [B, T, H] (decode: [N, H]) */
  DR_DECAY_HEAD = 1   /* alpha [H] */
} dr_decay_layout;

/* Sizes of one call. batch, seqlen, num_heads, head_dim_k, head_dim_v, num_seqs and in_dtype as in dr_dims;
 * num_heads must be a multiple of num_k_heads. strided = 0: q, k and v are dense; 1: the element strides
 * between consecutive tokens of a batch row and between batch rows (decode: between sequences) are given,
 * under the rules of dr_dims_v2 (heads and channels dense, non-negative, multiples of 16 bytes; token strides at
 * most 2^24 elements). At most 65536 heads. A kernel has at most 2^32 - 1 work items, which bounds the
 * (sequence, head) pairs of a call: about 5.5 million for the prefill (its workgroups have 768; float32 inputs take
 * d_v / 32 of them a head, d_v / 16 with d_k = 128), 8.3 million chunks of heads for the gradients, 16.7 million heads for the step; larger ones are refused (DR_ERR_UNSUPPORTED). */
typedef struct dr_decay_dims {
  int64_t batch;
  int64_t seqlen;
  int64_t num_heads;
  int64_t num_k_heads;
  int64_t head_dim_k;
  int64_t head_dim_v;
  int64_t num_seqs;
  int32_t in_dtype;
  int32_t decay_layout;
  int32_t strided;
  int32_t reserved; /* 0 */
  int64_t q_token_stride, q_batch_stride;
  int64_t k_token_stride, k_batch_stride;
  int64_t v_token_stride, v_batch_stride;
} dr_decay_dims;

/*
 * Bytes of workspace that a call of dr_decay_fwd (backward == 0) or dr_decay_bwd (backward != 0) with these dims takes;
 * packed: whether it has cu_seqlens. May be 0. Nothing in a workspace is kept from one call for the next.
 * Both calls take it as `workspace`, `workspace_bytes` (device memory, 16-byte aligned, not in use by another call
 * until this one is over on the stream). With NULL it comes from the library's pool, stream-ordered; while the
 * stream is being captured a call that needs any is then refused (DR_ERR_UNSUPPORTED).
 */
int dr_decay_workspace(const dr_decay_dims* dims, int packed, int backward, int64_t* bytes);

/*
 * Prefill.
 *   q, k       [B, T, Hk, d_k]  in_dtype;   v [B, T, H, d_v] in_dtype
 *   alpha      float32, [B, T, H] or [H]
 *   S0, cu_seqlens, o, S_T as in dr_chunk_fwd (o or S_T may be NULL, S_T may alias S0)
 *   opts       NULL, or state_idx / num_slots and snapshots / snapshot_every (a positive multiple of 64)
 *              as in dr_chunk_fwd_ex; the input preparation fields must be zero
 * Sequences that are too few to fill the GPU are cut into segments whose own states are formed
 * first; the workspace holds one state per segment and head. A call that needs no segments takes none (packed
 * sequences: a few integers per sequence).
 */
int dr_decay_fwd(const void* q, const void* k, const void* v, const float* alpha, const float* S0,
                 const int32_t* cu_seqlens, float* o, float* S_T, const dr_decay_dims* dims, const dr_opts* opts,
                 void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * One token for each of N sequences x H heads, the states updated in place.
 *   q, k [N, Hk, d_k], v [N, H, d_v] in_dtype;  alpha float32 [N, H] or [H];  S [N, H, d_k, d_v] (or the pool,
 *   with opts->state_idx: a slot outside it gives o = 0 and touches no state, two
 *   sequences naming the same slot race);  o [N, H, d_v] float32
 * dims: batch = num_seqs = N, seqlen = 1. Uses no other device memory.
 */
int dr_decay_step(const void* q, const void* k, const void* v, const float* alpha, float* S, float* o,
                  const dr_decay_dims* dims, const dr_opts* opts, hipStream_t stream);

/*
 * Gradients of dr_decay_fwd for dO = dL/do [B, T, H, d_v] and dS_T = dL/dS_T [N, H, d_k, d_v] (NULL: zero), float32
 * and dense, in the shapes of the inputs:
 *   dq, dk [B, T, Hk, d_k] (summed over the value heads of a query/key head), dv [B, T, H, d_v],
 *   dalpha [B, T, H], or [H] summed over all tokens,  dS0 [N, H, d_k, d_v] or NULL
 * The call forms the states and the state gradients at every 64th token (float32 inputs: every 32nd) itself; they and
 * the partial sums are its workspace: 8 d_k d_v bytes per 64 (32) tokens and head, and with shared heads 8 d_k
 * bytes per token and head. No atomics: the same call gives the same bits. Rows of tokens past
 * cu_seqlens[N] are not written.
 */
int dr_decay_bwd(const void* q, const void* k, const void* v, const float* alpha, const float* S0,
                 const int32_t* cu_seqlens, const float* dO, const float* dS_T, float* dq, float* dk, float* dv,
                 float* dalpha, float* dS0, const dr_decay_dims* dims, void* workspace, int64_t workspace_bytes,
                 hipStream_t stream);

/*
 * 8-bit state cache: fp32 states (of any recurrence of this library: a decode pool, a prefill's final states
 * or snapshots) written at a quarter of their size, and read back. A row is the d_v values of one key channel of
 * one head; it is held as d_v codes and one float32 scale, and stands for code * scale.
 *   DR_CACHE_INT8   scale = max(amax * r, 2^-126) with r the float32 number next to 1/127, the product rounded to
 *                   float32; code = the integer nearest to x / scale (the exact quotient,
 *                   ties to even)
 *   DR_CACHE_E4M3   scale = the least power of two, 2^-126 at the least, with amax <= 448 scale; code = x / scale
 *                   rounded to OCP e4m3 (nearest, ties to even)
 * A row that holds a NaN or an infinity gets a NaN scale and zero codes: the whole row reads back as NaN.
 * What is read back is code * scale rounded to float32: magnitudes from about 3.3e38 on may come back as infinities.
 */
typedef enum dr_cache_format { DR_CACHE_INT8 = 0, DR_CACHE_E4M3 = 1 } dr_cache_format;

/*
 * count      states moved by the call; at most 16.7 million workgroups of 16 KiB of one head (DR_ERR_UNSUPPORTED)
 * num_states rows of S [num_states, H, d_k, d_v]; num_slots rows of codes [num_slots, H, d_k, d_v] (1 byte each)
 *            and scales [num_slots, H, d_k]
 * state_idx  [count] int32 (device): row of S of each state, NULL: row n (num_states >= count)
 * slot_idx   [count] int32 (device): row of the cache of each state, NULL: row n (num_slots >= count)
 */
typedef struct dr_cache_dims {
  int64_t count;
  int64_t num_states;
  int64_t num_slots;
  int64_t num_heads;
  int64_t head_dim_k;
  int64_t head_dim_v;
  int32_t format;
  int32_t reserved; /* 0 */
} dr_cache_dims;

/* Writes state_idx[n] of S to slot_idx[n] of the cache. A state row outside S counts as the zero state (a sequence
 * with no stored state); a slot outside the cache is skipped. Slots that nobody names are left as they
 * are; two states with the same slot race (undefined). */
int dr_state_pack(const float* S, const int32_t* state_idx, uint8_t* codes, float* scales, const int32_t* slot_idx,
                  const dr_cache_dims* dims, hipStream_t stream);

/* Reads slot_idx[n] of the cache into state_idx[n] of S. A slot outside the cache gives the zero state; a state row
 * outside S is skipped. Rows that nobody names are left as they are. One slot may be read into many rows;
 * the same row named twice races (undefined). */
int dr_state_unpack(const uint8_t* codes, const float* scales, const int32_t* slot_idx, float* S,
                    const int32_t* state_idx, const dr_cache_dims* dims, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTARULE_DECAY_H */
