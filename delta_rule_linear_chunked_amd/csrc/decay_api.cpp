// C ABI of the decayed linear attention and the 8-bit state cache: argument checks, launch planning
// and dispatch. Every check runs on the host before any launch; no device memory is read here.
#include <climits>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>
#include <utility>

#include "../../include/deltarule_decay.h"
#include "decay.hpp"
#include "host.hpp"
#include "state_cache.hpp"

using dr::host_fail;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool head_dim_ok(int64_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
const char* const kTooLarge = "problem too large: more than 2^31 - 1 workgroups or 2^32 - 1 work items per kernel";
int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

using Named = std::pair<const void*, const char*>;
int check_ptrs(std::initializer_list<Named> required, std::initializer_list<Named> optional) {
  for (const Named& x : required)
    if (x.first == nullptr) return host_fail(DR_ERR_NULL, "`%s` is NULL", x.second);
  for (const auto* list : {&required, &optional})
    for (const Named& x : *list)
      if (!aligned16(x.first)) return host_fail(DR_ERR_LAYOUT, "`%s` is not 16-byte aligned", x.second);
  return DR_OK;
}

int check_dims(const dr_decay_dims* d, const int32_t* cu, bool decode) {
  if (d == nullptr) return host_fail(DR_ERR_NULL, "dims is NULL");
  if (d->in_dtype != DR_F32 && d->in_dtype != DR_BF16)
    return host_fail(DR_ERR_DTYPE, "in_dtype %d is neither DR_F32 nor DR_BF16", d->in_dtype);
  if (d->decay_layout != DR_DECAY_TOKEN && d->decay_layout != DR_DECAY_HEAD)
    return host_fail(DR_ERR_SHAPE, "decay_layout %d is neither DR_DECAY_TOKEN nor DR_DECAY_HEAD", d->decay_layout);
  if ((d->strided != 0 && d->strided != 1) || d->reserved != 0)
    return host_fail(DR_ERR_SHAPE, "strided must be 0 or 1 and reserved 0");
  if (d->batch < 0 || d->seqlen < 0 || d->num_heads < 1 || d->num_k_heads < 1 || d->num_seqs < 0)
    return host_fail(DR_ERR_SHAPE, "bad sizes: batch=%lld seqlen=%lld heads=%lld key heads=%lld seqs=%lld",
                     (long long)d->batch, (long long)d->seqlen, (long long)d->num_heads, (long long)d->num_k_heads,
                     (long long)d->num_seqs);
  if (d->num_heads % d->num_k_heads != 0)
    return host_fail(DR_ERR_SHAPE, "num_heads (%lld) is not a multiple of num_k_heads (%lld)", (long long)d->num_heads,
                     (long long)d->num_k_heads);
  if (!head_dim_ok(d->head_dim_k) || !head_dim_ok(d->head_dim_v))
    return host_fail(DR_ERR_UNSUPPORTED, "head sizes d_k=%lld d_v=%lld: each must be 16, 32, 64 or 128",
                     (long long)d->head_dim_k, (long long)d->head_dim_v);
  // (each factor is bounded first, so that the products below stay within 64 bits)
  const int64_t lim = (int64_t)1 << 31;
  if (d->num_heads > (int64_t)1 << 16)
    return host_fail(DR_ERR_UNSUPPORTED, "%lld heads: at most 65536", (long long)d->num_heads);
  if (d->num_heads >= lim || d->num_seqs >= lim || d->batch >= lim || d->seqlen >= lim ||
      d->num_seqs * d->num_heads >= lim || d->batch * d->seqlen >= lim)
    return host_fail(DR_ERR_SHAPE, "problem too large for 32-bit token or head counts");
  if (d->strided) {
    const int64_t st[6] = {d->q_token_stride, d->q_batch_stride, d->k_token_stride,
                           d->k_batch_stride, d->v_token_stride, d->v_batch_stride};
    static const char* names[6] = {"q token", "q batch", "k token", "k batch", "v token", "v batch"};
    const int64_t esz = d->in_dtype == DR_BF16 ? 2 : 4;
    for (int i = 0; i < 6; ++i) {
      if (st[i] < 0) return host_fail(DR_ERR_SHAPE, "%s stride %lld is negative", names[i], (long long)st[i]);
      // (a chunk's rows are reached with 32-bit offsets from its first one)
      const int64_t most = i % 2 == 0 ? (int64_t)1 << 24 : (int64_t)1 << 40;
      if (st[i] > most || (st[i] * esz) % 16 != 0)
        return host_fail(DR_ERR_LAYOUT, "%s stride %lld is not a multiple of 16 bytes (or is beyond %lld)", names[i],
                         (long long)st[i], (long long)most);
    }
  }
  if (decode) {
    if (d->num_seqs != d->batch || d->seqlen != 1)
      return host_fail(DR_ERR_SHAPE, "a step has num_seqs equal to batch and seqlen 1, got %lld, %lld and %lld",
                       (long long)d->num_seqs, (long long)d->batch, (long long)d->seqlen);
  } else if (cu != nullptr) {
    if (d->batch != 1)
      return host_fail(DR_ERR_SHAPE, "packed sequences (cu_seqlens) need batch == 1, got %lld", (long long)d->batch);
  } else if (d->num_seqs != d->batch) {
    return host_fail(DR_ERR_SHAPE, "num_seqs (%lld) must equal batch (%lld) without cu_seqlens", (long long)d->num_seqs,
                     (long long)d->batch);
  }
  return DR_OK;
}

int check_opts(const dr_opts* o, bool prefill) {
  if (o == nullptr) return DR_OK;
  if (o->l2norm_qk != 0 || o->alpha_dtype != DR_F32 || o->alpha_act != DR_ACT_NONE || o->gate_act != DR_ACT_NONE)
    return host_fail(DR_ERR_UNSUPPORTED, "the decayed linear attention takes its inputs as they are: no input preparation");
  if (o->state_idx) {
    if (!aligned16(o->state_idx)) return host_fail(DR_ERR_LAYOUT, "state_idx must be 16-byte aligned");
    if (o->num_slots < 0) return host_fail(DR_ERR_SHAPE, "num_slots (%lld) is negative", (long long)o->num_slots);
    if (o->num_slots > INT32_MAX) return host_fail(DR_ERR_UNSUPPORTED, "num_slots above 2^31 - 1");
  }
  if (o->snapshots) {
    if (!prefill) return host_fail(DR_ERR_SHAPE, "snapshots are a prefill option");
    if (!aligned16(o->snapshots)) return host_fail(DR_ERR_LAYOUT, "snapshots must be 16-byte aligned");
    if (o->snapshot_every <= 0 || o->snapshot_every % 64 != 0)
      return host_fail(DR_ERR_SHAPE, "snapshot_every (%lld) must be a positive multiple of 64", (long long)o->snapshot_every);
    if (o->snapshot_every > INT32_MAX) return host_fail(DR_ERR_UNSUPPORTED, "snapshot_every too large");
  }
  return DR_OK;
}

void set_dims(dr::DecayParams& p, const dr_decay_dims* d) {
  p.T = d->seqlen;
  p.H = (int32_t)d->num_heads;
  p.Hk = (int32_t)d->num_k_heads;
  p.DK = (int32_t)d->head_dim_k;
  p.DV = (int32_t)d->head_dim_v;
  p.a_tok = d->decay_layout == DR_DECAY_TOKEN;
  p.nseq = (int32_t)d->num_seqs;
  if (d->strided) {
    p.q_ts = d->q_token_stride; p.q_bs = d->q_batch_stride;
    p.k_ts = d->k_token_stride; p.k_bs = d->k_batch_stride;
    p.v_ts = d->v_token_stride; p.v_bs = d->v_batch_stride;
  } else {
    p.q_ts = p.k_ts = d->num_k_heads * d->head_dim_k;
    p.v_ts = d->num_heads * d->head_dim_v;
    p.q_bs = p.k_bs = d->seqlen * p.q_ts;
    p.v_bs = d->seqlen * p.v_ts;
  }
}

// An integer from the environment, for tuning and tests (0: not set).
int64_t env_int(const char* name) {
  const char* e = getenv(name);
  return e ? atoll(e) : 0;
}

// Segments and column blocks. A workgroup of the main pass fills a CU and carries one segment of one head; a
// segment's own state, needed when a sequence has more than one, costs it 0.42 of the main pass again. In units of a
// token's time (0.034 us in bf16) the call takes about
//   (rounds of 256 workgroups) x (tokens of a segment + 256) x (1 or 1.42) + (0 or 250 + 8 x segments)
// with the launches and the joining walk last; the segment length with the least is taken. Measured, us (all inputs
// bf16, d = 128, but the third): 4 x 4096 tokens, 16 heads: 1024 tokens 135, 512 154, 2048 169, whole sequences
// 184; 1000 tokens, 4 heads: 128 tokens 23, 256 30, whole 43; 3 x 1333 tokens, 6 heads, fp32, d = 64 / 32: 128 tokens 30, 64 39,
// 256 38, whole 84; 512 tokens, 16 heads: whole 24, 128 tokens 25.
// The backward's state passes take 32 columns per workgroup, two of which share a CU with one for each direction; a
// token takes them 0.012 us in bf16, 0.04 in fp32, which scales the launches' share. 4000 tokens, 4 heads, d = 64,
// bf16: 256 tokens 42, 128 49, 1024 59, whole 81; 4 x 4096, 16 heads, d = 128: whole 593, 2048 664.
// Packed calls are the least known: only the total length is on the host, and neither the join's traffic nor the
// backward's second state pass is in the formula. 12 sequences in 32768 tokens, 16 / 4 heads, d = 128: 307 to 333 at the
// planned 896 tokens, 295 at 1024; backward, 5 sequences in 7777 tokens, 12 / 3 heads, d = 64 / 128: 198 to 210 at the
// planned 576, 173 with whole sequences.
dr::DecayPlan plan_decay(const dr_decay_dims* d, bool packed, bool backward) {
  dr::DecayPlan pl{};
  const int64_t tiles = d->head_dim_v / 16, pairs = d->num_seqs * d->num_heads, T = d->seqlen;
  const bool bf16 = d->in_dtype == DR_BF16;
  // all columns in one workgroup (fp32 data, three times as large, in one or two tiles)
  const int most = bf16 ? (int)tiles : tiles >= 2 && d->head_dim_k < 128 ? 2 : 1;
  const int64_t blocks = backward ? (tiles + 1) / 2 : tiles / most;
  const double start = backward ? 128 : 256, again = !backward ? 1.42 : bf16 ? 2 : 1.65;
  const double launches = backward && bf16 ? 800 : 250, step = backward && bf16 ? 25 : 8;
  int64_t seg = (T + 63) / 64 * 64;
  double best = 0;
  // (the limit on the workgroups of a call that is cut keeps the segments' states within 1 GiB, at d = 128; smaller
  // states and packed calls with many sequences end there far below it. From 16 on not every value of n is tried)
  const auto many = [&](int64_t n) { return (packed ? (n + d->num_seqs) * d->num_heads : n * pairs) * blocks > 16384; };
  for (int64_t n = 1; n == 1 || (n * 128 < T + 128 && !many(n)); n += 1 + n / 16) {
    const int64_t s = ((T + n - 1) / n + 63) / 64 * 64, nseg = s > 0 ? (T + s - 1) / s : 1;
    // (packed lengths are not known here: half a segment per sequence for their ragged ends)
    const double wgs = (packed && s > 0 ? (double)T / s + 0.5 * d->num_seqs : (double)d->num_seqs * nseg) * d->num_heads * blocks;
    // (packed: half a round more than the expected number, which is all that is known)
    double rounds = packed || wgs > 8192 ? wgs / 256 + 0.5 : (double)(int64_t)((wgs + 255) / 256);
    if (rounds < 1) rounds = 1;
    const double cost = rounds * (s + start) * (nseg > 1 ? again : 1.0) + (nseg > 1 ? launches + step * nseg : 0.0);
    if (best == 0 || cost < best) {
      best = cost;
      seg = s;
    }
  }
  if (const int64_t s = env_int("DR_DECAY_SEG"))
    if (s > 0 && s <= INT32_MAX - 63) seg = (s + 63) / 64 * 64;
  if (seg < 64) seg = 64;
  pl.seg = seg;
  pl.nseg = (T + seg - 1) / seg;
  if (pl.nseg < 1) pl.nseg = 1;
  pl.slots = packed ? T / seg + d->num_seqs : d->num_seqs * pl.nseg;
  // fewer columns per workgroup while that still finds idle CUs (a chunk of 16, 32 or 128 columns takes 1.9, 2.6 and 4.2 us)
  pl.ct = most;
  const int64_t heads = packed ? (T / seg + 1) * d->num_heads : pairs * pl.nseg;
  while (pl.ct > 1 && heads * (tiles / pl.ct) < 256 && heads * (tiles / pl.ct) * 2 <= 256) pl.ct /= 2;
  if (const int64_t c = env_int("DR_DECAY_CT"))
    if ((c == 1 || c == 2 || c == 4 || c == 8) && c <= most) pl.ct = (int)c;
  return pl;
}

// A call's workspace: 256-byte aligned pieces one behind the other.
struct Space {
  int64_t size = 0;
  int64_t take(int64_t bytes) {
    const int64_t at = size;
    size += round256(bytes);
    return at;
  }
  // segments: their own states and decays (r: of the reverse pass); packed: tables; backward: states and state
  // gradients at chunk boundaries, shared heads' partial sums, tokens' gradients of a decay per head
  int64_t part, g, rpart, rg, tab, cs, ds, pq, pk, da;
};

Space fwd_space(const dr_decay_dims* d, const dr::DecayPlan& pl, bool packed) {
  Space s{};
  const int64_t nh = pl.slots * d->num_heads;
  if (pl.nseg > 1) {
    s.part = s.take(nh * d->head_dim_k * d->head_dim_v * 4);
    s.g = s.take(nh * 8);
  }
  if (packed) s.tab = s.take((pl.slots + 3 * d->num_seqs + 2) * 4);
  return s;
}

int64_t bwd_slots(const dr_decay_dims* d, bool packed) {
  const int64_t chunk = dr::decay_bwd_chunk(d->in_dtype == DR_BF16);
  return packed ? d->seqlen / chunk + d->num_seqs : d->num_seqs * ((d->seqlen + chunk - 1) / chunk);
}

Space bwd_space(const dr_decay_dims* d, const dr::DecayPlan& pl, bool packed) {
  Space s{};
  const int64_t H = d->num_heads, hsz = d->head_dim_k * d->head_dim_v, tokens = d->batch * d->seqlen;
  const int64_t cslots = bwd_slots(d, packed);
  s.cs = s.take(cslots * H * hsz * 4);
  s.ds = s.take(cslots * H * hsz * 4);
  if (pl.nseg > 1) {
    s.part = s.take(pl.slots * H * hsz * 4);
    s.g = s.take(pl.slots * H * 8);
    s.rpart = s.take(pl.slots * H * hsz * 4);
    s.rg = s.take(pl.slots * H * 8);
  }
  if (d->num_k_heads != H) {
    s.pq = s.take(tokens * H * d->head_dim_k * 4);
    s.pk = s.take(tokens * H * d->head_dim_k * 4);
  }
  if (d->decay_layout == DR_DECAY_HEAD) s.da = s.take(tokens * H * 4);
  if (packed) s.tab = s.take((pl.slots + cslots + 4 * d->num_seqs + 3) * 4);
  return s;
}

}  // namespace

extern "C" {

int dr_decay_workspace(const dr_decay_dims* dims, int packed, int backward, int64_t* bytes) {
  dr::host_clear_error();
  const int32_t some = 0;  // (only whether there are offsets counts)
  const int st = check_dims(dims, packed ? &some : nullptr, false);
  if (st) return st;
  if (bytes == nullptr) return host_fail(DR_ERR_NULL, "`bytes` is NULL");
  const dr::DecayPlan pl = plan_decay(dims, packed != 0, backward != 0);
  *bytes = backward ? bwd_space(dims, pl, packed != 0).size : fwd_space(dims, pl, packed != 0).size;
  return DR_OK;
}

int dr_decay_fwd(const void* q, const void* k, const void* v, const float* alpha, const float* S0,
                 const int32_t* cu_seqlens, float* o, float* S_T, const dr_decay_dims* dims, const dr_opts* opts,
                 void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_dims(dims, cu_seqlens, false);
  if (st) return st;
  if (dims->batch * dims->seqlen > 0) {
    st = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {alpha, "alpha"}}, {{o, "o"}});
    if (st) return st;
  }
  st = check_ptrs({}, {{S0, "S0"}, {S_T, "S_T"}, {cu_seqlens, "cu_seqlens"}});
  if (st) return st;
  st = check_opts(opts, true);
  if (st) return st;
  st = dr::host_check_offsets(cu_seqlens, dims->num_seqs, dims->seqlen, stream);
  if (st) return st;
  if (dims->num_seqs == 0) return DR_OK;
  const bool packed = cu_seqlens != nullptr;
  const dr::DecayPlan pl = plan_decay(dims, packed, false);
  dr::DecayParams p{};
  set_dims(p, dims);
  p.q = q; p.k = k; p.v = v; p.alpha = alpha; p.S0 = S0; p.cu = cu_seqlens; p.o = o; p.S = S_T;
  if (opts) {
    p.sidx = opts->state_idx;
    p.nslots = opts->num_slots;
    p.snap = opts->snapshots;
    p.snap_chunks = opts->snapshots ? (int32_t)(opts->snapshot_every / 64) : 0;
  }
  if (pl.slots * dims->num_heads * (dims->head_dim_v / 16) > INT32_MAX - 8 || pl.seg > INT32_MAX)
    return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  p.seg = (int32_t)pl.seg;
  p.nseg = (int32_t)pl.nseg;
  p.slots = (int32_t)pl.slots;
  if (!dr::decay_fwd_fits(p, pl)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  const Space sp = fwd_space(dims, pl, packed);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("decay prefill", sp.size, workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  if (pl.nseg > 1) {
    p.part = reinterpret_cast<float*>(ws + sp.part);
    p.gpart = reinterpret_cast<double*>(ws + sp.g);
  }
  if (packed) {
    p.slot_seq = reinterpret_cast<int32_t*>(ws + sp.tab);
    p.slot_first = p.slot_seq + pl.slots;
    p.cu_ok = p.slot_first + dims->num_seqs + 1;
    p.snap_first = p.cu_ok + dims->num_seqs + 1;
  }
  const hipError_t e = dr::launch_decay_fwd(p, pl, dims->in_dtype == DR_BF16, stream);
  const hipError_t ef = owned ? hipFreeAsync(ws, stream) : hipSuccess;
  if (e != hipSuccess) return host_fail(DR_ERR_HIP, "decay prefill launch failed: %s", hipGetErrorString(e));
  if (ef != hipSuccess) return host_fail(DR_ERR_HIP, "decay prefill workspace release failed: %s", hipGetErrorString(ef));
  return DR_OK;
}

int dr_decay_step(const void* q, const void* k, const void* v, const float* alpha, float* S, float* o,
                  const dr_decay_dims* dims, const dr_opts* opts, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_dims(dims, nullptr, true);
  if (st) return st;
  st = check_opts(opts, false);
  if (st) return st;
  if (dims->num_seqs == 0) return DR_OK;
  st = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {alpha, "alpha"}, {S, "S"}, {o, "o"}}, {});
  if (st) return st;
  dr::DecayParams p{};
  set_dims(p, dims);
  p.q = q; p.k = k; p.v = v; p.alpha = alpha; p.S = S; p.o = o;
  if (opts) {
    p.sidx = opts->state_idx;
    p.nslots = opts->num_slots;
  }
  if (dims->num_seqs * dims->num_heads * (dims->head_dim_v / 16) > INT32_MAX)
    return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  if (!dr::decay_step_fits(p)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  const hipError_t e = dr::launch_decay_step(p, dims->in_dtype == DR_BF16, stream);
  if (e != hipSuccess) return host_fail(DR_ERR_HIP, "decay step launch failed: %s", hipGetErrorString(e));
  return DR_OK;
}

int dr_decay_bwd(const void* q, const void* k, const void* v, const float* alpha, const float* S0,
                 const int32_t* cu_seqlens, const float* dO, const float* dS_T, float* dq, float* dk, float* dv,
                 float* dalpha, float* dS0, const dr_decay_dims* dims, void* workspace, int64_t workspace_bytes,
                 hipStream_t stream) {
  dr::host_clear_error();
  int st = check_dims(dims, cu_seqlens, false);
  if (st) return st;
  const int64_t tokens = dims->batch * dims->seqlen, H = dims->num_heads, N = dims->num_seqs;
  if (tokens > 0) {
    st = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {alpha, "alpha"}, {dO, "dO"}, {dq, "dq"}, {dk, "dk"}, {dv, "dv"}}, {});
    if (st) return st;
  }
  const bool per_head = dims->decay_layout == DR_DECAY_HEAD;
  if (tokens > 0 || per_head) {
    st = check_ptrs({{dalpha, "dalpha"}}, {});
    if (st) return st;
  }
  st = check_ptrs({}, {{S0, "S0"}, {cu_seqlens, "cu_seqlens"}, {dS_T, "dS_T"}, {dS0, "dS0"}});
  if (st) return st;
  st = dr::host_check_offsets(cu_seqlens, N, dims->seqlen, stream);
  if (st) return st;
  const bool packed = cu_seqlens != nullptr, bf16 = dims->in_dtype == DR_BF16;
  if (N == 0 && !per_head) return DR_OK;
  const dr::DecayPlan pl = plan_decay(dims, packed, true);
  const int64_t chunk = dr::decay_bwd_chunk(bf16);
  const int64_t cslots = bwd_slots(dims, packed);
  if (pl.slots * H * (dims->head_dim_v / 16) > INT32_MAX - 8 || cslots * H > INT32_MAX - 8 || pl.seg > INT32_MAX ||
      tokens * dims->num_k_heads * (dims->head_dim_k / 4) / 256 >= INT32_MAX)
    return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  dr::DecayParams p{};
  set_dims(p, dims);
  p.q = q; p.k = k; p.v = v; p.alpha = alpha; p.S0 = S0; p.cu = cu_seqlens;
  p.dO = dO; p.dST = dS_T; p.dq = dq; p.dk = dk; p.dv = dv; p.dalpha = dalpha; p.dS0 = dS0;
  p.seg = (int32_t)pl.seg;
  p.nseg = (int32_t)pl.nseg;
  p.slots = (int32_t)pl.slots;
  p.cslots = (int32_t)cslots;
  p.bwd_chunk = (int32_t)chunk;
  p.nbatch = (int32_t)dims->batch;
  if (!dr::decay_bwd_fits(p, pl)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  const Space sp = bwd_space(dims, pl, packed);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("decay backward", sp.size, workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  auto f = [&](int64_t off) { return reinterpret_cast<float*>(ws + off); };
  p.cs = f(sp.cs);
  p.ds = f(sp.ds);
  if (pl.nseg > 1) {
    p.part = f(sp.part);
    p.gpart = reinterpret_cast<double*>(ws + sp.g);
    p.rpart = f(sp.rpart);
    p.rgpart = reinterpret_cast<double*>(ws + sp.rg);
  }
  if (dims->num_k_heads != H) {
    p.pq = f(sp.pq);
    p.pk = f(sp.pk);
  }
  if (per_head) {
    p.head_da = dalpha;
    p.dalpha = f(sp.da);
  }
  if (packed) {
    p.slot_seq = reinterpret_cast<int32_t*>(ws + sp.tab);
    p.slot_first = p.slot_seq + pl.slots;
    p.cu_ok = p.slot_first + N + 1;
    p.chunk_first = p.cu_ok + N + 1;
    p.chunk_seq = p.chunk_first + N + 1;
  }
  const hipError_t e = dr::launch_decay_bwd(p, pl, bf16, stream);
  const hipError_t ef = owned ? hipFreeAsync(ws, stream) : hipSuccess;
  if (e != hipSuccess) return host_fail(DR_ERR_HIP, "decay backward launch failed: %s", hipGetErrorString(e));
  if (ef != hipSuccess) return host_fail(DR_ERR_HIP, "decay backward workspace release failed: %s", hipGetErrorString(ef));
  return DR_OK;
}

static int cache_checks(const void* S, const int32_t* state_idx, const void* codes, const float* scales,
                        const int32_t* slot_idx, const dr_cache_dims* d) {
  if (d == nullptr) return host_fail(DR_ERR_NULL, "dims is NULL");
  if (d->format != DR_CACHE_INT8 && d->format != DR_CACHE_E4M3)
    return host_fail(DR_ERR_DTYPE, "format %d is neither DR_CACHE_INT8 nor DR_CACHE_E4M3", d->format);
  if (d->reserved != 0) return host_fail(DR_ERR_SHAPE, "reserved must be 0");
  if (d->count < 0 || d->num_states < 0 || d->num_slots < 0 || d->num_heads < 1)
    return host_fail(DR_ERR_SHAPE, "bad sizes: count=%lld states=%lld slots=%lld heads=%lld", (long long)d->count,
                     (long long)d->num_states, (long long)d->num_slots, (long long)d->num_heads);
  if (!head_dim_ok(d->head_dim_k) || !head_dim_ok(d->head_dim_v))
    return host_fail(DR_ERR_UNSUPPORTED, "head sizes d_k=%lld d_v=%lld: each must be 16, 32, 64 or 128",
                     (long long)d->head_dim_k, (long long)d->head_dim_v);
  if (d->num_states > INT32_MAX || d->num_slots > INT32_MAX || d->num_heads > INT32_MAX || d->count > INT32_MAX ||
      d->count * d->num_heads > INT32_MAX / 4 || !dr::cache_fits(d->count * d->num_heads, (int)(d->head_dim_k * d->head_dim_v)))
    return host_fail(DR_ERR_UNSUPPORTED, "%lld states of %lld heads: too many for one call", (long long)d->count,
                     (long long)d->num_heads);
  if (state_idx == nullptr && d->num_states < d->count)
    return host_fail(DR_ERR_SHAPE, "%lld states for a count of %lld", (long long)d->num_states, (long long)d->count);
  if (slot_idx == nullptr && d->num_slots < d->count)
    return host_fail(DR_ERR_SHAPE, "%lld slots for a count of %lld", (long long)d->num_slots, (long long)d->count);
  int st = DR_OK;
  if (d->count > 0) st = check_ptrs({{S, "S"}, {codes, "codes"}, {scales, "scales"}}, {});
  if (st) return st;
  return check_ptrs({}, {{state_idx, "state_idx"}, {slot_idx, "slot_idx"}});
}

static dr::CacheParams cache_params(const float* S, const int32_t* state_idx, const uint8_t* codes, const float* scales,
                                    const int32_t* slot_idx, const dr_cache_dims* d) {
  dr::CacheParams p{};
  p.S = const_cast<float*>(S);
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<float*>(scales);
  p.state_idx = state_idx;
  p.slot_idx = slot_idx;
  p.count = d->count;
  p.nstates = d->num_states;
  p.nslots = d->num_slots;
  p.H = (int32_t)d->num_heads;
  p.DK = (int32_t)d->head_dim_k;
  p.DV = (int32_t)d->head_dim_v;
  return p;
}

int dr_state_pack(const float* S, const int32_t* state_idx, uint8_t* codes, float* scales, const int32_t* slot_idx,
                  const dr_cache_dims* dims, hipStream_t stream) {
  dr::host_clear_error();
  const int st = cache_checks(S, state_idx, codes, scales, slot_idx, dims);
  if (st || dims->count == 0) return st;
  const hipError_t e = dr::launch_state_pack(cache_params(S, state_idx, codes, scales, slot_idx, dims),
                                             dims->format == DR_CACHE_E4M3, stream);
  if (e != hipSuccess) return host_fail(DR_ERR_HIP, "state pack launch failed: %s", hipGetErrorString(e));
  return DR_OK;
}

int dr_state_unpack(const uint8_t* codes, const float* scales, const int32_t* slot_idx, float* S,
                    const int32_t* state_idx, const dr_cache_dims* dims, hipStream_t stream) {
  dr::host_clear_error();
  const int st = cache_checks(S, state_idx, codes, scales, slot_idx, dims);
  if (st || dims->count == 0) return st;
  const hipError_t e = dr::launch_state_unpack(cache_params(S, state_idx, codes, scales, slot_idx, dims),
                                               dims->format == DR_CACHE_E4M3, stream);
  if (e != hipSuccess) return host_fail(DR_ERR_HIP, "state unpack launch failed: %s", hipGetErrorString(e));
  return DR_OK;
}

}  // extern "C"
