// C ABI of the selective scan, the short convolution and the norm: argument checks, launch planning and dispatch. Every
// check runs on the host before any launch; no device memory is read here.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>

#include "../../include/deltarule_scan.h"
#include "host.hpp"
#include "scan.hpp"

using dr::host_fail;

namespace {

const char* const kTooLarge = "problem too large: more than 2^31 - 1 workgroups or 2^32 - 1 work items per kernel";
constexpr int64_t kTokens = ((int64_t)1 << 31) - 1024, kStride = (int64_t)1 << 40, kTokenStride = (int64_t)1 << 24;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

struct Ptr {
  const void* p;
  const char* name;
  int64_t align;
  bool need;
};
int check_ptrs(std::initializer_list<Ptr> list) {
  for (const Ptr& x : list) {
    if (x.p == nullptr && x.need) return host_fail(DR_ERR_NULL, "`%s` is NULL", x.name);
    if (reinterpret_cast<uintptr_t>(x.p) % (uintptr_t)x.align != 0)
      return host_fail(DR_ERR_LAYOUT, "`%s` is not %d-byte aligned", x.name, (int)x.align);
  }
  return DR_OK;
}
bool aligned16(std::initializer_list<const void*> list) {
  for (const void* p : list)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}
int check_dtype(int32_t t) {
  return t == DR_F32 || t == DR_BF16 ? DR_OK : host_fail(DR_ERR_DTYPE, "in_dtype %d is neither DR_F32 nor DR_BF16", t);
}
int64_t esize(int32_t t) { return t == DR_BF16 ? 2 : 4; }

// Sizes that every call over tokens has (a step: batch = num_seqs, seqlen 1).
int check_tokens(int64_t batch, int64_t seqlen, int64_t channels, int64_t seqs, const void* cu, bool step) {
  if (batch < 0 || seqlen < 0 || channels < 1 || seqs < 0)
    return host_fail(DR_ERR_SHAPE, "bad sizes: batch=%lld seqlen=%lld channels=%lld seqs=%lld", (long long)batch,
                     (long long)seqlen, (long long)channels, (long long)seqs);
  if (channels > (int64_t)1 << 20) return host_fail(DR_ERR_UNSUPPORTED, "%lld channels: at most 2^20", (long long)channels);
  if (batch > kTokens || seqlen > kTokens || seqs > kTokens || (seqlen > 0 && batch > kTokens / seqlen))
    return host_fail(DR_ERR_SHAPE, "problem too large: more than 2^31 - 1024 tokens or sequences");
  if (step) {
    if (seqs != batch || seqlen != 1)
      return host_fail(DR_ERR_SHAPE, "a step has num_seqs equal to batch and seqlen 1, got %lld, %lld and %lld",
                       (long long)seqs, (long long)batch, (long long)seqlen);
  } else if (cu != nullptr) {
    if (batch != 1) return host_fail(DR_ERR_SHAPE, "packed sequences (cu_seqlens) need batch == 1, got %lld", (long long)batch);
  } else if (seqs != batch) {
    return host_fail(DR_ERR_SHAPE, "num_seqs (%lld) must equal batch (%lld) without cu_seqlens", (long long)seqs, (long long)batch);
  }
  return DR_OK;
}
int check_stride(int64_t s, int64_t unit, const char* name, int64_t most = kStride) {
  if (s < 0) return host_fail(DR_ERR_SHAPE, "%s stride %lld is negative", name, (long long)s);
  if (s > most || s % unit != 0)
    return host_fail(DR_ERR_LAYOUT, "%s stride %lld is not a multiple of %lld elements (or is beyond %lld)", name, (long long)s, (long long)unit, (long long)most);
  return DR_OK;
}
int check_opts(const dr_opts* o) {
  if (o == nullptr) return DR_OK;
  if (o->l2norm_qk != 0 || o->alpha_dtype != DR_F32 || o->alpha_act != DR_ACT_NONE || o->gate_act != DR_ACT_NONE)
    return host_fail(DR_ERR_UNSUPPORTED, "these calls take their inputs as they are: no input preparation");
  if (o->snapshots) return host_fail(DR_ERR_UNSUPPORTED, "these calls take no snapshots");
  if (o->state_idx) {
    if (!aligned16({o->state_idx})) return host_fail(DR_ERR_LAYOUT, "state_idx must be 16-byte aligned");
    if (o->num_slots < 0) return host_fail(DR_ERR_SHAPE, "num_slots (%lld) is negative", (long long)o->num_slots);
    if (o->num_slots > INT32_MAX) return host_fail(DR_ERR_UNSUPPORTED, "num_slots above 2^31 - 1");
  }
  return DR_OK;
}
int64_t env_int(const char* name) {
  const char* e = getenv(name);
  return e ? atoll(e) : 0;
}
template <class P>
void set_opts(P& p, const dr_opts* o) {
  if (o == nullptr) return;
  p.sidx = o->state_idx;
  p.nslots = o->num_slots;
}
int done(hipError_t e, const char* what) {
  return e == hipSuccess ? DR_OK : host_fail(DR_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
}
int done(hipError_t e, bool owned, void* ws, hipStream_t stream, const char* what) {
  const hipError_t ef = owned ? hipFreeAsync(ws, stream) : hipSuccess;
  if (e != hipSuccess) return done(e, what);
  return ef == hipSuccess ? DR_OK : host_fail(DR_ERR_HIP, "%s workspace release failed: %s", what, hipGetErrorString(ef));
}

// ------------------------------------------------------------------------------------------------ convolution
int check_conv(const dr_conv_dims* d, const void* cu, bool step) {
  if (d == nullptr) return host_fail(DR_ERR_NULL, "dims is NULL");
  int st = check_dtype(d->in_dtype);
  if (st) return st;
  if (d->activation != DR_CONV_NONE && d->activation != DR_CONV_SILU)
    return host_fail(DR_ERR_UNSUPPORTED, "activation %d is neither DR_CONV_NONE nor DR_CONV_SILU", d->activation);
  if (d->width < 2 || d->width > 4) return host_fail(DR_ERR_UNSUPPORTED, "width %lld: 2, 3 or 4", (long long)d->width);
  st = check_tokens(d->batch, d->seqlen, d->channels, d->num_seqs, cu, step);
  if (!st) st = check_stride(d->x_token_stride, 1, "x token", kTokenStride);
  return st ? st : check_stride(d->x_batch_stride, 1, "x batch");
}
// Vectors of channels need aligned rows; below 32 of them most lanes of a wave would be idle, and single channels do better.
bool conv_vectors(const dr_conv_dims* d, std::initializer_list<const void*> ptrs) {
  const int64_t unit = 16 / esize(d->in_dtype);
  return d->channels % unit == 0 && d->channels >= 32 * unit && d->x_token_stride % unit == 0 && d->x_batch_stride % unit == 0 &&
         aligned16(ptrs);
}
dr::ConvParams conv_params(const dr_conv_dims* d, int64_t vec, bool backward) {
  dr::ConvParams p{};
  p.T = d->seqlen;
  p.x_ts = d->x_token_stride;
  p.x_bs = d->x_batch_stride;
  p.C = (int32_t)d->channels;
  p.nbatch = (int32_t)d->batch;
  p.nseq = (int32_t)d->num_seqs;
  p.silu = d->activation;
  // Alone, bf16 (fp32) outputs of 16 MiB take 11.7 (8.1) us around the caches and 13.5 (9.4) with ordinary stores, 32 MiB 19.0 (13.1) and 21.0
  // (13.0), 64 MiB 27.2 (22.2) and 37.9 (33.4), 128 MiB 58.8 (55.4) and 62.2 (58.8). With a reader of the output behind it 16 MiB 19.0 and
  // 19.6, 32 MiB 35.0 and 34.5, 64 MiB 62.6 and 57.3, 128 MiB 110.7 and 109.6: the reader pays for what the convolution saves.
  p.streamed = d->batch * d->seqlen * d->channels * esize(d->in_dtype) > (int64_t)32 << 20;
  p.cblocks = (int32_t)ceil_div(d->channels, 64 * vec);
  // tokens of a wave: as many as still leave 16 waves to a CU, so that the inputs read twice stay few
  const int64_t most = backward ? 64 : 32;
  int64_t run = 8;
  while (run < most && d->batch * ceil_div(d->seqlen, 2 * run) * p.cblocks >= 4096) run *= 2;
  p.run = (int32_t)run;
  p.runs = (int32_t)ceil_div(d->seqlen, run);
  return p;
}
int64_t conv_blocks(const dr::ConvParams& p) { return ceil_div((int64_t)p.nbatch * p.runs, dr::CONV_WAVES); }
bool conv_fits(const dr::ConvParams& p) {
  return dr::launch_fits((conv_blocks(p) + ceil_div(p.nseq, dr::CONV_WAVES)) * p.cblocks + 8, 64 * dr::CONV_WAVES);
}
// (a run may be as short as 8 tokens and a workgroup's share of the channels as narrow as one vector block)
int64_t conv_space(const dr_conv_dims* d) {
  int64_t most = 0;
  for (const int64_t vec : {(int64_t)1, (int64_t)4}) {
    const dr::ConvParams p = conv_params(d, vec, true);
    const int64_t n = conv_blocks(p) * (d->width + 1) * d->channels * 4;
    if (n > most) most = n;
  }
  return round256(most);
}

// ------------------------------------------------------------------------------------------------ scan
int check_scan(const dr_scan_dims* d, const void* cu, bool step) {
  if (d == nullptr) return host_fail(DR_ERR_NULL, "dims is NULL");
  int st = check_dtype(d->in_dtype);
  if (st) return st;
  if (d->softplus != 0 && d->softplus != 1) return host_fail(DR_ERR_SHAPE, "softplus must be 0 or 1, got %d", d->softplus);
  if (d->state_dim != 16 && d->state_dim != 32 && d->state_dim != 64)
    return host_fail(DR_ERR_UNSUPPORTED, "state_dim %lld: 16, 32 or 64", (long long)d->state_dim);
  if (d->groups > 65536) return host_fail(DR_ERR_UNSUPPORTED, "%lld groups: at most 65536", (long long)d->groups);
  if (d->groups < 1) return host_fail(DR_ERR_SHAPE, "groups (%lld) must be positive", (long long)d->groups);
  st = check_tokens(d->batch, d->seqlen, d->channels, d->num_seqs, cu, step);
  if (st) return st;
  if (d->channels % d->groups != 0)
    return host_fail(DR_ERR_SHAPE, "channels (%lld) are not a multiple of groups (%lld)", (long long)d->channels, (long long)d->groups);
  const int64_t row = 16 / esize(d->in_dtype);
  // (rows of a chunk are reached with 32-bit offsets from its first one)
  const struct { int64_t s, unit, most; const char* name; } strides[] = {
      {d->x_token_stride, 1, kTokenStride, "x token"}, {d->x_batch_stride, 1, kStride, "x batch"},
      {d->dt_token_stride, 1, kTokenStride, "dt token"}, {d->dt_batch_stride, 1, kStride, "dt batch"},
      {d->b_token_stride, row, kTokenStride, "B token"}, {d->b_batch_stride, row, kStride, "B batch"},
      {d->c_token_stride, row, kTokenStride, "C token"}, {d->c_batch_stride, row, kStride, "C batch"},
      {d->z_token_stride, 1, kTokenStride, "z token"}, {d->z_batch_stride, 1, kStride, "z batch"}};
  for (const auto& s : strides) {
    st = check_stride(s.s, s.unit, s.name, s.most);
    if (st) return st;
  }
  return DR_OK;
}

// Segments and kernels, by times in us as measured (bf16, 16 states, with z).
// A wave walks a segment of 32 channels x 16 states: 0.17 a token, also where two share a SIMD for half of the time, and k waves a
// SIMD take 0.85 k times as long. A sequence that is cut costs 0.6 of the main pass again (the segments' own states), what
// 20 tokens of each segment cost, and 8. 1 x 8192 tokens, 2048 channels: segments of 64 171, 128 147, 256 144, 512 169, 1024 306, whole 1396.
// With a workgroup's waves along the tokens the decays are formed once: a workgroup takes 6 for 128 tokens of 32 channels x 16
// states and fills a CU. 4 x 2048 tokens, 2048 channels: 103, in segments 129; 64 x 256 tokens: 213, a wave a sequence 133.
// Backward: 0.62 a token, 0.1 of it again for a cut sequence and what 10 tokens cost. 1 x 8192 tokens, 2048 channels: segments of 64 366,
// 128 323, 256 308, 512 454, whole 5066.
struct ScanCost {
  double token, again;
  double waves;  // of a segment
};
// So many segments as give every SIMD 1 to 8 waves, or whole sequences.
double few_segments(const dr_scan_dims* d, const ScanCost& c, bool packed, double own, int64_t* seg) {
  const int64_t T = d->seqlen;
  // (packed: as many whole segments as the tokens fill, and half of one at each sequence's end)
  const double ends = packed ? 0.5 * d->num_seqs : 0, rows = packed ? 1 : (double)d->num_seqs;
  auto load = [&](double n) {
    const double k = std::ceil((rows * n + ends) * c.waves / 1024);
    return k > 1 ? 0.85 * k : 1.0;
  };
  double best = load(1) * (ceil_div(T, 16) * 16) * c.token;  // (whole tiles: 37 tokens, 2048 channels 11.6, along the tokens 9.2; 24 tokens 8.9, 9.3)
  *seg = ceil_div(T, 8) * 8;
  for (const int k : {1, 2, 3, 4, 6, 8}) {  // so many waves a SIMD
    double n = std::floor((k * 1024 / c.waves - ends) / rows);
    if (n > (double)(T / 16)) n = (double)(T / 16);
    if (n < 2) continue;
    const int64_t s = ceil_div(ceil_div(T, (int64_t)n), 16) * 16;
    const double cost = load(std::ceil((double)T / s)) * (s + own) * c.token * c.again + 8;
    if (cost < best) {
      best = cost;
      *seg = s;
    }
  }
  return best;
}
// A packed row whose sequences' ends alone fill the GPU. The host knows its tokens and the number of its sequences, not their lengths. One of them may
// hold nearly all tokens, so a row that is not cut counts as one walk over all of them, and segments as if every sequence were cut: the
// tokens, and 20 more for each slot, at the rate of a full GPU, one segment behind them, and 0.25 for each step of a join over the
// whole row. Slots: at each sequence's end half a segment, and no fewer than there are sequences.
// 32768 tokens, 2048 channels, 64 sequences: segments of 64 507, 128 456, 256 458, 512 552, 1024 601; backward 1426, 1360, 1359, 1475, 1637.
// 300 sequences, one of them with 20000 tokens: 601, 506, 459, 493, 759, whole 3714; backward 1654, 1536, 1477, 1434, 1528, whole 14979.
// 2000 sequences, none cut: 497, whole 483; backward 2185, whole 1879 (the states' pass forms what a segment sends forward for each).
double many_segments(const dr_scan_dims* d, const ScanCost& c, int64_t* seg) {
  const double T = (double)d->seqlen, n = (double)d->num_seqs;
  double best = std::ceil(T / 16) * 16 * c.token;
  *seg = ceil_div(d->seqlen, 8) * 8;
  for (int64_t s = 16; s < d->seqlen; s *= 2) {
    if (T / s * c.waves > 8192) continue;  // (8 waves a SIMD; more would only add to the join)
    const double slots = std::fmax(n, T / s + 0.5 * n);
    const double cost = (0.85 * (T + 20 * slots) * c.waves / 1024 + s + 20) * c.token * c.again + 0.25 * T / s + 8;
    if (cost < best) {
      best = cost;
      *seg = s;
    }
  }
  return best;
}
dr::ScanPlan plan_scan(const dr_scan_dims* d, bool packed, bool backward) {
  dr::ScanPlan pl{};
  const int64_t T = d->seqlen, SL = d->state_dim / 16, tiles = d->groups * ceil_div(d->channels / d->groups, dr::SCAN_TILE);
  const ScanCost c{backward ? 0.62 : 0.17, backward ? 1.1 : 1.6, (double)(tiles * SL)};
  int64_t seg;
  const bool many = packed && 0.5 * d->num_seqs * c.waves >= 1024;
  const double best = many ? many_segments(d, c, &seg) : few_segments(d, c, packed, backward ? 10 : 20, &seg);
  const int64_t force = env_int("DR_SCAN_BLOCK");  // for tuning and tests: 1 wherever sequences are whole, 2 never
  // (packed: as if each sequence had all tokens, so that a row of several comes here only where it is short)
  const double block = std::ceil((double)d->num_seqs * tiles / 256) * (ceil_div(T * SL, 128) * 6.0 + 1);
  if (!backward && force != 2 && (block < best || force == 1)) {
    pl.block = true;
    seg = ceil_div(T, 8) * 8;
  }
  if (const int64_t s = env_int("DR_SCAN_SEG"))
    if (s > 0 && s <= INT32_MAX - 8) seg = ceil_div(s, 8) * 8;
  if (seg < 8) seg = 8;
  pl.seg = seg;
  pl.nseg = ceil_div(T, seg);
  if (pl.nseg < 1) pl.nseg = 1;
  if (pl.nseg > 1) pl.block = false;
  pl.slots = packed ? T / seg + d->num_seqs : d->num_seqs * pl.nseg;
  return pl;
}
int64_t grad_blocks(const dr_scan_dims* d) { return ceil_div(d->channels / d->groups, dr::scan_grad_channels((int)d->state_dim)); }
// Sizes of all launches of a call.
bool scan_fits(const dr_scan_dims* d, const dr::ScanPlan& pl, bool backward) {
  const int64_t tiles = d->groups * ceil_div(d->channels / d->groups, dr::SCAN_TILE), N = d->state_dim;
  if (pl.slots > INT32_MAX || pl.seg > INT32_MAX) return false;
  if (pl.block && !dr::launch_fits(pl.slots * tiles + 8, 64 * dr::SCAN_BLOCK_WAVES)) return false;
  if (!dr::launch_fits(pl.slots * tiles, (int)(64 * (N / 16))) || !dr::launch_fits(d->num_seqs * ceil_div(d->channels * (N / 4), 256), 256))
    return false;
  return !backward || (dr::launch_fits(pl.slots * d->groups * grad_blocks(d), 256) &&
                       dr::launch_fits(ceil_div(d->batch * d->seqlen * d->groups * 2 * N, 256), 256));
}
// A call's workspace: 256-byte aligned pieces one behind the other.
struct Space {
  int64_t size = 0;
  int64_t take(int64_t bytes) {
    const int64_t at = size;
    size += round256(bytes);
    return at;
  }
  int64_t part, sumd, tab, rpart, ck, ckd, pA, pD, pBC;
};
Space scan_space(const dr_scan_dims* d, const dr::ScanPlan& pl, bool packed, bool backward) {
  Space s{};
  const int64_t C = d->channels, cn = C * d->state_dim;
  if (pl.nseg > 1) {
    s.part = s.take(pl.slots * cn * 4);
    s.sumd = s.take(pl.slots * C * 4);
    if (backward) s.rpart = s.take(pl.slots * cn * 4);
  }
  if (packed) s.tab = s.take((pl.slots + 2 * d->num_seqs + 2) * 4);
  if (backward) {
    const int64_t chunks = dr::scan_chunks(d->seqlen, pl.slots, pl.seg, packed);
    s.ck = s.take(chunks * cn * 4);
    s.ckd = s.take(chunks * C * 4);
    s.pA = s.take(pl.slots * cn * 4);
    s.pD = s.take(pl.slots * C * 8);
    s.pBC = s.take(grad_blocks(d) * d->batch * d->seqlen * d->groups * d->state_dim * 8);
  }
  return s;
}
// Whether the sizes of a workspace stay within 64 bits.
bool scan_space_fits(const dr_scan_dims* d, const dr::ScanPlan& pl, bool packed) {
  const double chunks = packed ? (double)d->seqlen / 8 + 5 * (double)pl.slots : (double)pl.slots * (double)(pl.seg / 8 + 4);
  return chunks * (double)d->channels * (double)d->state_dim * 8 < 4e18 &&
         (double)grad_blocks(d) * (double)d->batch * (double)d->seqlen * (double)d->groups * (double)d->state_dim * 8 < 4e18;
}
dr::ScanParams scan_params(const dr_scan_dims* d) {
  dr::ScanParams p{};
  p.T = d->seqlen;
  p.C = (int32_t)d->channels;
  p.G = (int32_t)d->groups;
  p.Cg = p.C / p.G;
  p.tiles = (int32_t)ceil_div(p.Cg, dr::SCAN_TILE);
  p.cblocks = (int32_t)grad_blocks(d);
  p.nseq = (int32_t)d->num_seqs;
  p.nbatch = (int32_t)d->batch;
  p.softplus = d->softplus;
  p.x_ts = d->x_token_stride; p.x_bs = d->x_batch_stride;
  p.dt_ts = d->dt_token_stride; p.dt_bs = d->dt_batch_stride;
  p.b_ts = d->b_token_stride; p.b_bs = d->b_batch_stride;
  p.c_ts = d->c_token_stride; p.c_bs = d->c_batch_stride;
  p.z_ts = d->z_token_stride; p.z_bs = d->z_batch_stride;
  return p;
}
void set_plan(dr::ScanParams& p, const dr::ScanPlan& pl, const Space& sp, unsigned char* ws, bool packed) {
  p.seg = (int32_t)pl.seg;
  p.nseg = (int32_t)pl.nseg;
  p.slots = (int32_t)pl.slots;
  if (pl.nseg > 1) {
    p.part = reinterpret_cast<float*>(ws + sp.part);
    p.sumd = reinterpret_cast<float*>(ws + sp.sumd);
  }
  if (packed) {
    p.slot_seq = reinterpret_cast<int32_t*>(ws + sp.tab);
    p.slot_first = p.slot_seq + pl.slots;
    p.cu_ok = p.slot_first + p.nseq + 1;
  }
}

// ------------------------------------------------------------------------------------------------ norm
int check_norm(const dr_norm_dims* d) {
  if (d == nullptr) return host_fail(DR_ERR_NULL, "dims is NULL");
  int st = check_dtype(d->in_dtype);
  if (st) return st;
  if (d->out != DR_NORM_VALUES && d->out != DR_NORM_INT8 && d->out != DR_NORM_E4M3)
    return host_fail(DR_ERR_DTYPE, "out %d is none of dr_norm_out", d->out);
  if (d->reserved != 0) return host_fail(DR_ERR_SHAPE, "reserved must be 0");
  if (d->rows < 0 || d->channels < 1)
    return host_fail(DR_ERR_SHAPE, "bad sizes: rows=%lld channels=%lld", (long long)d->rows, (long long)d->channels);
  if (d->channels > dr::NORM_MOST) return host_fail(DR_ERR_UNSUPPORTED, "%lld channels: at most %d", (long long)d->channels, dr::NORM_MOST);
  if (d->rows > kStride) return host_fail(DR_ERR_UNSUPPORTED, "%lld rows: at most 2^40", (long long)d->rows);
  if (!(d->eps >= 0) || std::isinf(d->eps)) return host_fail(DR_ERR_SHAPE, "eps must be finite and not negative");
  st = check_stride(d->x_row_stride, 1, "x row");
  return st ? st : check_stride(d->residual_row_stride, 1, "residual row");
}
dr::NormParams norm_params(const dr_norm_dims* d, bool backward) {
  dr::NormParams p{};
  p.rows = d->rows;
  p.C = (int32_t)d->channels;
  p.x_rs = d->x_row_stride;
  p.r_rs = d->residual_row_stride;
  p.eps = d->eps;
  const bool few = dr::norm_few(d->rows, d->channels, backward);
  p.few = few;
  // (two for each CU keep the backward's sums few)
  p.nwg = (int32_t)dr::norm_groups(d->rows, d->channels, few, backward ? 512 : 2048);
  return p;
}

}  // namespace

extern "C" {

int dr_conv_fwd(const void* x, const float* weight, const float* bias, const void* state, const int32_t* cu_seqlens,
                void* y, void* state_T, const dr_conv_dims* dims, const dr_opts* opts, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_conv(dims, cu_seqlens, false);
  if (!st) st = check_opts(opts);
  if (st) return st;
  const int64_t e = esize(dims->in_dtype), tokens = dims->batch * dims->seqlen;
  st = check_ptrs({{x, "x", e, tokens > 0}, {weight, "weight", 16, true}, {bias, "bias", 16, false}, {state, "state", e, false},
                   {cu_seqlens, "cu_seqlens", 16, false}, {y, "y", e, tokens > 0}, {state_T, "state_T", e, false}});
  if (!st) st = dr::host_check_offsets(cu_seqlens, dims->num_seqs, dims->seqlen, stream);
  if (st || dims->num_seqs == 0) return st;
  const bool bf16 = dims->in_dtype == DR_BF16, vec = conv_vectors(dims, {x, state, y, state_T});
  dr::ConvParams p = conv_params(dims, dr::conv_vec(bf16, vec, false), false);
  if (!conv_fits(p)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  set_opts(p, opts);
  p.x = x; p.w = weight; p.bias = bias; p.state = state; p.cu = cu_seqlens; p.y = y; p.state_T = state_T;
  return done(dr::launch_conv_fwd(p, (int)dims->width, bf16, vec, stream), "convolution");
}

int dr_conv_step(const void* x, const float* weight, const float* bias, void* state, void* y, const dr_conv_dims* dims,
                 const dr_opts* opts, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_conv(dims, nullptr, true);
  if (!st) st = check_opts(opts);
  if (st || dims->num_seqs == 0) return st;
  const int64_t e = esize(dims->in_dtype);
  st = check_ptrs({{x, "x", e, true}, {weight, "weight", 16, true}, {bias, "bias", 16, false}, {state, "state", e, true}, {y, "y", e, true}});
  if (st) return st;
  const bool bf16 = dims->in_dtype == DR_BF16, vec = conv_vectors(dims, {x, state, y});
  dr::ConvParams p = conv_params(dims, dr::conv_vec(bf16, vec, false), false);
  if (!dr::launch_fits(ceil_div(p.nseq, dr::CONV_WAVES) * p.cblocks, 256)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  p.run = 1;
  // sequences of a wave: 512 x 4096 channels, bf16: 1 13.1 us, 2 9.9, 4 9.1, 8 11.5; 64 sequences: 4.7, 5.1, 6.3, 8.5
  while (p.run < 8 && (int64_t)p.nseq * p.cblocks >= 2048 * p.run) p.run *= 2;
  set_opts(p, opts);
  p.x = x; p.w = weight; p.bias = bias; p.state_T = state; p.y = y;
  return done(dr::launch_conv_step(p, (int)dims->width, bf16, vec, stream), "convolution step");
}

int dr_conv_workspace(const dr_conv_dims* dims, int packed, int64_t* bytes) {
  dr::host_clear_error();
  const int32_t some = 0;  // (only whether there are offsets counts)
  const int st = check_conv(dims, packed ? &some : nullptr, false);
  if (st) return st;
  if (bytes == nullptr) return host_fail(DR_ERR_NULL, "`bytes` is NULL");
  *bytes = conv_space(dims);
  return DR_OK;
}

int dr_conv_bwd(const void* x, const float* weight, const float* bias, const void* state, const int32_t* cu_seqlens,
                const void* dy, const void* dstate_T, void* dx, float* dweight, float* dbias, void* dstate,
                const dr_conv_dims* dims, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_conv(dims, cu_seqlens, false);
  if (st) return st;
  const int64_t e = esize(dims->in_dtype), tokens = dims->batch * dims->seqlen;
  st = check_ptrs({{x, "x", e, tokens > 0}, {weight, "weight", 16, true}, {bias, "bias", 16, false}, {state, "state", e, false},
                   {cu_seqlens, "cu_seqlens", 16, false}, {dy, "dy", e, tokens > 0}, {dstate_T, "dstate_T", e, false},
                   {dx, "dx", e, tokens > 0}, {dweight, "dweight", 16, true}, {dbias, "dbias", 16, false}, {dstate, "dstate", e, false}});
  if (!st) st = dr::host_check_offsets(cu_seqlens, dims->num_seqs, dims->seqlen, stream);
  if (st) return st;
  const bool bf16 = dims->in_dtype == DR_BF16, vec = conv_vectors(dims, {x, state, dy, dstate_T, dx, dstate});
  dr::ConvParams p = conv_params(dims, dr::conv_vec(bf16, vec, true), true);
  if (dims->num_seqs == 0) p.runs = 0;  // (the weights' gradients are zeros)
  if (!conv_fits(p)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("convolution backward", conv_space(dims), workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  p.x = x; p.w = weight; p.bias = bias; p.state = state; p.cu = cu_seqlens; p.dy = dy; p.dstate_T = dstate_T;
  p.dx = dx; p.dw = dweight; p.db = dbias; p.dstate = dstate;
  p.part = reinterpret_cast<float*>(ws);
  return done(dr::launch_conv_bwd(p, (int)dims->width, bf16, vec, stream), owned, ws, stream, "convolution backward");
}

int dr_scan_workspace(const dr_scan_dims* dims, int packed, int backward, int64_t* bytes) {
  dr::host_clear_error();
  const int32_t some = 0;
  const int st = check_scan(dims, packed ? &some : nullptr, false);
  if (st) return st;
  if (bytes == nullptr) return host_fail(DR_ERR_NULL, "`bytes` is NULL");
  const dr::ScanPlan pl = plan_scan(dims, packed != 0, backward != 0);
  if (!scan_space_fits(dims, pl, packed != 0)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  *bytes = scan_space(dims, pl, packed != 0, backward != 0).size;
  return DR_OK;
}

int dr_scan_fwd(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                const void* z, const float* dt_bias, const float* S0, const int32_t* cu_seqlens, void* y, float* S_T,
                const dr_scan_dims* dims, const dr_opts* opts, void* workspace, int64_t workspace_bytes,
                hipStream_t stream) {
  dr::host_clear_error();
  int st = check_scan(dims, cu_seqlens, false);
  if (!st) st = check_opts(opts);
  if (st) return st;
  const int64_t e = esize(dims->in_dtype);
  const bool some = dims->batch * dims->seqlen > 0, packed = cu_seqlens != nullptr;
  st = check_ptrs({{x, "x", e, some}, {dt, "dt", e, some}, {A, "A", 16, true}, {B, "B", 16, some}, {C, "C", 16, some},
                   {D, "D", 16, false}, {z, "z", e, false}, {dt_bias, "dt_bias", 16, false}, {S0, "S0", 16, false},
                   {cu_seqlens, "cu_seqlens", 16, false}, {y, "y", e, some}, {S_T, "S_T", 16, false}});
  if (!st) st = dr::host_check_offsets(cu_seqlens, dims->num_seqs, dims->seqlen, stream);
  if (st || dims->num_seqs == 0) return st;
  const dr::ScanPlan pl = plan_scan(dims, packed, false);
  if (!scan_fits(dims, pl, false) || !scan_space_fits(dims, pl, packed)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  const Space sp = scan_space(dims, pl, packed, false);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("selective scan", sp.size, workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  dr::ScanParams p = scan_params(dims);
  set_opts(p, opts);
  set_plan(p, pl, sp, ws, packed);
  p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = dt_bias; p.S0 = S0; p.cu = cu_seqlens;
  p.y = y; p.S = S_T;
  return done(dr::launch_scan_fwd(p, pl, (int)dims->state_dim, dims->in_dtype == DR_BF16, stream), owned, ws, stream, "selective scan");
}

int dr_scan_step(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                 const void* z, const float* dt_bias, float* S, void* y, const dr_scan_dims* dims, const dr_opts* opts,
                 hipStream_t stream) {
  dr::host_clear_error();
  int st = check_scan(dims, nullptr, true);
  if (!st) st = check_opts(opts);
  if (st || dims->num_seqs == 0) return st;
  const int64_t e = esize(dims->in_dtype);
  st = check_ptrs({{x, "x", e, true}, {dt, "dt", e, true}, {A, "A", 16, true}, {B, "B", 16, true}, {C, "C", 16, true},
                   {D, "D", 16, false}, {z, "z", e, false}, {dt_bias, "dt_bias", 16, false}, {S, "S", 16, true}, {y, "y", e, true}});
  if (st) return st;
  const int64_t groups = dims->num_seqs * ceil_div(dims->channels, dr::scan_step_channels((int)dims->state_dim));
  if (!dr::launch_fits(groups, 256))
    return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  dr::ScanParams p = scan_params(dims);
  set_opts(p, opts);
  // sequences of a workgroup: 512 x 4096 channels, 16 states: 1 64.8 us, 2 52.6, 4 51.1, 8 53.1; 8 sequences: 3.2, 3.6, 4.4, 6.0
  p.run = 1;
  while (p.run < dr::SCAN_STEP_RUN && groups >= 4096 * p.run) p.run *= 2;
  p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = dt_bias; p.S = S; p.y = y;
  return done(dr::launch_scan_step(p, (int)dims->state_dim, dims->in_dtype == DR_BF16, stream), "selective scan step");
}

int dr_scan_bwd(const void* x, const void* dt, const float* A, const void* B, const void* C, const float* D,
                const void* z, const float* dt_bias, const float* S0, const int32_t* cu_seqlens, const void* dy,
                const float* dS_T, void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz,
                float* ddt_bias, float* dS0, const dr_scan_dims* dims, void* workspace, int64_t workspace_bytes,
                hipStream_t stream) {
  dr::host_clear_error();
  int st = check_scan(dims, cu_seqlens, false);
  if (st) return st;
  const int64_t e = esize(dims->in_dtype);
  const bool some = dims->batch * dims->seqlen > 0, packed = cu_seqlens != nullptr;
  st = check_ptrs({{x, "x", e, some}, {dt, "dt", e, some}, {A, "A", 16, true}, {B, "B", 16, some}, {C, "C", 16, some},
                   {D, "D", 16, false}, {z, "z", e, false}, {dt_bias, "dt_bias", 16, false}, {S0, "S0", 16, false},
                   {cu_seqlens, "cu_seqlens", 16, false}, {dy, "dy", e, some}, {dS_T, "dS_T", 16, false},
                   {dx, "dx", e, some}, {ddt, "ddt", e, some}, {dA, "dA", 16, true}, {dB, "dB", e, some}, {dC, "dC", e, some},
                   {dD, "dD", 16, D != nullptr}, {dz, "dz", e, some && z != nullptr}, {ddt_bias, "ddt_bias", 16, dt_bias != nullptr},
                   {dS0, "dS0", 16, false}});
  if (!st) st = dr::host_check_offsets(cu_seqlens, dims->num_seqs, dims->seqlen, stream);
  if (st) return st;
  const dr::ScanPlan pl = plan_scan(dims, packed, true);
  if (!scan_fits(dims, pl, true) || !scan_space_fits(dims, pl, packed)) return host_fail(DR_ERR_UNSUPPORTED, kTooLarge);
  const Space sp = scan_space(dims, pl, packed, true);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("selective scan backward", sp.size, workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  dr::ScanParams p = scan_params(dims);
  set_plan(p, pl, sp, ws, packed);
  auto f = [&](int64_t off) { return reinterpret_cast<float*>(ws + off); };
  if (pl.nseg > 1) p.rpart = f(sp.rpart);
  p.ck = f(sp.ck); p.ckd = f(sp.ckd); p.pA = f(sp.pA); p.pD = f(sp.pD); p.pBC = f(sp.pBC);
  p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = dt_bias; p.S0 = S0; p.cu = cu_seqlens;
  p.dy = dy; p.dST = dS_T; p.dx = dx; p.ddt = ddt; p.dA = dA; p.dB = dB; p.dC = dC; p.dD = D ? dD : nullptr;
  p.dz = dz; p.dbias = dt_bias ? ddt_bias : nullptr; p.dS0 = dS0;
  return done(dr::launch_scan_bwd(p, (int)dims->state_dim, dims->in_dtype == DR_BF16, stream), owned, ws, stream, "selective scan backward");
}

int dr_norm_fwd(const void* x, const void* residual, const float* weight, void* y, float* scales, void* h,
                const dr_norm_dims* dims, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_norm(dims);
  if (st || dims->rows == 0) return st;
  const int64_t e = esize(dims->in_dtype);
  const bool codes = dims->out != DR_NORM_VALUES;
  st = check_ptrs({{x, "x", e, true}, {residual, "residual", e, false}, {weight, "weight", 16, true}, {y, "y", codes ? 1 : e, true},
                   {scales, "scales", 16, codes}, {h, "h", e, false}});
  if (st) return st;
  if (residual == nullptr && h != nullptr) return host_fail(DR_ERR_SHAPE, "h is the sum with a residual: there is none");
  if (!codes && scales != nullptr) return host_fail(DR_ERR_SHAPE, "scales are an output of the 8-bit formats");
  const int64_t unit = 16 / e;
  const bool vec = dims->channels % unit == 0 && dims->x_row_stride % unit == 0 &&
                   (residual == nullptr || dims->residual_row_stride % unit == 0) && aligned16({x, residual, y, h});
  dr::NormParams p = norm_params(dims, false);
  p.x = x; p.r = residual; p.w = weight; p.y = y; p.scales = scales; p.h = h;
  return done(dr::launch_norm_fwd(p, dims->out, dims->in_dtype == DR_BF16, vec, stream), "norm");
}

int dr_norm_workspace(const dr_norm_dims* dims, int64_t* bytes) {
  dr::host_clear_error();
  const int st = check_norm(dims);
  if (st) return st;
  if (bytes == nullptr) return host_fail(DR_ERR_NULL, "`bytes` is NULL");
  *bytes = round256((int64_t)norm_params(dims, true).nwg * dims->channels * 4);
  return DR_OK;
}

int dr_norm_bwd(const void* h, const float* weight, const void* dy, const void* dh, void* dx, float* dweight,
                const dr_norm_dims* dims, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  dr::host_clear_error();
  int st = check_norm(dims);
  if (st) return st;
  if (dims->out != DR_NORM_VALUES) return host_fail(DR_ERR_UNSUPPORTED, "the 8-bit outputs have no gradient");
  const int64_t e = esize(dims->in_dtype);
  const bool some = dims->rows > 0;
  st = check_ptrs({{h, "h", e, some}, {weight, "weight", 16, true}, {dy, "dy", e, some}, {dh, "dh", e, false}, {dx, "dx", e, some},
                   {dweight, "dweight", 16, true}});
  if (st) return st;
  dr::NormParams p = norm_params(dims, true);
  unsigned char* ws = nullptr;
  bool owned = false;
  st = dr::host_space("norm backward", round256((int64_t)p.nwg * p.C * 4), workspace, workspace_bytes, 16, stream, &ws, &owned);
  if (st) return st;
  const int64_t unit = 16 / e;
  const bool vec = dims->channels % unit == 0 && dims->x_row_stride % unit == 0 && aligned16({h, dy, dh, dx});
  p.x = h; p.w = weight; p.dy = dy; p.dh = dh; p.dx = dx; p.dw = dweight;
  p.part = reinterpret_cast<float*>(ws);
  return done(dr::launch_norm_bwd(p, dims->in_dtype == DR_BF16, vec, stream), owned, ws, stream, "norm backward");
}

}  // extern "C"
