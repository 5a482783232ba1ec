// C ABI entry points of the attention with modified scores (declared in
// include/mcs.h): host-side validation, workspace layout and launches.
#include <math.h>

#include <algorithm>
#include <cmath>

#include "mcs_internal.h"

using namespace mcs;

namespace {

constexpr int kMaxGroup = 128;            // query heads of one KV head: one 128-row tile holds a token's
constexpr int kMaxDocQueryTiles = 1 << 16;  // tiles of a document mask's bitmaps: over query tiles
constexpr int kMaxDocKeyTiles = 1 << 12;    // and over key tiles (the dQ kernel has 1 KB left for it)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t align256(size_t x) { return (x + 255) / 256 * 256; }
bool finite(float x) { return x == x && !isinf(x); }

mcs_status check_heads(int Hq, int Hkv, int d, float scale, float cap) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1) return MCS_ERR_INVALID_ARG;
  if (!finite(scale) || (scale > 0.f && (scale < 1e-12f || scale > 1e12f))) return MCS_ERR_INVALID_ARG;
  if (!finite(cap) || cap < 0.f || (cap > 0.f && cap < 1e-6f) || cap > 1e20f) return MCS_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MCS_ERR_UNSUPPORTED;
  if (Hq / Hkv > kMaxGroup) return MCS_ERR_UNSUPPORTED;
  return MCS_OK;
}

mcs_status check_attn(const mcs_attn_shape* s) {
  if (!s || s->B < 1 || s->Nq < 1 || s->Nk < 1) return MCS_ERR_INVALID_ARG;
  if ((s->flags & ~(MCS_ATTN_CAUSAL | MCS_ATTN_D_FROM_O)) != 0) return MCS_ERR_INVALID_ARG;
  const mcs_status st = check_heads(s->Hq, s->Hkv, s->d, s->scale, s->cap);
  if (st != MCS_OK) return st;
  if (static_cast<long long>(s->B) * s->Nq >= (1ll << 31) / s->Hq ||
      static_cast<long long>(s->B) * s->Nk >= (1ll << 31) / s->Hkv)
    return MCS_ERR_INVALID_ARG;
  return MCS_OK;
}

mcs_status check_opts(const mcs_attn_shape* s, const mcs_attn_opts* o) {
  if (!o) return MCS_OK;
  if (!aligned4(o->slopes) || !aligned4(o->prefix) || !aligned4(o->doc_q) || !aligned4(o->doc_k))
    return MCS_ERR_INVALID_ARG;
  if (o->prefix && !(s->flags & MCS_ATTN_CAUSAL)) return MCS_ERR_INVALID_ARG;
  if ((o->doc_q == nullptr) != (o->doc_k == nullptr)) return MCS_ERR_INVALID_ARG;
  if (o->doc_q) {
    const int tokens = 128 / (s->Hq / s->Hkv);
    if ((static_cast<long long>(s->Nk) + 127) / 128 > kMaxDocKeyTiles ||
        (static_cast<long long>(s->Nq) + tokens - 1) / tokens > kMaxDocQueryTiles)
      return MCS_ERR_UNSUPPORTED;
  }
  return MCS_OK;
}

float scale_of(float scale, int d) { return scale > 0.f ? scale : static_cast<float>(1.0 / sqrt(static_cast<double>(d))); }

CapFn cap_fn(float scale, float cap) {
  CapFn f{};
  const double ratio = static_cast<double>(scale) / cap, cl = cap * 1.4426950408889634074;
  if (!(cap > 0.f)) return f;
  f.on = 1;
  f.cl = static_cast<float>(cl);
  f.icl = static_cast<float>(1.0 / cl);
  const double p3[5] = {1.0, kTanhP0, kTanhP1, kTanhP2, kTanhP3}, p2[4] = {1.0, kTanhR0, kTanhR1, kTanhR2};
  auto coefficients = [&](double pre) {  // false: one of them is no normal fp32 number
    const double k = ratio / pre;
    f.pre = static_cast<float>(pre);
    f.k2 = static_cast<float>(2.0 * k * 1.4426950408889634074);
    f.z2 = static_cast<float>((0.4 / k) * (0.4 / k));
    f.z3 = static_cast<float>((0.625 / k) * (0.625 / k));
    bool normal = std::isfinite(f.z3);
    double pow = cl * k;
    for (int i = 0; i < 5; ++i, pow *= k * k) {
      f.a[i] = static_cast<float>(p3[i] * pow);
      normal = normal && std::isnormal(f.a[i]);
      if (i < 4) f.b[i] = static_cast<float>(p2[i] * pow);
    }
    return normal;
  };
  if (!coefficients(1.0)) coefficients(ldexp(1.0, ilogb(ratio) + 1));
  return f;
}

ExParams ex_params(const mcs_attn_shape* s, const mcs_attn_opts* o) {
  ExParams p{};
  p.B = s->B; p.Hq = s->Hq; p.Hkv = s->Hkv; p.g = s->Hq / s->Hkv; p.Nq = s->Nq; p.Nk = s->Nk;
  p.scale = scale_of(s->scale, s->d);
  p.cap = s->cap;
  p.causal = (s->flags & MCS_ATTN_CAUSAL) != 0;
  if (o) {
    p.slopes = o->slopes;
    p.prefix = o->prefix;
    p.doc_q = o->doc_q;
    p.doc_k = o->doc_k;
  }
  return p;
}

// How the forward fills the GPU: tiles, key splits and the order of work.
struct FwdPlan {
  int tpt, Tq, Tk, single, nsplit, chunk;
};

// A CTA takes two query tiles that share their key tiles, or one (single), half
// of its keys to each slot. While a wave has room the keys are split further and
// a second launch joins the parts, in about three steps' time (a step, one key
// tile per slot, takes 2 us). The shorter of the two counts of steps wins: with 8
// heads of 1024 tokens, d = 128, single takes 15.7 us where pairs take 20.7.
// Pairs win a tie, since they read K and V half as often: 12 heads of 390
// queries over 32760 keys take 98.5 us in pairs, 101.6 single. Where single tiles
// are more than a wave, they have to take at most three quarters of the steps:
// waves blend into one another and twice the loads show. (d = 128, heads x
// queries x keys, single and pairs: half the steps, 40 x 868 x 2048: 51 and 76 us;
// three quarters, 64 x 740 x 2048: 74 and 81; 0.83, 100 x 740 x 740: 69 and 62;
// 0.97, 100 x 1124 x 1124: 121 and 106.) A causal mask without a long context
// before the queries makes the jobs' lengths differ, which blends them more: 24 x
// 2020 x 2020, three quarters: 50 and 43.5; pairs, then.
constexpr int kJoinSteps = 3;

FwdPlan fwd_plan(int B, int Hkv, int g, int Nq, int Nk, int d, bool causal) {
  FwdPlan f;
  f.tpt = 128 / g;
  f.Tq = (Nq + f.tpt - 1) / f.tpt;
  f.Tk = (Nk + 127) / 128;
  const long long heads = static_cast<long long>(B) * Hkv;
  // steps of the slowest SM, and the splits that lead there
  auto cost = [&](bool single, int* nsplit) {
    const long long ctas = heads * (single ? f.Tq : (f.Tq + 1) / 2);
    const int steps = single ? (f.Tk + 1) / 2 : f.Tk;
    *nsplit = static_cast<int>(std::max(1ll, std::min<long long>(kSms / ctas, steps)));
    const int each = (steps + *nsplit - 1) / *nsplit;
    if (steps - each < kJoinSteps) *nsplit = 1;
    return (ctas * *nsplit + kSms - 1) / kSms * (*nsplit > 1 ? each + kJoinSteps : steps);
  };
  int one = 1;
  const long long pairs = cost(false, &f.nsplit);
  const long long ones = cost(true, &one);
  const bool even = !causal || Nk / 2 >= Nq;
  f.single = heads * f.Tq <= kSms ? ones < pairs : even && 4 * ones <= 3 * pairs;
  if (f.single) f.nsplit = one;
  // K and V of a chunk's heads take half of the 126 MB L2 at most
  const size_t head = static_cast<size_t>(Nk) * d * 4;
  const long long fit = static_cast<long long>((size_t(64) << 20) / head);
  f.chunk = static_cast<int>(std::max(1ll, std::min<long long>(fit, static_cast<long long>(B) * Hkv)));
  return f;
}

// Jobs of a document mask: their order matters where there are more than SMs;
// its entries, four times a job's number, are 32-bit.
bool order_matters(long long jobs) { return jobs > kSms && jobs < (1ll << 28); }

// workspace: status | document tiles | partials of the key splits
struct FwdWs {
  size_t k_ids, k_ranges, q_ranges, order, counts, part_lse, part_o, total;
};

FwdWs fwd_layout(const FwdPlan& f, int B, int Hkv, int d) {
  FwdWs w;
  size_t off = MCS_STATUS_BYTES;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  w.k_ids = take(static_cast<size_t>(B) * f.Tk * 512);
  w.k_ranges = take(static_cast<size_t>(B) * f.Tk * 16);
  w.q_ranges = take(static_cast<size_t>(B) * f.Tq * 16);
  w.order = take(static_cast<size_t>(B) * f.Tq * 4 + 4);
  w.counts = take(static_cast<size_t>(B) * f.Tq * 16);
  const size_t rows = f.nsplit > 1 ? static_cast<size_t>(f.nsplit) * B * Hkv * f.Tq * 128 : 0;
  w.part_lse = take(rows * 4);
  w.part_o = take(rows * d * 4);
  w.total = off;
  return w;
}

// workspace: status | document tiles | statistics of the packed rows
struct BwdWs {
  size_t k_ids, k_ranges, q_ids, q_ranges, order, k_order, counts, stats, part_kv, total;
  int kv_splits;
};

// A key tile's CTA sweeps all Tq query tiles (1.6 us each, 1.5 times as long as
// a query CTA's key tile). Its sweep is split among several CTAs where they fit
// the first wave and save at least five tiles' time (joining the parts costs
// about 5 us), or where it would last twice an SM's share of the whole (many
// query heads to a KV head).
int kv_splits(const FwdPlan& f, int B, int Hkv) {
  const long long heads = static_cast<long long>(B) * Hkv, keys = heads * f.Tk, queries = heads * f.Tq;
  if (keys + queries < kSms) {
    const int most = static_cast<int>(std::min<long long>({(kSms - queries) / keys, f.Tq / 2, 16}));
    return most > 1 && f.Tq - f.Tq / most >= 5 ? most : 1;
  }
  const double sweep = 1.5 * f.Tq, share = static_cast<double>(keys) * (1.5 + 1.0) * f.Tq / kSms;
  return sweep > 2 * share ? std::min({static_cast<int>(ceil(sweep / share)), f.Tq / 2, 16}) : 1;
}

BwdWs bwd_layout(const FwdPlan& f, int B, int Hkv, int Nk, int d) {
  BwdWs w;
  size_t off = MCS_STATUS_BYTES;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  w.k_ids = take(static_cast<size_t>(B) * f.Tk * 512);
  w.k_ranges = take(static_cast<size_t>(B) * f.Tk * 16);
  w.q_ids = take(static_cast<size_t>(B) * f.Tq * 512);
  w.q_ranges = take(static_cast<size_t>(B) * f.Tq * 16);
  w.order = take(static_cast<size_t>(B) * f.Tq * 4 + 4);
  w.k_order = take(static_cast<size_t>(B) * f.Tk * 4 + 4);
  w.counts = take(static_cast<size_t>(B) * (f.Tq + f.Tk) * 16);
  w.stats = take(static_cast<size_t>(B) * Hkv * f.Tq * 1024);
  w.kv_splits = kv_splits(f, B, Hkv);
  w.part_kv = take(w.kv_splits > 1 ? static_cast<size_t>(w.kv_splits) * 2 * B * Nk * Hkv * d * 4 : 0);
  w.total = off;
  return w;
}

ExTile tile_params(const ExParams& p, const FwdPlan& f, int d) {
  ExTile t{};
  t.B = p.B; t.Hq = p.Hq; t.Hkv = p.Hkv; t.g = p.g; t.tpt = f.tpt; t.Nq = p.Nq; t.Nk = p.Nk;
  t.Tq = f.Tq; t.Tk = f.Tk;
  t.nsplit = f.nsplit; t.single = f.single; t.chunk = f.chunk;
  t.scale = p.scale;
  t.cap = cap_fn(p.scale, p.cap);
  t.mul = t.cap.on ? 1.f : static_cast<float>(p.scale * 1.4426950408889634074);
  t.causal = p.causal;
  t.slopes = p.slopes;
  t.prefix = p.prefix;
  t.doc_q = p.doc_q;
  t.doc_k = p.doc_k;
  t.status = p.status;
  t.wait_limit_ns = kWaitLimitNs;
  t.debug_flags = debug_flags();
  return t;
}

mcs_status ok_or_cuda(cudaError_t e) { return e == cudaSuccess ? MCS_OK : MCS_ERR_CUDA; }

mcs_status check_decode(const mcs_decode_shape* s) {
  if (!s || s->B < 1 || s->C < 1 || s->P < 0) return MCS_ERR_INVALID_ARG;
  const mcs_status st = check_heads(s->Hq, s->Hkv, s->d, s->scale, s->cap);
  if (st != MCS_OK) return st;
  if (static_cast<long long>(s->B) * s->C >= (1ll << 31) / s->Hkv || s->P >= (1ll << 31) / s->Hkv ||
      static_cast<long long>(s->B) * s->Hq >= (1ll << 31) || static_cast<long long>(s->P) + s->C >= (1ll << 31))
    return MCS_ERR_INVALID_ARG;
  return MCS_OK;
}

// How single tokens fill the GPU. Two CTAs to an SM; the keys are cut so that
// about eight waves of them cover the batch (lengths differ, and a late long
// request should not run alone), in chunks of at least 512 keys, less only
// where the batch would not fill one wave. A single request has nothing to be
// balanced against: its length, whatever the cache could hold, is cut into the
// fewest waves that leave less than 3 % of the slots empty (75600 keys, d = 128:
// 8 KV heads 57 us, 64 in chunks of 512; 40 KV heads in three waves 239, in one,
// as clusters of 7 that do not pack into it, 340). Chunks of up to 512 keys fill
// one wave as far as they go.
struct DecodePlan {
  int gsplit, chunk, nsplit, cluster;
  FwdPlan pre;
};

DecodePlan decode_plan(const mcs_decode_shape* s) {
  DecodePlan f{};
  const int g = s->Hq / s->Hkv;
  f.gsplit = (g + 31) / 32;
  const long long jobs = static_cast<long long>(s->B) * s->Hkv * f.gsplit, slots = 2 * kSms;
  auto cut = [&](long long ctas) {  // chunk for about `ctas` CTAs, whole blocks of the four warps
    const long long per_job = std::max(1ll, ctas / jobs);
    return ((s->C + per_job - 1) / per_job + 63) / 64 * 64;
  };
  if (s->B == 1) {
    int waves = 1;
    while (waves < 8 && cut(slots) > 512 && 100 * (waves * slots / jobs * jobs) < 97 * waves * slots) ++waves;
    f.chunk = static_cast<int>(std::max(64ll, cut(waves * slots)));
  } else {
    f.chunk = static_cast<int>(std::max(64ll, std::max(cut(8 * slots), std::min(512ll, cut(slots)))));
  }
  f.nsplit = (s->C + f.chunk - 1) / f.chunk;
  f.cluster = s->P == 0 && f.nsplit > 1 && f.nsplit <= 8 && f.chunk <= 512 && jobs * f.nsplit <= slots;
  if (s->P > 0) f.pre = fwd_plan(1, s->Hkv, g, s->B, s->P, s->d, false);
  return f;
}

// workspace: status | parts of the cache's keys | parts of the prefix
struct DecodeWs {
  size_t part_lse, part_o, pre_lse, pre_o, total;
};

DecodeWs decode_layout(const DecodePlan& f, const mcs_decode_shape* s) {
  DecodeWs w;
  size_t off = MCS_STATUS_BYTES;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const bool parts = (f.nsplit > 1 && !f.cluster) || s->P > 0;
  const size_t rows = parts ? static_cast<size_t>(s->B) * s->Hq * f.nsplit : 0;
  const size_t pre = s->P > 0 ? static_cast<size_t>(f.pre.nsplit) * s->Hkv * f.pre.Tq * 128 : 0;
  w.part_lse = take(rows * 4);
  w.part_o = take(rows * s->d * 4);
  w.pre_lse = take(pre * 4);
  w.pre_o = take(pre * s->d * 4);
  w.total = off;
  return w;
}

mcs_status decode_call(const mcs_decode_shape* s, const void* q, const void* kp, const void* vp, const void* k,
                       const void* v, const int32_t* lens, const float* slopes, void* o, float* lse, void* ws,
                       size_t ws_bytes, cudaStream_t stream) {
  if (!q || !k || !v || !lens || !o || !ws || (s->P > 0 && (!kp || !vp))) return MCS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(kp) || !aligned16(vp) ||
      !aligned4(lens) || !aligned4(slopes) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return MCS_ERR_INVALID_ARG;
  const DecodePlan f = decode_plan(s);
  const DecodeWs w = decode_layout(f, s);
  if (ws_bytes < w.total) return MCS_ERR_INVALID_ARG;
  const mcs_status st = check_device();
  if (st != MCS_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const float scale = scale_of(s->scale, s->d);
  DecodeParams p{};
  p.B = s->B; p.Hq = s->Hq; p.Hkv = s->Hkv; p.g = s->Hq / s->Hkv; p.C = s->C;
  p.nsplit = f.nsplit; p.chunk = f.chunk; p.gsplit = f.gsplit;
  p.cap = cap_fn(scale, s->cap);
  p.mul = p.cap.on ? 1.f : static_cast<float>(scale * 1.4426950408889634074);
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.lens = lens;
  p.slopes = slopes;
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.status = static_cast<int*>(ws);
  const bool parts = (f.nsplit > 1 && !f.cluster) || s->P > 0;
  p.cluster = f.cluster;
  if (parts) {
    p.part_lse = reinterpret_cast<float*>(base + w.part_lse);
    p.part_o = reinterpret_cast<float*>(base + w.part_o);
  }
  if (s->P > 0) {
    // the prefix: one batch row whose tokens are the requests, every key valid
    ExParams e{};
    e.B = 1; e.Hq = s->Hq; e.Hkv = s->Hkv; e.g = p.g; e.Nq = s->B; e.Nk = s->P;
    e.scale = scale;
    e.cap = s->cap;
    e.slopes = slopes;
    e.status = p.status;
    CUtensorMap tq, tk, tv;
    if (tiles_map(&tq, q, 1, s->B, s->Hq, s->d, p.g, f.pre.tpt) != MCS_OK ||
        tiles_map(&tk, kp, 1, s->P, s->Hkv, s->d, 1, 128) != MCS_OK ||
        tiles_map(&tv, vp, 1, s->P, s->Hkv, s->d, 1, 128) != MCS_OK)
      return MCS_ERR_CUDA;
    ExTile t = tile_params(e, f.pre, s->d);
    t.lens = lens;
    t.P = s->P;
    t.C = s->C;
    t.part_lse = reinterpret_cast<float*>(base + w.pre_lse);
    t.part_o = reinterpret_cast<float*>(base + w.pre_o);
    if (launch_ex_fwd(s->d, &tq, &tk, &tv, t, stream) != cudaSuccess) return MCS_ERR_CUDA;
    p.pre_lse = t.part_lse;
    p.pre_o = t.part_o;
    p.pre_parts = f.pre.nsplit;
    p.pre_tiles = f.pre.Tq;
    p.pre_tpt = f.pre.tpt;
  }
  if (launch_decode(s->d, p, stream) != cudaSuccess) return MCS_ERR_CUDA;
  return parts ? ok_or_cuda(launch_decode_combine(s->d, p, stream)) : MCS_OK;
}

}  // namespace

extern "C" {

size_t mcs_attn_workspace_bytes(const mcs_attn_shape* s, mcs_op op) {
  if (check_attn(s) != MCS_OK) return 0;
  if (op != MCS_OP_DENSE_EX && op != MCS_OP_DENSE_BWD) return 0;
  const FwdPlan f = fwd_plan(s->B, s->Hkv, s->Hq / s->Hkv, s->Nq, s->Nk, s->d, s->flags & MCS_ATTN_CAUSAL);
  return op == MCS_OP_DENSE_EX ? fwd_layout(f, s->B, s->Hkv, s->d).total
                               : bwd_layout(f, s->B, s->Hkv, s->Nk, s->d).total;
}

mcs_status mcs_dense_ex(const mcs_attn_shape* s, const mcs_attn_opts* opts, const void* q, const void* k,
                        const void* v, void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  mcs_status st = check_attn(s);
  if (st != MCS_OK) return st;
  if (!q || !k || !v || !o || !ws) return MCS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return MCS_ERR_INVALID_ARG;
  if ((st = check_opts(s, opts)) != MCS_OK) return st;
  if (ws_bytes < mcs_attn_workspace_bytes(s, MCS_OP_DENSE_EX)) return MCS_ERR_INVALID_ARG;
  if ((st = check_device()) != MCS_OK) return st;
  ExParams p = ex_params(s, opts);
  p.status = static_cast<int*>(ws);
  const FwdPlan f = fwd_plan(p.B, p.Hkv, p.g, p.Nq, p.Nk, s->d, p.causal);
  const FwdWs w = fwd_layout(f, p.B, p.Hkv, s->d);
  uint8_t* base = static_cast<uint8_t*>(ws);
  CUtensorMap tq, tk, tv;
  if (tiles_map(&tq, q, p.B, p.Nq, p.Hq, s->d, p.g, f.tpt) != MCS_OK ||
      tiles_map(&tk, k, p.B, p.Nk, p.Hkv, s->d, 1, 128) != MCS_OK ||
      tiles_map(&tv, v, p.B, p.Nk, p.Hkv, s->d, 1, 128) != MCS_OK)
    return MCS_ERR_CUDA;
  ExTile t = tile_params(p, f, s->d);
  t.o = static_cast<uint16_t*>(o);
  t.lse = lse;
  if (p.doc_q) {
    int* ids = reinterpret_cast<int*>(base + w.k_ids);
    int4* kr = reinterpret_cast<int4*>(base + w.k_ranges);
    int4* qr = reinterpret_cast<int4*>(base + w.q_ranges);
    if (launch_ex_doc_tiles(t, ids, kr, nullptr, qr, stream) != cudaSuccess) return MCS_ERR_CUDA;
    t.k_ids = ids;
    t.k_ranges = kr;
    t.q_ranges = qr;
    if (order_matters(static_cast<long long>(p.B) * p.Hkv * (f.single ? f.Tq : (f.Tq + 1) / 2))) {
      int* order = reinterpret_cast<int*>(base + w.order);
      int4* counts = reinterpret_cast<int4*>(base + w.counts);
      if (launch_ex_doc_order(t, f.single ? 1 : 2, counts, order, nullptr, stream) != cudaSuccess) return MCS_ERR_CUDA;
      t.order = order;
    }
  }
  if (f.nsplit > 1) {
    t.part_lse = reinterpret_cast<float*>(base + w.part_lse);
    t.part_o = reinterpret_cast<float*>(base + w.part_o);
  }
  if (launch_ex_fwd(s->d, &tq, &tk, &tv, t, stream) != cudaSuccess) return MCS_ERR_CUDA;
  return f.nsplit > 1 ? ok_or_cuda(launch_ex_combine(s->d, t, f.nsplit, stream)) : MCS_OK;
}

mcs_status mcs_dense_bwd(const mcs_attn_shape* s, const mcs_attn_opts* opts, const void* q, const void* k,
                         const void* v, const void* o, const float* lse, const void* d_o, void* dq, void* dk,
                         void* dv, void* ws, size_t ws_bytes, cudaStream_t stream) {
  mcs_status st = check_attn(s);
  if (st != MCS_OK) return st;
  if (!q || !k || !v || !o || !lse || !d_o || !dq || !dk || !dv || !ws) return MCS_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(d_o) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return MCS_ERR_INVALID_ARG;
  if ((st = check_opts(s, opts)) != MCS_OK) return st;
  if (ws_bytes < mcs_attn_workspace_bytes(s, MCS_OP_DENSE_BWD)) return MCS_ERR_INVALID_ARG;
  if ((st = check_device()) != MCS_OK) return st;
  ExParams p = ex_params(s, opts);
  p.status = static_cast<int*>(ws);
  const FwdPlan f = fwd_plan(p.B, p.Hkv, p.g, p.Nq, p.Nk, s->d, p.causal);
  const BwdWs w = bwd_layout(f, p.B, p.Hkv, p.Nk, s->d);
  uint8_t* base = static_cast<uint8_t*>(ws);
  CUtensorMap tq, tg, tk, tv;
  const int qbox = 64 % p.g == 0 ? f.tpt / 2 : f.tpt;
  if (tiles_map(&tq, q, p.B, p.Nq, p.Hq, s->d, p.g, qbox) != MCS_OK ||
      tiles_map(&tg, d_o, p.B, p.Nq, p.Hq, s->d, p.g, qbox) != MCS_OK ||
      tiles_map(&tk, k, p.B, p.Nk, p.Hkv, s->d, 1, 128) != MCS_OK ||
      tiles_map(&tv, v, p.B, p.Nk, p.Hkv, s->d, 1, 128) != MCS_OK)
    return MCS_ERR_CUDA;
  ExTile t = tile_params(p, f, s->d);
  t.qbox = qbox;
  t.kv_splits = w.kv_splits;
  t.kv_size = static_cast<size_t>(p.B) * p.Nk * p.Hkv * s->d;
  if (w.kv_splits > 1) t.part_kv = reinterpret_cast<float*>(base + w.part_kv);
  t.dq = static_cast<uint16_t*>(dq);
  t.dk = static_cast<uint16_t*>(dk);
  t.dv = static_cast<uint16_t*>(dv);
  float* stats = reinterpret_cast<float*>(base + w.stats);
  t.stats = stats;
  t.lse_in = lse;
  t.o_in = static_cast<const uint16_t*>(o);
  t.do_in = static_cast<const uint16_t*>(d_o);
  if (p.doc_q) {
    int* kid = reinterpret_cast<int*>(base + w.k_ids);
    int* qid = reinterpret_cast<int*>(base + w.q_ids);
    int4* kr = reinterpret_cast<int4*>(base + w.k_ranges);
    int4* qr = reinterpret_cast<int4*>(base + w.q_ranges);
    if (launch_ex_doc_tiles(t, kid, kr, qid, qr, stream) != cudaSuccess) return MCS_ERR_CUDA;
    t.k_ids = kid;
    t.k_ranges = kr;
    t.q_ids = qid;
    t.q_ranges = qr;
    if (order_matters(static_cast<long long>(p.B) * p.Hkv * std::max(f.Tq, f.Tk))) {
      int* order = reinterpret_cast<int*>(base + w.order);
      int* k_order = reinterpret_cast<int*>(base + w.k_order);
      int4* counts = reinterpret_cast<int4*>(base + w.counts);
      if (launch_ex_doc_order(t, 1, counts, order, k_order, stream) != cudaSuccess) return MCS_ERR_CUDA;
      t.order = order;
      t.k_order = k_order;
    }
  }
  t.stats_out = stats;
  t.d_from_o = (s->flags & MCS_ATTN_D_FROM_O) != 0;
  if (t.d_from_o && launch_ex_row_stats(s->d, t, stream) != cudaSuccess) return MCS_ERR_CUDA;
  return ok_or_cuda(launch_ex_bwd(s->d, &tq, &tg, &tk, &tv, t, stream));
}

size_t mcs_decode_workspace_bytes(const mcs_decode_shape* s) {
  if (check_decode(s) != MCS_OK) return 0;
  return decode_layout(decode_plan(s), s).total;
}

mcs_status mcs_decode(const mcs_decode_shape* s, const void* q, const void* k, const void* v, const int32_t* lens,
                      const float* slopes, void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const mcs_status st = check_decode(s);
  if (st != MCS_OK) return st;
  if (s->P != 0) return MCS_ERR_INVALID_ARG;
  return decode_call(s, q, nullptr, nullptr, k, v, lens, slopes, o, lse, ws, ws_bytes, stream);
}

mcs_status mcs_decode_shared(const mcs_decode_shape* s, const void* q, const void* kp, const void* vp,
                             const void* k, const void* v, const int32_t* lens, const float* slopes, void* o,
                             float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const mcs_status st = check_decode(s);
  if (st != MCS_OK) return st;
  if (s->P < 1) return MCS_ERR_INVALID_ARG;
  return decode_call(s, q, kp, vp, k, v, lens, slopes, o, lse, ws, ws_bytes, stream);
}

}  // extern "C"
