// Attention with modified scores, forward (mcs_dense_ex), and the shared
// prefix of mcs_decode_shared: online softmax over key tiles of 128, both
// products on the tensor cores (tcgen05, operands by TMA, accumulators in
// TMEM).
//
// A CTA has two slots, each with a 128-row query tile, a score tile S, an
// output accumulator O and eight softmax warps. The UMMA
// warp alternates between them,
//   S_0(i) = Q_0 K^T | O_1 += P_1(i-1) V | S_1(i) = Q_1 K^T | O_0 += P_0(i) V,
// so one slot's softmax runs while the tensor pipe computes the other's
// products. Two ways to fill the slots:
//   pair    two consecutive query tiles that share every key tile;
//   single  one query tile whose even key tiles go to slot 0 and odd ones to
//           slot 1 (few rows over many keys); slot 0 joins the halves at the end
//           through shared memory. With (m, l, O) of each slot, m = max(m0, m1):
//           l = sum_t l_t 2^(m_t - m), O = sum_t O_t 2^(m_t - m).
//
// TMEM (512 columns): S_0 | S_1 (128 each) | O_0 | O_1 (D each). P_t (bf16
// pairs, the TS-form A operand of O_t += P_t V) overwrites S_t where d = 128. With
// d = 64 it has columns of its own, and S(i + 1) is computed while the softmax
// works on S(i).
//
// Masks: a key tile is skipped, whole, or partial. Causal and prefix masks
// bound the tile range and give each row a key limit; a document mask skips
// tiles whose range of ids cannot meet the query tiles' (bitmap built at the
// start), and compares ids element by element in partial tiles only.
//
// Softmax: eight warps per slot, two threads per row (64 keys of the tile each),
// whose maxima meet in shared memory so that both use one running maximum.
//
// What bounds it: a slot's step is a chain of 3700 cycles at d = 128 (softmax
// 2130, of which the exponentials are 1550 where the special-function unit needs
// 1083; O += P V and S 512 each; hand-overs 570) and two slots overlap, so the
// tensor pipe works 2048 of them. 37 heads of 8192 tokens, d = 128, on GPUs at
// their power limit: 1.06 to 1.26 ms, 1010 to 1200 TFLOP/s of the 1684 that a
// plain product reaches; capped scores 1.44 to 1.6, biased 1.17 to 1.4; d = 64,
// where the exponentials are as many for half the products, 0.95 to 1.12 ms.
//
// P is rounded to bf16, the products' operand type: each value by up to 2^-8 of
// itself, which moves o by up to 0.0012 (relative, sharp scores; less where many
// terms average it) beside the 0.0017 of o's own rounding. The row sums l take P
// before it.
#include "attn_ex.cuh"

namespace mcs {

namespace {

constexpr int kThreads = kExThreads;
constexpr int kLaunchRegs = kExLaunchRegs;
constexpr int kLowRegs = kExLowRegs;
constexpr int kSoftRegs = kExSoftRegs;
// A row's running maximum moves only when a tile exceeds it by this much in
// log2 units (a factor 16): probabilities stay below 16, where bf16 is as exact
// as below 1, and most tiles leave O alone.
constexpr float kRescale = 4.0f;

// Whether the two tiles of a pair take their own lists of key tiles side by side, n0 and n1 long, instead of the n that
// either needs.
__device__ __forceinline__ bool apart_pays(int n, int n0, int n1) {
  return 4 * n > 5 * max(n0, n1) && min(n0, n1) > 0;
}
// Pairs of query tiles beyond half of an SM's share of all steps, of which there are fewer than this, are cut.
constexpr int kMostCuts = 2 * kSms;

// 2^x for x <= 2^21 on the FMA pipe. t = x + 1.5 2^23, rounded down, holds n =
// floor(x) in its low bits; 2^(x - n) is a polynomial of degree 5 with p(0) = 1,
// fitted to [0, 1] by iteratively reweighted least squares (relative error at most
// 9.5e-8). It is multiplied by 2^n, whose bits are made of n: added to the
// polynomial's exponent field instead, n would turn a NaN into a number. x < -126
// gives exactly 0, NaN stays NaN.
__device__ __forceinline__ void exp2_fma(float& x0, float& x1) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x0));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x1));
  const uint64_t x = f2_pack(x0, x1), shift = f2_pack(12582912.f, 12582912.f);
  uint64_t t;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(t) : "l"(x), "l"(shift));
  const uint64_t r = f2_add(x, f2_sub(shift, t));
  uint64_t p = f2_fma(f2_pack(.00186713017f, .00186713017f), r, f2_pack(.00901702978f, .00901702978f));
  p = f2_fma(p, r, f2_pack(.0557999127f, .0557999127f));
  p = f2_fma(p, r, f2_pack(.240164444f, .240164444f));
  p = f2_fma(p, r, f2_pack(.693151295f, .693151295f));
  p = f2_fma(p, r, f2_pack(1.f, 1.f));
  float t0, t1;
  f2_unpack(t, t0, t1);
  const float n0 = __uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u);
  const float n1 = __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u);
  f2_unpack(f2_mul(p, f2_pack(n0, n1)), x0, x1);
}

template <int D>
struct FwdCfg {
  // With d = 64 the accumulators leave 128 TMEM columns for P, so S(i + 1) need not wait for O += P(i) V.
  static constexpr bool AHEAD = D == 64;
  static constexpr int KB = D / 64;
  static constexpr uint32_t TILE = 128u * D * 2u;
  static constexpr int NS = D == 128 ? 2 : 4;  // K/V stages
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + NS * TILE;
  // q_full, k_full[NS], v_full[NS], v_ok[NS], k_empty[NS], v_empty[NS], s_full[2], s_read[2], p_full[2], p_empty[2], drain
  static constexpr uint32_t NBAR = 1 + 5 * NS + 8 + 1;
  static constexpr uint32_t OFF_MAX = OFF_BAR + (NBAR * 8 + 32 + 15) / 16 * 16;  // [parity][slot][half][row]
  static constexpr uint32_t OFF_BITS = OFF_MAX + 2 * 2 * 2 * 128 * 8;
  static constexpr uint32_t SMEM = OFF_BITS + 1024;  // and five bits for each key tile under a document mask
};

}  // namespace

template <int D, bool CAP, bool BIAS, bool DOC>
__global__ void __launch_bounds__(kThreads, 1)
    ex_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const ExTile p) {
  using C = FwdCfg<D>;
  // An eighth of the exponentials on the FMA pipe: 2 to 4 % less time for plain and biased scores (4096 tokens, 16/4
  // heads, causal, biased: 88.5 us, 92 without; a quarter: 92). With a cap's arithmetic or a document mask's
  // comparisons beside them they cost up to 4 %.
  constexpr bool SHARE = !CAP && !DOC;
  next_may_start();
  await_previous();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = q_full + 1;           // [stage]
  uint64_t* v_full = k_full + C::NS;       // [stage]
  uint64_t* v_ok = v_full + C::NS;         // [stage]: V's padded rows are clear (document masks)
  uint64_t* k_empty = v_ok + C::NS;        // [stage]: every S from it is computed
  uint64_t* v_empty = k_empty + C::NS;     // [stage]: every O += P V from it is done
  uint64_t* s_full = v_empty + C::NS;      // [slot]: S(i) computed
  uint64_t* s_read = s_full + 2;           // [slot]: S(i) is in registers (AHEAD)
  uint64_t* p_full = s_read + 2;           // [slot]: P(i) written (and O rescaled)
  uint64_t* p_empty = p_full + 2;          // [slot]: O += P(i) V done
  uint64_t* drain_bar = p_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* count = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform to the compiler too
  const int lane = threadIdx.x & 31;
  bool single = p.single;
  const int per = single ? 1 : 2;  // query tiles of a job
  const int groups = (p.Tq + per - 1) / per;
  // Work order: splits of one job side by side; then, for causal masks, the
  // heads of a chunk (whose K and V fit L2 together) with the longest query
  // tiles first, else the query tiles of one head.
  int u = blockIdx.x;
  const int split = u % p.nsplit;
  u /= p.nsplit;
  int job, bh, part = 0;
  const int BH = p.B * p.Hkv;
  if (DOC && p.order) {  // the jobs with the most key tiles first
    bh = ordered_job(p, p.order, groups, u, &job, &part);
    if (bh < 0) return;
    if (part) single = true;  // a long pair, whose tiles have a CTA each
  } else if (p.causal) {
    const int per_chunk = p.chunk * groups;
    const int ch = u / per_chunk, in = u % per_chunk;
    const int heads = min(p.chunk, BH - ch * p.chunk);
    bh = ch * p.chunk + in % heads;
    job = groups - 1 - in / heads;
  } else {
    job = u % groups;
    bh = u / groups;
  }
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int qt0 = job * per + (part >> 1);
  const bool has1 = !single && qt0 + 1 < p.Tq;  // slot 1 has a query tile of its own
  const int prefix = p.prefix ? p.prefix[b] : 0;
  // keys below limit(position) pass the causal and prefix masks
  auto limit = [&](int pos) { return p.causal ? min(p.Nk, max(max(pos + 1, prefix), 0)) : p.Nk; };
  auto last_tok = [&](int qt) { return min(p.Nq, (qt + 1) * p.tpt) - 1; };
  const int off = p.Nk - p.Nq;  // position of token 0
  const int T0 = (limit(off + last_tok(qt0)) + 127) >> 7;
  const int T = has1 ? (limit(off + last_tok(qt0 + 1)) + 127) >> 7 : T0;
  const int lo = static_cast<int>(static_cast<long long>(split) * T / p.nsplit);
  const int hi = static_cast<int>(static_cast<long long>(split + 1) * T / p.nsplit);
  const int4 none = make_int4(0x7fffffff, static_cast<int>(0x80000000), 0, 0);
  int4 r0 = none, r1 = none;
  if (DOC) {
    r0 = p.q_ranges[b * p.Tq + qt0];
    if (has1) r1 = p.q_ranges[b * p.Tq + qt0 + 1];
  }

  const int rt = p.tpt * p.g;
  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};
  // The loads of list entries j0 .. j1 - 1 (their tiles from `it`), for one thread.
  auto load_q = [&]() {
    const int tiles = has1 ? 2 : 1;
    mbar_arrive_expect_tx(q_full, tiles * C::KB * rt * 128);
    for (int t = 0; t < tiles; ++t)
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
        tma_load_4d(&tm_q, q_full, sQ + t * C::TILE + kb * 16384, kb * 64, hk * p.g, (qt0 + t) * p.tpt, b);
  };
  auto load_kv = [&](EntryIter& it, int j0, int j1) {
    for (int j = j0; j < j1; ++j) {
      const int s = j % C::NS;
      const int kt = it.next();
      if ((p.debug_flags & 1) && j == 0) continue;  // test knob: never deliver tile 0
      if (j >= C::NS && !mbar_wait(&k_empty[s], ((j / C::NS) & 1) ^ 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
      mbar_arrive_expect_tx(&k_full[s], C::TILE);
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
        tma_load_4d(&tm_k, &k_full[s], sK + s * C::TILE + kb * 16384, kb * 64, hk, kt * 128, b);
      if (j >= C::NS && !mbar_wait(&v_empty[s], ((j / C::NS) & 1) ^ 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
      mbar_arrive_expect_tx(&v_full[s], C::TILE);
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
        tma_load_4d(&tm_v, &v_full[s], sV + s * C::TILE + kb * 16384, kb * 64, hk, kt * 128, b);
    }
  };
  // without a document mask the list is known, and the first loads run beside the rest of the set-up
  const int early = DOC ? 0 : max(0, min(hi - lo, C::NS));

  if (warp == 1 && elect_one()) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    mbar_init(q_full, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_ok[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_read[t], 256);
      mbar_init(&p_full[t], 256);
      mbar_init(&p_empty[t], 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    count[0] = count[1] = count[2] = 0;
    count[3] = single;
    fence_mbar_init();
    if (early > 0) {
      load_q();
      EntryIter it{TileIter{0u, 0u, lo, lo}, TileIter{}, 0, true};
      load_kv(it, 0, early);
    }
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // rows that no load writes (g does not divide 128) stay zero
  if (rt < 128) {
    for (int i = threadIdx.x; i < per * C::KB * (128 - rt) * 8; i += kThreads) {
      const int c = i & 7, row = rt + (i >> 3) % (128 - rt), blk = (i >> 3) / (128 - rt);
      *reinterpret_cast<uint4*>(sQ + blk * 16384 + row * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // key tiles of this CTA and of its slots; the CTA's list holds what either slot needs
  TileBits tiles(smem_u32(smem + C::OFF_BITS), p.Tk);
  int n = hi - lo, n0 = min(hi, T0) - lo, n1 = has1 ? n : 0;
  if (DOC) {
    tiles.build<true>(count, p.k_ranges + static_cast<size_t>(b) * p.Tk, lo, hi, r0, r1);
    n = count[0];
    n0 = count[1];
    n1 = count[2];
  }
  if (n0 < 0) n0 = 0;
  if (single) n1 = n >> 1, n0 = n - n1;
  // Two query tiles of different documents need different key tiles: beyond a fifth of them the slots go through their
  // own lists side by side instead of waiting for each other in one.
  const bool zip = DOC && !single && apart_pays(n, n0, n1);
  if (zip) n = n0 + n1;
  const bool apart = single || zip;  // no tile serves both slots
  const TileIter first{DOC ? tiles.meet : 0u, DOC && !zip ? tiles.meet2 : 0u, lo, lo};
  const TileIter second{tiles.meet2, 0u, lo, lo};
  const EntryIter entries{first, second, zip ? min(n0, n1) : 0, !zip || n0 > n1};

  // read again where it is needed, since a register for it would spill another
  const uint32_t mode_at = smem_u32(count + 3);
  auto one_tile = [&]() { return DOC ? lds32(mode_at) != 0 : single; };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
    if (warp == 0) {
      // ---------------------------------------------------------------- UMMA issuer
      if (n > 0 && elect_one()) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, false, true);
        const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dV = sdesc_sw128(smem_u32(sV), 16384, 1024);
        // S_t = Q_t K^T with the CTA's list entry j
        auto issue_s = [&](int t, int j) {
          const uint64_t dQt = sdesc_advance(dQ, one_tile() ? 0 : t * C::TILE);
          const uint64_t dKs = sdesc_advance(dK, (j % C::NS) * C::TILE);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_bf16_ss(tmem + t * 128, sdesc_advance(dQt, o), sdesc_advance(dKs, o), IDESC_S, kk > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[t]);
        };
        auto issue_o = [&](int t, int i, int j) {
          const uint64_t dVs = sdesc_advance(dV, (j % C::NS) * C::TILE);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(tmem + 256 + t * D,
                         C::AHEAD ? tmem + 384 + t * 64 + kk * 8 : tmem + t * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                         sdesc_advance(dVs, kk * 2048), IDESC_O,
                         (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&p_empty[t]);
        };
        auto wait = [&](uint64_t* bar, int k) { return mbar_wait(bar, k & 1, wctx, MCS_WHERE_ATTN_MMA); };
        // V of list entry j. Under a document mask, once the warp that clears padded rows is done with it, in tiles
        // without padding too: no stage is released before that warp has left it, so it is never a phase behind.
        auto v_there = [&](int j) {
          const int s = j % C::NS;
          return wait(&v_full[s], j / C::NS) && (!DOC || wait(&v_ok[s], j / C::NS));
        };
        TileIter it = first;
        const int steps = one_tile() ? (n + 1) >> 1 : zip ? max(n0, n1) : n;
        // the slots' list entries of a step
        auto entry0 = [&](int step) { return one_tile() ? 2 * step : zip ? step + min(step, n1) : step; };
        auto entry1 = [&](int step) { return one_tile() ? 2 * step + 1 : zip ? step + min(step + 1, n0) : step; };
        int i0 = 0, i1 = 0;     // the slots' steps
        int behind = -1;        // slot 1's list entry whose O += P V is to come
        bool ok = wait(q_full, 0);
        // step's slots (1, 2)
        auto look = [&](int step) {
          const int j0 = entry0(step), j1 = entry1(step);
          int f = 0;
          if (DOC && zip) {
            f = (step < n0 ? 1 : 0) | (step < n1 ? 2 : 0);
          } else if (DOC && !one_tile()) {
            if (j0 >= n) return 0;
            const int kt = it.next() - lo;
            f = (tile_bit(tiles.meet, kt) ? 1 : 0) | (tile_bit(tiles.meet2, kt) ? 2 : 0);
          } else {
            f = (j0 < (one_tile() ? n : n0) ? 1 : 0) | (j1 < (one_tile() || has1 ? n : 0) ? 2 : 0);
          }
          return f;
        };
        int flags = look(0);
        if constexpr (C::AHEAD) {
          // S of a step, then the products of the step before
          int prev = 0, o0 = 0, o1 = 0;
          for (int step = 0; ok && step <= steps; ++step) {
            const int j0 = entry0(step), j1 = entry1(step);
            const int p0 = entry0(step - 1), p1 = entry1(step - 1);
            const int now = flags;
            if (now & 1) {
              if (!(ok = wait(&k_full[j0 % C::NS], j0 / C::NS) && (i0 == 0 || wait(&s_read[0], i0 - 1)))) break;
              tc_fence_after();
              issue_s(0, j0);
              if (apart || !(now & 2)) umma_commit(&k_empty[j0 % C::NS]);
              ++i0;
            }
            if (now & 2) {
              if (!(ok = wait(&k_full[j1 % C::NS], j1 / C::NS) && (i1 == 0 || wait(&s_read[1], i1 - 1)))) break;
              tc_fence_after();
              issue_s(1, j1);
              umma_commit(&k_empty[j1 % C::NS]);
              ++i1;
            }
            flags = look(step + 1);
            if (prev & 1) {
              if (!(ok = v_there(p0) && wait(&p_full[0], o0))) break;
              tc_fence_after();
              issue_o(0, o0, p0);
              if (apart || !(prev & 2)) umma_commit(&v_empty[p0 % C::NS]);
              ++o0;
            }
            if (prev & 2) {
              if (!(ok = v_there(p1) && wait(&p_full[1], o1))) break;
              tc_fence_after();
              issue_o(1, o1, p1);
              umma_commit(&v_empty[p1 % C::NS]);
              ++o1;
            }
            prev = now;
          }
        } else
        // UMMAs run in order, so S_t(i + 1) overwrites P_t(i) only after the product that reads it
        for (int step = 0; ok && step <= steps; ++step) {
          const int j0 = entry0(step), j1 = entry1(step);
          const int now = flags;
          const bool a0 = now & 1, a1 = now & 2;
          if (a0) {
            if (!(ok = wait(&k_full[j0 % C::NS], j0 / C::NS))) break;
            tc_fence_after();
            issue_s(0, j0);
            if (apart || !a1) umma_commit(&k_empty[j0 % C::NS]);
          }
          if (behind >= 0) {
            if (!(ok = v_there(behind) && wait(&p_full[1], i1 - 1))) break;
            tc_fence_after();
            issue_o(1, i1 - 1, behind);
            umma_commit(&v_empty[behind % C::NS]);
            behind = -1;
          }
          if (a1) {
            if (!(ok = wait(&k_full[j1 % C::NS], j1 / C::NS))) break;
            tc_fence_after();
            issue_s(1, j1);
            umma_commit(&k_empty[j1 % C::NS]);
            behind = j1;
            ++i1;
          }
          flags = look(step + 1);  // beside the softmax that the next product waits for
          if (a0) {
            if (!(ok = v_there(j0) && wait(&p_full[0], i0))) break;
            tc_fence_after();
            issue_o(0, i0, j0);
            if (apart || !a1) umma_commit(&v_empty[j0 % C::NS]);
            ++i0;
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- TMA producer
      if (n > 0 && elect_one()) {
        if (early == 0) load_q();
        EntryIter it = entries;
        it.a.cur += early;
        load_kv(it, early, n);
      }
      __syncwarp();
    } else if (warp == 2 && DOC) {
      // ---------------------------------------------------------------- padded keys
      EntryIter it = entries;
      for (int j = 0; j < n; ++j) {
        const int s = j % C::NS;
        if (!mbar_wait_warp(&v_full[s], (j / C::NS) & 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
        const int kt = it.next();
        hold_cleaner(p);
        if (tile_bit(tiles.pads, kt - lo)) {
          zero_padded_rows<C::KB>(sV + s * C::TILE, p.k_ids + (static_cast<size_t>(b) * p.Tk + kt) * 128);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ok[s]);
      }
      __syncwarp();
    }
    named_barrier_sync<1, kThreads>();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
  } else {
    // ---------------------------------------------------------------- softmax + epilogue of slot t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int t = (warp - 4) >> 3;           // slot
    const int half = ((warp - 4) >> 2) & 1;  // keys 64 half .. 64 half + 63 of each tile
    const int wq = warp & 3;                 // TMEM lane quarter this warp may access
    const int row = wq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_addr + t * 128 + half * 64;
    const uint32_t tP = C::AHEAD ? tmem + lane_addr + 384 + t * 64 + half * 32 : tS;
    const uint32_t tO = tmem + lane_addr + 256 + t * D + half * (D / 2);  // this half's output columns
    const int nt = t == 0 ? n0 : n1;
    const int qt = one_tile() ? qt0 : qt0 + t;
    const int tok = qt * p.tpt + row / p.g;
    const int head = hk * p.g + row % p.g;
    const bool row_valid = row < rt && tok < p.Nq && (t == 0 || one_tile() || has1);
    const int pos = p.lens ? p.P + min(max(row_valid ? p.lens[tok] : 0, 0), p.C) - 1 : off + tok;
    const int lim = limit(pos) - half * 64;
    const int lim_all = limit(off + qt * p.tpt);  // keys that every row of the tile sees
    const uint32_t whole = t == 0 || one_tile() ? tiles.whole : tiles.whole2;
    int my_doc = DOC && row_valid ? p.doc_q[static_cast<size_t>(b) * p.Nq + tok] : -2;
    if (my_doc < 0) my_doc = -2;  // a padded query matches no key
    const float mul = p.mul;  // what turns a score into log2 units
    const float slope = BIAS && row_valid ? slope_of(p.slopes, head) * kLog2e / mul : 0.f;
    if (BIAS && row_valid) check_slope(p.slopes, head, p.status);
    const uint64_t mul2 = f2_pack(mul, mul);
    // the words of this row and half, and of the other half
    const uint32_t my_max = smem_u32(smem + C::OFF_MAX) + ((t * 2 + half) * 128 + row) * 8;
    const uint32_t other_max = smem_u32(smem + C::OFF_MAX) + ((t * 2 + (half ^ 1)) * 128 + row) * 8;
    const int pair_bar = 2 + t * 4 + wq;  // the two warps that share these rows
    TileIter it = first;
    if (DOC && !one_tile()) it = TileIter{t == 0 ? tiles.meet : tiles.meet2, 0u, lo, lo};
    if (one_tile() && t == 1 && nt > 0) it.next();
    float m = -CUDART_INF_F;  // running max, log2 units (the same in both halves)
    float l = 0.f;            // this half's sum
    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      const int kt = it.next();
      if (one_tile() && i + 1 < nt) it.next();
      // where the tile's documents differ: the ids of keys `lane` and 32 + `lane` of this half, under way while S is
      const bool mixed = DOC && !tile_bit(whole, kt - lo);
      int id0 = 0, id1 = 0;
      if (mixed) {
        const int* at = p.k_ids + (static_cast<size_t>(b) * p.Tk + kt) * 128 + half * 64 + lane;
        id0 = __ldg(at);
        id1 = __ldg(at + 32);
      }
      ok = ok && mbar_wait_warp(&s_full[t], i & 1, wctx, MCS_WHERE_ATTN_SOFTMAX);
      tc_fence_after();
      float sv[64];  // after a failed wait: whatever the columns hold
      tmem_ld32(tS, sv);
      tmem_ld32(tS + 32, sv + 32);
      tmem_wait_ld();
      if (C::AHEAD) {
        tc_fence_before();
        mbar_arrive(&s_read[t]);
      }
      float shift = 0.f;  // log2 units that the whole row of this tile lacks
      if (CAP) cap_scores<64>(sv, p.cap);
      if (BIAS) {
        shift = add_bias<64>(sv, slope, static_cast<float>(pos - kt * 128 - half * 64)) * mul;
      }
      if (mixed || (kt + 1) * 128 > lim_all) {
        const int valid = lim - kt * 128;
        if (mixed) {
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            const int id = __shfl_sync(0xffffffffu, c < 32 ? id0 : id1, c & 31);  // padding: -1, which no query has
            sv[c] = (c < valid && id == my_doc) ? sv[c] : -CUDART_INF_F;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) sv[c] = c < valid ? sv[c] : -CUDART_INF_F;
        }
      }
      float mc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a = sv[k * 16];
#pragma unroll
        for (int e = 1; e < 15; e += 2) a = fmax3(a, sv[k * 16 + e], sv[k * 16 + e + 1]);
        mc[k] = fmaxf(a, sv[k * 16 + 15]);
      }
      const float half_max = fmaf(fmaxf(fmax3(mc[0], mc[1], mc[2]), mc[3]), mul, shift);
      // Both warps meet here in every step, with the step's own word on whether their waits held, and leave the loop
      // in the same step if one did not.
      sts_pair(my_max + (i & 1) * 4096, half_max, ok ? 0.f : 1.f);
      asm volatile("barrier.sync %0, 64;" ::"r"(pair_bar) : "memory");
      const float2 other = lds_pair(other_max + (i & 1) * 4096);
      ok = ok && other.y == 0.f;
      if (!ok) break;
      const float mx = fmaxf(half_max, other.x);
      // a row that has seen no valid key keeps m = -inf, l = 0 and P = 0
      const bool need = i == 0 ? mx > m : mx > m + kRescale;
      const float m_old = m;
      m = need ? mx : m;
      const float e0 = m == -CUDART_INF_F ? 0.f : shift - m;
      const uint64_t e2 = f2_pack(e0, e0);
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        uint32_t pk[16];
        float* v = sv + 32 * h2;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(v[2 * q], v[2 * q + 1]), mul2, e2), x0, x1);
          if (SHARE && q % 8 == 7) {
            exp2_fma(x0, x1);
          } else {
            x0 = fast_exp2(x0);
            x1 = fast_exp2(x1);
          }
          v[2 * q] = x0;
          v[2 * q + 1] = x1;
          pk[q] = pack_bf16(v[2 * q], v[2 * q + 1]);
        }
        if (C::AHEAD && h2 == 0 && i > 0) {  // O += P(i-1) V has read P(i-1), and O may be scaled
          ok = mbar_wait_warp(&p_empty[t], (i - 1) & 1, wctx, MCS_WHERE_ATTN_SOFTMAX);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st16u(tP + h2 * 16, pk);
      }
      if (!ok) continue;  // the other half learns of it in the next step
      if (i > 0 && __any_sync(0xffffffffu, need)) {
        // O += P(i-1) V ran before S(i) (AHEAD: before this step's P), so O may be scaled here; O += P(i) V waits for p_full
        const float alpha = need ? fast_exp2(m_old - m) : 1.f;
        l *= alpha;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float ov[16];
          tmem_ld16(tO + c * 16, ov);
          tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(ov[e] * alpha);
          tmem_st16u(tO + c * 16, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
      // the sum of this half's P, beside the products that wait for it
      {
        uint64_t a[16];
#pragma unroll
        for (int q = 0; q < 16; ++q)
          a[q] = f2_add(f2_pack(sv[2 * q], sv[2 * q + 1]), f2_pack(sv[2 * q + 32], sv[2 * q + 33]));
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) {
#pragma unroll
          for (int q = 0; q < w; ++q) a[q] = f2_add(a[q], a[q + w]);
        }
        float s0, s1;
        f2_unpack(a[0], s0, s1);
        l += s0 + s1;
      }
    }
    // ---------------------------------------------------------------- epilogue of slot t
    const bool fin = ok && (nt == 0 || mbar_wait_warp(&p_empty[t], (nt - 1) & 1, wctx, MCS_WHERE_ATTN_EPILOGUE));
    // the row's sum: both halves', exchanged like the maxima (every warp takes part, whatever happened)
    // a loop left early wrote the other parity's words
    sts_pair(my_max + (nt & 1) * 4096, l, 0.f);
    asm volatile("barrier.sync %0, 64;" ::"r"(pair_bar) : "memory");
    l += lds_pair(other_max + (nt & 1) * 4096).x;
    // One query tile for both slots: slot 1 hands its sums over in the K/V ring, which nobody reads any more once both
    // slots' last products are done, and slot 0 joins them. Every warp takes part, whatever happened.
    float* handed = reinterpret_cast<float*>(smem + C::OFF_K) + half * (D / 2) * 128 + row;  // [column][row]
    const bool join = one_tile() && n1 > 0;
    if (join) {
      named_barrier_sync<10, 512>();
      if (t == 1) {
        sts_pair(my_max, m, l);
        tc_fence_after();
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          float ov[32];
          tmem_ld32(tO + cc * 32, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) handed[(cc * 32 + e) * 128] = ov[e];
        }
      }
      named_barrier_sync<10, 512>();
    }
    if (fin && (t == 0 || has1)) {
      // the row's place again (hidden from the compiler, which would hold it in registers through the loop)
      int row2 = row;
      asm volatile("" : "+r"(row2));
      const int tok = qt * p.tpt + row2 / p.g, head = hk * p.g + row2 % p.g;
      const bool row_valid = row2 < rt && tok < p.Nq;
      tc_fence_after();
      const bool partial = p.part_o != nullptr;
      float w0 = 1.f, w1 = 0.f;
      if (join) {
        const float2 ml = lds_pair(my_max + 2 * 128 * 8);  // slot 1's
        const float both = fmaxf(m, ml.x), top = top_or_zero(both);
        w0 = fast_exp2(m - top);
        w1 = fast_exp2(ml.x - top);
        l = l * w0 + ml.y * w1;
        m = both;
      }
      const float inv = l == 0.f ? 0.f : w0 / l, inv1 = l == 0.f ? 0.f : w1 / l;
      const float lse2 = l == 0.f ? -CUDART_INF_F : m + log2f(l);
      const size_t bht = static_cast<size_t>(bh) * p.Tq + qt;
      const size_t slice = static_cast<size_t>(split) * BH * p.Tq;
      if (row_valid && half == 0) {
        if (partial) p.part_lse[(slice + bht) * 128 + row] = lse2;
        else if (p.lse) p.lse[(static_cast<size_t>(b) * p.Hq + head) * p.Nq + tok] = lse2 * kLn2;
      }
      uint16_t* orow = p.o + ((static_cast<size_t>(b) * p.Nq + tok) * p.Hq + head) * D + half * (D / 2);
      float* prow = p.part_o + ((slice + bht) * 128 + row) * D + half * (D / 2);
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        float ov[32];
        if (nt > 0) {
          tmem_ld32(tO + cc * 32, ov);
          tmem_wait_ld();
        }
        if (!row_valid) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = l == 0.f ? 0.f : ov[e] * inv;
        if (join) {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = l == 0.f ? 0.f : fmaf(handed[(cc * 32 + e) * 128], inv1, ov[e]);
        }
        if (partial) {
          float4* d4 = reinterpret_cast<float4*>(prow + cc * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) d4[e] = make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
        } else {
          uint4* d4 = reinterpret_cast<uint4*>(orow + cc * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            d4[e] = make_uint4(pack_bf16(ov[8 * e], ov[8 * e + 1]), pack_bf16(ov[8 * e + 2], ov[8 * e + 3]),
                               pack_bf16(ov[8 * e + 4], ov[8 * e + 5]), pack_bf16(ov[8 * e + 6], ov[8 * e + 7]));
        }
      }
    }
    __syncwarp();
    // the softmax warps return their registers before the first warpgroup takes its own back
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
    named_barrier_sync<1, kThreads>();
  }

  // ------------------------------------------------------------------ teardown
  // All roles have left their loops. After an abort, wait (bounded) for copies
  // and UMMAs this CTA issued, then free TMEM.
  __syncthreads();
  if (*abort_flag) {
    volatile int never = 0;
    const WaitCtx drain_ctx{&never, nullptr, 50000000ull};
    if (threadIdx.x == 32 && n > 0) {
      // both parities of every load barrier: the phase that a load in flight completes is one of the two
      for (int j = 0; j < 1 + 2 * C::NS; ++j) {
        mbar_wait(&q_full[j], 0, drain_ctx, MCS_WHERE_DRAIN);
        mbar_wait(&q_full[j], 1, drain_ctx, MCS_WHERE_DRAIN);
      }
    }
    if (warp == 0 && lane == 0) {
      umma_commit(drain_bar);
      mbar_wait(drain_bar, 0, drain_ctx, MCS_WHERE_DRAIN);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

// Joins the splits of the keys: with lse2_s and o_s of split s,
// lse2 = log2 sum_s 2^lse2_s and o = sum_s 2^(lse2_s - lse2) o_s. One warp per
// row, lane l holds d/32 columns; the splits are summed in their order.
template <int D>
__global__ void __launch_bounds__(128) ex_combine(const ExTile p, int parts) {
  next_may_start();
  await_previous();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);  // (b, tok, head)
  if (r >= static_cast<long long>(p.B) * p.Nq * p.Hq) return;
  const int head = r % p.Hq, tok = r / p.Hq % p.Nq, b = r / p.Hq / p.Nq;
  const size_t at = ((static_cast<size_t>(b) * p.Hkv + head / p.g) * p.Tq + tok / p.tpt) * 128 + tok % p.tpt * p.g +
                    head % p.g;
  const size_t slice = static_cast<size_t>(p.B) * p.Hkv * p.Tq * 128;
  float m = -CUDART_INF_F, l = 0.f, o[E] = {};
  // four parts at a time, so that their loads overlap
  for (int s0 = 0; s0 < parts; s0 += 4) {
    float ls[4], v[4][E];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ls[k] = -CUDART_INF_F;
      if (s0 + k < parts) {
        ls[k] = p.part_lse[(s0 + k) * slice + at];
        const float* src = p.part_o + ((s0 + k) * slice + at) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = src[e];
      }
    }
    const float mn = fmaxf(m, fmaxf(fmaxf(ls[0], ls[1]), fmaxf(ls[2], ls[3])));
    const float top = top_or_zero(mn), a = fast_exp2(m - top);
    m = mn;
    l *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ls[k] == -CUDART_INF_F) continue;
      const float w = fast_exp2(ls[k] - top);
      l += w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[k][e], o[e]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(r) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[(static_cast<size_t>(b) * p.Hq + head) * p.Nq + tok] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// Document ids as the tiles read them. Key tiles: ids of 128 keys (-1 past Nk and
// for padding) and their range. Query tiles: the range over the tile's tokens
// and, for the backward pass, the id of every packed row (-2 for padding and
// empty rows). One CTA of 128 threads per tile.
__global__ void __launch_bounds__(128) ex_doc_tiles(const ExTile p, int* k_ids, int4* k_ranges, int* q_ids,
                                                    int4* q_ranges) {
  next_may_start();
  await_previous();
  __shared__ int s_min, s_max, s_pad;
  const int b = blockIdx.x / (p.Tk + p.Tq), at_b = blockIdx.x % (p.Tk + p.Tq);
  const bool key = at_b < p.Tk;
  const int tile = key ? at_b : at_b - p.Tk;
  if (threadIdx.x == 0) s_min = 0x7fffffff, s_max = static_cast<int>(0x80000000), s_pad = 0;
  __syncthreads();
  const int i = threadIdx.x;
  const int n = key ? p.Nk : p.Nq;
  const int tok = key ? tile * 128 + i : tile * p.tpt + i / p.g;
  const bool in = tok < n && (key || i < p.tpt * p.g);
  const int id = in ? (key ? p.doc_k : p.doc_q)[static_cast<size_t>(b) * n + tok] : -1;
  const size_t at = static_cast<size_t>(b) * (key ? p.Tk : p.Tq) + tile;
  if (key) k_ids[at * 128 + i] = id < 0 ? -1 : id;
  else if (q_ids) q_ids[at * 128 + i] = id < 0 ? -2 : id;
  if (id >= 0) {
    atomicMin(&s_min, id);
    atomicMax(&s_max, id);
  } else if (in) {
    s_pad = 1;  // every writer writes the same
  }
  __syncthreads();
  if (i == 0) (key ? k_ranges : q_ranges)[at] = make_int4(s_min, s_max, s_pad, 0);
}

// What the jobs of a document mask have to do, one warp per job: job i of request
// b is `per` query tiles (their key tiles) or, behind the query jobs, one key
// tile (its query tiles). counts[b jobs + i] = (steps, tiles of the first and of
// the second query tile).
__global__ void __launch_bounds__(256) ex_doc_counts(const ExTile p, int per, int q_all, int all, int4* counts) {
  next_may_start();
  await_previous();
  const int job = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (job >= all) return;
  const bool key = job >= q_all;
  const int at = key ? job - q_all : job;
  const int jobs = key ? p.Tk : (p.Tq + per - 1) / per;
  const int b = at / jobs, i = at % jobs, off = p.Nk - p.Nq;
  const int prefix = p.prefix ? p.prefix[b] : 0;
  const int4 none = make_int4(0x7fffffff, static_cast<int>(0x80000000), 0, 0);
  const int4* ranges = key ? p.q_ranges + static_cast<size_t>(b) * p.Tq : p.k_ranges + static_cast<size_t>(b) * p.Tk;
  int lo = 0, hi = key ? p.Tq : p.Tk;
  int4 r0, r1 = none;
  if (key) {
    r0 = p.k_ranges[static_cast<size_t>(b) * p.Tk + i];
    if (p.causal && i * 128 >= prefix) lo = min(p.Tq, max(0, i * 128 - off) / p.tpt);
  } else {
    r0 = p.q_ranges[static_cast<size_t>(b) * p.Tq + i * per];
    if (per == 2 && i * per + 1 < p.Tq) r1 = p.q_ranges[static_cast<size_t>(b) * p.Tq + i * per + 1];
    const int last = off + min(p.Nq, (i + 1) * per * p.tpt) - 1;
    if (p.causal) hi = (min(p.Nk, max(max(last + 1, prefix), 0)) + 127) >> 7;
  }
  int n0 = 0, n1 = 0, n = 0;
  for (int t0 = lo; t0 < hi; t0 += 256) {  // eight tiles a lane, whose loads overlap
    int4 r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = t0 + e * 32 + lane;
      r[e] = t < hi ? ranges[t] : none;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int a0 = docs_meet(r[e], r0), a1 = docs_meet(r[e], r1);
      n0 += a0;
      n1 += a1;
      n += a0 | a1;
    }
  }
  n0 = __reduce_add_sync(0xffffffffu, n0);
  n1 = __reduce_add_sync(0xffffffffu, n1);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) counts[job] = make_int4(apart_pays(n, n0, n1) ? max(n0, n1) : n, n0, n1, 0);
}

// Order of these jobs, those with the most steps first: the documents' lengths
// differ, and a long job that starts last runs alone. A pair of query tiles that
// takes more than half of an SM's share of the whole is cut into its tiles: each
// goes to both slots of a CTA of its own, with half of its key tiles to a slot.
// (Documents of 6000 tokens on average in 32760, 2 heads: the longest pair has 123
// steps, and cutting takes 270 instead of 365 us. Cut everywhere, calls whose jobs
// are many and short take 20 % longer: twice as many set-ups.) A counting sort by
// one CTA for the query jobs and one for the key tiles: order[0] entries
// b jobs + i, times 4, plus 0 or the tile's number, 1 or 2.
__global__ void __launch_bounds__(1024) ex_doc_order(const ExTile p, int per, const int4* counts, int* q_order,
                                                     int* k_order) {
  next_may_start();
  await_previous();
  __shared__ int bins[4096 + 1];
  __shared__ int sums[32];
  __shared__ int4 cut[kMostCuts];  // a cut job, its tiles' bins, whether there is a second
  __shared__ int cuts, seconds;
  __shared__ unsigned long long total_steps;
  const bool key = blockIdx.x == 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_jobs = (p.Tq + per - 1) / per, jobs = key ? p.Tk : q_jobs, all = jobs * p.B;
  if (key) counts += q_jobs * p.B;
  int* order = key ? k_order : q_order;
  const int step = ((key ? p.Tq : p.Tk) + 4095) / 4096;  // steps per bin
  auto bin = [&](int n) { return 4096 - n / step; };
  for (int i = threadIdx.x; i <= 4096; i += 1024) bins[i] = 0;
  if (threadIdx.x == 0) cuts = seconds = 0, total_steps = 0;
  __syncthreads();
  // whole-number sums: the atomics' order changes nothing but the order of equal jobs
  unsigned long long some = 0;
  for (int at = threadIdx.x; at < all; at += 1024) some += counts[at].x;
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) some += __shfl_xor_sync(0xffffffffu, some, w);
  if (lane == 0) atomicAdd(&total_steps, some);
  __syncthreads();
  // n > share / (2 SMs), so there are fewer than kMostCuts of them (each is there for every head)
  const unsigned long long share = total_steps * p.Hkv;
  auto long_job = [&](int n) { return per == 2 && !key && static_cast<unsigned long long>(n) * kMostCuts > share; };
  for (int at = threadIdx.x; at < all; at += 1024) {
    const int4 n = counts[at];
    if (long_job(n.x)) {
      const int second = at % jobs * 2 + 1 < p.Tq;
      const int4 c = make_int4(at, bin((n.y + 1) / 2), bin((n.z + 1) / 2), second);
      cut[atomicAdd(&cuts, 1)] = c;
      atomicAdd(&bins[c.y], 1);
      if (second) {
        atomicAdd(&bins[c.z], 1);
        atomicAdd(&seconds, 1);
      }
    } else {
      atomicAdd(&bins[bin(n.x)], 1);
    }
  }
  __syncthreads();
  // exclusive sums of the bins, four to a thread (the last bin, empty jobs, comes after them)
  int mine[4], total = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    mine[e] = bins[threadIdx.x * 4 + e];
    total += mine[e];
  }
  int incl = total;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, w);
    if (lane >= w) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = incl - total;
  for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bins[threadIdx.x * 4 + e] = before;
    before += mine[e];
  }
  if (threadIdx.x == 1023) bins[4096] = before;
  if (threadIdx.x == 0) order[0] = all + seconds;
  __syncthreads();
  // Equal jobs land about in order (neighbours share their tiles in L2); the order decides when they run, not what
  // they compute.
  ++order;
  for (int i = threadIdx.x; i < cuts; i += 1024) {
    const int4 c = cut[i];
    order[atomicAdd(&bins[c.y], 1)] = c.x * 4 + 1;
    if (c.w) order[atomicAdd(&bins[c.z], 1)] = c.x * 4 + 2;
  }
  for (int at = threadIdx.x; at - static_cast<int>(threadIdx.x) < all; at += 1024) {
    if (at < all) {
      const int n = counts[at].x;
      if (!long_job(n)) order[atomicAdd(&bins[bin(n)], 1)] = at * 4;
    }
    __syncthreads();
  }
}

template <int D, bool CAP, bool BIAS, bool DOC>
cudaError_t launch_fwd(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const ExTile& p,
                       cudaStream_t s) {
  auto kern = ex_fwd_kernel<D, CAP, BIAS, DOC>;
  const unsigned bits = DOC ? (p.Tk + 31) / 32 * 20u : 0u;
  const unsigned smem = FwdCfg<D>::SMEM + bits;
  static KernelReady ready;
  const cudaError_t e = make_ready(ready, kern, FwdCfg<D>::SMEM + 2560, kLaunchRegs);  // 2^12 tiles
  if (e != cudaSuccess) return e;
  const int per = p.single ? 1 : 2;
  long long grid = static_cast<long long>(p.B) * p.Hkv * ((p.Tq + per - 1) / per) * p.nsplit;
  if (p.order && per == 2) grid += std::min<long long>(grid, kMostCuts);  // CTAs for the second tiles of cut pairs
  return launch_in_sequence(kern, static_cast<unsigned>(grid), kThreads, smem, s, DOC, *tq, *tk, *tv, p);
}

}  // namespace

cudaError_t launch_ex_fwd(int d, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const ExTile& p,
                          cudaStream_t s) {
  return with_options(d, p, [&](auto D, auto CAP, auto BIAS, auto DOC) {
    return launch_fwd<D.value, CAP.value, BIAS.value, DOC.value>(tq, tk, tv, p, s);
  });
}

cudaError_t launch_ex_combine(int d, const ExTile& p, int parts, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.B) * p.Nq * p.Hq + 3) / 4);
  return launch_in_sequence(d == 64 ? ex_combine<64> : ex_combine<128>, grid, 128, 0, s, true, p, parts);
}

cudaError_t launch_ex_doc_order(const ExTile& p, int per, int4* counts, int* q_order, int* k_order, cudaStream_t s) {
  const int q_all = p.B * ((p.Tq + per - 1) / per), all = q_all + (k_order ? p.B * p.Tk : 0);
  const cudaError_t e = launch_in_sequence(ex_doc_counts, (all + 7) / 8, 256, 0, s, true, p, per, q_all, all, counts);
  if (e != cudaSuccess) return e;
  return launch_in_sequence(ex_doc_order, k_order ? 2 : 1, 1024, 0, s, true, p, per, counts, q_order, k_order);
}

cudaError_t launch_ex_doc_tiles(const ExTile& p, int* k_ids, int4* k_ranges, int* q_ids, int4* q_ranges,
                                cudaStream_t s) {
  return launch_in_sequence(ex_doc_tiles, p.B * (p.Tk + p.Tq), 128, 0, s, false, p, k_ids, k_ranges, q_ids, q_ranges);
}

}  // namespace mcs
