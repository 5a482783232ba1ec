// Attention with modified scores, gradients (mcs_dense_bwd), on the tensor
// cores. With P = 2^(s - lse) and D_i = sum_j P_ij dP_ij (= d_o_i . o_i),
//   dP = d_o V^T,  dS = P (dP - D) (1 - t^2),
//   dV = P^T d_o,  dK = scale dS^T Q,  dQ = scale dS K.
//
// First D, by a sweep of two products (ex_delta_kernel) or from the given o
// (ex_row_stats). Then two kinds of CTAs in one launch: dK and dV are sums over queries, dQ over
// keys, so a single sweep would have to add one of them into global memory from many
// CTAs, in an order that changes from run to run. Here every sum is one CTA's,
// in a fixed order, at the price of seven products per tile instead of five.
//
//   dkv_tile: a CTA owns 128 keys of a KV head, K and V resident, and
//     streams packed query tiles (so the heads that share the KV head are
//     summed in the accumulators). Scores are computed transposed, keys on
//     TMEM lanes: S^T = K Q^T, dP^T = V d_o^T. P^T and dS^T (bf16) overwrite
//     them and are the TS-form A operands of dV += P^T d_o, dK += dS^T Q.
//     The tile's two halves of 64 query rows take turns, each with its own
//     columns of S^T and dP^T: dV_h(i) S_h(i+1) dK_h(i) dP_h(i+1) for h = 0, 1, so
//     that a half's chain (P from S, dS from dP, and their barriers) runs beside
//     the other half's products. With whole tiles in one chain the tensor pipe
//     waited 1500 of every 3500 cycles; halves cost the N = 64 products 48
//     cycles for 32 cycles of work.
//     Where these CTAs are few, the query tiles are split among several, whose
//     fp32 parts ex_sum_parts adds.
//   dq_tile: a CTA owns one packed query tile and streams key tiles:
//     S = Q K^T, dP = d_o V^T, dS over dP, dQ += dS K. S(i+1) and dP(i+1) are
//     computed while the softmax works on tile i (dP has two buffers).
//
// Four threads work on a row of a tile, 32 of its columns each.
//
// What bounds it: the products (67 % of the tensor pipe's time in the launch of
// dK, dV and dQ) and the exponentials (56 % of the special-function unit's in the
// sweep). 37 heads of 8192 tokens, d = 128: 4.1 ms, 770 TFLOP/s on the formulas'
// five products, of the 1684 that a plain product reaches; with D from the given o
// 3.1 to 3.4 ms; capped scores 5.5 and 4.2 ms, d = 64 3.1 and 2.35 (the
// exponentials and the roundings of P and dS are as many for half the products).
//
// P and dS are rounded to bf16, the products' operand type: each value by up to
// 2^-8 of itself, 0.0017 (relative, rms) in dV, and in dK and dQ, which with the
// results' own rounding makes 0.0024.
#include <algorithm>

#include "attn_ex.cuh"

namespace mcs {

namespace {

constexpr int kThreads = kExThreads;
constexpr int kSoftThreads = 512;

template <int D>
struct DkvCfg {
  static constexpr int KB = D / 64;
  static constexpr uint32_t TILE = 128u * D * 2u;
  static constexpr int NS = D == 128 ? 2 : 4;  // stages of Q, d_o and their rows' statistics
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = TILE;
  static constexpr uint32_t OFF_Q = 2 * TILE;
  static constexpr uint32_t OFF_G = OFF_Q + NS * TILE;
  static constexpr uint32_t OFF_STAT = OFF_G + NS * TILE;     // [stage]: -lse (log2 units) [128], D [128]
  static constexpr uint32_t OFF_ROW = OFF_STAT + NS * 1024;   // slope [128], token in the tile [128]
  static constexpr uint32_t OFF_BAR = OFF_ROW + 1024;
  // kv_full, q_full[NS][2], g_full[NS][2], q_empty[NS][2], g_empty[NS][2], qg_ok[NS], s_full[2], dp_full[2],
  // p_full[2], ds_full[2], done
  static constexpr uint32_t NBAR = 1 + 9 * NS + 9;
  static constexpr uint32_t OFF_BITS = OFF_BAR + (NBAR * 8 + 32 + 15) / 16 * 16;
  static constexpr uint32_t SMEM = OFF_BITS + 1024;
};

template <int D>
struct DqCfg {
  static constexpr int KB = D / 64;
  static constexpr uint32_t TILE = 128u * D * 2u;
  static constexpr int NK = D == 128 ? 3 : 4;  // K stages: read by S(i) and, a tile later, by dQ(i)
  static constexpr int NV = D == 128 ? 2 : 4;  // V stages: read by dP(i) alone
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_G = TILE;
  static constexpr uint32_t OFF_K = 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NK * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + NV * TILE;
  // qg_full, k_full[NK], k_ok[NK], k_empty[NK], v_full[NV], v_empty[NV], s_full, s_read, dp_full[2], ds_full[2], done
  static constexpr uint32_t NBAR = 1 + 3 * NK + 2 * NV + 2 + 2 + 2 + 1;
  static constexpr uint32_t OFF_BITS = OFF_BAR + (NBAR * 8 + 32 + 15) / 16 * 16;
  static constexpr uint32_t SMEM = OFF_BITS + 1024;
};

// Zeroes rows rt .. 127 of `tiles` consecutive tiles (rows that no load writes).
template <int KB>
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int tiles, int rt) {
  for (int i = threadIdx.x; i < tiles * KB * (128 - rt) * 8; i += kThreads) {
    const int c = i & 7, row = rt + (i >> 3) % (128 - rt), blk = (i >> 3) / (128 - rt);
    *reinterpret_cast<uint4*>(tile + blk * 16384 + row * 128 + c * 16) = make_uint4(0, 0, 0, 0);
  }
}

// Stores N fp32 columns of one thread's TMEM row, times f, as bf16.
template <int N>
__device__ __forceinline__ void store_row(uint32_t taddr, bool have, bool valid, float f, uint16_t* dst) {
  constexpr int W = N < 32 ? N : 32;
#pragma unroll
  for (int cc = 0; cc < N / W; ++cc) {
    float v[W];
    if (have) {
      if constexpr (W == 32) tmem_ld32(taddr + cc * 32, v);
      else tmem_ld16(taddr, v);
      tmem_wait_ld();
    }
    if (!valid) continue;
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = have ? v[e] * f : 0.f;
    uint4* d4 = reinterpret_cast<uint4*>(dst + cc * 32);
#pragma unroll
    for (int e = 0; e < W / 8; ++e)
      d4[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                         pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
  }
}

// The same as fp32.
template <int N>
__device__ __forceinline__ void store_part(uint32_t taddr, bool have, bool valid, float* dst) {
#pragma unroll
  for (int cc = 0; cc < N / 32; ++cc) {
    float v[32];
    if (have) {
      tmem_ld32(taddr + cc * 32, v);
      tmem_wait_ld();
    }
    if (!valid) continue;
    float4* d4 = reinterpret_cast<float4*>(dst + cc * 32);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      d4[e] = have ? make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Frees TMEM once every role has left; after an abort, waits (bounded) for what is in flight.
__device__ __forceinline__ void teardown(volatile int* abort_flag, uint64_t* done, uint64_t* loads, int nloads,
                                         uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (*abort_flag) {
    volatile int never = 0;
    const WaitCtx drain_ctx{&never, nullptr, 50000000ull};
    if (warp == 1 && lane == 0) {
      // both parities of every load barrier: the phase that the loads in flight complete is one of the two
      for (int s = 0; s < nloads; ++s) {
        mbar_wait(&loads[s], 0, drain_ctx, MCS_WHERE_DRAIN);
        mbar_wait(&loads[s], 1, drain_ctx, MCS_WHERE_DRAIN);
      }
    }
    if (warp == 0 && lane == 0) {
      umma_commit(done);
      mbar_wait(done, 0, drain_ctx, MCS_WHERE_DRAIN);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Per packed row: -lse in log2 units (less slope times the row's token in the tile, which the dK/dV tiles' bias counts
// on) and D, as [B Hkv, Tq][2][128]; an empty row, like a row whose lse is -inf, gets (-inf, 0), which makes its P zero.
// Two ways to D:
//   ex_delta_kernel  D = sum_j P dP in fp32, a sweep of two products more (the default);
//   ex_row_stats     D = d_o . o from the given o, where the caller asks for that.
// o is rounded to bf16, which puts the second off by up to 2^-9 |d_o| |o|, and dP - D cancels where few keys carry a row's
// P: because it sees few, because scores are sharp, or because a distance bias leaves the near ones. In dQ, by itself,
// in 64 bits with d = 128 (relative, over all rows; dS in bf16 brings 0.0017 and so does the result's own rounding):
//   keys of a row             2       4      16      64     256    1024    4096
//   scores of spread 1    .0028   .0017   .0008   .0004   .0003   .0002   .0002
//   spread 2              .0043   .0029   .0018   .0014   .0008   .0007   .0005
//   spread 6              .0085   .0061   .0044   .0038   .0033   .0033   .0031
// and 0.0015 with 10 heads' slopes from 0.6 to 0.004 and scores of spread 2, however long the rows are. It saves the sweep:
// forward and gradients of 8192 tokens, 12 heads, capped, 1.97 instead of 2.48 ms.
// ex_row_stats: one CTA per tile, 16 bytes of a row per lane; reading o and d_o once from HBM is the bound.
template <int D>
__global__ void __launch_bounds__(256) ex_row_stats(const ExTile p) {
  next_may_start();
  await_previous();
  constexpr int LANES = D / 8;             // of a row
  constexpr int PASS = 256 / LANES;        // rows at a time
  const int qt = blockIdx.x % p.Tq, bh = blockIdx.x / p.Tq;
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int c = threadIdx.x % LANES;
  float* out = p.stats_out + static_cast<size_t>(blockIdx.x) * 256;
#pragma unroll 4
  for (int r0 = 0; r0 < 128; r0 += PASS) {
    const int row = r0 + threadIdx.x / LANES;
    const int t = row / p.g, tok = qt * p.tpt + t, head = hk * p.g + row - t * p.g;
    float nl = -CUDART_INF_F, s = 0.f;
    if (t < p.tpt && tok < p.Nq) {
      const float L = p.lse_in[(static_cast<size_t>(b) * p.Hq + head) * p.Nq + tok];
      const size_t at = ((static_cast<size_t>(b) * p.Nq + tok) * p.Hq + head) * D + c * 8;
      const uint4 x = *reinterpret_cast<const uint4*>(p.o_in + at), y = *reinterpret_cast<const uint4*>(p.do_in + at);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
      if (L != -CUDART_INF_F) {  // NaN passes on
        nl = -L * kLog2e;
        if (p.slopes) nl = fmaf(-slope_of(p.slopes, head) * kLog2e, static_cast<float>(t), nl);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
          s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
        }
      }
    }
#pragma unroll
    for (int w = LANES / 2; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (c == 0) {
      out[row] = nl;
      out[128 + row] = s;
    }
  }
}

}  // namespace

template <int D, bool CAP, bool BIAS, bool DOC>
__device__ __forceinline__ void dkv_tile(const CUtensorMap& tm_q, const CUtensorMap& tm_g, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const ExTile& p, int cta) {
  using C = DkvCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sG = smem + C::OFF_G;
  float* row_slope = reinterpret_cast<float*>(smem + C::OFF_ROW);
  float* row_tok = row_slope + 128;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = kv_full + 1;           // [stage][half of the tile's rows]: Q and the statistics
  uint64_t* g_full = q_full + 2 * C::NS;    // [stage][half]: d_o
  uint64_t* q_empty = g_full + 2 * C::NS;   // [stage][half]
  uint64_t* g_empty = q_empty + 2 * C::NS;  // [stage][half]
  uint64_t* qg_ok = g_empty + 2 * C::NS;    // [stage]: padded rows of Q and d_o are clear (document masks)
  uint64_t* s_full = qg_ok + C::NS;         // [half], as the next three
  uint64_t* dp_full = s_full + 2;
  uint64_t* p_full = dp_full + 2;
  uint64_t* ds_full = p_full + 2;
  uint64_t* done = ds_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* count = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform to the compiler too
  const int lane = threadIdx.x & 31;
  // causal: the first key tiles meet the most queries and go first, the heads of a chunk side by side
  const int BH = p.B * p.Hkv;
  const int split = cta % p.kv_splits;  // the query tiles' part
  cta /= p.kv_splits;
  int kt, bh;
  if (DOC && p.k_order) {  // the tiles with the most work first
    int part;
    bh = ordered_job(p, p.k_order, p.Tk, cta, &kt, &part);
  } else if (p.causal) {
    const int per_chunk = p.chunk * p.Tk;
    const int ch = cta / per_chunk, in = cta % per_chunk;
    const int heads = min(p.chunk, BH - ch * p.chunk);
    bh = ch * p.chunk + in % heads;
    kt = in / heads;
  } else {
    kt = cta % p.Tk;
    bh = cta / p.Tk;
  }
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int off = p.Nk - p.Nq;
  const int prefix = p.prefix ? p.prefix[b] : 0;
  // query tiles lo .. Tq - 1 reach these keys
  int lo = 0;
  if (p.causal && kt * 128 >= prefix) lo = min(p.Tq, max(0, kt * 128 - off) / p.tpt);
  const int rest = p.Tq - lo;
  const int hi = lo + static_cast<int>(static_cast<long long>(rest) * (split + 1) / p.kv_splits);
  lo += static_cast<int>(static_cast<long long>(rest) * split / p.kv_splits);
  const int4 none = make_int4(0x7fffffff, static_cast<int>(0x80000000), 0, 0);
  const int4 mine = DOC ? p.k_ranges[static_cast<size_t>(b) * p.Tk + kt] : none;
  const int rt = p.tpt * p.g;
  const bool halves = p.qbox < p.tpt;  // a tile loads as two boxes of 64 rows

  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};
  auto load_resident = [&]() {
    mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb) {
      tma_load_4d(&tm_k, kv_full, sK + kb * 16384, kb * 64, hk, kt * 128, b);
      tma_load_4d(&tm_v, kv_full, sV + kb * 16384, kb * 64, hk, kt * 128, b);
    }
  };
  // the loads of list entries j0 .. j1 - 1 (their tiles from `it`), for one thread
  auto load_queries = [&](TileIter& it, int j0, int j1) {
    bool ok = true;
    for (int j = j0; j < j1 && ok; ++j) {
      const int s = j % C::NS;
      const int qt = it.next();
      if ((p.debug_flags & 17) && j == 0) continue;  // test knob: never deliver tile 0
      const uint32_t parity = ((j / C::NS) & 1) ^ 1;
      const float* stats = p.stats + (static_cast<size_t>(bh) * p.Tq + qt) * 256;
      uint8_t* sS = smem + C::OFF_STAT + s * 1024;
      auto free = [&](uint64_t* empty, int h) {
        return j < C::NS || mbar_wait(&empty[2 * s + h], parity, wctx, MCS_WHERE_ATTN_PRODUCER);
      };
      auto box = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int h) {
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_4d(map, bar, dst + s * C::TILE + kb * 16384 + h * 8192, kb * 64, hk * p.g,
                      qt * p.tpt + h * p.qbox, b);
      };
      if (halves) {
#pragma unroll
        for (int h = 0; h < 2 && ok; ++h) {
          if (!(ok = free(q_empty, h))) break;
          mbar_arrive_expect_tx(&q_full[2 * s + h], C::KB * 8192 + 512);
          box(&tm_q, &q_full[2 * s + h], sQ, h);
          bulk_load(&q_full[2 * s + h], sS + h * 256, stats + h * 64, 256);
          bulk_load(&q_full[2 * s + h], sS + 512 + h * 256, stats + 128 + h * 64, 256);
          if (!(ok = free(g_empty, h))) break;
          mbar_arrive_expect_tx(&g_full[2 * s + h], C::KB * 8192);
          box(&tm_g, &g_full[2 * s + h], sG, h);
        }
      } else {  // a half's border cuts a token: the first half's barriers take the whole tile
        if (!(ok = free(q_empty, 0) && free(q_empty, 1))) break;
        mbar_arrive_expect_tx(&q_full[2 * s], C::KB * rt * 128 + 1024);
        box(&tm_q, &q_full[2 * s], sQ, 0);
        bulk_load(&q_full[2 * s], sS, stats, 1024);
        if (!(ok = free(g_empty, 0) && free(g_empty, 1))) break;
        mbar_arrive_expect_tx(&g_full[2 * s], C::KB * rt * 128);
        box(&tm_g, &g_full[2 * s], sG, 0);
      }
    }
  };
  // without a document mask the list is known, and the first loads run beside the rest of the set-up
  const int early = DOC ? 0 : max(0, min(hi - lo, C::NS));

  if (warp == 1 && elect_one()) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_g);
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::NS; ++s) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&q_full[2 * s + h], 1);
        mbar_init(&g_full[2 * s + h], 1);
        mbar_init(&q_empty[2 * s + h], 1);
        mbar_init(&g_empty[2 * s + h], 1);
      }
      mbar_init(&qg_ok[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&dp_full[h], 1);
      mbar_init(&p_full[h], kSoftThreads / 2);
      mbar_init(&ds_full[h], kSoftThreads / 2);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    count[0] = count[1] = count[2] = 0;
    fence_mbar_init();
    if (early > 0) {
      load_resident();
      TileIter it{0u, 0u, lo, lo};
      load_queries(it, 0, early);
    }
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (threadIdx.x < 128) {
    row_slope[threadIdx.x] = p.slopes ? slope_of(p.slopes, hk * p.g + threadIdx.x % p.g) * kLog2e : 0.f;
    row_tok[threadIdx.x] = static_cast<float>(threadIdx.x / p.g);
  }
  if (rt < 128) {
    zero_tail_rows<C::KB>(sQ, 2 * C::NS, rt);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int n = hi - lo;
  TileBits tiles(smem_u32(smem + C::OFF_BITS), p.Tq);
  if (DOC) {
    tiles.build<false>(count, p.q_ranges + static_cast<size_t>(b) * p.Tq, lo, hi, mine, none);
    n = count[0];
  }
  const TileIter first{DOC ? tiles.meet : 0u, 0u, lo, lo};

  if (warp < 4) {
    if (warp == 0) {
      // ---------------------------------------------------------------- UMMA issuer
      if (n > 0 && elect_one()) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64, false, false);
        constexpr uint32_t IDESC_A = idesc_bf16_f32(128, D, false, true);
        const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dV = sdesc_sw128(smem_u32(sV), 16, 1024);
        const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dG = sdesc_sw128(smem_u32(sG), 16, 1024);
        const uint64_t dQm = sdesc_sw128(smem_u32(sQ), 16384, 1024), dGm = sdesc_sw128(smem_u32(sG), 16384, 1024);
        // 64 columns at `to` = A B^T over d (both K-major), B the 64 query rows at `bb`
        auto scores = [&](uint32_t to, uint64_t a, uint64_t bb, uint64_t* bar) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_bf16_ss(to, sdesc_advance(a, o), sdesc_advance(bb, o), IDESC_S, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar);
        };
        // acc += (the bf16 tile over the 64 score columns at `from`) times the 64 query rows at `bb`
        auto accumulate = [&](uint32_t acc, uint32_t from, uint64_t bb, bool start) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ts(acc, from + (kk >> 1) * 32 + (kk & 1) * 8, sdesc_advance(bb, kk * 2048), IDESC_A,
                         (!start || kk > 0) ? 1u : 0u);
        };
        auto wait = [&](uint64_t* bar, int k) { return mbar_wait(bar, k & 1, wctx, MCS_WHERE_ATTN_MMA); };
        // Q or d_o of list entry j, half h; `pad`: once the padded rows are clear. Of a tile without padding the
        // clearing warp's word is awaited before its first release only (below), when it has long been given.
        auto ready = [&](uint64_t* full, int j, int h, bool pad) {
          const int s = j % C::NS;
          const bool there = wait(&full[halves ? 2 * s + h : 2 * s], j / C::NS) && (!pad || wait(&qg_ok[s], j / C::NS));
          tc_fence_after();
          return there;
        };
        TileIter it = first;
        bool pad = DOC && tile_bit(tiles.pads, it.next() - lo);
        bool ok = wait(kv_full, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = ready(q_full, 0, h, pad))) break;
          scores(tmem + h * 64, dK, sdesc_advance(dQ, h * 8192), &s_full[h]);
          if (!(ok = ready(g_full, 0, h, pad))) break;
          scores(tmem + 128 + h * 64, dV, sdesc_advance(dG, h * 8192), &dp_full[h]);
        }
        for (int i = 0; ok && i < n; ++i) {
          const uint32_t at = (i % C::NS) * C::TILE, nx = ((i + 1) % C::NS) * C::TILE;
          if (DOC && i + 1 < n) pad = tile_bit(tiles.pads, it.next() - lo);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // no stage is released before the clearing warp has left it, so that warp is never a phase behind
            if (!(ok = wait(&p_full[h], i) && (!DOC || h > 0 || wait(&qg_ok[i % C::NS], i / C::NS)))) break;
            tc_fence_after();
            accumulate(tmem + 256, tmem + h * 64, sdesc_advance(dGm, at + h * 8192), i == 0 && h == 0);
            umma_commit(&g_empty[2 * (i % C::NS) + h]);
            if (i + 1 < n) {
              if (!(ok = ready(q_full, i + 1, h, pad))) break;
              scores(tmem + h * 64, dK, sdesc_advance(dQ, nx + h * 8192), &s_full[h]);
            }
            if (!(ok = wait(&ds_full[h], i))) break;
            tc_fence_after();
            accumulate(tmem + 384, tmem + 128 + h * 64, sdesc_advance(dQm, at + h * 8192), i == 0 && h == 0);
            umma_commit(&q_empty[2 * (i % C::NS) + h]);
            if (i + 1 < n) {
              if (!(ok = ready(g_full, i + 1, h, pad))) break;
              scores(tmem + 128 + h * 64, dV, sdesc_advance(dG, nx + h * 8192), &dp_full[h]);
            } else if (h == 1) {
              umma_commit(done);
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- TMA producer
      if (n > 0 && elect_one()) {
        if (early == 0) load_resident();
        TileIter it = first;
        it.cur += early;
        load_queries(it, early, n);
      }
      __syncwarp();
    } else if (warp == 2 && DOC) {
      // ---------------------------------------------------------------- padded queries
      TileIter it = first;
      for (int j = 0; j < n; ++j) {
        const int s = j % C::NS;
        bool there = true;
        for (int h = 0; h < (halves ? 2 : 1) && there; ++h)
          there = mbar_wait_warp(&q_full[2 * s + h], (j / C::NS) & 1, wctx, MCS_WHERE_ATTN_PRODUCER) &&
                  mbar_wait_warp(&g_full[2 * s + h], (j / C::NS) & 1, wctx, MCS_WHERE_ATTN_PRODUCER);
        if (!there) break;
        const int qt = it.next();
        hold_cleaner(p);
        if (tile_bit(tiles.pads, qt - lo)) {
          const size_t at = static_cast<size_t>(b) * p.Tq + qt;
          zero_padded_rows<C::KB>(sQ + s * C::TILE, p.q_ids + at * 128);
          zero_padded_rows<C::KB>(sG + s * C::TILE, p.q_ids + at * 128);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qg_ok[s]);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- P and dS, then the epilogue
    const int quarter = (warp - 4) >> 2;  // query rows 32 quarter .. 32 quarter + 31 of each tile
    const int half = quarter >> 1;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const int key = kt * 128 + row;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_addr + quarter * 32;
    const uint32_t tP = tS + 128;
    const bool key_valid = key < p.Nk;
    const int my_doc = DOC ? p.k_ids[(static_cast<size_t>(b) * p.Tk + kt) * 128 + row] : 0;  // padding: -1
    const bool all_rows = !p.causal || key < prefix;
    const bool all_keys = !p.causal || kt * 128 + 127 < prefix;
    const float mul = p.mul;
    const uint64_t mul2 = f2_pack(mul, mul);
    const float im = 1.f / mul;
    const float4* tok4 = reinterpret_cast<const float4*>(row_tok) + quarter * 8;
    const float4* sl4 = reinterpret_cast<const float4*>(row_slope) + quarter * 8;
    TileIter it = first;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int s = i % C::NS;
      const int qt = it.next();
      // where the tile's documents differ: the id of row `lane` of this quarter, under way while S is
      const bool mixed = DOC && !tile_bit(tiles.whole, qt - lo);
      int id = 0;
      if (mixed) id = __ldg(p.q_ids + (static_cast<size_t>(b) * p.Tq + qt) * 128 + quarter * 32 + lane);
      const float4* nl4 = reinterpret_cast<const float4*>(smem + C::OFF_STAT + s * 1024) + quarter * 8;
      const float4* dl4 = nl4 + 32;
      // this key's place among the tile's tokens: token c sees it when c >= at
      const int at_i = key - off - qt * p.tpt;
      const float at = static_cast<float>(at_i);
      const bool partial = mixed || (!all_keys && kt * 128 + 127 > off + qt * p.tpt);
      // the statistics of this stage, then the scores
      if (!mbar_wait_warp(&q_full[halves ? 2 * s + half : 2 * s], (i / C::NS) & 1, wctx, MCS_WHERE_ATTN_SOFTMAX) ||
          !mbar_wait_warp(&s_full[half], i & 1, wctx, MCS_WHERE_ATTN_SOFTMAX)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float pv[32];  // score, P, then with a cap P (t^2 - 1)
      float w[32];   // t^2 - 1
      tmem_ld32(tS, pv);
      tmem_wait_ld();
      if (CAP) {
        cap_scores<32>(pv, p.cap);
#pragma unroll
        for (int c = 0; c < 32; c += 2) f2_unpack(cap_slope2(f2_pack(pv[c], pv[c + 1]), p.cap), w[c], w[c + 1]);
      }
      if (BIAS) {
        // The statistics hold nl - slope token. With token >= key the bias is -slope (token - at), of which
        // slope at is left; else slope (token - at), and otherwise the two cases element by element.
        const bool after = __all_sync(0xffffffffu, at_i <= 0);
        const bool before = __all_sync(0xffffffffu, at_i >= p.tpt - 1);
        const float at_m = at * im;
        if (after) {
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 sl = sl4[c >> 2];
            const uint64_t at2 = f2_pack(at_m, at_m);
            f2_unpack(f2_fma(f2_pack(sl.x, sl.y), at2, f2_pack(pv[c], pv[c + 1])), pv[c], pv[c + 1]);
            f2_unpack(f2_fma(f2_pack(sl.z, sl.w), at2, f2_pack(pv[c + 2], pv[c + 3])), pv[c + 2], pv[c + 3]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 tk = tok4[c >> 2], sl = sl4[c >> 2];
            const float d0 = tk.x - at, d1 = tk.y - at, d2 = tk.z - at, d3 = tk.w - at;
            pv[c] = fmaf(sl.x * im, tk.x - (before ? -d0 : fabsf(d0)), pv[c]);
            pv[c + 1] = fmaf(sl.y * im, tk.y - (before ? -d1 : fabsf(d1)), pv[c + 1]);
            pv[c + 2] = fmaf(sl.z * im, tk.z - (before ? -d2 : fabsf(d2)), pv[c + 2]);
            pv[c + 3] = fmaf(sl.w * im, tk.w - (before ? -d3 : fabsf(d3)), pv[c + 3]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 nl = nl4[c >> 2];
        float x0, x1, x2, x3;
        f2_unpack(f2_fma(f2_pack(pv[c], pv[c + 1]), mul2, f2_pack(nl.x, nl.y)), x0, x1);
        f2_unpack(f2_fma(f2_pack(pv[c + 2], pv[c + 3]), mul2, f2_pack(nl.z, nl.w)), x2, x3);
        pv[c] = fast_exp2(x0);
        pv[c + 1] = fast_exp2(x1);
        pv[c + 2] = fast_exp2(x2);
        pv[c + 3] = fast_exp2(x3);
      }
      if (partial) {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 tk = tok4[c >> 2];
          bool v0 = all_rows || tk.x >= at, v1 = all_rows || tk.y >= at;
          bool v2 = all_rows || tk.z >= at, v3 = all_rows || tk.w >= at;
          if (mixed) {  // padded queries hold -2, which no key's id equals
            // every lane takes part in the shuffles: none stands behind a condition that differs between lanes
            const int i0 = __shfl_sync(0xffffffffu, id, c), i1 = __shfl_sync(0xffffffffu, id, c + 1);
            const int i2 = __shfl_sync(0xffffffffu, id, c + 2), i3 = __shfl_sync(0xffffffffu, id, c + 3);
            v0 = v0 && i0 == my_doc;
            v1 = v1 && i1 == my_doc;
            v2 = v2 && i2 == my_doc;
            v3 = v3 && i3 == my_doc;
          }
          pv[c] = v0 ? pv[c] : 0.f;
          pv[c + 1] = v1 ? pv[c + 1] : 0.f;
          pv[c + 2] = v2 ? pv[c + 2] : 0.f;
          pv[c + 3] = v3 ? pv[c + 3] : 0.f;
          if (CAP) {  // a padded key's scores may be NaN
            w[c] = v0 ? w[c] : 0.f;
            w[c + 1] = v1 ? w[c + 1] : 0.f;
            w[c + 2] = v2 ? w[c + 2] : 0.f;
            w[c + 3] = v3 ? w[c + 3] : 0.f;
          }
        }
      }
      {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(pv[2 * c], pv[2 * c + 1]);
        tmem_st16u(tS, pk);  // over scores that this thread has read
      }
      if (CAP) {
#pragma unroll
        for (int c = 0; c < 32; c += 2)
          f2_unpack(f2_mul(f2_pack(pv[c], pv[c + 1]), f2_pack(w[c], w[c + 1])), pv[c], pv[c + 1]);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[half]);
      if (!mbar_wait_warp(&dp_full[half], i & 1, wctx, MCS_WHERE_ATTN_SOFTMAX)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld32(tP, w);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const float4 dl = dl4[c >> 2];
        f2_unpack(f2_mul(f2_pack(pv[c], pv[c + 1]), dp_less_d<CAP>(f2_pack(w[c], w[c + 1]), f2_pack(dl.x, dl.y))), w[c],
                  w[c + 1]);
        f2_unpack(f2_mul(f2_pack(pv[c + 2], pv[c + 3]), dp_less_d<CAP>(f2_pack(w[c + 2], w[c + 3]), f2_pack(dl.z, dl.w))),
                  w[c + 2], w[c + 3]);
      }
      if (partial) {  // a padded key's V may be NaN
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pv[c] == 0.f ? 0.f : w[c];
      }
      {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(w[2 * c], w[2 * c + 1]);
        tmem_st16u(tP, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&ds_full[half]);
    }
    const bool fin = ok && (n == 0 || mbar_wait_warp(done, 0, wctx, MCS_WHERE_ATTN_EPILOGUE));
    if (fin) {
      tc_fence_after();
      const size_t at = ((static_cast<size_t>(b) * p.Nk + key) * p.Hkv + hk) * D;
      // quarters 0 and 1 store the two halves of dV's columns, 2 and 3 those of dK's
      const int c0 = (quarter & 1) * (D / 2);
      if (p.part_kv)
        store_part<D / 2>(tmem + lane_addr + (quarter < 2 ? 256 : 384) + c0, n > 0, key_valid,
                          p.part_kv + (quarter < 2 ? 0 : p.kv_splits * p.kv_size) + split * p.kv_size + at + c0);
      else if (quarter < 2) store_row<D / 2>(tmem + lane_addr + 256 + c0, n > 0, key_valid, 1.f, p.dv + at + c0);
      else store_row<D / 2>(tmem + lane_addr + 384 + c0, n > 0, key_valid, p.scale, p.dk + at + c0);
    }
    __syncwarp();
  }
  teardown(abort_flag, done, kv_full, n > 0 ? 1 + 4 * C::NS : 0, tmem);
}

template <int D, bool CAP, bool BIAS, bool DOC, bool DELTA>
__device__ __forceinline__ void dq_tile(const CUtensorMap& tm_q, const CUtensorMap& tm_g, const CUtensorMap& tm_k,
                                        const CUtensorMap& tm_v, const ExTile& p, int cta) {
  using C = DqCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sG = smem + C::OFF_G;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* qg_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = qg_full + 1;
  uint64_t* v_full = k_full + C::NK;
  uint64_t* k_ok = v_full + C::NV;  // K's padded rows are clear (document masks)
  uint64_t* k_empty = k_ok + C::NK;
  uint64_t* v_empty = k_empty + C::NK;
  uint64_t* s_full = v_empty + C::NV;
  uint64_t* s_read = s_full + 1;
  uint64_t* dp_full = s_read + 1;  // [buffer]
  uint64_t* ds_full = dp_full + 2;  // [buffer]
  uint64_t* done = ds_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* count = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int BH = p.B * p.Hkv;
  int qt, bh;
  if (DOC && p.order) {
    int part;
    bh = ordered_job(p, p.order, p.Tq, cta, &qt, &part);
  } else if (p.causal) {  // the last query tiles see the most keys and go first
    const int per_chunk = p.chunk * p.Tq;
    const int ch = cta / per_chunk, in = cta % per_chunk;
    const int heads = min(p.chunk, BH - ch * p.chunk);
    bh = ch * p.chunk + in % heads;
    qt = p.Tq - 1 - in / heads;
  } else {
    qt = cta % p.Tq;
    bh = cta / p.Tq;
  }
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int off = p.Nk - p.Nq;
  const int prefix = p.prefix ? p.prefix[b] : 0;
  auto limit = [&](int pos) { return p.causal ? min(p.Nk, max(max(pos + 1, prefix), 0)) : p.Nk; };
  const int hi = (limit(off + min(p.Nq, (qt + 1) * p.tpt) - 1) + 127) >> 7;
  const int4 none = make_int4(0x7fffffff, static_cast<int>(0x80000000), 0, 0);
  const int4 mine = DOC ? p.q_ranges[static_cast<size_t>(b) * p.Tq + qt] : none;
  const int rt = p.tpt * p.g;

  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};
  auto load_resident = [&]() {
    mbar_arrive_expect_tx(qg_full, 2 * C::KB * rt * 128);
#pragma unroll
    for (int kb = 0; kb < C::KB; ++kb)
      for (int h = 0; h < p.tpt / p.qbox; ++h) {
        const int tok = qt * p.tpt + h * p.qbox;
        tma_load_4d(&tm_q, qg_full, sQ + kb * 16384 + h * 8192, kb * 64, hk * p.g, tok, b);
        tma_load_4d(&tm_g, qg_full, sG + kb * 16384 + h * 8192, kb * 64, hk * p.g, tok, b);
      }
  };
  // the loads of list entries j0 .. j1 - 1 (their tiles from `it`), for one thread
  auto load_keys = [&](TileIter& it, int j0, int j1) {
    for (int j = j0; j < j1; ++j) {
      const int sk = j % C::NK, sv = j % C::NV;
      const int kt = it.next();
      if (j >= C::NK && !mbar_wait(&k_empty[sk], ((j / C::NK) & 1) ^ 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
      if (!((p.debug_flags & (DELTA ? 65 : 33)) && j == 0)) {  // test knob: never deliver tile 0
        mbar_arrive_expect_tx(&k_full[sk], C::TILE);
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_4d(&tm_k, &k_full[sk], sK + sk * C::TILE + kb * 16384, kb * 64, hk, kt * 128, b);
      }
      if (j >= C::NV && !mbar_wait(&v_empty[sv], ((j / C::NV) & 1) ^ 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
      mbar_arrive_expect_tx(&v_full[sv], C::TILE);
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
        tma_load_4d(&tm_v, &v_full[sv], sV + sv * C::TILE + kb * 16384, kb * 64, hk, kt * 128, b);
    }
  };
  // without a document mask the list is known, and the first loads run beside the rest of the set-up
  const int early = DOC ? 0 : max(0, min(hi, C::NV));

  if (warp == 1 && elect_one()) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    mbar_init(qg_full, 1);
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_ok[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, kSoftThreads);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&dp_full[s], 1);
      mbar_init(&ds_full[s], kSoftThreads);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    count[0] = count[1] = count[2] = 0;
    fence_mbar_init();
    if (early > 0) {
      load_resident();
      TileIter it{0u, 0u, 0, 0};
      load_keys(it, 0, early);
    }
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (rt < 128) {
    zero_tail_rows<C::KB>(sQ, 2, rt);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int n = hi;
  TileBits tiles(smem_u32(smem + C::OFF_BITS), p.Tk);
  if (DOC) {
    tiles.build<false>(count, p.k_ranges + static_cast<size_t>(b) * p.Tk, 0, hi, mine, none);
    n = count[0];
  }
  const TileIter first{DOC ? tiles.meet : 0u, 0u, 0, 0};
  // TMEM: S | dP 0 | dQ | dP 1
  auto dp_buf = [&](int i) { return tmem + ((i & 1) ? 384u : 128u); };

  if (warp < 4) {
    if (warp == 0) {
      // ---------------------------------------------------------------- UMMA issuer
      if (n > 0 && elect_one()) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t IDESC_A = idesc_bf16_f32(128, D, false, true);
        const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dG = sdesc_sw128(smem_u32(sG), 16, 1024);
        const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024), dV = sdesc_sw128(smem_u32(sV), 16, 1024);
        const uint64_t dKm = sdesc_sw128(smem_u32(sK), 16384, 1024);
        auto scores = [&](uint32_t to, uint64_t a, uint64_t bb, uint64_t* bar) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_bf16_ss(to, sdesc_advance(a, o), sdesc_advance(bb, o), IDESC_S, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar);
        };
        auto wait = [&](uint64_t* bar, int k) { return mbar_wait(bar, k & 1, wctx, MCS_WHERE_ATTN_MMA); };
        TileIter it = first;
        // S(j) and dP(j): S is free once the softmax has read S(j - 1), dP's buffer once dQ(j - 2) was issued
        auto both = [&](int j) {
          if (j > 0 && !wait(s_read, j - 1)) return false;
          if (!wait(&k_full[j % C::NK], j / C::NK)) return false;
          if (DOC && tile_bit(tiles.pads, it.next()) && !wait(&k_ok[j % C::NK], j / C::NK)) return false;
          tc_fence_after();
          scores(tmem, dQ, sdesc_advance(dK, (j % C::NK) * C::TILE), s_full);
          if (!wait(&v_full[j % C::NV], j / C::NV)) return false;
          tc_fence_after();
          scores(dp_buf(j), dG, sdesc_advance(dV, (j % C::NV) * C::TILE), &dp_full[j & 1]);
          umma_commit(&v_empty[j % C::NV]);
          return true;
        };
        bool ok = wait(qg_full, 0) && both(0);
        for (int i = 0; ok && i < n; ++i) {
          if (i + 1 < n && !both(i + 1)) break;
          // no stage is released before the clearing warp has left it, so that warp is never a phase behind
          if (!wait(&ds_full[i & 1], i >> 1) || (DOC && !wait(&k_ok[i % C::NK], i / C::NK))) break;
          tc_fence_after();
          const uint64_t bb = sdesc_advance(dKm, (i % C::NK) * C::TILE);
#pragma unroll
          for (int kk = 0; kk < (DELTA ? 0 : 8); ++kk)
            umma_bf16_ts(tmem + 256, dp_buf(i) + (kk >> 1) * 32 + (kk & 1) * 8, sdesc_advance(bb, kk * 2048),
                         IDESC_A, (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&k_empty[i % C::NK]);
          if (i + 1 == n) umma_commit(done);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- TMA producer
      if (n > 0 && elect_one()) {
        if (early == 0) load_resident();
        TileIter it = first;
        it.cur += early;
        load_keys(it, early, n);
      }
      __syncwarp();
    } else if (warp == 2 && DOC) {
      // ---------------------------------------------------------------- padded keys
      TileIter it = first;
      for (int j = 0; j < n; ++j) {
        const int s = j % C::NK;
        if (!mbar_wait_warp(&k_full[s], (j / C::NK) & 1, wctx, MCS_WHERE_ATTN_PRODUCER)) break;
        const int kt = it.next();
        hold_cleaner(p);
        if (tile_bit(tiles.pads, kt)) {
          const size_t at = static_cast<size_t>(b) * p.Tk + kt;
          zero_padded_rows<C::KB>(sK + s * C::TILE, p.k_ids + at * 128);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_ok[s]);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- dS, then the epilogue
    const int quarter = (warp - 4) >> 2;  // keys 32 quarter .. 32 quarter + 31 of each tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const int tok = qt * p.tpt + row / p.g;
    const int head = hk * p.g + row % p.g;
    const bool row_valid = row < rt && tok < p.Nq;
    const float* st = p.stats + (static_cast<size_t>(bh) * p.Tq + qt) * 256;
    const float lse = row_valid ? p.lse_in[(static_cast<size_t>(b) * p.Hq + head) * p.Nq + tok] : -CUDART_INF_F;
    const float negl = lse == -CUDART_INF_F ? lse : -lse * kLog2e, delta = DELTA ? 0.f : st[128 + row];
    uint64_t d2 = 0;  // DELTA: the sum of P dP, over even and odd columns
    // DELTA: a row with a single key has D = dP to the bit, and so dS = 0 (the products give the same dP whichever operand
    // it is that stands on the lanes, which the tests check). Such a key's tile is partial for the row: the sum of dP
    // over the valid keys of partial tiles, and the number of keys (two for a whole tile).
    float one = 0.f;
    int keys = 0;
    const uint64_t negl2 = f2_pack(negl, negl), delta2 = f2_pack(delta, delta);
    const int pos = off + tok;
    const int lim = limit(pos) - quarter * 32;
    const int lim_all = limit(off + qt * p.tpt);
    const int my_doc = DOC ? p.q_ids[(static_cast<size_t>(b) * p.Tq + qt) * 128 + row] : 0;  // padding: -2
    const float mul = p.mul;
    const float slope = BIAS && row_valid ? slope_of(p.slopes, head) * kLog2e / mul : 0.f;
    if (BIAS && row_valid) check_slope(p.slopes, head, p.status);
    const uint64_t mul2 = f2_pack(mul, mul);
    TileIter it = first;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int kt = it.next();
      // where the tile's documents differ: the id of key `lane` of this quarter, under way while S is
      const bool mixed = DOC && !tile_bit(tiles.whole, kt);
      int id = 0;
      if (mixed) id = __ldg(p.k_ids + (static_cast<size_t>(b) * p.Tk + kt) * 128 + quarter * 32 + lane);
      const bool partial = mixed || (kt + 1) * 128 > lim_all;
      if (!mbar_wait_warp(s_full, i & 1, wctx, MCS_WHERE_ATTN_SOFTMAX)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float pv[32];  // score, P, then with a cap P (t^2 - 1)
      float w[32];   // t^2 - 1
      tmem_ld32(tmem + lane_addr + quarter * 32, pv);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(s_read);
      if (CAP) {
        cap_scores<32>(pv, p.cap);
#pragma unroll
        for (int c = 0; c < (DELTA ? 0 : 32); c += 2) f2_unpack(cap_slope2(f2_pack(pv[c], pv[c + 1]), p.cap), w[c], w[c + 1]);
      }
      uint64_t e2 = negl2;
      if (BIAS) {
        const float e = fmaf(add_bias<32>(pv, slope, static_cast<float>(pos - kt * 128 - quarter * 32)), mul, negl);
        e2 = f2_pack(e, e);
      }
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(pv[c], pv[c + 1]), mul2, e2), x0, x1);
        pv[c] = fast_exp2(x0);
        pv[c + 1] = fast_exp2(x1);
      }
      if (CAP && !DELTA) {
#pragma unroll
        for (int c = 0; c < 32; c += 2)
          f2_unpack(f2_mul(f2_pack(pv[c], pv[c + 1]), f2_pack(w[c], w[c + 1])), pv[c], pv[c + 1]);
      }
      int found = 0;  // DELTA: this row's keys of a mixed tile
      if (partial) {
        const int valid = lim - kt * 128;
        if (mixed) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int i_c = __shfl_sync(0xffffffffu, id, c);  // every lane takes part
            const bool in = c < valid && i_c == my_doc;
            pv[c] = in ? pv[c] : 0.f;
            if (DELTA) found += in;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) pv[c] = c < valid ? pv[c] : 0.f;
        }
      }
      const uint32_t tP = dp_buf(i) + lane_addr + quarter * 32;
      if (!mbar_wait_warp(&dp_full[i & 1], (i >> 1) & 1, wctx, MCS_WHERE_ATTN_SOFTMAX)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld32(tP, w);
      tmem_wait_ld();
      if (partial) {  // a padded key's V, a padded query's d_o may be NaN
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pv[c] == 0.f ? 0.f : w[c];
      }
      if (DELTA) {
        if (partial) {
#pragma unroll
          for (int c = 0; c < 32; ++c) one += w[c];
        }
        keys += !partial ? 2 : mixed ? found : min(max(lim - kt * 128, 0), 32);
#pragma unroll
        for (int c = 0; c < 32; c += 2) d2 = f2_fma(f2_pack(pv[c], pv[c + 1]), f2_pack(w[c], w[c + 1]), d2);
      } else {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float a, b2;
          f2_unpack(f2_mul(f2_pack(pv[c], pv[c + 1]), dp_less_d<CAP>(f2_pack(w[c], w[c + 1]), delta2)), a, b2);
          pk[c / 2] = pack_bf16(a, b2);
        }
        tmem_st16u(tP, pk);  // over dP columns that this thread has read
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&ds_full[i & 1]);
    }
    const bool fin = ok && (n == 0 || mbar_wait_warp(done, 0, wctx, MCS_WHERE_ATTN_EPILOGUE));
    if (DELTA) {
      // the four quarters' sums, added in order; the ring has no reader or writer left
      float* sums = reinterpret_cast<float*>(sK);
      float even, odd;
      f2_unpack(d2, even, odd);
      sums[quarter * 128 + row] = even + odd;
      sums[512 + quarter * 128 + row] = one;
      reinterpret_cast<int*>(sums)[1024 + quarter * 128 + row] = keys;
      named_barrier_sync<2, 512>();
      if (fin && quarter == 0) {
        const bool live = negl != -CUDART_INF_F;  // NaN passes on
        float* out = p.stats_out + (static_cast<size_t>(bh) * p.Tq + qt) * 256;
        out[row] = BIAS && live ? fmaf(-slope_of(p.slopes, head) * kLog2e, static_cast<float>(row / p.g), negl) : negl;
        const int* nk = reinterpret_cast<const int*>(sums) + 1024 + row;
        const float* from = sums + ((nk[0] + nk[128]) + (nk[256] + nk[384]) == 1 ? 512 : 0) + row;
        out[128 + row] = live ? (from[0] + from[128]) + (from[256] + from[384]) : 0.f;
      }
    } else if (fin) {
      tc_fence_after();
      // each quarter of the warps stores its quarter of the columns
      const int c0 = quarter * (D / 4);
      uint16_t* dst = p.dq + ((static_cast<size_t>(b) * p.Nq + tok) * p.Hq + head) * D + c0;
      store_row<D / 4>(tmem + lane_addr + 256 + c0, n > 0, row_valid, p.scale, dst);
    }
    __syncwarp();
  }
  teardown(abort_flag, done, qg_full, n > 0 ? 1 + C::NK + C::NV : 0, tmem);
}

template <int D, bool CAP, bool BIAS, bool DOC>
__global__ void __launch_bounds__(kThreads, 1)
    ex_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_g,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const ExTile p) {
  next_may_start();
  await_previous();
  const int keys = p.B * p.Hkv * p.Tk * p.kv_splits;
  if (static_cast<int>(blockIdx.x) < keys) dkv_tile<D, CAP, BIAS, DOC>(tm_q, tm_g, tm_k, tm_v, p, blockIdx.x);
  else dq_tile<D, CAP, BIAS, DOC, false>(tm_q, tm_g, tm_k, tm_v, p, blockIdx.x - keys);
}

// The rows' statistics with D summed from P dP in fp32 (see ex_row_stats).
template <int D, bool CAP, bool BIAS, bool DOC>
__global__ void __launch_bounds__(kThreads, 1)
    ex_delta_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_g,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const ExTile p) {
  next_may_start();
  await_previous();
  dq_tile<D, CAP, BIAS, DOC, true>(tm_q, tm_g, tm_k, tm_v, p, blockIdx.x);
}

namespace {

// dV and dK as the sums of their parts over the query tiles, in the parts' order; four values per thread.
__global__ void __launch_bounds__(256) ex_sum_parts(const ExTile p) {
  next_may_start();
  await_previous();
  const size_t quads = p.kv_size / 4;
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= 2 * quads) return;
  const bool key = i >= quads;
  const size_t at = key ? i - quads : i;
  const float4* src = reinterpret_cast<const float4*>(p.part_kv) + (key ? p.kv_splits * quads : 0) + at;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < p.kv_splits; ++s) {
    const float4 x = src[s * quads];
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
  }
  const float f = key ? p.scale : 1.f;
  reinterpret_cast<uint2*>(key ? p.dk : p.dv)[at] = make_uint2(pack_bf16(a.x * f, a.y * f), pack_bf16(a.z * f, a.w * f));
}

template <int D, bool CAP, bool BIAS, bool DOC>
cudaError_t launch_bwd(const CUtensorMap* tq, const CUtensorMap* tg, const CUtensorMap* tk, const CUtensorMap* tv,
                       const ExTile& p, cudaStream_t s) {
  static KernelReady ready;
  auto kern = ex_bwd_kernel<D, CAP, BIAS, DOC>;
  constexpr unsigned most_kv = DkvCfg<D>::SMEM + 24576, most_q = DqCfg<D>::SMEM + 1536;  // 2^16 and 2^12 tiles
  const cudaError_t e = make_ready(ready, kern, std::max(most_kv, most_q), 0);
  if (e != cudaSuccess) return e;
  const unsigned smem = std::max(DkvCfg<D>::SMEM + (DOC ? (p.Tq + 31) / 32 * 12u : 0u),
                                 DqCfg<D>::SMEM + (DOC ? (p.Tk + 31) / 32 * 12u : 0u));
  if (!p.d_from_o) {
    static KernelReady ready_delta;
    auto delta = ex_delta_kernel<D, CAP, BIAS, DOC>;
    const cudaError_t e2 = make_ready(ready_delta, delta, most_q, 0);
    if (e2 != cudaSuccess) return e2;
    const unsigned smem_delta = DqCfg<D>::SMEM + (DOC ? (p.Tk + 31) / 32 * 12u : 0u);
    const cudaError_t e3 = launch_in_sequence(delta, p.B * p.Hkv * p.Tq, kThreads, smem_delta, s, DOC, *tq, *tg, *tk,
                                              *tv, p);
    if (e3 != cudaSuccess) return e3;
  }
  const cudaError_t e4 = launch_in_sequence(kern, p.B * p.Hkv * (p.Tk * p.kv_splits + p.Tq), kThreads, smem, s, true, *tq,
                                            *tg, *tk, *tv, p);
  if (e4 != cudaSuccess || !p.part_kv) return e4;
  return launch_in_sequence(ex_sum_parts, static_cast<unsigned>((p.kv_size / 2 + 255) / 256), 256, 0, s, true, p);
}

}  // namespace

cudaError_t launch_ex_row_stats(int d, const ExTile& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.B) * p.Hkv * p.Tq;
  return launch_in_sequence(d == 64 ? ex_row_stats<64> : ex_row_stats<128>, grid, 256, 0, s, p.doc_q != nullptr, p);
}

cudaError_t launch_ex_bwd(int d, const CUtensorMap* tq, const CUtensorMap* tg, const CUtensorMap* tk,
                          const CUtensorMap* tv, const ExTile& p, cudaStream_t s) {
  return with_options(d, p, [&](auto D, auto CAP, auto BIAS, auto DOC) {
    return launch_bwd<D.value, CAP.value, BIAS.value, DOC.value>(tq, tg, tk, tv, p, s);
  });
}

}  // namespace mcs
