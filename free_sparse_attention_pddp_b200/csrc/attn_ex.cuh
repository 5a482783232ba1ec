// Shared by the kernels of the attention with modified scores: packed query
// tiles, tile lists, the score's cap and bias, padded rows.
//
// Packed query tiles. The g = Hq / Hkv query heads of a KV head meet the same
// keys, so a 128-row tile holds TPT = floor(128 / g) tokens times g heads: row
// r is head r % g of token tile * TPT + r / g. One product then serves the
// whole group, a short query keeps its rows full, and a causal tile's diagonal
// is only TPT tokens wide. Rows from TPT * g on (g not a power of two) and of
// tokens past Nq are empty.
#pragma once
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "mcs_ptx.cuh"

namespace mcs {

// Calls f with the head size and the call's options as compile-time constants.
// One kernel per combination: the options' code in one body overflows the
// instruction cache (with all of it the capped dK/dV and dQ passes ran 1.29
// times as long on 37 heads of 8192 tokens).
template <typename F>
cudaError_t with_options(int d, const ExTile& p, F f) {
  using T = std::true_type;
  using N = std::false_type;
  auto pick = [&](auto D) {
    const int which = (p.cap.on ? 4 : 0) + (p.slopes ? 2 : 0) + (p.k_ranges ? 1 : 0);
    switch (which) {
      case 0: return f(D, N{}, N{}, N{});
      case 1: return f(D, N{}, N{}, T{});
      case 2: return f(D, N{}, T{}, N{});
      case 3: return f(D, N{}, T{}, T{});
      case 4: return f(D, T{}, N{}, N{});
      case 5: return f(D, T{}, N{}, T{});
      case 6: return f(D, T{}, T{}, N{});
      default: return f(D, T{}, T{}, T{});
    }
  };
  if (d == 64) return pick(std::integral_constant<int, 64>{});
  return pick(std::integral_constant<int, 128>{});
}

// CTA of the tile kernels: warp 0 issues the UMMAs, warp 1 the TMA loads, warp
// 2 clears padded rows, warp 3 only completes their warpgroup; 16 softmax warps,
// four to each SM sub-partition, so that one warp's TMEM loads, barriers and
// dependent arithmetic hide behind the others' exponentials. (37 heads of 8192
// tokens, d = 128, forward, against 8 softmax warps of twice the columns, when
// both were built: capped scores 10 % and biased 7 % faster, plain the same.) In the
// forward kernel setmaxnreg moves registers from the first warpgroup to the
// softmax; the gradients' kernel runs at the launch's count.
constexpr int kExThreads = 640;
constexpr int kExLaunchRegs = 96;
constexpr int kExLowRegs = 64;
constexpr int kExSoftRegs = 104;
static_assert(128 * kExLowRegs + 512 * kExSoftRegs <= kExThreads * kExLaunchRegs, "register split");

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int ID, int NTHREADS>
__device__ __forceinline__ void named_barrier_sync() {
  asm volatile("barrier.sync %0, %1;" ::"n"(ID), "n"(NTHREADS) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float2 lds_pair(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_pair(uint32_t addr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// What a maximum of -inf is counted from: the weights of parts that saw no key
// are 2^-inf = 0, and NaN sums come through.
__device__ __forceinline__ float top_or_zero(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// Tiles from `cur` on in order; with bitmaps (shared-memory addresses), those
// that are in one of them (bit 0 of word 0 is tile `base`).
struct TileIter {
  uint32_t bits, bits2;  // 0: every tile, no second bitmap
  int cur, base;
  __device__ __forceinline__ uint32_t word(int w) const {
    return bits2 ? lds32(bits + w * 4) | lds32(bits2 + w * 4) : lds32(bits + w * 4);
  }
  __device__ __forceinline__ int next() {
    if (!bits) return cur++;
    int i = cur - base;
    uint32_t w = word(i >> 5) >> (i & 31);
    while (!w) {  // the caller asks for no more tiles than there are
      i = (i | 31) + 1;
      w = word(i >> 5);
    }
    i += __ffs(w) - 1;
    cur = base + i + 1;
    return base + i;
  }
};

// The entries of a forward CTA's K/V ring in order: one list of tiles or, zipped,
// a's and b's tiles in turn for as long as both have some.
struct EntryIter {
  TileIter a, b;
  int both;     // zipped: tiles of the shorter list, else 0
  bool a_long;  // whose tiles remain
  int i = 0;
  __device__ __forceinline__ int next() {
    const bool from_a = i < 2 * both ? !(i & 1) : a_long;
    ++i;
    return from_a ? a.next() : b.next();
  }
};

// Document ids of a tile: smallest and largest id of its rows that are not
// padding (an empty tile: INT_MAX, INT_MIN) and whether any row is padding.
__device__ __forceinline__ bool docs_meet(int4 a, int4 b) { return a.x <= b.y && b.x <= a.y; }
__device__ __forceinline__ bool docs_same(int4 a, int4 b) {  // every pair of rows is valid
  return a.x == a.y && b.x == b.y && a.x == b.x && !a.z && !b.z;
}

// What a document mask makes of tiles lo .. hi - 1, as bitmaps in shared memory:
// those whose documents meet the CTA's tile, those of whose pairs with it every
// one is valid, and those with padding. `two`: for two tiles at once, the second
// one's bitmaps behind the first one's.
struct TileBits {
  uint32_t meet, whole, pads, meet2, whole2;  // shared-memory addresses
  __device__ __forceinline__ TileBits(uint32_t at, int tiles) {
    const int w = ((tiles + 31) >> 5) * 4;
    meet = at;
    whole = at + w;
    pads = at + 2 * w;
    meet2 = at + 3 * w;
    whole2 = at + 4 * w;
  }
  // All threads of the CTA call it. counts: three shared words, zero before: tiles that meet either, `mine`, `mine2`.
  template <bool TWO>
  __device__ __forceinline__ void build(int* counts, const int4* ranges, int lo, int hi, int4 mine, int4 mine2) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int w = warp; w * 32 < hi - lo; w += warps) {
      const int t = lo + w * 32 + lane;
      int4 r = make_int4(0x7fffffff, static_cast<int>(0x80000000), 0, 0);
      if (t < hi) r = ranges[t];
      const uint32_t m = __ballot_sync(0xffffffffu, docs_meet(r, mine));
      const uint32_t a = __ballot_sync(0xffffffffu, docs_same(r, mine));
      const uint32_t z = __ballot_sync(0xffffffffu, r.z != 0);
      uint32_t m2 = 0, a2 = 0;
      if (TWO) {
        m2 = __ballot_sync(0xffffffffu, docs_meet(r, mine2));
        a2 = __ballot_sync(0xffffffffu, docs_same(r, mine2));
      }
      if (lane == 0) {
        sts32(meet + w * 4, m);
        sts32(whole + w * 4, a);
        sts32(pads + w * 4, z);
        if (TWO) {
          sts32(meet2 + w * 4, m2);
          sts32(whole2 + w * 4, a2);
        }
        atomicAdd(&counts[0], __popc(m | m2));  // whole-number sums: their order is free
        atomicAdd(&counts[1], __popc(m));
        atomicAdd(&counts[2], __popc(m2));
      }
    }
    __syncthreads();
  }
};
__device__ __forceinline__ bool tile_bit(uint32_t bits, int i) { return (lds32(bits + (i >> 5) * 4) >> (i & 31)) & 1u; }

// s[c] <- cap log2(e) tanh(k s[c]), the capped score in log2 units, in place (s times
// f.pre first, where that is not 1). |k s| <= 0.625: s Q(s^2) with Q from x + x z P(z), z = x^2, P of degree 3
// fitted to (tanh(x)/x - 1)/z by iteratively reweighted least squares on the
// relative error of tanh (1.3e-7 at most); up to 0.4 degree 2 is as exact. The
// factors k and cap log2(e) are in Q's coefficients: six (five) packed FMAs per
// pair. Beyond, 1 - 2 / (1 + 2^(2 |x| log2 e)), whose approximate exponential and
// reciprocal leave about 2e-7. A warp takes the widest form that one of its 16
// columns needs: scores of trained models mostly lie well inside the cap, and
// the polynomials cost no MUFU slot (two for the last form, in kernels that
// already use one per score).
__device__ __forceinline__ float cap_far(float s, const CapFn& f) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(fabsf(s) * f.k2)));
  return copysignf(fmaf(-2.f * f.cl, r, f.cl), s);
}
template <int N>
__device__ __forceinline__ void cap_scores(float* s, const CapFn& f) {
  constexpr int W = N < 16 ? N : 16;
  if (f.pre != 1.f) {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] *= f.pre;
  }
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += W) {
    float* v = s + c0;
    uint64_t z[W / 2];
    float big = 0.f;
#pragma unroll
    for (int c = 0; c < W / 2; ++c) {
      const uint64_t x = f2_pack(v[2 * c], v[2 * c + 1]);
      z[c] = f2_mul(x, x);
      float z0, z1;
      f2_unpack(z[c], z0, z1);
      big = fmax3(big, z0, z1);
    }
    if (__all_sync(0xffffffffu, big <= f.z2)) {
      const uint64_t b0 = f2_pack(f.b[0], f.b[0]), b1 = f2_pack(f.b[1], f.b[1]);
      const uint64_t b2 = f2_pack(f.b[2], f.b[2]), b3 = f2_pack(f.b[3], f.b[3]);
#pragma unroll
      for (int c = 0; c < W / 2; ++c)
        f2_unpack(f2_mul(f2_pack(v[2 * c], v[2 * c + 1]), f2_fma(f2_fma(f2_fma(b3, z[c], b2), z[c], b1), z[c], b0)),
                  v[2 * c], v[2 * c + 1]);
    } else {
      const uint64_t a0 = f2_pack(f.a[0], f.a[0]), a1 = f2_pack(f.a[1], f.a[1]), a2 = f2_pack(f.a[2], f.a[2]);
      const uint64_t a3 = f2_pack(f.a[3], f.a[3]), a4 = f2_pack(f.a[4], f.a[4]);
      const bool far = !__all_sync(0xffffffffu, big <= f.z3);
#pragma unroll
      for (int c = 0; c < W / 2; ++c) {
        const float s0 = v[2 * c], s1 = v[2 * c + 1];
        f2_unpack(f2_mul(f2_pack(s0, s1), f2_fma(f2_fma(f2_fma(f2_fma(a4, z[c], a3), z[c], a2), z[c], a1), z[c], a0)),
                  v[2 * c], v[2 * c + 1]);
        if (far) {
          float z0, z1;
          f2_unpack(z[c], z0, z1);
          v[2 * c] = z0 <= f.z3 ? v[2 * c] : cap_far(s0, f);
          v[2 * c + 1] = z1 <= f.z3 ? v[2 * c + 1] : cap_far(s1, f);
        }
      }
    }
  }
}

// tanh^2 - 1 from a capped score: minus the cap's slope, so that no square of the cap is needed
__device__ __forceinline__ uint64_t cap_slope2(uint64_t y, const CapFn& f) {
  const uint64_t t = f2_mul(y, f2_pack(f.icl, f.icl));
  return f2_fma(t, t, f2_pack(-1.f, -1.f));
}
// dP - D; its negative beside the cap's negative slope
template <bool CAP>
__device__ __forceinline__ uint64_t dp_less_d(uint64_t dp, uint64_t d) {
  return CAP ? f2_sub(d, dp) : f2_sub(dp, d);
}

// A head's slope, within +-64. The tiles add the bias as slope (c - base) with the two products rounded by themselves
// (add_bias below, the statistics of dK/dV), which leaves up to 2^-15 |slope| in a score, 2^-9 at the bound; and
// within it no distance makes the bias infinite.
constexpr float kMaxSlope = 64.f;
__device__ __forceinline__ float slope_of(const float* slopes, int head) {
  return fminf(fmaxf(slopes[head], -kMaxSlope), kMaxSlope);
}
// Reports a slope outside the bound, or NaN.
__device__ __forceinline__ void check_slope(const float* slopes, int head, int* status) {
  if (!(fabsf(slopes[head]) <= kMaxSlope)) record_status(status, MCS_ERR_INVALID_ARG, head);
}

// Distance bias of a row: s[c] <- s[c] - slope |base - c| - r, where `base` is the
// distance at c = 0 and the returned r is the same for the whole row. Where the
// warp's distances all have one sign the bias is linear in c, and r = -slope base
// leaves one FMA with an immediate per score.
template <int N>
__device__ __forceinline__ float add_bias(float* s, float slope, float base) {
  const bool pos = __all_sync(0xffffffffu, base >= static_cast<float>(N - 1));
  const bool neg = __all_sync(0xffffffffu, base <= 0.f);
  if (pos || neg) {
    const float sl = pos ? slope : -slope;
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(sl, static_cast<float>(c), s[c]);
    return -sl * base;
  }
#pragma unroll
  for (int c = 0; c < N; ++c) s[c] = fmaf(-slope, fabsf(base - static_cast<float>(c)), s[c]);
  return 0.f;
}

// CTA u of an ordered launch: chunk by chunk of heads (whose K and V fit L2
// together), the B x jobs jobs in their order, the chunk's heads side by side.
// Returns b Hkv + head (-1: no work is left for this CTA), the job and its part:
// 0 the whole job, 1 and 2 the first and the second query tile of a pair.
__device__ __forceinline__ int ordered_job(const ExTile& p, const int* order, int jobs, int u, int* job, int* part) {
  const int most = min(p.Hkv, max(1, p.chunk / p.B)), all = order[0];
  const int ch = u / (most * all), in = u % (most * all);
  const int heads = min(most, p.Hkv - ch * most);
  if (heads <= 0 || in >= heads * all) return -1;
  const int entry = order[1 + in / heads], at = entry >> 2;
  *part = entry & 3;
  *job = at % jobs;
  return at / jobs * p.Hkv + ch * most + in % heads;
}

// Test knob: the warp that clears padded rows falls 20 us behind in every tile, which is ten steps.
__device__ __forceinline__ void hold_cleaner(const ExTile& p) {
  if (p.debug_flags & 8) __nanosleep(20000);
}

// Zeroes the rows of a swizzled tile (KB column blocks of 128 rows x 128 bytes)
// whose document id is negative, so that whatever padding holds (NaN) meets
// the zero probabilities of its row as zero. One warp; `ids`: 128 document ids.
template <int KB>
__device__ __forceinline__ void zero_padded_rows(uint8_t* tile, const int* ids) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t m = __ballot_sync(0xffffffffu, ids[w * 32 + lane] < 0);
    while (m) {
      const int r = w * 32 + __ffs(m) - 1;
      m &= m - 1;
      if (lane < KB * 8)
        *reinterpret_cast<uint4*>(tile + (lane >> 3) * 16384 + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
}

}  // namespace mcs
