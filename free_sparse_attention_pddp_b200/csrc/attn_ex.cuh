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

#include "mcs_ptx.cuh"

namespace mcs {

// CTA of the tile kernels: warp 0 issues the UMMAs, warp 1 the TMA loads, warp
// 2 clears padded rows, warp 3 only completes their warpgroup; 16 softmax warps,
// four to each SM sub-partition, so that one warp's TMEM loads, barriers and
// dependent arithmetic hide behind the others' exponentials. (With 8 softmax
// warps of twice the columns the forward kernel ran at 1004 instead of XXXX
// TFLOP/s on 37 heads of 8192 tokens, d = 128.) setmaxnreg moves registers from
// the first warpgroup to the softmax.
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

// Tiles lo .. hi - 1 in order; with a bitmap (bit 0 of word 0: tile lo's
// 32-aligned start), only those whose bit is set.
struct TileIter {
  const uint32_t* bits;  // null: every tile
  int cur, base;         // next candidate; tile of bit 0
  __device__ __forceinline__ int next() {
    if (!bits) return cur++;
    int i = cur - base;
    uint32_t w = bits[i >> 5] >> (i & 31);
    while (!w) {  // the caller asks for no more tiles than there are
      i = (i | 31) + 1;
      w = bits[i >> 5];
    }
    i += __ffs(w) - 1;
    cur = base + i + 1;
    return base + i;
  }
};

// Document ids of a tile: smallest and largest id of its rows that are not
// padding (an empty tile: INT_MAX, INT_MIN) and whether any row is padding.
__device__ __forceinline__ bool docs_meet(int4 a, int4 b) { return a.x <= b.y && b.x <= a.y; }
__device__ __forceinline__ bool docs_same(int4 a, int4 b) {  // every pair of rows is valid
  return a.x == a.y && b.x == b.y && a.x == b.x && !a.z && !b.z;
}

// Sets, for tiles lo .. hi - 1, the bits of those whose documents meet `mine`
// (or `mine2`), and returns their number to every thread. All threads of the
// CTA call it. `count` is a shared word that is zero before.
__device__ __forceinline__ int build_tile_bits(uint32_t* bits, int* count, const int4* ranges, int lo, int hi,
                                               int4 mine, int4 mine2) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int w = warp; w * 32 < hi - lo; w += warps) {
    const int t = lo + w * 32 + lane;
    bool on = false;
    if (t < hi) {
      const int4 r = ranges[t];
      on = docs_meet(r, mine) || docs_meet(r, mine2);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, on);
    if (lane == 0) {
      bits[w] = m;
      if (m) atomicAdd(count, __popc(m));  // a whole-number sum: its order is free
    }
  }
  __syncthreads();
  return *count;
}

// tanh(x) of 2 n arguments that are k times the values of s, in place.
// |x| <= 0.625: x + x z P(z), z = x^2, P of degree 3 fitted to (tanh(x)/x - 1)/z
// by iteratively reweighted least squares on the relative error of tanh
// (1.3e-7 at most); beyond, 1 - 2 / (1 + 2^(2 x log2 e)), whose approximate
// exponential and reciprocal leave about 2e-7. A warp takes the second form
// only if one of its values needs it: scores of trained models mostly lie well
// inside the cap, and the polynomial costs no MUFU slot (two for the other
// form, in kernels that already use one per score).
template <int N>
__device__ __forceinline__ void tanh_scaled(float* s, float k) {
  float big = 0.f;
#pragma unroll
  for (int c = 0; c < N; ++c) big = fmaxf(big, fabsf(s[c]));
  const bool far = __any_sync(0xffffffffu, !(big * k <= 0.625f));
  const uint64_t kk = f2_pack(k, k);
  const uint64_t c0 = f2_pack(-0.333323412f, -0.333323412f), c1 = f2_pack(0.133081745f, 0.133081745f);
  const uint64_t c2 = f2_pack(-0.0519478787f, -0.0519478787f), c3 = f2_pack(0.0151953385f, 0.0151953385f);
  if (!far) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint64_t x = f2_mul(f2_pack(s[c], s[c + 1]), kk);
      const uint64_t z = f2_mul(x, x);
      const uint64_t p = f2_fma(f2_fma(f2_fma(c3, z, c2), z, c1), z, c0);
      f2_unpack(f2_fma(f2_mul(x, z), p, x), s[c], s[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float x = s[c] * k, z = x * x;
      const float p = fmaf(fmaf(fmaf(0.0151953385f, z, -0.0519478787f), z, 0.133081745f), z, -0.333323412f);
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(fabsf(x) * (2.f * kLog2e))));
      const float t = copysignf(fmaf(-2.f, r, 1.f), x);
      s[c] = fabsf(x) <= 0.625f ? fmaf(x * z, p, x) : t;
    }
  }
}

// tanh_scaled over N values, 32 at a time
template <int N>
__device__ __forceinline__ void tanh_all(float* s, float k) {
#pragma unroll
  for (int c = 0; c < N; c += 32) tanh_scaled<32>(s + c, k);
}

// s[c] <- mul * s[c] - slope * |base - c * step| for c < N (log2 units). `base` is the
// distance at c = 0. Where the warp's distances all have one sign the bias is
// linear in c: two packed FMAs per pair.
template <int N>
__device__ __forceinline__ void add_bias(float* s, float mul, float slope, float base, float step) {
  const float end = base - step * (N - 1);
  const bool pos = __all_sync(0xffffffffu, base >= 0.f && end >= 0.f);
  const bool neg = __all_sync(0xffffffffu, base <= 0.f && end <= 0.f);
  if (pos || neg) {
    const float sl = pos ? slope : -slope;
    const uint64_t m2 = f2_pack(mul, mul), t0 = f2_pack(-sl * base, -sl * base), s2 = f2_pack(sl * step, sl * step);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint64_t b = f2_fma(s2, f2_pack(static_cast<float>(c), static_cast<float>(c + 1)), t0);
      f2_unpack(f2_fma(m2, f2_pack(s[c], s[c + 1]), b), s[c], s[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(mul, s[c], -slope * fabsf(fmaf(-step, static_cast<float>(c), base)));
  }
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
