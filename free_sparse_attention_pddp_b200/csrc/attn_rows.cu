// Single tokens over a cache, one warp per row: the plainest form of
// mcs_decode and mcs_decode_shared.
//
// A warp walks its row's partners 32 at a time. Lane l forms the score of
// partner l (an fp32 dot product over d), the warp keeps a running maximum and
// sum, and each lane accumulates d/32 columns of the output.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "mcs_ptx.cuh"

namespace mcs {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ uint16_t to_bf(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// dot product of a row in shared memory (fp32) with a bf16 row in global memory
template <int D>
__device__ __forceinline__ float dot(const float* a, const uint16_t* row) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w = reinterpret_cast<const uint4*>(row)[c];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(a[c * 8 + 2 * e], __uint_as_float(u[e] << 16), s);
      s = fmaf(a[c * 8 + 2 * e + 1], __uint_as_float(u[e] & 0xffff0000u), s);
    }
  }
  return s;
}

// score from the scaled product; t receives tanh(x / cap) (0 without a cap)
__device__ __forceinline__ float score(float x, float cap, float slope, float dist, float& t) {
  t = 0.f;
  if (cap > 0.f) {
    t = tanhf(x / cap);
    x = cap * t;
  }
  return x - slope * dist;
}

template <int D>
struct RowAcc {
  static constexpr int E = D / 32;  // columns of a lane
  float a[E] = {};
  __device__ void scale(float f) {
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] *= f;
  }
  __device__ void add(float w, const uint16_t* row, int lane) {
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = fmaf(w, bf(row[lane * E + e]), a[e]);
  }
  __device__ void store(uint16_t* row, int lane, float f) const {
#pragma unroll
    for (int e = 0; e < E; ++e) row[lane * E + e] = to_bf(a[e] * f);
  }
};

template <int D>
__global__ void rows_decode(const DecodeParams p) {
  __shared__ float sq[kWarps][D];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + w;  // (b, h)
  if (row >= static_cast<long long>(p.B) * p.Hq) return;
  const int h = row % p.Hq, b = row / p.Hq, hk = h / p.g;
  for (int c = lane; c < D; c += 32) sq[w][c] = bf(p.q[row * D + c]);
  __syncwarp();
  int n = p.lens[b];
  if (n < 0 || n > p.C) {
    if (lane == 0) record_status(p.status, MCS_ERR_BAD_INDEX, n);
    n = n < 0 ? 0 : p.C;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  const int pos = p.P + n - 1;
  float m = -CUDART_INF_F, l = 0.f;
  RowAcc<D> acc;
  for (int part = 0; part < 2; ++part) {
    const int keys = part ? n : p.P, base = part ? p.P : 0;
    const uint16_t* K = part ? p.k + static_cast<size_t>(b) * p.C * p.Hkv * D : p.kp;
    const uint16_t* V = part ? p.v + static_cast<size_t>(b) * p.C * p.Hkv * D : p.vp;
    for (int j0 = 0; j0 < keys; j0 += 32) {
      const int j = j0 + lane;
      float s = -CUDART_INF_F, t;
      if (j < keys)
        s = score(p.scale * dot<D>(sq[w], K + (static_cast<size_t>(j) * p.Hkv + hk) * D), p.cap, slope,
                  fabsf(static_cast<float>(pos - base - j)), t);
      const float mn = fmaxf(m, warp_max(s));
      const float pr = expf(s - mn), alpha = expf(m - mn);
      m = mn;
      l = l * alpha + warp_sum(pr);
      acc.scale(alpha);
      for (int e = 0; e < 32 && j0 + e < keys; ++e)
        acc.add(__shfl_sync(0xffffffffu, pr, e), V + (static_cast<size_t>(j0 + e) * p.Hkv + hk) * D, lane);
    }
  }
  acc.store(p.o + row * D, lane, l > 0.f ? 1.f / l : 0.f);
  if (p.lse && lane == 0) p.lse[row] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
}

unsigned blocks(long long rows) { return static_cast<unsigned>((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_decode_rows(int d, const DecodeParams& p, cudaStream_t s) {
  const unsigned n = blocks(static_cast<long long>(p.B) * p.Hq);
  if (d == 64) rows_decode<64><<<n, kWarps * 32, 0, s>>>(p);
  else rows_decode<128><<<n, kWarps * 32, 0, s>>>(p);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace mcs
