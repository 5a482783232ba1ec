// One token per request over a cache (mcs_decode), and the join of its parts
// with those of a shared prefix (mcs_decode_shared, whose prefix runs on the
// forward kernel with all requests' rows packed into tiles).
//
// What bounds it: reading K and V once from HBM. The g query heads of a KV
// head are the 16 rows of mma.sync m16n8k16 tiles, which is arithmetic enough
// (g multiply-adds per byte) without tcgen05's 128-row tiles.
//
// A CTA takes one request, one KV head and one chunk of its keys. Its four
// warps are independent: each streams every fourth block of 16 keys through
// its own cp.async ring in shared memory (no block barrier in the loop) and
// keeps its own running maximum, sum and output; the four are joined at the
// end, the chunks by decode_combine or, where at most eight chunks of every
// request fit one wave, by the CTAs themselves as a cluster (one launch: 9 us
// instead of 12 from Python for a single request's 480 keys). Keys past the request's length are never
// read (cp.async fills zeros), so the cache may hold anything there.
//
// 1 request of 75600 keys (8 KV heads, 40 query heads, d = 128): 51 us for 310 MB,
// 6.1 TB/s of the 6.46 that a copy reaches, and 5 us for the join; 64 requests
// of ragged lengths run at a copy's rate. Up to 16 query heads to a KV head take one
// 16-row tile; up to 32 two, which is arithmetic beyond the loads (16 requests of
// 16384 keys of one KV head, d = 128: 16 heads 38 us, 32 heads 56); more go to several
// CTAs, each of which reads the cache (64 heads 89, 128 heads 153 us).
//
// P is split into two bf16 terms for P V: the products are free here, and the
// output keeps fp32 accuracy.
#include "attn_ex.cuh"

namespace mcs {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 16;      // keys of a block
constexpr int kStages = 3;      // blocks in a warp's ring
constexpr float kRescale = 4.0f;  // as in the forward kernel

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// `addr` of this CTA's shared memory in the cluster's CTA `rank`, and 16 bytes from there
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_load(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// length of request b, bounded to [0, C]
__device__ __forceinline__ int request_len(const DecodeParams& p, int b) { return min(max(p.lens[b], 0), p.C); }

// keys of a request's chunks; a single request's are its length's share, whole blocks of the four warps
__device__ __forceinline__ int chunk_keys(const DecodeParams& p, int len) {
  return p.B > 1 ? p.chunk : max(64, ((len + p.nsplit - 1) / p.nsplit + 63) / 64 * 64);
}

template <int D, int MT>
struct DecCfg {
  static constexpr int ROW = D * 2;                        // bytes of a key
  static constexpr int STAGE = 2 * kBlock * ROW;           // K and V of a block
  static constexpr int RING = kStages * STAGE;             // one warp's ring
  static constexpr int OUT = kWarps * MT * 16 * (D + 4) * 4;  // the warps' outputs at the end
  static constexpr int STAT = kWarps * MT * 16 * 8;
  static constexpr int SMEM = (kWarps * RING > OUT ? kWarps * RING : OUT) + STAT;
};

}  // namespace

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const DecodeParams p) {
  await_previous();
  using C = DecCfg<D, MT>;
  constexpr int NT = D / 8;   // output column tiles
  constexpr int KS = D / 16;  // k steps of the scores
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int u = blockIdx.x;
  const int chunk = u % p.nsplit;
  u /= p.nsplit;
  const int r0 = u % p.gsplit * (MT * 16);  // first head of the group that this CTA takes
  u /= p.gsplit;
  const int hk = u % p.Hkv, b = u / p.Hkv;
  const int len = request_len(p, b);
  if (threadIdx.x == 0 && chunk == 0 && r0 == 0 && hk == 0 && len != p.lens[b])
    record_status(p.status, MCS_ERR_BAD_INDEX, p.lens[b]);
  const int keys = chunk_keys(p, len), k0 = chunk * keys, k1 = min(len, k0 + keys);
  if (k0 >= k1 && p.part_o) return;  // nothing of this request: the join does not look here
  // in a cluster every chunk takes part in the join, an empty one with lse = -inf
  const int rows = min(p.g - r0, MT * 16);
  const int head0 = hk * p.g + r0;

  // blocks warp, warp + 4, ... of the chunk
  const int nblk = (max(k1 - k0, 0) + kBlock - 1) / kBlock;
  const int mine = (nblk - warp + kWarps - 1) / kWarps;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  const size_t row_stride = static_cast<size_t>(p.Hkv) * D;
  const size_t head_at = static_cast<size_t>(b) * p.C * row_stride + static_cast<size_t>(hk) * D;
  auto load = [&](int i) {
    const uint32_t dst = ring + i % kStages * C::STAGE;
    const int key0 = k0 + (warp + i * kWarps) * kBlock;
    constexpr int CH = D / 8;  // 16-byte pieces of a row
#pragma unroll
    for (int e = 0; e < kBlock * CH / 32; ++e) {
      const int x = e * 32 + lane, r = x / CH, c = x % CH;
      const bool in = key0 + r < k1;
      const size_t src = head_at + static_cast<size_t>(in ? key0 + r : k0) * row_stride + c * 8;
      const uint32_t at = r * C::ROW + ((c ^ (r & 7)) << 4);
      cp_async16(dst + at, p.k + src, in);
      cp_async16(dst + kBlock * C::ROW + at, p.v + src, in);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < mine) load(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // query fragments: rows lane / 4 and + 8 of each 16-row tile
  uint32_t qa[MT][KS][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m * 16 + (lane >> 2) + (e & 1) * 8, c = ks * 16 + (lane & 3) * 2 + (e >> 1) * 8;
        qa[m][ks][e] = r < rows ? *reinterpret_cast<const uint32_t*>(
                                      p.q + (static_cast<size_t>(b) * p.Hq + head0 + r) * D + c)
                                : 0u;
      }
  float slope[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = m * 16 + (lane >> 2) + e * 8;
      slope[m][e] = p.slopes && r < rows ? slope_of(p.slopes, head0 + r) * kLog2e : 0.f;
      if (p.slopes && r < rows) check_slope(p.slopes, head0 + r, p.status);
    }
  float o[MT][NT][4] = {};
  float mx[MT][2], l[MT][2] = {};
#pragma unroll
  for (int m = 0; m < MT; ++m) mx[m][0] = mx[m][1] = -CUDART_INF_F;

  for (int i = 0; i < mine; ++i) {
    if (i + kStages - 1 < mine) load(i + kStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t sk = ring + i % kStages * C::STAGE, sv = sk + kBlock * C::ROW;
    const int key0 = k0 + (warp + i * kWarps) * kBlock;
    float s[MT][8] = {};  // two column tiles of 8 keys
    {
      const int r = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t kb[4];
        ldsm4(kb, sk + r * C::ROW + (((2 * ks + half) ^ (r & 7)) << 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(s[m], qa[m][ks], kb[0], kb[1]);
          mma16816(s[m] + 4, qa[m][ks], kb[2], kb[3]);
        }
      }
    }
    uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (p.cap.on) cap_scores<8>(s[m], p.cap);
      // element e: row (e >> 1) & 1, key 8 (e >> 2) + 2 (lane & 3) + (e & 1); in log2 units
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = key0 + 8 * (e >> 2) + 2 * (lane & 3) + (e & 1);
        const float bias = slope[m][(e >> 1) & 1] * static_cast<float>(len - 1 - j);
        s[m][e] = j < k1 ? fmaf(p.mul, s[m][e], -bias) : -CUDART_INF_F;
      }
      float alpha[2];
      bool move = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a = fmaxf(fmaxf(s[m][2 * e], s[m][2 * e + 1]), fmaxf(s[m][4 + 2 * e], s[m][5 + 2 * e]));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        alpha[e] = 1.f;
        if (a > mx[m][e] + kRescale) {
          alpha[e] = fast_exp2(mx[m][e] - a);
          mx[m][e] = a;
          move = true;
        }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[m][n][0] *= alpha[0];
          o[m][n][1] *= alpha[0];
          o[m][n][2] *= alpha[1];
          o[m][n][3] *= alpha[1];
        }
      }
      // every block holds a key, so both maxima are finite
#pragma unroll
      for (int e = 0; e < 8; ++e) s[m][e] = fast_exp2(s[m][e] - mx[m][(e >> 1) & 1]);
      l[m][0] = l[m][0] * alpha[0] + ((s[m][0] + s[m][1]) + (s[m][4] + s[m][5]));
      l[m][1] = l[m][1] * alpha[1] + ((s[m][2] + s[m][3]) + (s[m][6] + s[m][7]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s[m][2 * e], y = s[m][2 * e + 1];
        const uint32_t h = pack_bf16(x, y);
        hi[m][e] = h;
        lo[m][e] = pack_bf16(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
      }
    }
    {
      const int r = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t vb[4];
        ldsm4t(vb, sv + r * C::ROW + (((n + half) ^ (r & 7)) << 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816(o[m][n], hi[m], vb[0], vb[1]);
          mma16816(o[m][n + 1], hi[m], vb[2], vb[3]);
          mma16816(o[m][n], lo[m], vb[0], vb[1]);
          mma16816(o[m][n + 1], lo[m], vb[2], vb[3]);
        }
      }
    }
    __syncwarp();  // the ring's oldest block may be overwritten
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  next_may_start();  // not before: what waits beside the loop costs it 6 % (one request of 75600 keys)

  // join the four warps: outputs and (max, sum) of each row through shared memory
  float* out = reinterpret_cast<float*>(smem);
  float2* stat = reinterpret_cast<float2*>(smem + C::SMEM - C::STAT);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[m][e];
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      const int r = m * 16 + (lane >> 2) + e * 8;
      if ((lane & 3) == 0) stat[warp * MT * 16 + r] = make_float2(mx[m][e], t);
      float* dst = out + (warp * MT * 16 + r) * (D + 4) + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < NT; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
    }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat[w * MT * 16 + r].x);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    const float top = top_or_zero(M);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = stat[w * MT * 16 + r];
      const float f = fast_exp2(st.x - top);
      const float4 v = *reinterpret_cast<const float4*>(out + (w * MT * 16 + r) * (D + 4) + c);
      L = fmaf(f, st.y, L);
      a.x = fmaf(f, v.x, a.x);
      a.y = fmaf(f, v.y, a.y);
      a.z = fmaf(f, v.z, a.z);
      a.w = fmaf(f, v.w, a.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float lse2 = L == 0.f ? -CUDART_INF_F : M + log2f(L);
    a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
    if (p.cluster) {
      // over the merged warps' own sums: this thread has read what it overwrites, and the other threads of the row
      // read other columns
      *reinterpret_cast<float4*>(out + r * (D + 4) + c) = a;
      if (c == 0) out[r * (D + 4) + D] = lse2;
    } else if (p.part_o) {
      const size_t at = (static_cast<size_t>(b) * p.Hq + head0 + r) * p.nsplit + chunk;
      *reinterpret_cast<float4*>(p.part_o + at * D + c) = a;
      if (c == 0) p.part_lse[at] = lse2;
    } else {
      const size_t at = static_cast<size_t>(b) * p.Hq + head0 + r;
      *reinterpret_cast<uint2*>(p.o + at * D + c) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
      if (c == 0 && p.lse) p.lse[at] = lse2 * kLn2;
    }
  }
  if (p.cluster) {
    // the chunks of a request are the CTAs of a cluster: rows rank, rank + nsplit, ... from all of them, in order
    cluster_sync();
    for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c = x % (D / 4) * 4;
      if (r % p.nsplit != chunk) continue;
      float ls[8], M = -CUDART_INF_F;
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ls[k] = -CUDART_INF_F;
        if (k < p.nsplit) {
          const uint32_t at = cluster_address(smem_u32(out + r * (D + 4)), k);
          ls[k] = cluster_load(at + D * 4).x;
          v[k] = cluster_load(at + c * 4);
        }
        M = fmaxf(M, ls[k]);
      }
      float L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (ls[k] == -CUDART_INF_F) continue;
        const float f = fast_exp2(ls[k] - top_or_zero(M));
        L += f;
        a.x = fmaf(f, v[k].x, a.x);
        a.y = fmaf(f, v[k].y, a.y);
        a.z = fmaf(f, v[k].z, a.z);
        a.w = fmaf(f, v[k].w, a.w);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const size_t at = static_cast<size_t>(b) * p.Hq + head0 + r;
      *reinterpret_cast<uint2*>(p.o + at * D + c) =
          make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      if (c == 0 && p.lse) p.lse[at] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

namespace {

// Joins the chunks of a request's keys and, behind a shared prefix, the
// prefix's parts: one CTA per (request, head), its warps take the parts in
// turn, then the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(256) decode_combine(const DecodeParams p) {
  next_may_start();
  await_previous();
  constexpr int E = D / 32;
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int head = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq;
  const int len = request_len(p, b);
  const int keys = chunk_keys(p, len), chunks = (len + keys - 1) / keys;
  const int parts = p.pre_parts + chunks;
  const size_t own = (static_cast<size_t>(b) * p.Hq + head) * p.nsplit;
  // the prefix's parts lie in packed tiles: request b is token b of the one batch row
  const size_t pre = p.pre_parts ? (static_cast<size_t>(head / p.g) * p.pre_tiles + b / p.pre_tpt) * 128 +
                                       b % p.pre_tpt * p.g + head % p.g
                                 : 0;
  const size_t slice = static_cast<size_t>(p.Hkv) * p.pre_tiles * 128;
  float m = -CUDART_INF_F, l = 0.f, o[E] = {};
  // batches of 4 parts per warp, so that their loads overlap
  for (int s0 = warp * 4; s0 < parts; s0 += warps * 4) {
    float ls[4], v[4][E];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k;
      ls[k] = -CUDART_INF_F;
      if (s < parts) {
        const bool mine = s >= p.pre_parts;
        const size_t at = mine ? own + s - p.pre_parts : s * slice + pre;
        ls[k] = (mine ? p.part_lse : p.pre_lse)[at];
        const float* src = (mine ? p.part_o : p.pre_o) + at * D + lane * E;
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
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (warp == 0) {
    float M = -CUDART_INF_F;
    for (int w = 0; w < warps; ++w) M = fmaxf(M, s_m[w]);
    float L = 0.f, a[E] = {};
    for (int w = 0; w < warps; ++w) {
      const float f = fast_exp2(s_m[w] - top_or_zero(M));
      L = fmaf(f, s_l[w], L);
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = fmaf(f, s_o[w][lane * E + e], a[e]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + static_cast<size_t>(blockIdx.x) * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(a[e] * inv, a[e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[blockIdx.x] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
  }
}

template <int D, int MT>
cudaError_t launch(const DecodeParams& p, cudaStream_t s) {
  static KernelReady ready;
  const cudaError_t e = make_ready(ready, decode_kernel<D, MT>, DecCfg<D, MT>::SMEM, 0);
  if (e != cudaSuccess) return e;
  const long long grid = static_cast<long long>(p.B) * p.Hkv * p.gsplit * p.nsplit;
  if (p.cluster) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = DecCfg<D, MT>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.nsplit;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    note_launches(1);
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, decode_kernel<D, MT>, p);
    return launched == cudaSuccess ? launched : cudaGetLastError();
  }
  return launch_in_sequence(decode_kernel<D, MT>, static_cast<unsigned>(grid), kThreads, DecCfg<D, MT>::SMEM, s,
                            p.pre_parts > 0, p);
}

}  // namespace

cudaError_t launch_decode(int d, const DecodeParams& p, cudaStream_t s) {
  if (d == 64) return p.g > 16 ? launch<64, 2>(p, s) : launch<64, 1>(p, s);
  return p.g > 16 ? launch<128, 2>(p, s) : launch<128, 1>(p, s);
}

cudaError_t launch_decode_combine(int d, const DecodeParams& p, cudaStream_t s) {
  const int parts = p.pre_parts + p.nsplit;
  const int warps = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;
  const unsigned grid = static_cast<unsigned>(p.B) * p.Hq;
  return launch_in_sequence(d == 64 ? decode_combine<64> : decode_combine<128>, grid, warps * 32, 0, s, true, p);
}

}  // namespace mcs
