// Internal declarations shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/mcs.h"

// status block word indices (int32 words at the start of the workspace)
#define MCS_SW_STATUS 0
#define MCS_SW_DETAIL 1
#define MCS_SW_BAND_OVERFLOW 2
#define MCS_SW_REFINED 3
#define MCS_SW_TOPK_FULL 4
#define MCS_SW_LANCZOS_STEPS 5  // grouping: Lanczos steps summed over all nodes (a diagnostic)
#define MCS_SW_LANCZOS_NODES 6  // grouping: nodes that ran Lanczos

// where-codes recorded as the status detail when a bounded wait expires
enum {
  MCS_WHERE_ATTN_PRODUCER = 1,
  MCS_WHERE_ATTN_MMA = 2,
  MCS_WHERE_ATTN_SOFTMAX = 3,
  MCS_WHERE_ATTN_EPILOGUE = 4,
  MCS_WHERE_MASS_PRODUCER = 11,
  MCS_WHERE_MASS_MMA = 12,
  MCS_WHERE_MASS_CONSUMER = 13,
  MCS_WHERE_DRAIN = 20,
};

namespace mcs {

// Basis vectors of one Lanczos cycle in the grouping's node kernel (its shared
// memory holds that many): the most Krylov steps a fixed-step grouping takes.
constexpr int kPddpKrylovMax = 64;

// ATTN_ANCHOR_DENSE is ATTN_DENSE plus the anchor's exports (fp32 O_dense, the
// lse as an fp32 hi/lo pair) computed with the exact-exponent arithmetic the
// fp64 selection re-score relies on.
enum AttnMode { ATTN_DENSE = 0, ATTN_REUSE = 1, ATTN_ANCHOR_SPARSE = 2, ATTN_ANCHOR_DENSE = 3 };

struct AttnParams {
  int B, H, N;
  int h0, hc;       // heads [h0, h0 + hc) of this launch (hc == 0: all H); strides use H
  int G;            // query tiles per (b,h)
  int kv_count;     // keys per tile list: N (dense) or K (sparse)
  float scale_log2;    // softmax scale * log2(e), rounded to fp32
  float scale_log2_lo; // the rounding residual: scale * log2(e) - scale_log2 (used by ATTN_ANCHOR_DENSE)
  const uint16_t *q, *k, *v;     // bf16 [B,N,H,d] (read directly by the gathered modes)
  const int32_t* perm;           // [B,H,N] or null (identity query order)
  const int32_t* kv_idx;         // [B,H,G,K] (sparse modes)
  const uint16_t* resid_in;      // reuse: bf16 [B,H,N,d] perm order (nullable)
  const float* o_dense_in;       // anchor sparse: fp32 [B,H,G*128,d] perm order
  uint16_t* o;                   // bf16 [B,N,H,d] token order (dense, reuse)
  float* o_dense_out;            // anchor dense: fp32 [B,H,G*128,d] perm order (nullable)
  float* lse_out;                // token order [B,H,N] (nullable)
  float* lse_perm_out;           // perm order [B,H,G*128], NEGATED lse in log2 units, -inf past N (nullable)
  float* lse_perm_lo_out;        // same rows: -lse2 - lse_perm_out in fp32 (the low part; 0 past N; nullable)
  uint16_t* resid_out;           // anchor sparse: bf16 [B,H,N,d] perm order
  int* status;                   // status block
  uint64_t wait_limit_ns;
  int debug_flags;
};

struct MassParams {
  int B, H, N, G, h0, hn;  // heads [h0, h0+hn) of this chunk
  float scale_log2;
  const int32_t* perm;     // [B,H,N] (unused by the kernel; queries come in group order)
  const float* lse_perm;   // [B,H,G*128] negated lse in log2 units (-lse * log2 e), -inf past N
  float* mass;             // [B,hn,G,N] for the chunk
  int* status;
  uint64_t wait_limit_ns;
};

struct TopkParams {
  int B, H, N, G, K, d, h0, hn;
  double scale;            // softmax scale (natural), in fp64 as the caller's shape defines it
  const float* mass;       // [B,hn,G,N]
  const uint16_t* q;       // bf16 [B,N,H,d]
  const uint16_t* k;
  const int32_t* perm;
  const float* lse_perm;   // [B,H,G*128] negated lse in log2 units (high part)
  const float* lse_perm_lo;  // [B,H,G*128] its low part: -lse2 = lse_perm + lse_perm_lo (fp64 sum)
  int32_t* kv_idx;         // [B,H,G,K]
  int* status;
  float band_rel;          // relative half-width of the uncertain band
  int cand_cap;            // set by launch_topk: keys of one bin the two-sweep path holds in shared memory
  int force_full;          // test hook: every group takes the general seven-sweep path
};

// launchers (return cudaSuccess or the launch error)
// plain dense attention (ATTN_DENSE) at d = 128 over pairs of query tiles (attn_pair.cu)
cudaError_t launch_attention_pair(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                                  const AttnParams& p, cudaStream_t s);
cudaError_t launch_attention(int d, AttnMode mode, const CUtensorMap* tq, const CUtensorMap* tk,
                             const CUtensorMap* tv, const AttnParams& p, cudaStream_t s);
cudaError_t launch_mass(int d, const CUtensorMap* tqp, const CUtensorMap* tk, const MassParams& p,
                        cudaStream_t s);
cudaError_t launch_permute_queries(const uint16_t* q, const int32_t* perm, uint16_t* qp, int B, int H, int N, int G,
                                   int d, int* status, cudaStream_t s);
cudaError_t launch_topk(const TopkParams& p, cudaStream_t s);
// packed selection (uint32 [rows, ceil(N/32)]) <-> ascending index lists (int32 [rows, K])
size_t meta_pack_smem_bytes(int N);
cudaError_t launch_meta_pack(const int32_t* idx, uint32_t* mask, long long rows, int N, int K, int* status,
                             cudaStream_t s);
cudaError_t launch_meta_unpack(const uint32_t* mask, int32_t* idx, long long rows, int N, int K, int* status,
                               cudaStream_t s);

// PDDP grouping: enqueue the whole recursion (fp64) for all heads
struct PddpPlan;
// krylov_steps: 0 = principal direction to convergence; k > 0 = top Ritz vector after k Lanczos steps;
// whiten: group the per-channel standardised queries
cudaError_t pddp_run(int B, int H, int N, int d, const uint16_t* q, int32_t* perm, void* ws, size_t ws_bytes,
                     int* status, int krylov_steps, bool whiten, cudaStream_t s);
size_t pddp_workspace_bytes(int B, int H, int N, int d);

// ---- attention with modified scores (api_ex.cu, attn_ex*.cu) ----

struct ExParams {
  int B, Hq, Hkv, g, Nq, Nk;   // g = Hq / Hkv
  float scale;                 // softmax scale
  float cap;                   // 0: none
  int causal;
  const float* slopes;         // [Hq] or null
  const int32_t* prefix;       // [B] or null
  const int32_t *doc_q, *doc_k;  // [B,Nq], [B,Nk] or null
  int* status;
};

constexpr int kSms = 148;  // of a B200: the sizes of workspaces and launches follow from the shape alone

// The score cap: y(s) = cap log2(e) tanh(k pre s), k pre = scale / cap, for products s = q . k (cap_scores in
// attn_ex.cuh). pre is 1, or the power of two that brings k near 1 where the coefficients would leave fp32's range.
struct CapFn {
  int on;
  float pre;
  float k2, cl, icl;  // 2 k log2 e, cap log2 e and its inverse
  float z2, z3;       // (pre s)^2 up to which the coefficients b, and a, hold
  float a[5], b[4];   // y = x Q(x^2), x = pre s
};
// tanh(x) = x + x z P(z), z = x^2: the coefficients of P, degree 3
constexpr float kTanhP0 = -0.333323412f, kTanhP1 = 0.133081745f, kTanhP2 = -0.0519478787f, kTanhP3 = 0.0151953385f;
constexpr float kTanhR0 = -0.333318822f, kTanhR1 = 0.132776282f, kTanhR2 = -0.0477941821f;  // degree 2, |x| <= 0.4

// The tile kernels' view of a call (attn_ex_fwd.cu, attn_ex_bwd.cu).
struct ExTile {
  int B, Hq, Hkv, g, tpt, Nq, Nk;  // tpt: tokens of a packed query tile
  int qbox;                        // backward: tokens of a query map's box, tpt or (64 rows) tpt / 2
  int Tq, Tk;                      // query and key tiles
  int nsplit, single, chunk;       // forward: key splits, one-tile CTAs, heads per chunk of the work order
  float mul;                       // log2 units per score: scale log2 e, or 1 where the cap yields them
  CapFn cap;
  float scale;
  int causal;
  const float* slopes;
  const int32_t* prefix;
  const int32_t *doc_q, *doc_k;    // null without a document mask, and then so are the next five
  const int4 *q_ranges, *k_ranges;  // [B,Tq], [B,Tk]: smallest and largest id, any padding
  const int *q_ids, *k_ids;        // [B,Tq,128] (backward), [B,Tk,128]
  const int *order, *k_order;      // document mask: the order of the query jobs and of the key tiles (their number,
                                   // then 4 job + part), or null
  const int32_t* lens;             // shared prefix: the requests' lengths give the positions
  int P, C;
  uint16_t* o;                     // outputs, or the partials of the splits
  float* lse;
  const float* stats;              // backward: [B,Hkv,Tq][2][128], -lse in log2 units and d_o . o
  const float* lse_in;             // backward: the forward's lse,
  const uint16_t *o_in, *do_in;    // its o, and the gradient of o
  int kv_splits;                   // backward: CTAs that share a key tile's queries
  size_t kv_size;                  // elements of dk
  float* part_kv;                  // [2 (dv, dk)][kv_splits][B,Nk,Hkv,d], null unless kv_splits > 1
  float* stats_out;                // where the statistics go
  int d_from_o;                    // backward: D is d_o . o, else a sweep sums it from P dP
  uint16_t *dq, *dk, *dv;
  float *part_o, *part_lse;        // [parts][B,Hkv,Tq,128](,d), lse in log2 units
  int* status;
  uint64_t wait_limit_ns;
  int debug_flags;
};

cudaError_t launch_ex_fwd(int d, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const ExTile& p,
                          cudaStream_t s);
cudaError_t launch_ex_combine(int d, const ExTile& p, int parts, cudaStream_t s);
// packed rows' statistics, then the gradients; tg: the map of d_o
cudaError_t launch_ex_row_stats(int d, const ExTile& p, cudaStream_t s);
cudaError_t launch_ex_bwd(int d, const CUtensorMap* tq, const CUtensorMap* tg, const CUtensorMap* tk,
                          const CUtensorMap* tv, const ExTile& p, cudaStream_t s);
// order of the jobs (of `per` query tiles) and, unless null, of the key tiles: [B jobs], [B Tk]
cudaError_t launch_ex_doc_order(const ExTile& p, int per, int4* counts, int* q_order, int* k_order, cudaStream_t s);
cudaError_t launch_ex_doc_tiles(const ExTile& p, int* k_ids, int4* k_ranges, int* q_ids, int4* q_ranges,
                                cudaStream_t s);

struct DecodeParams {
  int B, Hq, Hkv, g, C;
  int nsplit, chunk;               // chunks of the keys, keys of a chunk
  int gsplit;                      // parts of a head group (32 heads each)
  int cluster;                     // the chunks of a request are one cluster, which joins them
  float mul;                       // as in ExTile
  CapFn cap;
  const uint16_t *q, *k, *v;
  const int32_t* lens;
  const float* slopes;
  uint16_t* o;
  float* lse;
  float *part_o, *part_lse;        // [B,Hq,nsplit](,d), lse in log2 units; null: o and lse directly
  const float *pre_o, *pre_lse;    // the shared prefix's parts, in ExTile's layout
  int pre_parts, pre_tiles, pre_tpt;
  int* status;
};

cudaError_t launch_decode(int d, const DecodeParams& p, cudaStream_t s);
cudaError_t launch_decode_combine(int d, const DecodeParams& p, cudaStream_t s);

// MCS_OK when the current device is an sm_100 GPU
mcs_status check_device();
// 4-D map of a bf16 [B, N, H, d] tensor, box {64, heads, tokens, 1}, 128-byte swizzle: `tokens` consecutive
// tokens of `heads` consecutive heads per load; tokens past N read as zero
mcs_status tiles_map(CUtensorMap* m, const void* base, int B, int N, int H, int d, int heads, int tokens);
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per bounded device wait

// Before a kernel's first launch on the current device: allow `smem` bytes of dynamic shared memory and, where
// `regs` is not 0, check the registers per thread that its setmaxnreg split counts on. `done` is one flag per device.
struct KernelReady {
  std::atomic<bool> done[64] = {};
};
template <typename Kernel>
cudaError_t make_ready(KernelReady& r, Kernel kern, unsigned smem, int regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && r.done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (regs && fa.numRegs != regs) return cudaErrorInvalidKernelImage;
  if (dev < 64) r.done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

// process-wide test knobs (see mcs_debug_set in api.cu)
int debug_flags();

// count of kernel launches this library made in the process (diagnostics)
void note_launches(int n);

// Launches a kernel that begins with await_previous(). `after`: behind another such
// kernel of the same call, whose end it awaits itself. (Forward and gradients of
// 2 x 601 tokens with documents and a cap, six launches: 62.6 us, 70.3 one after the
// other; 8 requests behind a shared prefix of 4096 keys, three launches: 19.0 and
// 23.6.) A call's first kernel starts after whatever the stream held before.
template <class... P, class... A>
cudaError_t launch_in_sequence(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                               bool after, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = after ? 1 : 0;
  note_launches(1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? e : cudaGetLastError();  // reported here, not to the next caller
}

}  // namespace mcs
