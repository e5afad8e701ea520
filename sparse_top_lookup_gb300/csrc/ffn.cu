// The gated feed-forward block and its backward pass:
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) * u,  y = h Wd^T
//   dh = dy Wd;  dg = dh * u * act'(g),  du = dh * act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h
//
// x [B, dim], Wg and Wu [F, dim], Wd [dim, F] (nn.Linear's layouts), bf16
// in, fp32 accumulation on the tcgen05 tensor cores.
//
// Every product runs through one kernel: clusters of two CTAs issue
// tcgen05.mma.cta_group::2 of M = 256 rows (128 in each CTA) and N = 256
// columns, K in slabs of 64 through a ring of shared-memory stages filled by
// TMA; 512 TMEM columns hold two accumulators, so a tile is multiplied while
// the one before it is written out by eight epilogue warps.  Operands are
// taken as they lie in memory: with K contiguous (K-major) or with M or N
// contiguous (MN-major: the products with a transposed operand), both with
// 128-byte swizzle.  What differs is the epilogue (Epi).
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "pkm_internal.cuh"
#include "tc_common.cuh"

namespace pkm {
namespace {

using namespace tc;

constexpr int FM = 128;                   // rows per CTA (the pair's MMA takes 2 * FM)
constexpr int FN = 256;                   // accumulator columns per tile
constexpr int FK = 64;                    // K per stage: one 128-byte swizzle row of bf16
constexpr int FA_BYTES = FM * FK * 2;     // 16 KiB
constexpr int FB_BYTES = FN / 2 * FK * 2; // 16 KiB: each CTA holds half of the columns
constexpr int FSTAGE_BYTES = FA_BYTES + FB_BYTES;
constexpr int FSTAGES = 6;
constexpr int FSMEM = FSTAGES * FSTAGE_BYTES + 1024;  // + alignment slack
constexpr int FEPI_WARPS = 8;
constexpr int FTHREADS = 64 + 32 * FEPI_WARPS;
static_assert(FSMEM <= 227 * 1024, "feed-forward shared memory");

enum Epi {
  kGate,    // accumulator columns: 128 of g, the same 128 of u; writes h (and g, u)
  kStore,   // C in bf16
  kAdd32,   // C added to an fp32 matrix
  kDGate    // accumulator: dh; reads g, u; writes dg, du, h
};

// One launch: `groups` products of one shape that differ in A and C (group i:
// a[i], b[i], c[i]), or one product whose K runs through `segs` pairs (a[i],
// b[i]) one after the other.
struct GemmArgs {
  CUtensorMap a[2], b[2];
  int M, N, K;        // of one product; K of one segment
  int segs, groups;   // at most one of them above 1
  int a_mn, b_mn;     // operand stored with M (N) contiguous
  int act;
  void* c[2];                       // kStore: bf16 [M, N]; kAdd32: fp32 [M, N]
  __nv_bfloat16 *g, *u, *h;         // kGate: written (g, u may be NULL)
  const __nv_bfloat16 *g_in, *u_in; // kDGate
  __nv_bfloat16 *dg, *du;
  int* status;
};

__device__ __forceinline__ float act_fwd(float g, int act) {
  switch (act) {
    case PKM_ACT_SILU:
      return __fdividef(g, 1.0f + __expf(-g));
    case PKM_ACT_GELU:
      return 0.5f * g * (1.0f + erff(g * 0.70710678f));
    case PKM_ACT_GELU_TANH: {
      // 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v))
      const float v2 = 1.59576912f * g * fmaf(0.044715f * g, g, 1.0f);
      return __fdividef(g, 1.0f + __expf(-v2));
    }
    default:
      return fmaxf(g, 0.0f);
  }
}

// act(g) and act'(g)
__device__ __forceinline__ float2 act_both(float g, int act) {
  switch (act) {
    case PKM_ACT_SILU: {
      const float s = __fdividef(1.0f, 1.0f + __expf(-g));
      return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
    }
    case PKM_ACT_GELU: {
      const float cdf = 0.5f * (1.0f + erff(g * 0.70710678f));
      return make_float2(g * cdf, fmaf(g * 0.39894228f, __expf(-0.5f * g * g), cdf));
    }
    case PKM_ACT_GELU_TANH: {
      const float g2 = g * g;
      const float s = __fdividef(1.0f, 1.0f + __expf(-1.59576912f * g * fmaf(0.044715f, g2, 1.0f)));
      return make_float2(g * s, s * fmaf(g * (1.0f - s), 1.59576912f * fmaf(0.134145f, g2, 1.0f),
                                         1.0f));
    }
    default:
      return make_float2(fmaxf(g, 0.0f), g > 0.0f ? 1.0f : 0.0f);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// 32 columns from column c0 of a row of an [., N] bf16 matrix (N a multiple of 8).
__device__ __forceinline__ void store32(__nv_bfloat16* row, int c0, int N, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c0 + 8 * j < N)
      *reinterpret_cast<uint4*>(row + c0 + 8 * j) =
          make_uint4(pack2(v[8 * j], v[8 * j + 1]), pack2(v[8 * j + 2], v[8 * j + 3]),
                     pack2(v[8 * j + 4], v[8 * j + 5]), pack2(v[8 * j + 6], v[8 * j + 7]));
}
__device__ __forceinline__ void load32(const __nv_bfloat16* row, int c0, int N, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (c0 + 8 * j < N) x = __ldg(reinterpret_cast<const uint4*>(row + c0 + 8 * j));
    v[8 * j] = lo_bf16(x.x), v[8 * j + 1] = hi_bf16(x.x);
    v[8 * j + 2] = lo_bf16(x.y), v[8 * j + 3] = hi_bf16(x.y);
    v[8 * j + 4] = lo_bf16(x.z), v[8 * j + 5] = hi_bf16(x.z);
    v[8 * j + 6] = lo_bf16(x.w), v[8 * j + 7] = hi_bf16(x.w);
  }
}

// Tile t of `groups` x (tm_count x tn_count): bands of 8 row tiles, within a
// band row tiles fastest, so the tiles that run at one time share operands in L2.
__device__ __forceinline__ void tile_at(int t, int tm_count, int tn_count, int& grp, int& tm,
                                        int& tn) {
  const int per = tm_count * tn_count;
  grp = t / per;
  t -= grp * per;
  const int band = t / (8 * tn_count);
  const int rows = min(8, tm_count - 8 * band);
  t -= band * 8 * tn_count;
  tn = t / rows;
  tm = band * 8 + t - tn * rows;
}

template <int kEpi>
__global__ void __launch_bounds__(FTHREADS, 1)
ffn_gemm_kernel(const __grid_constant__ GemmArgs p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * FSTAGES + 4 + 1];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  constexpr int kTileN = kEpi == kGate ? FN / 2 : FN;  // output columns per tile
  const int tm_count = (p.M + 2 * FM - 1) / (2 * FM), tn_count = (p.N + kTileN - 1) / kTileN;
  const uint32_t rank = cluster_ctarank();
  const int slot = (int)(blockIdx.x >> 1), slots = (int)(gridDim.x >> 1);
  const int tiles = tm_count * tn_count * p.groups;
  const int mine = slot < tiles ? (tiles - 1 - slot) / slots + 1 : 0;
  if (mine == 0) return;  // both CTAs of the cluster alike
  const int kb_seg = (p.K + FK - 1) / FK, kb_count = kb_seg * p.segs;

  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t stages_u32 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(&bars[0]);
  auto bar_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto bar_empty = [&](uint32_t s) { return bar0 + 8u * (FSTAGES + s); };
  auto bar_tfull = [&](uint32_t b) { return bar0 + 8u * (2 * FSTAGES + b); };
  auto bar_tempty = [&](uint32_t b) { return bar0 + 8u * (2 * FSTAGES + 2 + b); };
  const uint32_t bar_done = bar0 + 8u * (2 * FSTAGES + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < FSTAGES; ++s) {
      mbar_init(bar_full(s), 1);   // leader: its producer's expect_tx (both CTAs' bytes)
      mbar_init(bar_empty(s), 1);  // the leader's MMA commit, multicast to both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull(b), 1);                 // the leader's MMA commit, multicast
      mbar_init(bar_tempty(b), 2 * FEPI_WARPS);   // leader: the epilogue warps of both CTAs
    }
    mbar_init(bar_done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {  // one warp of each CTA allocates, jointly for the pair
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs' barriers exist before any remote arrival
  const uint32_t tmem = s_tmem_base;
  const Ctl ctl{&s_abort, p.status};

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int i = 0; ok && i < mine; ++i) {
        int grp, tm, tn;
        tile_at(slot + i * slots, tm_count, tn_count, grp, tm, tn);
        const int row0 = (2 * tm + (int)rank) * FM;
        // kGate: CTA 0 holds the tile's rows of Wg, CTA 1 those of Wu
        const int col0 = kEpi == kGate ? tn * kTileN : tn * FN + (int)rank * (FN / 2);
        for (int kb = 0; kb < kb_count; ++kb, ++it) {
          const uint32_t s = it % FSTAGES, ph = (it / FSTAGES) & 1u;
          if (!wait_phase_cluster(bar_empty(s), ph ^ 1u, ctl)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(bar_full(s), 2u * FSTAGE_BYTES);
          const int seg = kb / kb_seg, k0 = (kb - seg * kb_seg) * FK;
          const CUtensorMap* ma = &p.a[seg + grp];
          const CUtensorMap* mb = kEpi == kGate ? &p.b[rank] : &p.b[seg + grp];
          const uint32_t da = stages_u32 + s * FSTAGE_BYTES, db = da + FA_BYTES;
          const uint32_t fb = mapa_shared(bar_full(s), 0);
          if (p.a_mn) {
            tma_load_2d_cg2(da, ma, row0, k0, fb);
            tma_load_2d_cg2(da + FA_BYTES / 2, ma, row0 + 64, k0, fb);
          } else {
            tma_load_2d_cg2(da, ma, k0, row0, fb);
          }
          if (p.b_mn) {
            tma_load_2d_cg2(db, mb, col0, k0, fb);
            tma_load_2d_cg2(db + FB_BYTES / 2, mb, col0 + 64, k0, fb);
          } else {
            tma_load_2d_cg2(db, mb, k0, col0, fb);
          }
        }
      }
      // the leader's last releases of this CTA's stages land before it exits
      if (ok) {
        const uint32_t first = it > (uint32_t)FSTAGES ? it - FSTAGES : 0u;
        for (uint32_t j = first; j < it; ++j)
          wait_phase_drain(bar_empty(j % FSTAGES), (j / FSTAGES) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = idesc_bf16(2 * FM, FN) | (p.a_mn ? kIdescAMn : 0u) |
                             (p.b_mn ? kIdescBMn : 0u);
      // descriptor advance per 16 of K: 32 bytes along a swizzled row, or 16
      // rows of 128 bytes
      const uint32_t a_step = p.a_mn ? 128u : 2u, b_step = p.b_mn ? 128u : 2u;
      uint32_t it = 0;
      bool ok = true;
      for (int i = 0; ok && i < mine; ++i) {
        const uint32_t buf = i & 1u, use = i >> 1;
        if (!wait_phase_cluster(bar_tempty(buf), (use & 1u) ^ 1u, ctl)) break;
        tc_fence_after();
        for (int kb = 0; kb < kb_count; ++kb, ++it) {
          const uint32_t s = it % FSTAGES, ph = (it / FSTAGES) & 1u;
          if (!wait_phase_cluster(bar_full(s), ph, ctl)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = stages_u32 + s * FSTAGE_BYTES;
          const uint64_t a_desc = p.a_mn ? sw128_mn_desc(sa, FA_BYTES / 2) : sw128_desc(sa);
          const uint64_t b_desc = p.b_mn ? sw128_mn_desc(sa + FA_BYTES, FB_BYTES / 2)
                                         : sw128_desc(sa + FA_BYTES);
#pragma unroll
          for (int kk = 0; kk < FK / 16; ++kk)
            tc_mma_cg2(tmem + buf * FN, a_desc + a_step * kk, b_desc + b_step * kk, idesc,
                       (kb | kk) != 0);
          tc_commit_cg2_mc(bar_empty(s), 3);  // the stage is free again in both CTAs
        }
        if (!ok) break;
        tc_commit_cg2_mc(bar_tfull(buf), 3);  // the tile's sums are in both TMEMs
      }
      // every issued MMA completes before TMEM is released
      tc_commit_cg2_mc(bar_done, 1);
      wait_phase_drain(bar_done, 0);
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    for (int i = 0; i < mine; ++i) {
      int grp, tm, tn;
      tile_at(slot + i * slots, tm_count, tn_count, grp, tm, tn);
      const uint32_t buf = i & 1u, use = i >> 1;
      if (!__all_sync(0xffffffffu, wait_phase_cluster(bar_tfull(buf), use & 1u, ctl))) break;
      tc_fence_after();
      const uint32_t taddr = lane_addr + buf * FN;
      const int row = (2 * tm + (int)rank) * FM + quad * 32 + lane;
      const size_t at = (size_t)row * p.N;
      constexpr int kHalfN = kTileN / 2;
      for (int c = half * kHalfN; c < (half + 1) * kHalfN; c += 32) {
        const int c0 = tn * kTileN + c;
        if (c0 >= p.N) break;
        float v[32];
        tmem_ld32(taddr + c, v);
        if constexpr (kEpi == kGate) {
          float w[32];
          tmem_ld32(taddr + FN / 2 + c, w);
          if (row < p.M) {
            if (p.g) {
              store32(p.g + at, c0, p.N, v);
              store32(p.u + at, c0, p.N, w);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] *= act_fwd(v[j], p.act);
            store32(p.h + at, c0, p.N, w);
          }
        } else if constexpr (kEpi == kStore) {
          if (row < p.M) store32(static_cast<__nv_bfloat16*>(p.c[grp]) + at, c0, p.N, v);
        } else if constexpr (kEpi == kAdd32) {
          if (row < p.M) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.c[grp]) + at + c0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c0 + 4 * j < p.N) {
                float4 t = dst[j];
                t.x += v[4 * j], t.y += v[4 * j + 1], t.z += v[4 * j + 2], t.w += v[4 * j + 3];
                dst[j] = t;
              }
          }
        } else {
          if (row < p.M) {
            float g[32], u[32];
            load32(p.g_in + at, c0, p.N, g);
            load32(p.u_in + at, c0, p.N, u);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 a = act_both(g[j], p.act);
              g[j] = v[j] * u[j] * a.y;
              u[j] *= a.x;  // h
              v[j] *= a.x;  // du
            }
            store32(p.dg + at, c0, p.N, g);
            store32(p.du + at, c0, p.N, v);
            store32(p.h + at, c0, p.N, u);
          }
        }
      }
      // tile written: hand the TMEM buffer back to the leader's MMA warp
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(bar_tempty(buf), 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  // the leader's MMAs (which write both CTAs' TMEM and read both CTAs'
  // stages) are complete, and no CTA still arrives on the other's barriers
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// A [rows, cols] bf16 matrix in boxes of box_cols x box_rows, 128-byte swizzle.
bool encode2(CUtensorMap* m, const void* ptr, int rows, int cols, int box_cols, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An operand whose rows are M (N) and whose columns are K, or the transpose.
bool operand(CUtensorMap* m, const void* ptr, int rows, int cols, bool mn) {
  return encode2(m, ptr, rows, cols, 64, mn ? FK : FM);
}

template <int kEpi>
cudaError_t launch_gemm(const GemmArgs& p, cudaStream_t stream) {
  auto kernel = ffn_gemm_kernel<kEpi>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(FTHREADS);
  cfg.dynamicSmemBytes = FSMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static int max_clusters = 0;
  if (!max_clusters) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FSMEM);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    max_clusters = n;
  }
  const int tile_n = kEpi == kGate ? FN / 2 : FN;
  const int64_t tiles =
      (int64_t)((p.M + 2 * FM - 1) / (2 * FM)) * ((p.N + tile_n - 1) / tile_n) * p.groups;
  cfg.gridDim = dim3(2 * (unsigned)(tiles < max_clusters ? tiles : max_clusters));
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t gated_ffn_workspace_bytes(int B, int F) { return align256((size_t)B * F * 2); }
size_t gated_ffn_backward_workspace_bytes(int B, int F) { return 3 * align256((size_t)B * F * 2); }

cudaError_t launch_gated_ffn(const void* x, const void* w_gate, const void* w_up,
                             const void* w_down, int B, int dim, int F, int act, void* workspace,
                             void* y, void* gate, void* up, int* status, cudaStream_t stream) {
  GemmArgs p = {};
  p.segs = p.groups = 1;
  p.act = act;
  p.status = status;
  p.M = B, p.N = F, p.K = dim;
  p.g = static_cast<__nv_bfloat16*>(gate);
  p.u = static_cast<__nv_bfloat16*>(up);
  p.h = static_cast<__nv_bfloat16*>(workspace);
  if (!operand(&p.a[0], x, B, dim, false) || !operand(&p.b[0], w_gate, F, dim, false) ||
      !operand(&p.b[1], w_up, F, dim, false))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_gemm<kGate>(p, stream);
  if (e != cudaSuccess) return e;
  p.N = dim, p.K = F;
  p.c[0] = y;
  if (!operand(&p.a[0], workspace, B, F, false) || !operand(&p.b[0], w_down, dim, F, false))
    return cudaErrorInvalidValue;
  return launch_gemm<kStore>(p, stream);
}

cudaError_t launch_gated_ffn_backward(const void* x, const void* w_gate, const void* w_up,
                                      const void* w_down, const void* gate, const void* up,
                                      const void* dy, int B, int dim, int F, int act,
                                      void* workspace, void* dx, void* dw_gate, void* dw_up,
                                      void* dw_down, int grad_dtype, int* status,
                                      cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const size_t part = align256((size_t)B * F * 2);
  GemmArgs p = {};
  p.segs = p.groups = 1;
  p.act = act;
  p.status = status;
  p.g_in = static_cast<const __nv_bfloat16*>(gate);
  p.u_in = static_cast<const __nv_bfloat16*>(up);
  p.dg = reinterpret_cast<__nv_bfloat16*>(ws);
  p.du = reinterpret_cast<__nv_bfloat16*>(ws + part);
  p.h = reinterpret_cast<__nv_bfloat16*>(ws + 2 * part);
  // dh = dy Wd, then dg, du and h
  p.M = B, p.N = F, p.K = dim, p.b_mn = 1;
  if (!operand(&p.a[0], dy, B, dim, false) || !operand(&p.b[0], w_down, dim, F, true))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_gemm<kDGate>(p, stream);
  if (e != cudaSuccess) return e;
  if (dx) {  // dx = dg Wg + du Wu: one product of twice the depth
    p.N = dim, p.K = F, p.segs = 2;
    p.c[0] = dx;
    if (!operand(&p.a[0], p.dg, B, F, false) || !operand(&p.a[1], p.du, B, F, false) ||
        !operand(&p.b[0], w_gate, F, dim, true) || !operand(&p.b[1], w_up, F, dim, true))
      return cudaErrorInvalidValue;
    if ((e = launch_gemm<kStore>(p, stream)) != cudaSuccess) return e;
    p.segs = 1;
  }
  const bool add = grad_dtype == PKM_F32;
  p.a_mn = 1, p.K = B;
  if (dw_gate) {  // dWg = dg^T x and dWu = du^T x
    p.M = F, p.N = dim, p.groups = 2;
    p.c[0] = dw_gate, p.c[1] = dw_up;
    if (!operand(&p.a[0], p.dg, B, F, true) || !operand(&p.a[1], p.du, B, F, true) ||
        !operand(&p.b[0], x, B, dim, true))
      return cudaErrorInvalidValue;
    p.b[1] = p.b[0];
    e = add ? launch_gemm<kAdd32>(p, stream) : launch_gemm<kStore>(p, stream);
    if (e != cudaSuccess) return e;
    p.groups = 1;
  }
  if (dw_down) {  // dWd = dy^T h
    p.M = dim, p.N = F;
    p.c[0] = dw_down;
    if (!operand(&p.a[0], dy, B, dim, true) || !operand(&p.b[0], p.h, B, F, true))
      return cudaErrorInvalidValue;
    e = add ? launch_gemm<kAdd32>(p, stream) : launch_gemm<kStore>(p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkm

namespace {

// device status word for calls that pass none
__device__ int g_ffn_status;

bool ffn_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int ffn_status(int* status, int** out) {
  *out = status;
  if (status) return PKM_OK;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_ffn_status) != cudaSuccess) return PKM_ERR_CUDA;
  *out = static_cast<int*>(p);
  return PKM_OK;
}

int ffn_check(int B, int dim, int F, int act) {
  if (B < 0 || dim < 1 || F < 1) return PKM_ERR_INVALID;
  if (act < PKM_ACT_SILU || act > PKM_ACT_RELU || dim % 8 || F % 8) return PKM_ERR_UNSUPPORTED;
  // the kernels count tiles (of 128 x 128 at the smallest) and rows in 32 bits
  constexpr int most = INT32_MAX - 256;
  auto t = [](int n) { return ((int64_t)n + 127) / 128; };
  if (B > most || dim > most || F > most || t(B) * t(F) > most || t(B) * t(dim) > most ||
      2 * t(F) * t(dim) > most)
    return PKM_ERR_RANGE;
  return PKM_OK;
}

}  // namespace

extern "C" size_t pkm_gated_ffn_workspace_bytes(int B, int dim, int F) {
  if (B < 0 || dim < 1 || F < 1) return 0;
  return pkm::gated_ffn_workspace_bytes(B, F);
}

extern "C" size_t pkm_gated_ffn_backward_workspace_bytes(int B, int dim, int F) {
  if (B < 0 || dim < 1 || F < 1) return 0;
  return pkm::gated_ffn_backward_workspace_bytes(B, F);
}

extern "C" int pkm_gated_ffn(const void* x, const void* w_gate, const void* w_up,
                             const void* w_down, int B, int dim, int F, int act, void* workspace,
                             void* y, void* gate, void* up, int* status, void* stream) {
  int rc = ffn_check(B, dim, F, act);
  if (rc) return rc;
  if (B == 0) return PKM_OK;
  if (!x || !w_gate || !w_up || !w_down || !workspace || !y || !gate != !up)
    return PKM_ERR_INVALID;
  for (const void* p : {x, w_gate, w_up, w_down, (const void*)workspace, (const void*)y,
                        (const void*)gate, (const void*)up})
    if (!ffn_aligned16(p)) return PKM_ERR_ALIGN;
  int* st;
  if ((rc = ffn_status(status, &st))) return rc;
  return pkm::launch_gated_ffn(x, w_gate, w_up, w_down, B, dim, F, act, workspace, y, gate, up, st,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

extern "C" int pkm_gated_ffn_backward(const void* x, const void* w_gate, const void* w_up,
                                      const void* w_down, const void* gate, const void* up,
                                      const void* dy, int B, int dim, int F, int act,
                                      void* workspace, void* dx, void* dw_gate, void* dw_up,
                                      void* dw_down, int grad_dtype, int* status, void* stream) {
  int rc = ffn_check(B, dim, F, act);
  if (rc) return rc;
  if (grad_dtype != PKM_BF16 && grad_dtype != PKM_F32) return PKM_ERR_UNSUPPORTED;
  if (!dw_gate != !dw_up) return PKM_ERR_INVALID;
  if (B == 0) {  // no token: the weights' gradients are zero (fp32 ones: nothing is added)
    if (grad_dtype == PKM_F32) return PKM_OK;
    for (void* p : {dw_gate, dw_up, dw_down})
      if (p && cudaMemsetAsync(p, 0, (size_t)dim * F * 2, static_cast<cudaStream_t>(stream)) !=
                   cudaSuccess)
        return PKM_ERR_CUDA;
    return PKM_OK;
  }
  if (!x || !w_gate || !w_up || !w_down || !gate || !up || !dy || !workspace)
    return PKM_ERR_INVALID;
  for (const void* p : {x, w_gate, w_up, w_down, gate, up, dy, (const void*)workspace,
                        (const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                        (const void*)dw_down})
    if (!ffn_aligned16(p)) return PKM_ERR_ALIGN;
  int* st;
  if ((rc = ffn_status(status, &st))) return rc;
  return pkm::launch_gated_ffn_backward(x, w_gate, w_up, w_down, gate, up, dy, B, dim, F, act,
                                        workspace, dx, dw_gate, dw_up, dw_down, grad_dtype, st,
                                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}
