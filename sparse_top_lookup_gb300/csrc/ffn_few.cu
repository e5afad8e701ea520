// The feed-forward block for few tokens (T up to kFewTokens): every product reads its weights once
// and is bound by that, so the weights are the MMA's rows and the tokens its columns.
//
//   D [rows of weights, tokens] = W [rows, K] t [tokens, K]^T
//
// tcgen05.mma M = 128, N = tokens rounded up to 16.  A tile is R <= 128 rows of weights (the gate
// and up projections: R <= 64 of each, rows 0 .. and 64 ..), R chosen with the number of CTAs that
// share a tile's K so that all SMs stream the same number of bytes; the MMA always takes 128 rows
// of shared memory, and what lies behind the R ends up in rows of D that nobody reads.  The CTAs of
// a tile form a cluster and join their sums through shared memory, each for a share of the rows,
// in a fixed order.
//
// Bound by HBM, and at one token by latency: a ring of about 100 KB per SM keeps 15 MB of weights
// in flight, and the second kernel of a call starts while the first one runs (programmatic
// dependent launch; both fit on an SM): it fills its ring with weights and waits for the first
// only before it loads the tokens' rows.  Rings of 64 and 180 KB: 11.4 and 17 us at one token of
// 1024 x 4096 (captured; this one 12 then, 11 now), 31 and 42 at 37 of 2048 x 8192 (this one 28).
//
// Measured at 37 tokens of 2048 x 8192 (100 MB of weights, 14.8 us at the copy's rate): 28 us
// captured.  The gate's weights stream from 2.4 to 15 us at 5.4 TB/s and its results are out at
// 17.5; the second kernel's tokens are there at 20, its products done at 25.5, its results out at 28.
#include <cuda_bf16.h>
#include <stdint.h>

#include "ffn_common.cuh"
#include "pkm_internal.cuh"
#include "tc_common.cuh"

namespace pkm {
namespace {

using namespace tc;

constexpr int WK = 64;            // K per slab: one 128-byte swizzle row of bf16
constexpr int WTHREADS = 192;     // copies, MMAs, four warps for the sums
constexpr int kRingBytes = 104 * 1024;
constexpr int kStageBytes = 26 * 1024;  // about; at least one slab
constexpr int kFewStages = 8;     // at most

enum FewMode { kFewGate, kFewStore, kFewDGate };

struct FewArgs {
  CUtensorMap w[2], t[2];  // kFewGate: Wg and Wu against t[0]; else segment i: w[i] against t[i]
  CUtensorMap t3_map[2];   // t as [K / 64][tokens][64]
  int M, T, K, segs;       // rows of weights, tokens, K of a segment
  int w_mn;                // weights stored with M contiguous (R is 64 or 128)
  int R, lsh;              // rows of a tile; log2 of the CTAs that share it
  int npad, slabs, stages; // tokens rounded up; slabs of a stage
  int t3;                  // K is whole slabs: a stage's token slabs in one copy
  int act, keep, dependent;
  __nv_bfloat16 *out0, *out1, *out2;  // [T, M]: kFewGate h, g, u; kFewStore C; kFewDGate dg, du, h
  const __nv_bfloat16 *g_in, *u_in;   // kFewDGate
  int* status;  // may be NULL
};

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  // (volatile keeps it behind the barriers; no memory clobber, so that loads of several items
  // can be in flight past the stores of the ones before)
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

template <int kMode>
__global__ void __launch_bounds__(WTHREADS)
ffn_few_kernel(const __grid_constant__ FewArgs p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kFewStages + 1];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  const int S = 1 << p.lsh, rank = (int)blockIdx.x & (S - 1), m0 = (int)(blockIdx.x >> p.lsh) * p.R;
  const int kb_seg = (p.K + WK - 1) / WK, kb = kb_seg * p.segs;
  const int per = (kb + S - 1) >> p.lsh;
  const int k_lo = min(rank * per, kb), k_hi = min(k_lo + per, kb);
  const int slab_w = kMode == kFewGate ? 8192 + p.R * 128 : p.R * 128;  // bytes of a slab's weights
  const int slab_t = p.npad * 128;
  const int stage_bytes = p.slabs * (slab_w + slab_t);

  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t ring = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(&bars[0]);
  auto bar_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto bar_empty = [&](uint32_t s) { return bar0 + 8u * (kFewStages + s); };
  const uint32_t bar_done = bar0 + 8u * (2 * kFewStages);
  const uint32_t columns = p.npad <= 32 ? 32 : p.npad <= 64 ? 64 : 128;  // of TMEM

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem_base)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  const Ctl ctl{&s_abort, status_of(p.status)};
  // A call's first launch may begin, up to here, before the launch before it has ended; its second
  // begins when all of the first are here, after what came before, so it may read weights.
  if (!p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------ copies
    // (all lanes run the loops, one is elected for each copy: see ffn.cu)
    auto weights = [&](uint32_t s, int k) {  // slabs from k on into stage s
      const int n = min(p.slabs, k_hi - k);
      if (elect_one())
        mbar_expect_tx(bar_full(s),
                       (uint32_t)(n * ((kMode == kFewGate ? 2 : 1) * p.R * 128 + slab_t)));
      for (int j = 0; j < n; ++j, ++k) {
        const int seg = k >= kb_seg ? 1 : 0, k0 = (k - seg * kb_seg) * WK;
        const uint32_t dst = ring + s * stage_bytes + j * slab_w;
        if (kMode == kFewGate) {
          if (elect_one()) {
            tma_load_2d(dst, &p.w[0], k0, m0, bar_full(s));
            tma_load_2d(dst + 8192, &p.w[1], k0, m0, bar_full(s));
          }
        } else if (p.w_mn) {
          if (elect_one()) {
            tma_load_2d(dst, &p.w[seg], m0, k0, bar_full(s));
            if (p.R > 64) tma_load_2d(dst + 8192, &p.w[seg], m0 + 64, k0, bar_full(s));
          }
        } else {
          if (elect_one()) tma_load_2d(dst, &p.w[seg], k0, m0, bar_full(s));
        }
      }
    };
    auto tokens = [&](uint32_t s, int k) {
      const int n = min(p.slabs, k_hi - k);
      const uint32_t at = ring + s * stage_bytes + p.slabs * slab_w;
      if (p.t3 && n == p.slabs && (k + n <= kb_seg || k >= kb_seg)) {
        const int seg = k >= kb_seg ? 1 : 0;
        if (elect_one())
          tma_load_3d(at, &p.t3_map[kMode == kFewGate ? 0 : seg], 0, 0, k - seg * kb_seg,
                      bar_full(s));
        return;
      }
      for (int j = 0; j < n; ++j, ++k) {
        const int seg = k >= kb_seg ? 1 : 0, k0 = (k - seg * kb_seg) * WK;
        if (elect_one())
          tma_load_2d(at + j * slab_t, &p.t[kMode == kFewGate ? 0 : seg], k0, 0, bar_full(s));
      }
    };
    // the ring's first filling: weights, then (once the kernel before this one is done) tokens
    int issued = 0;
    for (int k = k_lo; k < k_hi && issued < p.stages; k += p.slabs, ++issued) weights(issued, k);
    if (p.dependent) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      asm volatile("fence.proxy.async;" ::: "memory");
    }
    for (int i = 0; i < issued; ++i) tokens(i, k_lo + i * p.slabs);
    uint32_t s = 0, ph = 0;
    for (int k = k_lo + p.stages * p.slabs; k < k_hi; k += p.slabs, ++issued) {
      if (!__all_sync(0xffffffffu, wait_phase(bar_empty(s), ph, ctl))) break;
      weights(s, k);
      tokens(s, k);
      if (++s == (uint32_t)p.stages) s = 0, ph ^= 1u;
    }
    // every copy lands before the ring is used for the sums (and before the CTA goes)
    for (int j = max(0, issued - p.stages); j < issued; ++j)
      wait_phase_drain(bar_full(j % p.stages), (uint32_t)(j / p.stages) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------ MMAs
    const uint32_t idesc = idesc_bf16(128, p.npad) | (p.w_mn ? kIdescAMn : 0u);
    const uint32_t w_step = p.w_mn ? 128u : 2u;
    uint32_t s = 0, ph = 0;
    for (int k = k_lo; k < k_hi; k += p.slabs) {
      if (!__all_sync(0xffffffffu, wait_phase(bar_full(s), ph, ctl))) break;
      tc_fence_after();
      const int n = min(p.slabs, k_hi - k);
      for (int j = 0; j < n; ++j) {
        const uint32_t wa = ring + s * stage_bytes + j * slab_w;
        const uint32_t ta = ring + s * stage_bytes + p.slabs * slab_w + j * slab_t;
        const uint64_t wd = p.w_mn ? sw128_mn_desc(wa, 64 * WK * 2) : sw128_desc(wa);
        const uint64_t td = sw128_desc(ta);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < WK / 16; ++kk)
            tc_mma(tmem, wd + w_step * kk, td + 2u * kk, idesc, (k - k_lo) + j + kk != 0);
          if (j + 1 == n) tc_commit(bar_empty(s));
        }
      }
      __syncwarp();
      if (++s == (uint32_t)p.stages) s = 0, ph ^= 1u;
    }
    if (elect_one()) tc_commit(bar_done);
    __syncwarp();
  }
  // this CTA's share of the rows, two at a time, rows fastest
  const int share = ((p.R + S - 1) >> p.lsh) + 1 & ~1;
  const int r0 = rank * share, rows = min(share, min(p.R, p.M - m0) - r0);
  const int half = (rows + 1) / 2, items = rows > 0 ? half * p.T : 0;
  if (kMode == kFewDGate && warp >= 2)
    for (int i = threadIdx.x - 64; i < items; i += 128) {
      const int t = i / half;
      const size_t o = (size_t)t * p.M + m0 + r0 + 2 * (i - t * half);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.g_in + o));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.u_in + o));
    }
  // every copy has landed and every MMA has read it: the ring takes the sums, [token][row] (those of a
  // call that gave up mean nothing, but its MMAs still end before their memory goes)
  if (!wait_phase(bar_done, 0, ctl)) wait_phase_drain(bar_done, 0);
  __syncwarp();
  tc_fence_after();
  __syncthreads();
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* d = reinterpret_cast<float*>(smem);
    for (int c = 0; c < p.npad; c += 16) {
      float v[16];
      tmem_ld16(lane_addr + c, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) d[(c + j) * 128 + row] = k_lo < k_hi ? v[j] : 0.0f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync();
  if (items > 0) {
    for (int i = threadIdx.x; i < items; i += WTHREADS) {
      const int t = i / half, r = r0 + 2 * (i - t * half);
      float2 a = make_float2(0.0f, 0.0f), b = a;
      const uint32_t at = ring + (t * 128 + r) * 4;
#pragma unroll 4
      for (int c = 0; c < S; ++c) {
        const uint32_t from = S > 1 ? mapa_shared(at, c) : at;
        const float2 x = ld_cluster2(from);
        a.x += x.x, a.y += x.y;
        if (kMode == kFewGate) {
          const float2 y = ld_cluster2(from + 64 * 4);
          b.x += y.x, b.y += y.y;
        }
      }
      const size_t o = (size_t)t * p.M + m0 + r;
      auto put = [&](__nv_bfloat16* out, float x, float y) {
        *reinterpret_cast<uint32_t*>(out + o) = pack2(x, y);
      };
      if constexpr (kMode == kFewStore) {
        put(p.out0, a.x, a.y);
      } else if constexpr (kMode == kFewGate) {
        with_act(p.act, [&](auto tag) {
          constexpr int kAct = decltype(tag)::value;
          put(p.out0, act_fwd<kAct>(a.x) * b.x, act_fwd<kAct>(a.y) * b.y);
        });
        if (p.keep) {
          put(p.out1, a.x, a.y);
          put(p.out2, b.x, b.y);
        }
      } else {
        const uint32_t g = __ldg(reinterpret_cast<const uint32_t*>(p.g_in + o));
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p.u_in + o));
        with_act(p.act, [&](auto tag) {
          constexpr int kAct = decltype(tag)::value;
          const float2 x = act_both<kAct>(lo_bf16(g)), y = act_both<kAct>(hi_bf16(g));
          put(p.out0, a.x * lo_bf16(u) * x.y, a.y * hi_bf16(u) * y.y);
          put(p.out1, a.x * x.x, a.y * y.x);
          put(p.out2, lo_bf16(u) * x.x, hi_bf16(u) * y.x);
        });
      }
    }
  }
  // no CTA leaves while another reads its sums
  if (S > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns)
                 : "memory");
  }
}

// A [rows, cols] matrix, cols a multiple of 64, as [cols / 64][rows][64].
bool encode_slabs(CUtensorMap* m, const void* ptr, int rows, int cols, int box_rows, int slabs) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {WK, (cuuint64_t)rows, (cuuint64_t)cols / WK};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, WK * 2};
  const cuuint32_t box[3] = {WK, (cuuint32_t)box_rows, (cuuint32_t)slabs};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a tile and the CTAs that share it: the fewest bytes per CTA with every tile on the GPU
// at one time; fewer CTAs to a tile where that costs nothing.
void shape(FewArgs& p, int mode) {
  const int sms = sm_count(), kb = (p.K + WK - 1) / WK * p.segs;
  const int r_max = mode == kFewGate ? 64 : 128;
  int64_t best = -1;
  for (int lsh = 0; lsh <= 3; ++lsh) {
    const int S = 1 << lsh, per = (kb + S - 1) / S;
    if ((S - 1) * per >= kb) break;  // a CTA without a slab
    // (clusters of 8 do not fill every GPC)
    const int clusters = lsh == 3 ? sms * 15 / 16 / 8 : sms / S;
    int R = ((p.M + clusters - 1) / clusters + 7) / 8 * 8;
    if (p.w_mn) R = R > 64 ? 128 : 64;
    if (R > r_max) R = r_max;
    const int64_t tiles = (p.M + R - 1) / R, rounds = (tiles + clusters - 1) / clusters;
    // bytes of a CTA, its tokens' too, and a slab's own cost (about 2 KB more)
    const int64_t cost = rounds * per * ((mode == kFewGate ? 2 : 1) * R + p.npad + 16);
    if (best < 0 || cost < best) best = cost, p.R = R, p.lsh = lsh;
  }
  const int slab = (mode == kFewGate ? 8192 + p.R * 128 : p.R * 128) + p.npad * 128;
  p.slabs = kStageBytes / slab;
  if (p.slabs < 1) p.slabs = 1;
  p.stages = kRingBytes / (p.slabs * slab);
  if (p.stages > kFewStages) p.stages = kFewStages;
}

template <int kMode>
cudaError_t launch_few(FewArgs& p, const void* w0, const void* w1, const void* t0, const void* t1,
                       cudaStream_t stream) {
  p.npad = (p.T + 15) / 16 * 16;
  shape(p, kMode);
  p.t3 = p.K % WK == 0 && p.slabs > 1;
  const void *w[2] = {w0, w1}, *t[2] = {t0, t1};
  for (int i = 0; i < 2; ++i) {
    if (w[i] && !(p.w_mn ? encode_matrix(&p.w[i], w[i], p.K, p.M, 64, WK)
                         : encode_matrix(&p.w[i], w[i], p.M, p.K, WK, p.R)))
      return cudaErrorInvalidValue;
    if (t[i] && !encode_matrix(&p.t[i], t[i], p.T, p.K, WK, p.npad)) return cudaErrorInvalidValue;
    if (t[i] && p.t3 && !encode_slabs(&p.t3_map[i], t[i], p.T, p.K, p.npad, p.slabs))
      return cudaErrorInvalidValue;
  }
  const int slab_w = kMode == kFewGate ? 8192 + p.R * 128 : p.R * 128;
  const int stage = p.slabs * (slab_w + p.npad * 128);
  // behind the last slab's weights the MMA still reads up to 128 rows' worth
  const int behind = 16384 - slab_w - p.slabs * p.npad * 128;
  int bytes = p.stages * stage + (behind > 0 ? behind : 0);
  if (bytes < p.npad * 512) bytes = p.npad * 512;  // the sums
  auto kernel = ffn_few_kernel<kMode>;
  static int allowed = 0;
  if (!allowed) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRingBytes + 17 * 1024);
    if (e != cudaSuccess) return e;
    allowed = 1;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1 << p.lsh;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(WTHREADS);
  cfg.gridDim = dim3((unsigned)((p.M + p.R - 1) / p.R) << p.lsh);
  cfg.dynamicSmemBytes = bytes + 1024;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_ffn_few(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                           int B, int dim, int F, int act, void* h, void* y, void* gate, void* up,
                           int* status, cudaStream_t stream) {
  FewArgs p = {};
  p.act = act, p.status = status, p.segs = 1;
  p.T = B, p.M = F, p.K = dim;
  p.keep = gate != nullptr;
  p.out0 = static_cast<__nv_bfloat16*>(h);
  p.out1 = static_cast<__nv_bfloat16*>(gate);
  p.out2 = static_cast<__nv_bfloat16*>(up);
  cudaError_t e = launch_few<kFewGate>(p, w_gate, w_up, x, nullptr, stream);
  if (e != cudaSuccess) return e;
  p.M = dim, p.K = F, p.dependent = 1;
  p.out0 = static_cast<__nv_bfloat16*>(y);
  return launch_few<kFewStore>(p, w_down, nullptr, h, nullptr, stream);
}

cudaError_t launch_ffn_few_backward(const void* w_gate, const void* w_up, const void* w_down,
                                    const void* gate, const void* up, const void* dy, int B,
                                    int dim, int F, int act, void* dg, void* du, void* h, void* dx,
                                    int* status, cudaStream_t stream) {
  FewArgs p = {};
  p.act = act, p.status = status, p.segs = 1, p.w_mn = 1;
  p.T = B, p.M = F, p.K = dim;
  p.g_in = static_cast<const __nv_bfloat16*>(gate);
  p.u_in = static_cast<const __nv_bfloat16*>(up);
  p.out0 = static_cast<__nv_bfloat16*>(dg);
  p.out1 = static_cast<__nv_bfloat16*>(du);
  p.out2 = static_cast<__nv_bfloat16*>(h);
  cudaError_t e = launch_few<kFewDGate>(p, w_down, nullptr, dy, nullptr, stream);
  if (e != cudaSuccess || !dx) return e;
  p.M = dim, p.K = F, p.segs = 2, p.dependent = 1;
  p.out0 = static_cast<__nv_bfloat16*>(dx);
  return launch_few<kFewStore>(p, w_gate, w_up, dg, du, stream);
}

}  // namespace pkm
