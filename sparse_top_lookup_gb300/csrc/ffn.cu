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
// tcgen05.mma.cta_group::2 of M = 256 rows (128 in each CTA) and N = 256 or 128
// columns, K in slabs of 64 through a ring of shared-memory stages filled by
// TMA; TMEM holds two accumulators, so a tile is multiplied while the one
// before it is written out by eight epilogue warps.  Operands are
// taken as they lie in memory: with K contiguous (K-major) or with M or N
// contiguous (MN-major: the products with a transposed operand), both with
// 128-byte swizzle.  What differs is the epilogue (Epi): each warp turns 32
// columns of its 32 rows at a time into bf16 in its own shared-memory buffers
// and stores them by TMA (a thread's own 64 bytes of a row, stored directly,
// touch 32 lines per instruction: the forward gate took 745 us at 16384 x 2048 x
// 8192 that way, 600 this way).
//
// Roundings to bf16 besides the results': h, dg and du, which the tensor cores take as bf16 operands,
// and g and u, which the caller keeps in bf16 between the passes (fp32 would double what the gate
// stores and the backward gate loads, which bounds it).  Off the 64-bit results in the 2-norm: y
// 2.3e-3, gradients of a forward and a backward pass 3.5e-3, where one rounding at the end leaves 1.7e-3.
//
// Bound by the tensor pipe in long products: 92 to 95 % busy in the gate and in the backward
// pass's last four at 4096 x 2048 x 8192, 81 % in the down projection (128 tiles on 76 clusters),
// at the clock that 1400 W leaves.  Each SM takes 180 GB/s of operands from L2 then, about what L2
// gives all of them, so what an epilogue moves beside them costs time: the backward gate (five
// tensors through it) takes 424 us at 16384 x 2048 x 8192, of which the product alone is 266, the
// loads of g and u 70 and the stores of dg, du and h 85; its arithmetic is hidden.  g and u through
// registers took 469 us, h stored directly 508, g and u prefetched into L2 438, asked for two blocks
// ahead from tile to tile with blocks of their own for the results 433.
//
// The vocabulary loss's products run here too (launch_products; vocab_loss.cu says what its epilogues
// are for): tiles of 256, 192 or 128 columns, and for the logits two sets of epilogue warps.
//
// One launch takes several products (the backward pass's last four), so that
// small ones fill the GPU together.  Work is split evenly over the clusters
// (Plan): whole tiles while there is one for every cluster, then, where that
// pays, what is left in equal stretches of K slabs.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <chrono>

#include "ffn_common.cuh"
#include "gemm_tiles.cuh"
#include "pkm_internal.cuh"
#include "tc_common.cuh"

namespace pkm {
namespace {

using namespace tc;
using namespace tiles;

// Segment i of cluster c; false past the last.
template <int kEpi>
__device__ __forceinline__ bool seg_at(const Plan& p, int c, int i, Seg& s) {
  s.part = -1, s.parts = 0, s.first = 0;
  if (kEpi == kOut && p.lead) {
    s.k0 = 0, s.k1 = -1;
    const int mine = p.lead / p.clusters + (c < p.later);
    if (i < mine) {
      s.tile = i * p.clusters + c;
      return true;
    }
    i -= mine;
    const bool late = c >= p.later;
    if (late && i < p.sooner) {
      s.tile = p.lead + i * (p.clusters - p.later) + c - p.later;
    } else {
      if (late) i -= p.sooner;
      // (those that had more to do so far come last)
      s.tile = p.lead + p.sooner * (p.clusters - p.later) + i * p.clusters + p.clusters - 1 - c;
    }
    return s.tile < p.whole;
  }
  if (p.cut) {
    const int r = p.clusters - 1 - c;  // a tile's later stretches belong to lower clusters
    const int total = p.cut * p.kb;
    const int lo = min(r * p.w, total), hi = min(lo + p.w, total);
    const int t0 = lo / p.kb;
    const int mid = lo == t0 * p.kb ? lo : min(hi, (t0 + 1) * p.kb);  // where a tile begins
    const int n = (lo < mid) + (mid < hi);
    if (i < n) {
      if (i == 0 && lo < mid) {
        s.tile = p.cut0 + t0, s.k0 = lo - t0 * p.kb, s.k1 = mid - t0 * p.kb, s.part = r;
      } else {
        const int t = mid / p.kb;
        s.tile = p.cut0 + t, s.k0 = 0, s.k1 = hi - mid;
        s.first = r + 1;
        s.parts = ((t + 1) * p.kb - 1) / p.w - r;
      }
      return true;
    }
    i -= n;
  }
  // (every other round backwards: the clusters with the longest tiles of a launch, its first,
  // are the last to get a second one)
  const int t = i * p.clusters + (i & 1 ? p.clusters - 1 - c : c);
  s.tile = p.whole0 + t, s.k0 = 0, s.k1 = -1;
  return t < p.whole;
}

// A 32 x 32 block in shared memory as TMA stores it: rows of 64 bytes (bf16, 64-byte swizzle) or
// of 128 (fp32, 128-byte swizzle); 16-byte piece `piece` of row `row`.
__device__ __forceinline__ uint32_t at64(uint32_t buf, int row, int piece) {
  return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t at128(uint32_t buf, int row, int piece) {
  return buf + row * 128 + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ void sts(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Row `lane` of a block from 32 values.
__device__ __forceinline__ void put_row(uint32_t buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    sts(at64(buf, lane, j),
        make_uint4(pack2(v[8 * j], v[8 * j + 1]), pack2(v[8 * j + 2], v[8 * j + 3]),
                   pack2(v[8 * j + 4], v[8 * j + 5]), pack2(v[8 * j + 6], v[8 * j + 7])));
}
__device__ __forceinline__ void get_row(uint32_t buf, int lane, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 x = lds(at64(buf, lane, j));
    v[8 * j] = lo_bf16(x.x), v[8 * j + 1] = hi_bf16(x.x);
    v[8 * j + 2] = lo_bf16(x.y), v[8 * j + 3] = hi_bf16(x.y);
    v[8 * j + 4] = lo_bf16(x.z), v[8 * j + 5] = hi_bf16(x.z);
    v[8 * j + 6] = lo_bf16(x.w), v[8 * j + 7] = hi_bf16(x.w);
  }
}
// A block's store (one thread), each in a group of its own.
__device__ __forceinline__ void store_open(const CUtensorMap* map, uint32_t buf, int col, int row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(col), "r"(row), "r"(buf)
               : "memory");
}
__device__ __forceinline__ void commit_stores() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_block(const CUtensorMap* map, uint32_t buf, int col, int row) {
  store_open(map, buf, col, row);
  commit_stores();
}
__device__ __forceinline__ void add_block(const CUtensorMap* map, uint32_t buf, int col, int row) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(col), "r"(row), "r"(buf)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last kPending stores of this thread have read their blocks.
template <int kPending>
__device__ __forceinline__ void blocks_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void blocks_written() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void blocks_visible() {  // this thread's writes, to the stores
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Tile t: its product, row tile and column tile (tile_n columns).  Within a product, bands of 8
// row tiles, within a band row tiles fastest: tiles that run at one time share operands in L2.
// split: its stretch of K, where K is split.
template <int kEpi>
__device__ __forceinline__ const Prod& tile_at(const GemmArgs& p, int t, int tile_n, int& tm, int& tn,
                                               int& split) {
  int i = 0;
  while (i + 1 < p.prods && t >= p.prod[i].tiles) t -= p.prod[i++].tiles;
  const Prod& q = p.prod[i];
  const int tm_count = (q.M + 2 * FM - 1) / (2 * FM), tn_count = (q.N + tile_n - 1) / tile_n;
  split = 0;
  if (kEpi == kOut && q.splits > 1) {
    split = t / (tm_count * tn_count);
    t -= split * tm_count * tn_count;
  }
  const int band = t / (8 * tn_count);
  const int rows = min(8, tm_count - 8 * band);
  t -= band * 8 * tn_count;
  tn = t / rows;
  tm = band * 8 + t - tn * rows;
  return q;
}

// The slabs of K that a tile's segment takes.
template <int kEpi>
__device__ __forceinline__ void slabs_of(const Prod& q, const Seg& sg, int split, int& k0, int& k1) {
  const int kb = (q.K + FK - 1) / FK * q.segs;
  k0 = sg.k0, k1 = sg.k1 < 0 ? kb : sg.k1;
  if (kEpi == kOut && q.splits > 1) k0 = split * q.split_kb, k1 = min(k0 + q.split_kb, kb);
}

template <int kEpi, int kN>
__global__ void __launch_bounds__((Tile<kEpi, kN>::kThreads), 1)
ffn_gemm_kernel(const __grid_constant__ GemmArgs p) {
  extern __shared__ unsigned char smem_raw[];
  using Shape = Tile<kEpi, kN>;
  constexpr int FSTAGES = Shape::kStages, FSTAGE_BYTES = Shape::kStage;
  __shared__ __align__(8) uint64_t bars[2 * FSTAGES + 4 + 1 + 2 * FEPI_WARPS];
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_abort;

  // output columns per tile
  const int tile_n = any_width(kEpi) ? p.plan.width : kEpi == kGate ? kN / 2 : kN;
  const uint32_t rank = cluster_ctarank();
  const int slot = (int)(blockIdx.x >> 1);

  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t stages_u32 = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
    for (int i = 0; i < 2 * FEPI_WARPS; ++i) mbar_init(bar_done + 8u * (1 + i), 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {  // one warp of each CTA allocates, jointly for the pair
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem_base)),
                 "r"(2 * kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs' barriers exist before any remote arrival
  const uint32_t tmem = s_tmem_base;
  const Ctl ctl{&s_abort, status_of(p.status)};

  // Everything up to here may run before the launch before this one has ended (programmatic
  // dependent launch); no memory is read or written until it has.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool run = !p.only_if || *p.only_if != 0;

  // The two issuing warps run their loops with all lanes and elect one only around what it
  // issues: with the loop in one lane's branch a step took 0.22 us more or less whatever it
  // copied, as long as a slab's MMAs; so it takes 0.13.
  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    uint32_t s = 0, ph = 1, used = 0;
    const uint32_t full0 = mapa_shared(bar0, 0);  // the leader's barriers
    bool ok = true;
    Seg sg;
    for (int i = 0; run && ok && seg_at<kEpi>(p.plan, slot, i, sg); ++i) {
      int tm, tn, split, k_first, k1;
      const Prod& q = tile_at<kEpi>(p, sg.tile, tile_n, tm, tn, split);
      slabs_of<kEpi>(q, sg, split, k_first, k1);
      const int row0 = (2 * tm + (int)rank) * FM;
      // kGate: CTA 0 holds the tile's rows of Wg, CTA 1 those of Wu
      const int col0 = kEpi == kGate ? tn * tile_n : tn * tile_n + (int)rank * (tile_n / 2);
      const int kb_seg = (q.K + FK - 1) / FK;
      const bool a_mn = q.a_mn, b_mn = q.b_mn;
      int seg = k_first / kb_seg, k0 = (k_first - seg * kb_seg) * FK;
      for (int kb = k_first; kb < k1; ++kb) {
        if (!__all_sync(0xffffffffu, wait_phase_cluster(bar_empty(s), ph, ctl))) {
          ok = false;
          break;
        }
        const uint32_t da = stages_u32 + s * FSTAGE_BYTES, db = da + FA_BYTES;
        const uint32_t fb = full0 + 8u * s;
        const CUtensorMap* ma = &q.a[seg];
        const CUtensorMap* mb = kEpi == kGate ? &q.b[rank] : &q.b[seg];
        if (elect_one()) {
          // (any_width: boxes of 64 columns, the last of which may be half used; or tile_n / 2 rows)
          const int boxes = any_width(kEpi) ? (tile_n / 2 + 63) / 64 : kN / 128;
          if (rank == 0)
            mbar_expect_tx(bar_full(s), !any_width(kEpi) ? 2u * FSTAGE_BYTES
                                        : 2u * ((a_mn ? FM : q.a_rows) +
                                                (b_mn ? boxes * 64 : tile_n / 2)) * FK * 2);
          if (a_mn) {
            tma_load_2d_cg2(da, ma, row0, k0, fb);
            tma_load_2d_cg2(da + FA_BYTES / 2, ma, row0 + 64, k0, fb);
          } else {
            tma_load_2d_cg2(da, ma, k0, row0, fb);
          }
          if (b_mn) {
#pragma unroll
            for (int j = 0; j < kN / 128; ++j)
              if (j < boxes) tma_load_2d_cg2(db + j * 64 * FK * 2, mb, col0 + 64 * j, k0, fb);
          } else {
            tma_load_2d_cg2(db, mb, k0, col0, fb);
          }
        }
        __syncwarp();
        if (used < (uint32_t)FSTAGES) ++used;
        if (++s == (uint32_t)FSTAGES) s = 0, ph ^= 1u;
        k0 += FK;
        if (k0 >= q.K) k0 = 0, ++seg;
      }
    }
    // the leader's last releases of this CTA's stages land before it exits; if a wait gave up, the
    // copies on their way (the leader sees both CTAs', as far as it has got)
    if (!ok && rank != 0) let_copies_land();
    for (uint32_t j = 0; (ok || rank == 0) && j < used; ++j) {
      if (s == 0) s = FSTAGES, ph ^= 1u;
      --s;
      wait_phase_drain(ok ? bar_empty(s) : bar_full(s), ph ^ 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      uint32_t s = 0, ph = 0;
      bool ok = true;
      Seg sg;
      for (int i = 0; run && ok && seg_at<kEpi>(p.plan, slot, i, sg); ++i) {
        const uint32_t buf = i & 1u, use = i >> 1;
        if (!__all_sync(0xffffffffu, wait_phase_cluster(bar_tempty(buf), (use & 1u) ^ 1u, ctl)))
          break;
        tc_fence_after();
        int tm, tn, split, k0, k1;
        const Prod& q = tile_at<kEpi>(p, sg.tile, tile_n, tm, tn, split);
        slabs_of<kEpi>(q, sg, split, k0, k1);
        const bool a_mn = q.a_mn, b_mn = q.b_mn;
        const uint32_t idesc =
            idesc_bf16(2 * FM, any_width(kEpi) ? tile_n : kN) | (a_mn ? kIdescAMn : 0u) | (b_mn ? kIdescBMn : 0u);
        // descriptor advance per 16 of K: 32 bytes along a swizzled row, or 16 rows of 128 bytes
        const uint32_t a_step = a_mn ? 128u : 2u, b_step = b_mn ? 128u : 2u;
        for (int kb = k0; kb < k1; ++kb) {
          if (!__all_sync(0xffffffffu, wait_phase_cluster(bar_full(s), ph, ctl))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = stages_u32 + s * FSTAGE_BYTES;
          const uint64_t a_desc = a_mn ? sw128_mn_desc(sa, 64 * FK * 2) : sw128_desc(sa);
          const uint64_t b_desc = b_mn ? sw128_mn_desc(sa + FA_BYTES, 64 * FK * 2)
                                       : sw128_desc(sa + FA_BYTES);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < FK / 16; ++kk)
              tc_mma_cg2(tmem + buf * kN, a_desc + a_step * kk, b_desc + b_step * kk, idesc,
                         kb != k0 || kk != 0);
            tc_commit_cg2_mc(bar_empty(s), 3);  // the stage is free again in both CTAs
            // the tile's sums are in both TMEMs
            if (kb + 1 == k1) tc_commit_cg2_mc(bar_tfull(buf), 3);
          }
          __syncwarp();
          if (++s == (uint32_t)FSTAGES) s = 0, ph ^= 1u;
        }
      }
      // every issued MMA completes before TMEM is released
      if (elect_one()) tc_commit_cg2_mc(bar_done, 1);
      __syncwarp();
      wait_phase_drain(bar_done, 0);
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int set = (warp - 2) / FEPI_WARPS, ew = (warp - 2) % FEPI_WARPS;
    const int quad = warp & 3, half = ew >> 2;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t bufs = stages_u32 + FSTAGES * FSTAGE_BYTES + (warp - 2) * Shape::kOut;
    uint32_t nb = 0;  // next buffer of four; kDGate: bit k, the parity of set k's next loads
    uint32_t asked = 0;  // kDGate, lane 0: bit k, set k's loads are on their way
    bool ok = true;
    Seg sg;
    for (int i = set; run && ok && seg_at<kEpi>(p.plan, slot, i, sg); i += Shape::kSets) {
      int tm, tn, split;
      const Prod& q = tile_at<kEpi>(p, sg.tile, tile_n, tm, tn, split);
      const int M = q.M, N = q.N;
      const uint32_t buf = i & 1u, use = i >> 1;
      const uint32_t taddr = lane_addr + buf * kN;
      const int row0 = (2 * tm + (int)rank) * FM + quad * 32;  // of the warp
      const int row = row0 + lane;
      const int half_n = tile_n / 2;
      const int cols = min(half_n, N - tn * tile_n - half * half_n);  // may be <= 0
      const int col0 = tn * tile_n + half * half_n;
      const bool in = row < M;
      // this thread's part of a stretch's sums: [column / 4][row]
      const int prow = quad * 32 + lane;
      auto part_at = [&](int r) {
        return p.parts + ((size_t)(2 * r + rank) * (kN / 4)) * FM + prow;
      };
      auto flag_at = [&](int r) { return p.flags + (size_t)(2 * r + rank) * FEPI_WARPS + ew; };

      // kLoss, kProb, kExp: this thread's row; its target's column in this launch, or -1
      int at = -1;
      float ref = 0.0f, loss = 0.0f;
      bool live = false;
      if constexpr (of_logits(kEpi)) {
        if (in) {
          const int64_t t = p.target[row];
          if (t >= p.col0 && t < p.col0 + N) at = (int)(t - p.col0);
          if constexpr (kEpi != kLoss) ref = p.ref[row], live = p.factor[row] != 0.0f;
          if constexpr (kEpi == kProb) loss = p.loss[row];
        }
      }
      float scale = 1.0f, all = 1.0f;
      if constexpr (kEpi == kOut) {
        if (q.all_scale) all = *q.all_scale;
        if (q.row_scale && in) scale = q.row_scale[row];
      }

      // kDGate: chunk c's blocks of g and u into set (c / 32) & 1
      const uint32_t bar_set = bar_done + 8u * (1 + 2 * ew);
      auto ask = [&](int c) {
        const uint32_t k = (c >> 5) & 1, set = bufs + k * 3 * 2048;
        blocks_read<0>();  // the set's stores are done with it
        asked |= 1u << k;
        mbar_expect_tx(bar_set + 8u * k, 2 * 2048);
        tma_load_2d(set, &p.in[0], col0 + c, row0, bar_set + 8u * k);
        tma_load_2d(set + 2048, &p.in[1], col0 + c, row0, bar_set + 8u * k);
      };
      if (kEpi == kDGate && sg.part < 0 && row0 < M && lane == 0) {
        if (cols > 0) ask(0);
        if (cols > 32) ask(32);
      }
      __syncwarp();
      if (!(ok = __all_sync(0xffffffffu, wait_phase_cluster(bar_tfull(buf), use & 1u, ctl)))) break;
      tc_fence_after();
      if (row0 < M && cols > 0) {
        if (sg.part >= 0) {
          float4* dst = part_at(sg.part);
          for (int c = 0; c < cols; c += 32) {
#pragma unroll
            for (int q = 0; q < (kEpi == kGate ? 2 : 1); ++q) {
              const int tc = half * half_n + c + q * (kN / 2);
              float v[32];
              tmem_ld32(taddr + tc, v);
              if (in)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  __stcg(dst + (tc / 4 + j) * FM,
                         make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
            }
          }
          __threadfence();
          __syncwarp();
          if (lane == 0)
            asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(flag_at(sg.part)), "l"(p.epoch)
                         : "memory");
        } else {
          for (int r0 = 0; r0 < sg.parts; r0 += 32) {  // a lane waits for each part
            if (r0 + lane < sg.parts) {
              unsigned long long* flag = flag_at(sg.first + r0 + lane);
              const unsigned long long begun = globaltimer();
              unsigned long long f;
              do {
                asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(f) : "l"(flag) : "memory");
                if (f != p.epoch && globaltimer() - begun > WAIT_LIMIT_NS) {
                  s_abort = 1;
                  atomicExch(status_of(p.status), PKM_ERR_TIMEOUT);
                  break;
                }
              } while (f != p.epoch && !*ctl.abort);
              if (f != p.epoch) ok = false;
              *flag = 0;  // the next launch with this workspace starts afresh
            }
            ok = __all_sync(0xffffffffu, ok);
          }
          // accumulator columns tc .. tc + 31, with the other stretches' parts
          auto sums = [&](int tc, float (&v)[32]) {
            tmem_ld32(taddr + tc, v);
            for (int r = sg.first; r < sg.first + sg.parts; ++r) {
              const float4* src = part_at(r);
              if (in)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float4 t = __ldcg(src + (tc / 4 + j) * FM);
                  v[4 * j] += t.x, v[4 * j + 1] += t.y, v[4 * j + 2] += t.z, v[4 * j + 3] += t.w;
                }
            }
          };
          auto next_buf = [&] {
            const uint32_t b = bufs + nb * 2048;
            nb = (nb + 1) & 3;
            return b;
          };
          if constexpr (of_logits(kEpi)) {
            // (two blocks of a row go out together: each fence before a store costs what a block's
            // arithmetic does)
            float top = -INFINITY, sum = 0.0f;  // kLoss, kExp
#pragma unroll 1
            for (int i = 0; i < half_n / 32; ++i) {
              const int c = 32 * i, gc = col0 + c;
              if (!ok || c >= cols) break;
              float v[32];
              sums(half * half_n + c, v);
              if (kEpi != kProb && c + 32 > cols)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = c + j < cols ? v[j] : -INFINITY;
              const bool here = __any_sync(0xffffffffu, (unsigned)(at - gc) < 32u);
              if (kEpi != kProb && here)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (gc + j == at) v[j] = -INFINITY;
              float most = top;
              if constexpr (kEpi != kProb) {
                float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int j = 4; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
                most = fmaxf(fmaxf(most, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
              }
              if constexpr (kEpi == kLoss) {
                // (nothing but -inf yet, or +inf: powers against 0)
                ref = fabsf(most) < INFINITY ? most : 0.0f;
                sum *= top == -INFINITY ? 1.0f : ex2((top - ref) * kLog2e);
              }
              top = most;
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = ex2((v[j] - ref) * kLog2e);
              if constexpr (kEpi != kProb) {
                float more[4] = {};
#pragma unroll
                for (int j = 0; j < 32; ++j) more[j & 3] += v[j];
                sum += (more[0] + more[1]) + (more[2] + more[3]);
              }
              if constexpr (kEpi != kLoss) {
                if (here) {
                  // (a learnt token's is small: its loss still holds it, this logit and the log-sum-exp do not;
                  // kExp: what belongs here is known with the row's sum; beside a logit of +inf it is no number)
                  const float mine = kEpi == kExp ? 0.0f : ref == INFINITY ? NAN : expm1f(-loss);
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (gc + j == at) v[j] = mine;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = live ? v[j] : 0.0f;
                if (!(i & 1)) {
                  if (lane == 0) blocks_read<0>();  // the last stores are done with the two blocks
                  __syncwarp();
                }
                put_row(bufs + (i & 1) * 2048, lane, v);
                if ((i & 1) || c + 32 >= cols) {
                  blocks_visible();
                  __syncwarp();
                  if (lane == 0) {
                    if (i & 1) store_open(&q.out, bufs, gc - 32, row0);
                    store_open(&q.out, bufs + (i & 1) * 2048, gc, row0);
                    commit_stores();
                  }
                }
              }
            }
            if constexpr (kEpi != kProb)
              if (in && ok) p.row_parts[(int64_t)(2 * tn + half) * M + row] = make_float2(top, sum);
          } else
          for (int c = 0; ok && c < cols; c += 32) {
            const int tc = half * half_n + c, gc = col0 + c;
            float v[32];
            if constexpr (kEpi == kGate) {
              float w[32];
              sums(tc, v);
              sums(kN / 2 + tc, w);
              if (lane == 0) blocks_read<1>();
              __syncwarp();
              const uint32_t b0 = next_buf();
              uint32_t b1 = 0, b2 = 0;
              if (p.keep) {
                b1 = next_buf(), b2 = next_buf();
                put_row(b1, lane, v);
                put_row(b2, lane, w);
              }
              with_act(p.act, [&](auto tag) {
#pragma unroll
                for (int j = 0; j < 32; ++j) w[j] *= act_fwd<decltype(tag)::value>(v[j]);
              });
              put_row(b0, lane, w);
              blocks_visible();
              __syncwarp();
              if (lane == 0) {
                store_block(&q.out, b0, gc, row0);
                if (p.keep) {
                  store_block(&p.more[0], b1, gc, row0);
                  store_block(&p.more[1], b2, gc, row0);
                }
              }
            } else if constexpr (kEpi == kStore || kEpi == kOut) {
              sums(tc, v);
              if (kEpi == kOut && (q.row_scale || q.all_scale))
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = v[j] * scale * all;  // (their product may be out of range)
              if (!q.add32) {
                if (lane == 0) blocks_read<1>();  // (the last may be an fp32 block, two buffers)
                __syncwarp();
                const uint32_t b0 = next_buf();
                put_row(b0, lane, v);
                blocks_visible();
                __syncwarp();
                if (lane == 0) store_block(&q.out, b0, gc, row0);
              } else {
                // two buffers of twice the size (the blocks of a product before this one that
                // still lie in them are read first)
                if (lane == 0) blocks_read<0>();
                __syncwarp();
                const uint32_t b0 = bufs + (nb & 2) * 2048;
                nb = (nb + 2) & 3;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  sts(at128(b0, lane, j),
                      make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                 __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
                blocks_visible();
                __syncwarp();
                if (lane == 0) {
                  if (kEpi == kOut && q.add32 == 2)
                    store_block(&q.out, b0, gc, row0 + split * ((M + 31) / 32 * 32));
                  else
                    add_block(&q.out, b0, gc, row0);
                }
              }
            } else {
              const uint32_t k = (c >> 5) & 1, b0 = bufs + k * 3 * 2048, b1 = b0 + 2048,
                             b2 = b1 + 2048;
              sums(tc, v);
              if (!(ok = __all_sync(0xffffffffu, wait_phase(bar_set + 8u * k, (nb >> k) & 1u, ctl))))
                break;
              nb ^= 1u << k;
              asked &= ~(1u << k);
              float g[32], u[32];
              get_row(b0, lane, g);
              get_row(b1, lane, u);
              // the other set for the next chunk (its stores, of the chunk before, are read by now)
              if (lane == 0 && c >= 32 && c + 32 < cols) ask(c + 32);
              with_act(p.act, [&](auto tag) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float2 a = act_both<decltype(tag)::value>(g[j]);
                  g[j] = v[j] * u[j] * a.y;  // dg
                  v[j] *= a.x;               // du
                  u[j] *= a.x;               // h
                }
              });
              put_row(b0, lane, g);
              put_row(b1, lane, v);
              put_row(b2, lane, u);
              blocks_visible();
              __syncwarp();
              if (lane == 0) {
                store_block(&q.out, b0, gc, row0);
                store_block(&p.more[0], b1, gc, row0);
                store_block(&p.more[1], b2, gc, row0);
              }
              __syncwarp();
            }
          }
        }
      }
      // tile read: hand the TMEM buffer back to the leader's MMA warp
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(bar_tempty(buf), 0));
    }
    if (lane == 0) {
      for (uint32_t k = 0; kEpi == kDGate && k < 2; ++k)  // (gave up before they were needed)
        if (asked >> k & 1u) wait_phase_drain(bar_done + 8u * (1 + 2 * ew + k), (nb >> k) & 1u);
      blocks_written();
    }
  }

  tc_fence_before();
  __syncthreads();
  // the leader's MMAs (which write both CTAs' TMEM and read both CTAs'
  // stages) are complete, and no CTA still arrives on the other's barriers
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kN)
                 : "memory");
  }
}

// The value of this launch's flags.  The workspace is whatever its memory held before: a flag
// counts only if it has the launch's own 64-bit number, and is cleared when it has been seen (so
// a captured launch can be replayed).
unsigned long long next_epoch() {
  static std::atomic<unsigned long long> n(
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() *
      0x9E3779B97F4A7C15ull);
  const unsigned long long e = n.fetch_add(1, std::memory_order_relaxed);
  return e ? e : n.fetch_add(1, std::memory_order_relaxed);
}

// A slab's time by its accumulator columns, beside one of 256: 128 take about 0.66 (4096 x 1024 x 4096: 52 us
// against 39), 192 0.82.
double slab_time(int kN) { return kN == 256 ? 1.0 : kN == 192 ? 0.82 : 0.66; }

// The products of p in tiles of kN columns over at most `most` clusters, and about how long that
// takes, in slabs of a 256-column tile.
Plan plan_of(const GemmArgs& p, int epi, int kN, int most, double* cost) {
  const int tile_n = epi == kGate ? kN / 2 : kN;
  Plan pl = {};
  int64_t slabs = 0;
  int tiles = 0, longest = 0, first_tiles = 0, first_kb = 0, others = 0;
  for (int i = 0; i < p.prods; ++i) {
    const Prod& q = p.prod[i];
    int t = (q.M + 2 * FM - 1) / (2 * FM) * ((q.N + tile_n - 1) / tile_n);
    int kb = (q.K + FK - 1) / FK * q.segs;
    if (q.splits > 1) t *= q.splits, kb = q.split_kb;
    tiles += t;
    slabs += (int64_t)t * kb;
    longest = kb > longest ? kb : longest;
    if (i == 0)
      first_tiles = t, first_kb = kb;
    else
      others = kb > others ? kb : others;
  }
  const double slab = slab_time(kN);
  pl.width = kN;
  pl.clusters = tiles < most ? tiles : most;
  pl.whole = tiles;
  double rounds;  // in slabs; tiles of several lengths even out
  if (p.prods == 1)
    rounds = (double)((tiles + most - 1) / most) * longest;
  else
    rounds = (double)slabs / most + 0.5 * others > longest ? (double)slabs / most + 0.5 * others
                                                           : longest;
  if (epi == kOut && p.prods == 2 && first_kb > others && first_tiles > 0) {
    const int longer = tile_slabs(first_kb), shorter = tile_slabs(others);
    pl.lead = first_tiles;
    pl.later = first_tiles % pl.clusters;
    pl.sooner = pl.later ? (longer + shorter / 2) / shorter : 0;
    *cost = rounds * slab;
    return pl;
  }
  // Cutting: a tile into up to 4.  Parts cost about 6 us, 24 slabs' time, to write, to wait for
  // and to read (200 tokens, F = 8192, dim = 2048: 30 us whole, 20 cut in four).
  const int cut = p.prods == 1 ? tiles % most : first_tiles, kb = first_kb;
  if (cut && p.prod[0].splits <= 1 && (int64_t)cut * kb < INT32_MAX / 2) {
    int64_t w = ((int64_t)cut * kb + most - 1) / most;
    if (w < (kb + 3) / 4) w = (kb + 3) / 4;
    const int parts = (int)((kb + w - 1) / w);  // and one more where stretches straddle tiles
    const int rows = p.prod[0].M < 2 * FM ? p.prod[0].M : 2 * FM;
    const double extra = (14 + (6 + 3 * parts) * (rows / (2.0 * FM)) * (kN / 256.0)) / slab;
    double with;  // rounds, if it is cut
    if (p.prods == 1) {
      with = rounds - kb + w + extra;
    } else {
      const double rest = (double)(slabs - (int64_t)cut * kb) / most + 0.5 * others;
      with = w + extra + (rest > others ? rest : others);
    }
    if (w < kb && with < rounds) {
      rounds = with;
      pl.cut = cut, pl.kb = kb, pl.w = (int)w;
      pl.whole = tiles - cut;
      pl.cut0 = p.prods == 1 ? pl.whole : 0;
      pl.whole0 = p.prods == 1 ? 0 : cut;
      pl.clusters = pl.whole ? most : (int)(((int64_t)cut * kb + w - 1) / w);
    }
  }
  *cost = rounds * slab;
  return pl;
}

template <int kEpi, int kN>
cudaError_t launch_tiles(GemmArgs& p, cudaStream_t stream, int* most) {
  auto kernel = ffn_gemm_kernel<kEpi, kN>;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Tile<kEpi, kN>::kThreads);
  cfg.dynamicSmemBytes = Tile<kEpi, kN>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = most ? 1 : 2;
  if (most) {  // how many clusters run at one time
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Tile<kEpi, kN>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    *most = n < kMaxClusters ? n : kMaxClusters;
    return cudaSuccess;
  }
  cfg.gridDim = dim3(2 * (unsigned)p.plan.clusters);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// (B operands are encoded here, for the tile's width)
template <int kEpi>
cudaError_t launch_gemm(GemmArgs& p, const BOperand (&b)[kMaxProds][2], cudaStream_t stream,
                        int* half = nullptr) {
  static int most[2];
  if (!most[0]) {
    cudaError_t e = launch_tiles<kEpi, 256>(p, stream, &most[0]);
    if (e != cudaSuccess) return e;
  }
  int kN = 256;
  if constexpr (any_width(kEpi)) {
    double least = 0;
    for (int n = 256; n >= 128; n -= 64) {
      double cost;
      const Plan plan = plan_of(p, kEpi, n, most[0], &cost);
      if (n == 256 || cost < least) least = cost, p.plan = plan, kN = n;
    }
  } else {
    if (!most[1]) {
      cudaError_t e = launch_tiles<kEpi, 128>(p, stream, &most[1]);
      if (e != cudaSuccess) return e;
    }
    double c256, c128;
    const Plan p256 = plan_of(p, kEpi, 256, most[0], &c256);
    const Plan p128 = plan_of(p, kEpi, 128, most[1], &c128);
    kN = c256 <= c128 ? 256 : 128;
    p.plan = kN == 256 ? p256 : p128;
  }
  const int tile_n = kEpi == kGate ? kN / 2 : kN;
  if (half) *half = tile_n / 2;
  for (int i = 0; i < p.prods; ++i) {
    Prod& q = p.prod[i];
    q.tiles = (q.M + 2 * FM - 1) / (2 * FM) * ((q.N + tile_n - 1) / tile_n);
    if (q.splits > 1) q.tiles *= q.splits;
    for (int j = 0; j < (kEpi == kGate ? 2 : q.segs); ++j)
      if (!operand(&q.b[j], b[i][j].ptr, b[i][j].rows, b[i][j].cols, q.b_mn, kN / 2, b[i][j].pitch))
        return cudaErrorInvalidValue;
  }
  p.epoch = next_epoch();
  if constexpr (any_width(kEpi)) return launch_tiles<kEpi, 256>(p, stream, nullptr);
  else
    return kN == 256 ? launch_tiles<kEpi, 256>(p, stream, nullptr)
                     : launch_tiles<kEpi, 128>(p, stream, nullptr);
}

}  // namespace

namespace tiles {
cudaError_t launch_products(Epi epi, GemmArgs& p, const BOperand (&b)[kMaxProds][2], cudaStream_t stream,
                            int* half) {
  switch (epi) {
    case kOut: return launch_gemm<kOut>(p, b, stream, half);
    case kLoss: return launch_gemm<kLoss>(p, b, stream, half);
    case kProb: return launch_gemm<kProb>(p, b, stream, half);
    case kExp: return launch_gemm<kExp>(p, b, stream, half);
    default: return cudaErrorInvalidValue;
  }
}
}  // namespace tiles

size_t gated_ffn_workspace_bytes(int B, int F) {
  return align256((size_t)B * F * 2) + (B > kFewTokens ? kPartsBytes + kFlagsBytes : 0);
}
size_t gated_ffn_backward_workspace_bytes(int B, int F) {
  return 3 * align256((size_t)B * F * 2) + kPartsBytes + kFlagsBytes;
}

cudaError_t launch_gated_ffn(const void* x, const void* w_gate, const void* w_up,
                             const void* w_down, int B, int dim, int F, int act, void* workspace,
                             void* y, void* gate, void* up, int* status, cudaStream_t stream) {
  if (B <= kFewTokens)
    return launch_ffn_few(x, w_gate, w_up, w_down, B, dim, F, act, workspace, y, gate, up, status,
                          stream);
  GemmArgs p = {};
  p.prods = 1;
  p.act = act;
  p.status = status;
  p.keep = gate != nullptr;
  set_parts(p, static_cast<unsigned char*>(workspace) + align256((size_t)B * F * 2));
  Prod& q = p.prod[0];
  q.segs = 1;
  q.M = B, q.N = F, q.K = dim;
  if (!operand(&q.a[0], x, B, dim, false) || !result(&q.out, workspace, B, F) ||
      (gate && (!result(&p.more[0], gate, B, F) || !result(&p.more[1], up, B, F))))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_gemm<kGate>(p, {{{w_gate, F, dim}, {w_up, F, dim}}}, stream);
  if (e != cudaSuccess) return e;
  q.N = dim, q.K = F;
  if (!operand(&q.a[0], workspace, B, F, false) || !result(&q.out, y, B, dim))
    return cudaErrorInvalidValue;
  return launch_gemm<kStore>(p, {{{w_down, dim, F}}}, stream);
}

cudaError_t launch_gated_ffn_backward(const void* x, const void* w_gate, const void* w_up,
                                      const void* w_down, const void* gate, const void* up,
                                      const void* dy, int B, int dim, int F, int act,
                                      void* workspace, void* dx, void* dw_gate, void* dw_up,
                                      void* dw_down, int grad_dtype, int* status,
                                      cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const size_t part = align256((size_t)B * F * 2);
  void *dg = ws, *du = ws + part, *h = ws + 2 * part;
  GemmArgs p = {};
  p.prods = 1;
  p.act = act;
  p.status = status;
  set_parts(p, ws + 3 * part);
  const bool few = B <= kFewTokens;
  if (few) {
    cudaError_t e = launch_ffn_few_backward(w_gate, w_up, w_down, gate, up, dy, B, dim, F, act, dg,
                                            du, h, dx, status, stream);
    if (e != cudaSuccess) return e;
  } else {  // dh = dy Wd, then dg, du and h
    Prod& q = p.prod[0];
    q.segs = 1;
    q.M = B, q.N = F, q.K = dim, q.b_mn = 1;
    if (!operand(&q.a[0], dy, B, dim, false) || !result(&q.out, dg, B, F) ||
        !result(&p.more[0], du, B, F) || !result(&p.more[1], h, B, F) ||
        !result(&p.in[0], const_cast<void*>(gate), B, F) ||
        !result(&p.in[1], const_cast<void*>(up), B, F))
      return cudaErrorInvalidValue;
    cudaError_t e = launch_gemm<kDGate>(p, {{{w_down, dim, F}}}, stream);
    if (e != cudaSuccess) return e;
  }
  // the rest in one launch
  const bool add = grad_dtype == PKM_F32;
  BOperand b[kMaxProds][2] = {};
  p.prods = 0;
  auto weight = [&](const void* a, int rows, const void* bp, int cols, void* out) {
    Prod& q = p.prod[p.prods];  // out [rows, cols] = a^T b over the batch
    q = Prod{};
    q.segs = 1;
    q.M = rows, q.N = cols, q.K = B, q.a_mn = q.b_mn = 1, q.add32 = add;
    b[p.prods++][0] = {bp, B, cols};
    return operand(&q.a[0], a, B, rows, true) && result(&q.out, out, rows, cols, add);
  };
  auto input = [&] {  // dx = dg Wg + du Wu: one product of twice the depth
    Prod& q = p.prod[p.prods];
    q = Prod{};
    q.segs = 2;
    q.M = B, q.N = dim, q.K = F, q.b_mn = 1;
    b[p.prods][0] = {w_gate, F, dim};
    b[p.prods++][1] = {w_up, F, dim};
    return operand(&q.a[0], dg, B, F, false) && operand(&q.a[1], du, B, F, false) &&
           result(&q.out, dx, B, dim);
  };
  // longest tiles first: shorter ones fill the last rounds
  const bool first = 2 * (int64_t)F >= B;
  if (dx && !few && first && !input()) return cudaErrorInvalidValue;
  if (dw_gate && (!weight(dg, F, x, dim, dw_gate) || !weight(du, F, x, dim, dw_up)))
    return cudaErrorInvalidValue;
  if (dw_down && !weight(dy, dim, h, F, dw_down)) return cudaErrorInvalidValue;
  if (dx && !few && !first && !input()) return cudaErrorInvalidValue;
  return p.prods ? launch_gemm<kStore>(p, b, stream) : cudaSuccess;
}

}  // namespace pkm

namespace {

bool ffn_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ffn_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int ffn_check(int B, int dim, int F, int act) {
  if (B < 0 || dim < 1 || F < 1) return PKM_ERR_INVALID;
  if (act < PKM_ACT_SILU || act > PKM_ACT_RELU || dim % 8 || F % 8) return PKM_ERR_UNSUPPORTED;
  // the kernels count tiles (of 128 x 128 at the smallest) and rows in 32 bits
  constexpr int most = INT32_MAX - 256;
  auto t = [](int n) { return ((int64_t)n + 127) / 128; };
  if (B > most || dim > most || F > most || t(B) * t(F) > most / 4 || t(B) * t(dim) > most / 4 ||
      t(F) * t(dim) > most / 4)
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
  if (!ffn_aligned4(status)) return PKM_ERR_ALIGN;
  return pkm::launch_gated_ffn(x, w_gate, w_up, w_down, B, dim, F, act, workspace, y, gate, up, status,
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
  if (!ffn_aligned4(status)) return PKM_ERR_ALIGN;
  return pkm::launch_gated_ffn_backward(x, w_gate, w_up, w_down, gate, up, dy, B, dim, F, act,
                                        workspace, dx, dw_gate, dw_up, dw_down, grad_dtype, status,
                                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}
