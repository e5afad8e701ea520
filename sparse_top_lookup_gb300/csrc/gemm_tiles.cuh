// The products of ffn.cu's kernel (see there): what a launch takes, for the operators that run theirs
// through it.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "ffn_common.cuh"
#include "pkm_internal.cuh"
#include "tc_common.cuh"

namespace pkm {
namespace tiles {

constexpr int FM = 128;                   // rows per CTA (the pair's MMA takes 2 * FM)
constexpr int FK = 64;                    // K per stage: one 128-byte swizzle row of bf16
constexpr int FA_BYTES = FM * FK * 2;     // 16 KiB
constexpr int FEPI_WARPS = 8;             // of one epilogue set

enum Epi {
  kGate,   // accumulator columns: half of them g, the same half of u; writes h (and g, u)
  kStore,  // C in bf16, or (Prod::add32 1) added to an fp32 matrix
  kDGate,  // accumulator: dh; reads g, u; writes dg, du, h
  kOut,    // as kStore, with rows' factors, fp32 results and stretches of K (Prod)
  // accumulator: logits of a vocabulary; see vocab_loss.cu
  kLoss,   // row by row, half a tile's maximum and sum of powers beside the target's
  kProb,   // their gradient in bf16, from the rows' log-sum-exp
  kExp     // powers against a reference for the row in bf16, and as kLoss, with that reference
};
constexpr bool of_logits(int epi) { return epi == kLoss || epi == kProb || epi == kExp; }
// Those whose tiles' width is Plan::width, 256, 192 or 128 columns, whatever kN (256) their space is for.
constexpr bool any_width(int epi) { return of_logits(epi) || epi == kOut; }
// What goes with the epilogue and the tile's accumulator columns kN.
template <int kEpi, int kN>
struct Tile {
  static constexpr int kB = kN / 2 * FK * 2;  // bytes of a B slab: each CTA holds half the columns
  static constexpr int kStage = FA_BYTES + kB;
  // an epilogue warp's blocks of 32 x 32 bf16; kDGate: two sets of three (g, then dg; u, then du;
  // h), which cost it one stage (a stage less is 5 % of a long product, measured)
  static constexpr int kBlocks = kEpi == kDGate ? 6 : kEpi == kLoss ? 0 : of_logits(kEpi) ? 2 : 4;
  static constexpr int kOut = kBlocks * 2048;
  // Two sets of epilogue warps take tiles in turn, one for each TMEM buffer (with one, of two warps to a
  // scheduler, latencies bound the logits' tiles: 4.5 us of 256 x 256 whatever their depth)
  static constexpr int kSets = of_logits(kEpi) ? 2 : 1;
  static constexpr int kThreads = 64 + 32 * FEPI_WARPS * kSets;
  static constexpr int kStages = (kN == 256 ? 5 : 6) - (kEpi == kDGate) + (kEpi == kLoss);
  static constexpr int kSmem = kStages * kStage + FEPI_WARPS * kSets * kOut + 1024;  // + alignment
  static_assert(kSmem + 768 <= 227 * 1024, "feed-forward shared memory");
};

// How a launch's tiles are split over its clusters.  The products' tiles are numbered one product
// after the other.  `whole` of them, from tile whole0 on, are done whole, one per cluster and
// round.  `cut` of them, from cut0 on, of kb slabs each, are laid end to end and cut into
// stretches of w slabs (what a single product leaves after its last full round; or a launch's
// first product, when its few tiles are much longer than the others): a stretch begins with the
// end of a tile (its cluster writes those sums to memory: a part) and goes on with the beginning
// of the next, whose cluster adds the other stretches' parts, waits for them if it must, and
// writes the tile.  Stretches are done first, and a cluster waits only
// for clusters of lower numbers, which start before it and never wait before they have written
// their part.  Two products of kOut are dealt out by their tiles' lengths instead: the longer ones round by
// round, then shorter ones to the clusters that are done first, until all are level (in plain rounds
// the clusters with one long tile more had up to a tenth more to do than the average).
struct Plan {
  int clusters;
  int width;
  int whole0, whole;
  int cut0, cut, kb, w;  // cut 0: no tile is cut
  // lead > 0 (no tile is cut): two products, the first one's `lead` tiles longer than the second's; clusters
  // from `later` on have one of those less than the others, and `sooner` of the shorter ones first
  int lead, later, sooner;
};
struct Seg {
  int tile, k0, k1;  // k1 < 0: all of the tile's slabs
  int part;    // >= 0: the sums go to this part instead of the tile
  int parts;   // of the tile, to be added: [first, first + parts)
  int first;
};

// A product: K runs through `segs` pairs (a[i], b[i]) one after the other.
struct Prod {
  CUtensorMap a[2], b[2], out;
  int M, N, K;     // K of one segment
  int segs;
  int a_mn, b_mn;  // operand stored with M (N) contiguous
  int a_rows;      // any_width, not a_mn: rows of a's boxes, FM or all of fewer (rows past them are not stored)
  int add32;       // out is fp32: 1 added to, 2 (kOut) overwritten
  // kOut, splits > 1: K in so many stretches of split_kb slabs (the last may be shorter), whose sums go, in
  // fp32 (add32 2), to out's rows from split * (M rounded up to 32) on
  int splits, split_kb;
  // kOut: each row is multiplied by its own, then all by one, in fp32; or NULL
  const float *row_scale, *all_scale;
  int tiles;
};
constexpr int kMaxProds = 4;
struct GemmArgs {
  Prod prod[kMaxProds];
  CUtensorMap more[2];  // kGate (out: h): g, u; kDGate (out: dg): du, h
  CUtensorMap in[2];    // kDGate: g, u
  int prods, act, keep;  // keep: kGate writes g and u
  // kLoss, kProb, kExp: the tokens' targets (columns; those of this launch are [col0, col0 + N))
  const int64_t* target;
  int64_t col0;
  float2* row_parts;         // kLoss, kExp: [half a tile][row], maximum and sum
  const float* ref;          // kExp: [row]; kProb: the log-sum-exp
  const float* loss;         // kProb: [row]
  const float* factor;       // kProb, kExp: [row], a row of 0 is written as zeros
  const int* only_if;        // NULL, or a word on the device: nothing is done if it is 0
  Plan plan;
  float4* parts;                // [stretch][CTA of the pair][column / 4][row], FM rows
  unsigned long long* flags;    // [stretch][CTA of the pair][epilogue warp]
  unsigned long long epoch;     // a flag's value when its part is there
  int* status;  // may be NULL
};

// An operand whose rows are M (N) and whose columns are K, or the transpose; `rows` of it (64 for
// the transpose) are one CTA's in a slab.
inline bool operand(CUtensorMap* m, const void* ptr, int rows, int cols, bool mn, int box = FM,
                    int64_t pitch = 0) {
  return encode_matrix(m, ptr, rows, cols, 64, mn ? FK : box, pitch);
}
// A result [rows, cols] in blocks of 32 x 32, bf16 or fp32.
inline bool result(CUtensorMap* m, void* ptr, int rows, int cols, bool f32 = false, int64_t pitch = 0) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(pitch ? pitch : cols) * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr,
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Parts of cut tiles: [cluster][2][columns / 4][FM rows] float4, and their flags.
constexpr int kMaxClusters = 80, kMaxN = 256;
constexpr size_t kPartsBytes = (size_t)kMaxClusters * 2 * kMaxN * FM * 4;
constexpr size_t kFlagsBytes = (size_t)kMaxClusters * 2 * FEPI_WARPS * 8;
static_assert(kPartsBytes % 256 == 0 && kFlagsBytes % 256 == 0, "parts of the workspace are aligned");
inline void set_parts(GemmArgs& p, void* ws) {
  p.parts = static_cast<float4*>(ws);
  p.flags = reinterpret_cast<unsigned long long*>(static_cast<unsigned char*>(ws) + kPartsBytes);
}

// B operands are encoded here, for the tile's width.
struct BOperand {
  const void* ptr;
  int rows, cols;
  int64_t pitch;  // 0: cols
};
// What a tile of kOut takes, in slabs of K: at least its epilogue (131072 x 1024 from one token: 2048 tiles of
// one slab in 80 us, 3 us each on 76 clusters).
inline int tile_slabs(int kb) { return kb < 10 ? 10 : kb; }

// a of a product of any width, K contiguous.  Few rows have boxes of their own height: rows that are not there
// cost a copy as much as those that are (4 tokens, 131072 x 1024: loss 72 us in boxes of 128, 53 so).
inline bool rows_operand(Prod& q, const void* ptr, int rows, int cols, int64_t pitch = 0) {
  q.a_rows = rows < FM ? (rows + 7) / 8 * 8 : FM;
  return operand(&q.a[0], ptr, rows, cols, false, q.a_rows, pitch);
}

// Runs p's products, whose b operands are b (encoded for the tile's width that the plan takes).
// half: NULL, or the columns of half a tile (kLoss's row_parts).
cudaError_t launch_products(Epi epi, GemmArgs& p, const BOperand (&b)[kMaxProds][2], cudaStream_t stream,
                            int* half = nullptr);

}  // namespace tiles
}  // namespace pkm
