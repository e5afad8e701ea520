// The head's product and the softmax cross entropy over its vocabulary, a piece of the logits at a time:
//
//   z = x W^T,  lse = log sum exp z,  loss = lse - z[target]
//   dz = dloss (exp(z - lse) - [target]),  dx = dz W,  dW = dz^T x
//
// x [B, dim] and W [V, dim] in bf16, z in fp32 in the tensor cores' accumulators (ffn.cu's kernel,
// which all products here run through).  Loss: the epilogue reduces each row of a tile, half a tile's
// columns at a time, to its maximum and sum of powers beside the target's, and join_kernel adds those up.
// The target stays out of the sums, and its logit is a sum of its own on the CUDA cores (the tensor
// cores cut low bits off, 5e-7 of a logit of 12 over 1024 products), so that the loss of a token that
// the model knows, log(1 + what is left), is good relative to itself.
//
// Backward: z is computed again, and its epilogue writes dz / dloss = exp(z - lse) - [target] in bf16,
// piece by piece (of the tokens, and of the vocabulary within), then dx and dW of the piece in one
// launch.  The target's own, exp(-loss) - 1, comes from the forward's loss, or from lse and once more an
// fp32 sum for its logit, which leaves in it what lse is off by (2^-24 of it from its rounding alone).  dloss
// multiplies dx's rows in fp32, and x in dW's operand, over what most tokens' dloss is in a mean
// (common_factor, which multiplies dW in fp32): x is rounded once more only where tokens weigh differently.
//
// Training, where the logits are more than one round of tiles: a quarter of the products can be saved.  The
// loss's epilogue writes E = exp(z - r) in bf16 against a reference r of its own for each token, the
// target's logit, which is known before, and the sums are known after it: dz = dloss exp(r - lse) E beside
// the target, whose element the join writes.  That factor takes dloss's place, so nothing passes over E
// again; it may be 2^-100 of dloss, so the common factor stays out of it here too, and dx's rows are multiplied
// by the one and the other.  E holds for a row whose sum stays below 2^100; when one of a piece does not (its best
// logit is 69 above the target's), the join takes that row's maximum for its reference and raises a mark, and two
// launches that do nothing otherwise (7 us) do the piece again.  8192 x 2048 x 131072: 10.7 ms in two passes,
// 7.7 to 8.3 so (one GPU and another).
//
// Roundings besides the results': dz (E) and the scaled x, both bf16 operands of the tensor cores.  Off the
// 64-bit results in the 2-norm: dx and dW 2.4e-3 where powers are kept and 2.1e-3 in two passes of a
// mean's gradient (one rounding at the end 1.7e-3), the loss 9e-7.
//
// Bound by the tensor pipe in long products: a training step of 8192 x 2048 x 131072 runs at 1.6 to 1.7 PFLOP/s, 93
// to 99 % of what cuBLAS sustains under the power limit; 84 % of the pipe's cycles in dx and dW at 4096 x 1024 x
// 32000, 76 % in the logits (27 rounds of tiles where 26.3 would do, and an epilogue of 2.9 us a tile beside 5.2 of
// products).  Short products (dim below 512) by that epilogue; few tokens by W's reading and dW's writing.
#include <math.h>
#include <stdint.h>

#include "gemm_tiles.cuh"
#include "launch_common.cuh"
#include "num_common.cuh"
#include "pkm_internal.cuh"

namespace pkm {
namespace {

using namespace tiles;

constexpr int64_t kPieceBytes = 1ll << 30;   // of dz
constexpr int64_t kPartBytes = 128ll << 20;  // of the rows' parts
constexpr int kMostTokens = 32768;           // of a piece in the backward pass

// ---------------------------------------------------------------- small kernels

// Rows of 32 tokens: a block's warps share a token's parts, which lie [part][token].
constexpr int kJoinWarps = 32;

struct Partial {  // sum exp(v - top) = sum
  float top, sum;
};
__device__ __forceinline__ float power(float v, float ref) { return ex2((v - ref) * kLog2e); }
// What powers are taken against for a maximum of `top`: it itself, or 0 where all logits so far are -inf (powers
// of 0) or one is +inf (its power, and so the sum, is +inf; inf - inf would be no number).
__device__ __forceinline__ float reference(float top) { return fabsf(top) < INFINITY ? top : 0.0f; }
// (a part without a finite logit has top = -inf, and a sum of 0 or NaN)
__device__ __forceinline__ Partial joined(Partial a, Partial b) {
  const float top = fmaxf(a.top, b.top), ref = reference(top);
  return {top, (a.top == -INFINITY ? a.sum : a.sum * power(a.top, ref)) +
                   (b.top == -INFINITY ? b.sum : b.sum * power(b.top, ref))};
}

// The loss of one token, whose time is the weight's reading: a warp takes kOneRows rows of W at a time
// (16-byte loads, the next ones on their way), their products on the CUDA cores in fp32, and keeps
// the maximum and the sum, so a block writes one part.  With its join 17 us at 32000 x 1024 (65 MB, 10
// us at the copy's rate), 86 at 131072 x 2048 (79), where tiles of 256 tokens take 21 and 105; two tokens
// in this way take 20 and 113, four 26 and 131.
constexpr int kOneWarps = 8, kOneRows = 4, kOneBlocks = 4 * 152;
constexpr int kOneMostDim = 32768;  // (64 KiB of x in shared memory)

__device__ __forceinline__ float dot8(uint4 a, const float (&x)[8], float s) {
  s = fmaf(lo_bf16(a.x), x[0], fmaf(hi_bf16(a.x), x[1], s));
  s = fmaf(lo_bf16(a.y), x[2], fmaf(hi_bf16(a.y), x[3], s));
  s = fmaf(lo_bf16(a.z), x[4], fmaf(hi_bf16(a.z), x[5], s));
  return fmaf(lo_bf16(a.w), x[6], fmaf(hi_bf16(a.w), x[7], s));
}

__global__ void __launch_bounds__(32 * kOneWarps)
one_token_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w,
                 const int64_t* __restrict__ target, int vecs, int V, float2* parts) {
  extern __shared__ uint4 xs[];  // [vecs]
  __shared__ Partial rows[kOneWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_launch_ahead();
  for (int i = threadIdx.x; i < vecs; i += 32 * kOneWarps) xs[i] = x[i];
  const int64_t at = target[0];
  __syncthreads();
  Partial sum = {-INFINITY, 0.0f};
  const int64_t step = (int64_t)gridDim.x * kOneWarps * kOneRows;
  for (int64_t v0 = ((int64_t)blockIdx.x * kOneWarps + warp) * kOneRows; v0 < V; v0 += step) {
    auto load = [&](int i, uint4 (&a)[kOneRows]) {
#pragma unroll
      for (int r = 0; r < kOneRows; ++r) {
        a[r] = make_uint4(0, 0, 0, 0);
        if (i < vecs && v0 + r < V) a[r] = __ldcs(w + (v0 + r) * vecs + i);
      }
    };
    float z[kOneRows] = {};
    uint4 a[kOneRows], next[kOneRows];
    load(lane, a);
    for (int i = lane; i < vecs; i += 32) {
      load(i + 32, next);
      const uint4 u = xs[i];
      const float f[8] = {lo_bf16(u.x), hi_bf16(u.x), lo_bf16(u.y), hi_bf16(u.y),
                          lo_bf16(u.z), hi_bf16(u.z), lo_bf16(u.w), hi_bf16(u.w)};
#pragma unroll
      for (int r = 0; r < kOneRows; ++r) z[r] = dot8(a[r], f, z[r]), a[r] = next[r];
    }
    float top = sum.top;
#pragma unroll
    for (int r = 0; r < kOneRows; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z[r] += __shfl_xor_sync(0xffffffffu, z[r], o);
      if (v0 + r >= V || v0 + r == at) z[r] = -INFINITY;
      top = fmaxf(top, z[r]);
    }
    const float ref = reference(top);
    float s = sum.top == -INFINITY ? sum.sum : sum.sum * power(sum.top, ref);
#pragma unroll
    for (int r = 0; r < kOneRows; ++r) s += power(z[r], ref);
    sum = {top, s};
  }
  if (lane == 0) rows[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kOneWarps; ++i) sum = joined(sum, rows[i]);
    parts[blockIdx.x] = make_float2(sum.top, sum.sum);
  }
}

// A row of x times its factor, rounded, or zeros where that is 0 (what such a row holds does not
// matter); one warp.
__device__ __forceinline__ void scaled_row(const uint4* x, int vecs, float s, uint4* out) {
  constexpr int kBatch = 4;  // loads on their way
  for (int i0 = threadIdx.x & 31; i0 < vecs; i0 += 32 * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      v[u] = s != 0.0f && i0 + 32 * u < vecs ? x[i0 + 32 * u] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint4& a = v[u];
      a.x = pack2(s * lo_bf16(a.x), s * hi_bf16(a.x)), a.y = pack2(s * lo_bf16(a.y), s * hi_bf16(a.y));
      a.z = pack2(s * lo_bf16(a.z), s * hi_bf16(a.z)), a.w = pack2(s * lo_bf16(a.w), s * hi_bf16(a.w));
      if (i0 + 32 * u < vecs) out[i0 + 32 * u] = a;
    }
  }
}

// Where powers are kept, x's copy is multiplied by this beside its factors, which are between 1 and 2^-100 of
// what they are in two passes: bf16's range is 2^-126 to 2^127.
constexpr float kLift = 0x1p20f;

// Where powers are kept, x's copy is rounded with its row's factor anyway: the factor there also takes back what
// rounding to bf16 changed of the target's power (exact / rounded), as a rule the row's largest element of dz by
// far.  What is left of it is in the row's other elements (as much of each), and dW is 2.4e-3 off the 64-bit result
// in the 2-norm instead of 2.9e-3 (4096 x 1024 x 32000).
__device__ __forceinline__ float taken_back(float exact, __nv_bfloat16 rounded) {
  const float q = __fdiv_rn(exact, __bfloat162float(rounded));
  return q > 0.5f && q < 2.0f ? q : 1.0f;  // (0, infinities, NaN)
}

// What a piece's dloss are divided by in x's copy: that of its first token (of 32) that has one, if it is of a
// size that leaves the others in range; else 1.  One warp; the same in every warp.
__device__ __forceinline__ float common_factor(const int64_t* target, const float* dloss, int B, int V) {
  const int i = threadIdx.x & 31;
  float d = 0.0f;
  if (i < B) {
    const int64_t t = target[i];
    if (t >= 0 && t < V) d = fabsf(dloss[i]);
  }
  const unsigned some = __ballot_sync(0xffffffffu, d > 1e-18f && d < 1e18f);
  return some ? __shfl_sync(0xffffffffu, d, __ffs(some) - 1) : 1.0f;
}

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float s) {
  return fmaf(hi_bf16(a), hi_bf16(b), fmaf(lo_bf16(a), lo_bf16(b), s));
}
// x . w, over a warp; in every lane
__device__ __forceinline__ float dot_row(const uint4* x, const uint4* w, int vecs) {
  float s = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < vecs; i += 32) {
    const uint4 u = x[i], v = w[i];
    s = dot2(u.w, v.w, dot2(u.z, v.z, dot2(u.y, v.y, dot2(u.x, v.x, s))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

struct JoinArgs {
  const float2* parts;        // kLoss's or kExp's
  int count;                  // of parts
  const int64_t* target;
  int B, V;
  const uint4 *x, *w;         // rows of `vecs`
  int vecs;
  float *loss, *lse;
  int* status;
  // a training step's: dloss, x's scaled copies (or NULL), dx's factors
  const float* dloss;
  uint4* scaled;
  int scaled_vecs;            // from row to row
  float* row_scale;
  float* common;              // common_factor, for dW; kExps: it is there already
  // kExp: the reference, the target's logit, and the result, where the targets' elements are still to
  // come
  float* ref;
  const float* logit;
  __nv_bfloat16* exps;
  int64_t pitch;
  int* again;                 // raised when a row's sum is out of range
  const int* only_if;         // as GemmArgs'
};

// kExps: of kExp's parts, whose sums are against the row's reference; otherwise of kLoss's.
template <bool kExps>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const JoinArgs p) {
  __shared__ Partial rows[kJoinWarps][33];
  __shared__ float logits[32], scales[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t b0 = (int64_t)blockIdx.x * 32, b = b0 + lane;
  wait_for_launch_ahead();
  if (p.only_if && *p.only_if == 0) return;
  constexpr int kBatch = 8;
  Partial sum = {-INFINITY, 0.0f};
  if (b < p.B)
    for (int i0 = w; i0 < p.count; i0 += kBatch * kJoinWarps) {
      float2 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kJoinWarps;
        v[u] = make_float2(-INFINITY, 0.0f);
        if (i < p.count) v[u] = p.parts[(int64_t)i * p.B + b];
      }
      Partial more = {-INFINITY, 0.0f};
#pragma unroll
      for (int u = 0; u < kBatch; ++u) more.top = fmaxf(more.top, v[u].x);
      const float ref = reference(more.top);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        more.sum += kExps || v[u].x == -INFINITY ? v[u].y : v[u].y * power(v[u].x, ref);
      if (kExps)
        sum.top = fmaxf(sum.top, more.top), sum.sum += more.sum;
      else
        sum = joined(sum, more);
    }
  rows[w][lane] = sum;
  const float common = kExps ? *p.common : p.scaled ? common_factor(p.target, p.dloss, p.B, p.V) : 1.0f;
  if (!kExps && b0 + w < p.B) {
    const int64_t t = p.target[b0 + w];
    if (t >= 0 && t < p.V) {
      const float z = dot_row(p.x + (b0 + w) * p.vecs, p.w + t * p.vecs, p.vecs);
      if (lane == 0) logits[w] = z;
    }
  }
  __syncthreads();
  // warp w joins token b0 + w's, a part in each lane
  if (b0 + w < p.B) {
    sum = rows[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Partial other = {__shfl_xor_sync(0xffffffffu, sum.top, o),
                             __shfl_xor_sync(0xffffffffu, sum.sum, o)};
      if (kExps)
        sum = {fmaxf(sum.top, other.top), sum.sum + other.sum};
      else
        sum = joined(sum, other);
    }
  }
  if (b0 + w < p.B && lane == 0) {
    const int64_t mine = b0 + w, t = p.target[mine];
    const bool there = t >= 0 && t < p.V;
    if (t >= p.V && p.status) atomicExch(p.status, PKM_ERR_BAD_INDEX);
    const float zt = there ? kExps ? p.logit[mine] : logits[w] : -INFINITY;
    // both against one reference
    const float ref = kExps ? p.ref[mine] : reference(fmaxf(sum.top, zt));
    const float rest = kExps || sum.top == -INFINITY ? sum.sum : sum.sum * power(sum.top, ref);
    const float total = rest + power(zt, ref), lse = ref + logf(total);
    float loss = 0.0f, scale = there && p.scaled ? p.dloss[mine] : 0.0f, back = 1.0f;
    if (there) {
      // (of infinite logits: inf - inf is no number if the target's is one of them, a limit if it is not)
      if (total == INFINITY)
        loss = zt == INFINITY ? NAN : INFINITY;
      else
        loss = zt >= ref ? log1pf(rest * power(ref, zt)) : (ref - zt) + logf(total);
    }
    if (kExps) {
      // (below the range: a token whose target's logit is -inf, or that has none, has a reference that may lie far
      // above its logits; a target's own power is 1)
      if ((total >= 0x1p100f || total < 0x1p-100f) && zt != INFINITY && fabsf(sum.top) < INFINITY &&
          ref != sum.top) {
        p.ref[mine] = sum.top;
        *p.again = 1;
      }
      if (scale != 0.0f) {
        const float own = expm1f(-loss) * total;
        const __nv_bfloat16 rounded = __float2bfloat16(own);
        p.exps[mine * p.pitch + t] = rounded;
        scale = scale / common / total, back = taken_back(own, rounded);
      }
    }
    if (p.scaled) p.row_scale[mine] = scale, scales[w] = scale * back;
    p.loss[mine] = loss;
    if (p.lse) p.lse[mine] = lse;
  }
  if (!p.scaled) return;
  __syncwarp();
  if (!kExps && blockIdx.x == 0 && threadIdx.x == 0) *p.common = common;
  if (b0 + w < p.B)
    scaled_row(p.x + (b0 + w) * p.vecs, p.vecs, kExps ? scales[w] * kLift : scales[w] / common,
               p.scaled + (b0 + w) * p.scaled_vecs);
}

// Ahead of the backward pass's products: a token's factor (dloss, or 0 where its target is none), its row
// of x times that over the common one, the common one, and, unless loss is NULL, the token's loss from lse.
__global__ void __launch_bounds__(256)
rows_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w, const int64_t* __restrict__ target,
            const float* __restrict__ lse, const float* __restrict__ dloss, int B, int vecs, int V,
            float* scale, float* loss, uint4* out, int out_vecs, float* common, int* status) {
  const int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_launch_ahead();
  const float all = common_factor(target, dloss, B, V);
  if (blockIdx.x == 0 && threadIdx.x == 0) *common = all;
  if (b >= B) return;
  const int64_t t = target[b];
  const float s = t >= 0 && t < V ? dloss[b] : 0.0f;
  if ((threadIdx.x & 31) == 0) {
    scale[b] = s;
    if (t >= V && status) atomicExch(status, PKM_ERR_BAD_INDEX);
  }
  if (loss && t >= 0 && t < V) {
    // (below 0 where lse is that of other logits, rounded ones for instance: exp(z - lse) - 1 all the same)
    const float z = dot_row(x + b * vecs, w + t * vecs, vecs);
    if ((threadIdx.x & 31) == 0) loss[b] = lse[b] - z;
  }
  scaled_row(x + b * vecs, vecs, s / all, out + b * out_vecs);
}

// Ahead of a training step's products: a token's reference, the target's logit (of column 0 where it has
// none), and whether it has a gradient; the common factor, for dx, and over kLift for dW.
__global__ void __launch_bounds__(256)
reference_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w,
                 const int64_t* __restrict__ target, const float* __restrict__ dloss, int B, int vecs,
                 int V, float* ref, float* logit, float* factor, int* again, float* common) {
  const int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_launch_ahead();
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    const float all = common_factor(target, dloss, B, V);
    if (threadIdx.x == 0) *again = 0, common[0] = all, common[1] = all / kLift;
  }
  if (b >= B) return;
  const int64_t t = target[b];
  const bool there = t >= 0 && t < V;
  const float z = dot_row(x + b * vecs, w + (there ? t : 0) * vecs, vecs);
  if ((threadIdx.x & 31) == 0) {
    logit[b] = z;
    ref[b] = fabsf(z) < INFINITY ? z : 0.0f;
    factor[b] = there && dloss[b] != 0.0f ? 1.0f : 0.0f;
  }
}

// out [rows][vecs] = bf16(sum over `count` of in[i * stride + ...]), whose rows are in_vecs apart; 8 elements
// a thread
__global__ void __launch_bounds__(256)
round_kernel(const float4* __restrict__ in, int count, int64_t stride, int64_t total, unsigned vecs,
             unsigned in_vecs, uint4* out) {
  wait_for_launch_ahead();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = vecs == in_vecs ? 0 : i / vecs, at = i + row * (in_vecs - vecs);
    float4 a = in[2 * at], b = in[2 * at + 1];
    for (int j = 1; j < count; ++j) {
      const float4 c = in[2 * (j * stride + at)], d = in[2 * (j * stride + at) + 1];
      a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
      b.x += d.x, b.y += d.y, b.z += d.z, b.w += d.w;
    }
    out[i] = make_uint4(pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w));
  }
}

cudaError_t launch_round(const float* in, int count, int64_t stride, int64_t rows, int dim, int pitch,
                         void* out, cudaStream_t stream) {
  const int64_t total = rows * (dim / 8);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 152 * 8) blocks = 152 * 8;
  return launch_early(round_kernel, dim3((unsigned)blocks), 256, 0, stream,
                      reinterpret_cast<const float4*>(in), count, stride / 8, total, (unsigned)dim / 8,
                      (unsigned)pitch / 8, static_cast<uint4*>(out));
}

// ---------------------------------------------------------------- sizes

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t down(int64_t v, int64_t to) { return v / to * to; }
// Rows of the workspace are 128 bytes and their multiples apart: a TMA box's rows of 128 bytes lie in one
// line then (4096 x 192 x 32003, the logits' gradient: 121 us with rows of 64016 bytes, 90 so).
int pitch16(int columns) { return (int)up(columns, 64); }
int pitch32(int columns) { return (int)up(columns, 32); }

// Tokens of a piece of the loss: their parts (at most one for 64 columns) stay within kPartBytes.
int loss_tokens(int B, int V) {
  const int64_t per = 2 * up(V, 128) / 128 * 8;
  const int64_t n = down(kPartBytes / per, 256);
  return (int)(n < 256 ? 256 < B ? 256 : B : n < B ? n : B);
}
size_t loss_region(int B, int V) {
  const size_t parts = align256(2 * up(V, 128) / 128 * 8 * loss_tokens(B, V)), one = align256(8 * kOneBlocks);
  return parts > one ? parts : one;
}

// Few tokens before a large W: dx, which reads W, and dW, which writes as much, in launches of their own
// (131072 x 1024, 64 tokens: 77 and 84 us, both in one 197; 32000 x 512 16 and 16, 33).
bool apart(int tokens, int dim, int columns) { return tokens < 256 && (int64_t)columns * dim >= 1 << 25; }

// Where dx has few tiles, all of them as long as the vocabulary, each would be worked on long after
// dW is done: the columns are cut until a tile takes at most a cluster's share of the work (a third of it
// alone: 131072 x 2048, 64 tokens 125 -> 112 us).
constexpr int kPairs = 76;  // of SMs
int splits_of(int tokens, int dim, int columns) {
  auto t = [](int64_t n) { return (n + 255) / 256; };
  const int64_t slabs = (columns + FK - 1) / FK, dx_tiles = t(tokens) * t(dim);
  const int64_t dw = apart(tokens, dim, columns) ? 0 : t(columns) * t(dim) * tile_slabs((tokens + FK - 1) / FK);
  const int64_t work = dx_tiles * slabs + dw;
  int64_t longest = work / (apart(tokens, dim, columns) ? 3 * kPairs : kPairs);
  if (longest < 16) longest = 16;
  if (slabs <= longest) return 1;
  int64_t n = (slabs + longest - 1) / longest;
  if (n > 64) n = 64;
  const int64_t per = (slabs + n - 1) / n;
  return (int)((slabs + per - 1) / per);
}

// The backward pass's pieces.
struct Pieces {
  int tokens, columns;  // of a piece
  int pitch;            // of dz
  int splits;           // of the columns in dx, each with its own fp32 sums
  bool dx32, dw32;      // sums in fp32 over several pieces, or over the splits
  size_t dz, x, dxs, dws;  // bytes
};
Pieces pieces_of(int B, int dim, int V, int grad_dtype) {
  Pieces s = {};
  s.tokens = B < kMostTokens ? B : kMostTokens;
  int64_t columns = down(kPieceBytes / 2 / s.tokens, 256);
  if (columns < 256) columns = 256;
  s.columns = (int)(columns < V ? columns : V);
  s.pitch = pitch16(s.columns);
  s.splits = s.columns == V ? splits_of(s.tokens, dim, V) : 1;
  s.dx32 = s.columns < V || s.splits > 1;
  s.dw32 = s.tokens < B && grad_dtype == PKM_BF16;
  s.dz = align256((size_t)s.tokens * s.pitch * 2);
  s.x = align256((size_t)s.tokens * pitch16(dim) * 2);
  s.dxs = s.dx32 ? align256((size_t)up(s.tokens, 32) * s.splits * pitch32(dim) * 4) : 0;
  s.dws = s.dw32 ? align256((size_t)V * dim * 4) : 0;
  return s;
}

// A training step whose logits are one round of tiles is quicker in two passes: their product costs less than
// the reference's launch and the two in reserve (200 x 512 x 5000: 43 -> 37 us).
bool small_step(int B, int V) { return ((int64_t)B + 255) / 256 * (((int64_t)V + 255) / 256) <= kPairs; }

// A training step's pieces: all of a piece's E at once.  Several pieces need dW's sums in fp32 (unless dW
// is): where those would take as much as the rest of E, it is one piece (8192 x 2048 x 131072 on one GPU: two of
// 1 GiB and 1 GiB of sums 8.35 ms, one of 2 GiB 8.05).
int train_tokens(int B, int dim, int V, int grad_dtype) {
  const int64_t row = 2 * (int64_t)pitch16(V), sums = grad_dtype == PKM_BF16 ? 4 * (int64_t)V * dim : 0;
  if (row * B <= kPieceBytes + sums) return B;
  const int64_t n = down(kPieceBytes / row, 256);
  return (int)(n < 256 ? 256 : n);
}
struct TrainPieces {
  int tokens, pitch, splits;
  bool dw32;
  size_t exps, x, dxs, dws, parts, rows;  // bytes; rows: of one float a token
};
TrainPieces train_pieces_of(int B, int dim, int V, int grad_dtype) {
  TrainPieces s = {};
  s.tokens = train_tokens(B, dim, V, grad_dtype);
  if (s.tokens > B) s.tokens = B;
  s.pitch = pitch16(V);
  s.splits = splits_of(s.tokens, dim, V);
  s.dw32 = s.tokens < B && grad_dtype == PKM_BF16;
  s.exps = align256((size_t)s.tokens * s.pitch * 2);
  s.x = align256((size_t)s.tokens * pitch16(dim) * 2);
  s.dxs = s.splits > 1 ? align256((size_t)up(s.tokens, 32) * s.splits * pitch32(dim) * 4) : 0;
  s.dws = s.dw32 ? align256((size_t)V * dim * 4) : 0;
  s.parts = align256(2 * up(V, 128) / 128 * 8 * (size_t)s.tokens);
  s.rows = align256((size_t)s.tokens * 4);
  return s;
}
size_t train_region(int B, int dim, int V, int grad_dtype) {
  const TrainPieces s = train_pieces_of(B, dim, V, grad_dtype);
  return s.exps + s.x + s.dxs + s.dws + s.parts + 4 * s.rows + 256;
}

// The tokens' factors, their losses, and the common factor.
size_t scale_region(int B) { return align256((size_t)B * 8 + 4); }

size_t gemm_region() { return kPartsBytes + kFlagsBytes; }

}  // namespace

size_t vocab_loss_workspace_bytes(int B, int V) { return gemm_region() + loss_region(B, V); }

size_t vocab_loss_backward_workspace_bytes(int B, int dim, int V, int grad_dtype) {
  const Pieces s = pieces_of(B, dim, V, grad_dtype);
  const size_t head = scale_region(B) + s.dz + s.x;
  size_t most = head + s.dxs + s.dws;
  const size_t train = small_step(B, V) ? head + loss_region(B, V) : train_region(B, dim, V, grad_dtype);
  if (train > most) most = train;
  return gemm_region() + most;
}

namespace {

cudaError_t launch_one_token(const void* x, const void* w, const int64_t* target, int dim, int V,
                             float2* parts, int* count, cudaStream_t stream) {
  const int64_t groups = ((int64_t)V + kOneWarps * kOneRows - 1) / (kOneWarps * kOneRows);
  *count = (int)(groups < kOneBlocks ? groups : kOneBlocks);
  if ((size_t)2 * dim > kSharedUnasked) {
    cudaError_t e = cudaFuncSetAttribute(one_token_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         2 * kOneMostDim);
    if (e != cudaSuccess) return e;
  }
  return launch_early(one_token_kernel, dim3((unsigned)*count), 32 * kOneWarps, 2 * dim, stream,
                      static_cast<const uint4*>(x), static_cast<const uint4*>(w), target, dim / 8, V, parts);
}

// step: NULL, or a training step's arguments of the join (of all B tokens: one piece)
cudaError_t loss_pass(const void* x, const void* weight, const int64_t* target, int B, int dim, int V,
                      void* gemm, void* region, float* loss, float* lse, int* status,
                      const JoinArgs* step, cudaStream_t stream) {
  const int most = loss_tokens(B, V);
  for (int64_t b0 = 0; b0 < B; b0 += most) {
    const int n = (int)(B - b0 < most ? B - b0 : most);
    const void* xs = static_cast<const uint16_t*>(x) + b0 * dim;
    GemmArgs p = {};
    p.prods = 1;
    p.status = status;
    set_parts(p, gemm);
    Prod& q = p.prod[0];
    q.segs = 1;
    q.M = n, q.N = V, q.K = dim;
    p.target = target + b0;
    p.row_parts = static_cast<float2*>(region);
    if (!rows_operand(q, xs, n, dim)) return cudaErrorInvalidValue;
    int half = 0;
    JoinArgs j = step ? *step : JoinArgs{};
    cudaError_t e = n == 1 && dim <= kOneMostDim
                        ? launch_one_token(xs, weight, p.target, dim, V, p.row_parts, &j.count, stream)
                        : launch_products(kLoss, p, {{{weight, V, dim}}}, stream, &half);
    if (e != cudaSuccess) return e;
    if (half) j.count = (V + half - 1) / half;
    j.parts = p.row_parts;
    j.target = p.target, j.B = n, j.V = V;
    j.x = static_cast<const uint4*>(xs), j.w = static_cast<const uint4*>(weight), j.vecs = dim / 8;
    j.loss = loss + b0, j.lse = lse ? lse + b0 : nullptr, j.status = status;
    e = launch_early(join_kernel<false>, dim3((unsigned)(n + 31) / 32), 32 * kJoinWarps, 0, stream, j);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Where a piece's dx and dW go.
struct Out {
  void* dx;           // bf16, or NULL
  float* dxs;         // NULL, or dx's sums in fp32: of `splits` stretches of the columns, or of several pieces
  int splits;
  bool first_columns, last_columns;  // of the pieces that dxs joins
  void* dw;           // fp32 if dw32 > 0 (Prod::add32), or NULL
  int dw32;
  const float *dx_common, *common;  // that multiply dx (beside its rows' factors) and dW, or NULL
};
// dx = dz W and dW = dz^T xs, dz [n, cols] of `pitch` columns, W's rows those of the columns.
cudaError_t products(GemmArgs& p, const void* dz, int n, int cols, int64_t pitch, const void* w,
                     const void* xs, int dim, const float* row_scale, const Out& o, cudaStream_t stream) {
  BOperand b[kMaxProds][2] = {};
  p.prods = 0;
  auto into_dx = [&] {
    Prod& q = p.prod[p.prods];
    q = Prod{};
    q.segs = 1;
    q.M = n, q.N = dim, q.K = cols, q.b_mn = 1;
    q.row_scale = row_scale, q.all_scale = o.dx_common;
    int rows = n;
    if (o.dxs) q.add32 = o.first_columns ? 2 : 1;
    if (o.splits > 1) {
      const int slabs = (cols + FK - 1) / FK;
      q.splits = o.splits, q.split_kb = (slabs + o.splits - 1) / o.splits;
      rows = (int)up(n, 32) * o.splits;
    }
    b[p.prods++][0] = {w, cols, dim};
    return rows_operand(q, dz, n, cols, pitch) &&
           result(&q.out, o.dxs ? o.dxs : o.dx, rows, dim, o.dxs != nullptr, o.dxs ? pitch32(dim) : 0);
  };
  auto into_dw = [&] {
    Prod& q = p.prod[p.prods];
    q = Prod{};
    q.segs = 1;
    q.M = cols, q.N = dim, q.K = n, q.a_mn = q.b_mn = 1, q.add32 = o.dw32;
    q.all_scale = o.common;
    b[p.prods++][0] = {xs, n, dim, pitch16(dim)};
    return operand(&q.a[0], dz, n, cols, true, FM, pitch) && result(&q.out, o.dw, cols, dim, o.dw32 != 0);
  };
  cudaError_t e = cudaSuccess;
  if (apart(n, dim, cols)) {
    if (o.dx && !into_dx()) return cudaErrorInvalidValue;
    if (o.dx) e = launch_products(kOut, p, b, stream);
    if (e != cudaSuccess) return e;
    p.prods = 0;
    if (o.dw && !into_dw()) return cudaErrorInvalidValue;
  } else {  // longest tiles first
    const bool first = cols / o.splits > n;
    if (o.dx && first && !into_dx()) return cudaErrorInvalidValue;
    if (o.dw && !into_dw()) return cudaErrorInvalidValue;
    if (o.dx && !first && !into_dx()) return cudaErrorInvalidValue;
  }
  if (p.prods) e = launch_products(kOut, p, b, stream);
  if (e != cudaSuccess || !o.dx || !o.dxs || !o.last_columns) return e;
  return launch_round(o.dxs, o.splits, up(n, 32) * pitch32(dim), n, dim, pitch32(dim), o.dx, stream);
}

// loss: NULL, or the tokens' losses; scaled: their join has scaled x's rows already
cudaError_t gradient_pass(const void* x, const void* weight, const int64_t* target, const float* lse,
                          const float* loss, bool scaled, const float* dloss, int B, int dim, int V,
                          void* gemm, unsigned char* region, void* dx, void* dweight, int grad_dtype,
                          int* status, cudaStream_t stream) {
  const Pieces s = pieces_of(B, dim, V, grad_dtype);
  float *scale = reinterpret_cast<float*>(region), *from_lse = scale + B, *common = from_lse + B;
  unsigned char* dz = region + scale_region(B);
  unsigned char *xs = dz + s.dz, *dxs = xs + s.x, *dws = dxs + s.dxs;
  const uint16_t* w = static_cast<const uint16_t*>(weight);
  cudaError_t e;
  for (int64_t b0 = 0; b0 < B; b0 += s.tokens) {
    const int n = (int)(B - b0 < s.tokens ? B - b0 : s.tokens);
    const uint16_t* xb = static_cast<const uint16_t*>(x) + b0 * dim;
    if (!scaled) {
      e = launch_early(rows_kernel, dim3((unsigned)(n + 7) / 8), 256, 0, stream,
                       reinterpret_cast<const uint4*>(xb), reinterpret_cast<const uint4*>(w), target + b0,
                       lse + b0, dloss + b0, n, dim / 8, V, scale + b0, loss ? nullptr : from_lse + b0,
                       reinterpret_cast<uint4*>(xs), pitch16(dim) / 8, common, status);
      if (e != cudaSuccess) return e;
    }
    for (int64_t c0 = 0; c0 < V; c0 += s.columns) {
      const int cols = (int)(V - c0 < s.columns ? V - c0 : s.columns);
      const void* wc = w + c0 * dim;
      GemmArgs p = {};
      p.prods = 1;
      p.status = status;
      set_parts(p, gemm);
      Prod& q = p.prod[0];
      q.segs = 1;
      q.M = n, q.N = cols, q.K = dim;
      p.target = target + b0;
      p.col0 = c0;
      p.ref = lse + b0;
      p.loss = (loss ? loss : from_lse) + b0;
      p.factor = scale + b0;
      if (!rows_operand(q, xb, n, dim) || !result(&q.out, dz, n, cols, false, s.pitch))
        return cudaErrorInvalidValue;
      e = launch_products(kProb, p, {{{wc, cols, dim}}}, stream);
      if (e != cudaSuccess) return e;
      Out o = {};
      if (dx) o.dx = static_cast<uint16_t*>(dx) + b0 * dim;
      if (s.dx32) o.dxs = reinterpret_cast<float*>(dxs);
      o.splits = s.splits, o.first_columns = c0 == 0, o.last_columns = c0 + cols == V;
      o.common = common;
      if (dweight && grad_dtype == PKM_F32)
        o.dw = static_cast<float*>(dweight) + c0 * dim, o.dw32 = 1;
      else if (dweight && s.dw32)
        o.dw = reinterpret_cast<float*>(dws) + c0 * dim, o.dw32 = b0 ? 1 : 2;
      else if (dweight)
        o.dw = static_cast<uint16_t*>(dweight) + c0 * dim;
      e = products(p, dz, n, cols, s.pitch, wc, xs, dim, scale + b0, o, stream);
      if (e != cudaSuccess) return e;
    }
  }
  return dweight && s.dw32 ? launch_round(reinterpret_cast<const float*>(dws), 1, 0, V, dim, dim, dweight,
                                          stream)
                           : cudaSuccess;
}

cudaError_t train_pass(const void* x, const void* weight, const int64_t* target, const float* dloss,
                       int B, int dim, int V, void* gemm, unsigned char* region, float* loss, float* lse,
                       void* dx, void* dweight, int grad_dtype, int* status, cudaStream_t stream) {
  const TrainPieces s = train_pieces_of(B, dim, V, grad_dtype);
  unsigned char *exps = region, *xs = exps + s.exps, *dxs = xs + s.x, *dws = dxs + s.dxs;
  unsigned char* parts = dws + s.dws;
  float* ref = reinterpret_cast<float*>(parts + s.parts);
  float *factor = ref + s.rows / 4, *logit = factor + s.rows / 4, *scale = logit + s.rows / 4;
  int* again = reinterpret_cast<int*>(scale + s.rows / 4);
  float* common = reinterpret_cast<float*>(again + 2);
  cudaError_t e;
  for (int64_t b0 = 0; b0 < B; b0 += s.tokens) {
    const int n = (int)(B - b0 < s.tokens ? B - b0 : s.tokens);
    const uint16_t* xb = static_cast<const uint16_t*>(x) + b0 * dim;
    e = launch_early(reference_kernel, dim3((unsigned)(n + 7) / 8), 256, 0, stream,
                     reinterpret_cast<const uint4*>(xb), static_cast<const uint4*>(weight), target + b0,
                     dloss + b0, n, dim / 8, V, ref, logit, factor, again, common);
    if (e != cudaSuccess) return e;
    GemmArgs p = {};
    p.status = status;
    set_parts(p, gemm);
    p.target = target + b0;
    p.row_parts = reinterpret_cast<float2*>(parts);
    p.factor = factor;
    JoinArgs j = {};
    j.parts = p.row_parts, j.target = target + b0, j.B = n, j.V = V;
    j.x = reinterpret_cast<const uint4*>(xb), j.w = static_cast<const uint4*>(weight), j.vecs = dim / 8;
    j.loss = loss + b0, j.lse = lse + b0, j.status = status;
    p.ref = j.ref = ref;
    j.logit = logit, j.dloss = dloss + b0, j.row_scale = scale;
    j.exps = reinterpret_cast<__nv_bfloat16*>(exps), j.pitch = s.pitch;
    j.scaled = reinterpret_cast<uint4*>(xs), j.scaled_vecs = pitch16(dim) / 8;
    j.common = common;
    for (int pass = 0; pass < 2; ++pass) {
      p.prods = 1;
      Prod& q = p.prod[0];
      q = Prod{};
      q.segs = 1;
      q.M = n, q.N = V, q.K = dim;
      if (!rows_operand(q, xb, n, dim) || !result(&q.out, exps, n, V, false, s.pitch))
        return cudaErrorInvalidValue;
      int half = 0;
      if ((e = launch_products(kExp, p, {{{weight, V, dim}}}, stream, &half)) != cudaSuccess) return e;
      j.count = (V + half - 1) / half;
      j.again = again + pass;
      e = launch_early(join_kernel<true>, dim3((unsigned)(n + 31) / 32), 32 * kJoinWarps, 0, stream, j);
      if (e != cudaSuccess) return e;
      p.only_if = j.only_if = again;  // the second time
    }
    p.only_if = nullptr;
    Out o = {};
    if (dx) o.dx = static_cast<uint16_t*>(dx) + b0 * dim;
    if (s.splits > 1) o.dxs = reinterpret_cast<float*>(dxs);
    o.splits = s.splits, o.first_columns = o.last_columns = true;
    o.dw = dweight, o.dw32 = grad_dtype == PKM_F32;
    o.dx_common = common, o.common = common + 1;
    if (dweight && s.dw32) o.dw = dws, o.dw32 = b0 ? 1 : 2;
    e = products(p, exps, n, V, s.pitch, weight, xs, dim, scale, o, stream);
    if (e != cudaSuccess) return e;
  }
  return dweight && s.dw32 ? launch_round(reinterpret_cast<const float*>(dws), 1, 0, V, dim, dim, dweight,
                                          stream)
                           : cudaSuccess;
}

}  // namespace

cudaError_t launch_vocab_loss(const void* x, const void* weight, const int64_t* target, int B, int dim,
                              int V, void* workspace, float* loss, float* lse, int* status,
                              cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  return loss_pass(x, weight, target, B, dim, V, ws, ws + gemm_region(), loss, lse, status, nullptr, stream);
}

cudaError_t launch_vocab_loss_backward(const void* x, const void* weight, const int64_t* target,
                                       const float* lse, const float* loss, const float* dloss, int B,
                                       int dim, int V, void* workspace, void* dx, void* dweight,
                                       int grad_dtype, int* status, cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  return gradient_pass(x, weight, target, lse, loss, false, dloss, B, dim, V, ws, ws + gemm_region(), dx,
                       dweight, grad_dtype, status, stream);
}

cudaError_t launch_vocab_loss_train(const void* x, const void* weight, const int64_t* target,
                                    const float* dloss, int B, int dim, int V, void* workspace,
                                    float* loss, float* lse, void* dx, void* dweight, int grad_dtype,
                                    int* status, cudaStream_t stream) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  if (small_step(B, V)) {
    // (the parts of the loss lie where dx's sums will)
    unsigned char *region = ws + gemm_region(), *dz = region + scale_region(B);
    const Pieces s = pieces_of(B, dim, V, grad_dtype);
    JoinArgs step = {};
    step.dloss = dloss;
    step.scaled = reinterpret_cast<uint4*>(dz + s.dz), step.scaled_vecs = pitch16(dim) / 8;
    step.row_scale = reinterpret_cast<float*>(region), step.common = step.row_scale + 2 * (size_t)B;
    cudaError_t e = loss_pass(x, weight, target, B, dim, V, ws, dz + s.dz + s.x, loss, lse, status, &step,
                              stream);
    if (e != cudaSuccess) return e;
    return gradient_pass(x, weight, target, lse, loss, true, dloss, B, dim, V, ws, region, dx, dweight,
                         grad_dtype, status, stream);
  }
  return train_pass(x, weight, target, dloss, B, dim, V, ws, ws + gemm_region(), loss, lse, dx, dweight,
                    grad_dtype, status, stream);
}

}  // namespace pkm

namespace {

bool vocab_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int vocab_check(int B, int dim, int V) {
  if (B < 0 || dim < 1 || V < 1) return PKM_ERR_INVALID;
  if (dim % 8) return PKM_ERR_UNSUPPORTED;
  // the kernels count tiles (of 128 x 128 at the smallest) and rows in 32 bits
  constexpr int most = INT32_MAX - 256;
  auto t = [](int n) { return ((int64_t)n + 127) / 128; };
  if (B > most || dim > most || V > most || t(B) * t(V) > most / 4 || t(B) * t(dim) > most / 4 ||
      t(V) * t(dim) > most / 4)
    return PKM_ERR_RANGE;
  return PKM_OK;
}

int vocab_rc(cudaError_t e) { return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA; }

// What all three calls take.
int vocab_inputs(const void* x, const void* weight, const int64_t* target, const void* workspace,
                 const int* status) {
  if (!x || !weight || !target || !workspace) return PKM_ERR_INVALID;
  if (!vocab_aligned(x, 16) || !vocab_aligned(weight, 16) || !vocab_aligned(workspace, 16) ||
      !vocab_aligned(target, 8) || !vocab_aligned(status, 4))
    return PKM_ERR_ALIGN;
  return PKM_OK;
}

// No token: the weight's gradient is zero (an fp32 one: nothing is added).
int vocab_empty(int dim, int V, void* dweight, int grad_dtype, void* stream) {
  if (!dweight || grad_dtype == PKM_F32) return PKM_OK;
  if (!vocab_aligned(dweight, 16)) return PKM_ERR_ALIGN;
  return vocab_rc(cudaMemsetAsync(dweight, 0, (size_t)V * dim * 2, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" size_t pkm_vocab_loss_workspace_bytes(int B, int dim, int V) {
  return vocab_check(B, dim, V) || B == 0 ? 0 : pkm::vocab_loss_workspace_bytes(B, V);
}

extern "C" size_t pkm_vocab_loss_backward_workspace_bytes(int B, int dim, int V, int grad_dtype) {
  if (vocab_check(B, dim, V) || B == 0 || (grad_dtype != PKM_BF16 && grad_dtype != PKM_F32)) return 0;
  return pkm::vocab_loss_backward_workspace_bytes(B, dim, V, grad_dtype);
}

extern "C" int pkm_vocab_loss(const void* x, const void* weight, const int64_t* target, int B, int dim,
                              int V, void* workspace, float* loss, float* lse, int* status,
                              void* stream) {
  int rc = vocab_check(B, dim, V);
  if (rc || B == 0) return rc;
  if (!loss) return PKM_ERR_INVALID;
  if ((rc = vocab_inputs(x, weight, target, workspace, status))) return rc;
  if (!vocab_aligned(loss, 4) || !vocab_aligned(lse, 4)) return PKM_ERR_ALIGN;
  return vocab_rc(pkm::launch_vocab_loss(x, weight, target, B, dim, V, workspace, loss, lse, status,
                                         static_cast<cudaStream_t>(stream)));
}

namespace {

// loss: of the second call, which needs it
int vocab_backward(const void* x, const void* weight, const int64_t* target, const float* lse,
                   bool with_loss, const float* loss, const float* dloss, int B, int dim, int V,
                   void* workspace, void* dx, void* dweight, int grad_dtype, int* status, void* stream) {
  int rc = vocab_check(B, dim, V);
  if (rc) return rc;
  if (grad_dtype != PKM_BF16 && grad_dtype != PKM_F32) return PKM_ERR_UNSUPPORTED;
  if (B == 0) return vocab_empty(dim, V, dweight, grad_dtype, stream);
  if (!lse || !dloss || (with_loss && !loss)) return PKM_ERR_INVALID;
  if ((rc = vocab_inputs(x, weight, target, workspace, status))) return rc;
  if (!vocab_aligned(lse, 4) || !vocab_aligned(loss, 4) || !vocab_aligned(dloss, 4) ||
      !vocab_aligned(dx, 16) || !vocab_aligned(dweight, 16))
    return PKM_ERR_ALIGN;
  return vocab_rc(pkm::launch_vocab_loss_backward(x, weight, target, lse, loss, dloss, B, dim, V,
                                                  workspace, dx, dweight, grad_dtype, status,
                                                  static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" int pkm_vocab_loss_backward(const void* x, const void* weight, const int64_t* target,
                                       const float* lse, const float* dloss, int B, int dim, int V,
                                       void* workspace, void* dx, void* dweight, int grad_dtype,
                                       int* status, void* stream) {
  return vocab_backward(x, weight, target, lse, false, nullptr, dloss, B, dim, V, workspace, dx, dweight,
                        grad_dtype, status, stream);
}

extern "C" int pkm_vocab_loss_backward_with_loss(const void* x, const void* weight,
                                                 const int64_t* target, const float* lse,
                                                 const float* loss, const float* dloss, int B, int dim,
                                                 int V, void* workspace, void* dx, void* dweight,
                                                 int grad_dtype, int* status, void* stream) {
  return vocab_backward(x, weight, target, lse, true, loss, dloss, B, dim, V, workspace, dx, dweight,
                        grad_dtype, status, stream);
}

extern "C" int pkm_vocab_loss_train(const void* x, const void* weight, const int64_t* target,
                                    const float* dloss, int B, int dim, int V, void* workspace,
                                    float* loss, float* lse, void* dx, void* dweight, int grad_dtype,
                                    int* status, void* stream) {
  int rc = vocab_check(B, dim, V);
  if (rc) return rc;
  if (grad_dtype != PKM_BF16 && grad_dtype != PKM_F32) return PKM_ERR_UNSUPPORTED;
  if (B == 0) return vocab_empty(dim, V, dweight, grad_dtype, stream);
  if (!dloss || !loss || !lse) return PKM_ERR_INVALID;
  if ((rc = vocab_inputs(x, weight, target, workspace, status))) return rc;
  if (!vocab_aligned(loss, 4) || !vocab_aligned(lse, 4) || !vocab_aligned(dloss, 4) ||
      !vocab_aligned(dx, 16) || !vocab_aligned(dweight, 16))
    return PKM_ERR_ALIGN;
  return vocab_rc(pkm::launch_vocab_loss_train(x, weight, target, dloss, B, dim, V, workspace, loss, lse,
                                               dx, dweight, grad_dtype, status,
                                               static_cast<cudaStream_t>(stream)));
}
