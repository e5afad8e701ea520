// The sum of a residual stream and a block's (or a memory's) result, its root-mean-square norm,
// and their backward pass:
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * weight
//   g = dy * weight,  d = ds + rstd * (g - s * rstd^2 * mean(g * s)),  dweight = sum_b dy * s * rstd
//
// d is the gradient of s, so of x and of r alike.  Everything between the loads and the stores is
// fp32; y comes from the unrounded s.
//
// Bound by HBM in large batches: 16384 x 2048, bf16 all through, 40.6 us (97 % of the copy), fp32 stream
// with an fp8 result 68 (94 %); the backward pass 50 (80 %): its 16 warps an SM, of 120 registers, leave
// issue slots empty (58 % used) while loads are on their way.  Rows ahead in shared memory (61 to 69), more
// warps of fewer registers (61) and packed arithmetic (52) were slower.  Small ones by the launch (4 us).  The
// backward pass of rows above 8192 columns by its registers: the next row beside this one, four vectors of each a
// thread, spills (4096 x 16384 bf16 173 us, 46 % of the copy, an fp32 stream 428 and 32 %, fp32 all through
// 1165 and 14 %).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "launch_common.cuh"
#include "num_common.cuh"
#include "pkm_internal.cuh"

namespace pkm {
namespace {

constexpr int kNormMaxWarps = 16;  // of a block
constexpr int kVec = 8;            // elements a thread takes at a time

// kVec values as they lie in memory
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&v)[kVec]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float (&v)[kVec]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[kVec]) {
  Raw<T> r;
  r.load(p);
  r.get(v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// at element `at` of an array of dtype
__device__ __forceinline__ void store8(void* p, int dtype, int64_t at, const float (&v)[kVec]) {
  if (dtype == PKM_BF16)
    store8(static_cast<__nv_bfloat16*>(p) + at, v);
  else
    store8(static_cast<float*>(p) + at, v);
}

struct Sum {
  __device__ static float join(float a, float b) { return a + b; }
};
struct Max {
  __device__ static float join(float a, float b) { return fmaxf(a, b); }
};

// One value over the `warps` warps of a row's group (group g of its block, which meet at named
// barrier g + 1); every thread gets the same.  scratch: kNormMaxWarps floats of the group's own.
template <typename Op>
__device__ __forceinline__ float join_group(float v, int warps, int g, float* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::join(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % warps;
  if (lane == 0) scratch[w] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(32 * warps) : "memory");
  v = scratch[lane % warps];  // (warps: a power of two, so every value counts as often)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < warps) v = Op::join(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

constexpr int kNormThreads = 512;  // of a block at most: see shape_of

__device__ __forceinline__ float scale_of(float amax) {
  const float scale = __fdiv_rn(amax, 448.0f);
  return scale >= FLT_MIN ? scale : FLT_MIN;
}
__device__ __forceinline__ uint2 codes_of(const float (&v)[kVec], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = 0;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      w[j] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[4 * j + m], scale), __NV_SATFINITE, __NV_E4M3)
              << (8 * m);
  }
  return make_uint2(w[0], w[1]);
}

// A row whose mean of squares (and eps) lies below this, or past fp32, is summed scaled.  Squares below 2^-126
// have lost bits, of 16384 of them 2^-136 in the sum at most: this keeps 2^-36 of it clear.
constexpr float kLeastMean = 0x1p-100f;

struct NormArgs {
  const float* weight;
  float eps;
  int B, dim, warps;
  void* sum;
  int sum_dtype;
  void* y;
  int y_dtype;
  float* rstd;
};

// Row b of such a kind, by its group: s is scaled by a power of two, which brings the largest of it and of
// sqrt(eps) to 1, and read again each time (from registers these lines would cost the kernel, in all its rows, 8
// more of them).
template <typename X, typename R>
__device__ __noinline__ void scaled_norm_row(const X* x, const R* r, const NormArgs p, int64_t b, int g,
                                             float (*scratch)[kNormMaxWarps][kNormMaxWarps]) {
  const int t = threadIdx.x - g * 32 * p.warps, per = 32 * p.warps * kVec;
  const int64_t row = b * p.dim;
  auto load = [&](int c, float (&s)[kVec]) {
    load8(x + row + c, s);
    if (r) {
      float v[kVec];
      load8(r + row + c, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[j] += v[j];
    }
  };
  float most = 0.0f;
  for (int c = t * kVec; c < p.dim; c += per) {
    float s[kVec];
    load(c, s);
#pragma unroll
    for (int j = 0; j < kVec; ++j) most = fmaxf(most, fabsf(s[j]));
  }
  most = fmaxf(join_group<Max>(most, p.warps, g, scratch[1][g]), __fsqrt_rn(p.eps));
  float pre = 1.0f;
  if (most > 0.0f && most < INFINITY) {  // (zeros without eps and infinities have no scale)
    const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -126), 126);
    pre = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
  }
  float ss = 0.0f;
  for (int c = t * kVec; c < p.dim; c += per) {
    float s[kVec];
    load(c, s);
#pragma unroll
    for (int j = 0; j < kVec; ++j) ss = fmaf(s[j] * pre, s[j] * pre, ss);
  }
  ss = join_group<Sum>(ss, p.warps, g, scratch[0][g]);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)p.dim) + p.eps * pre * pre));
  if (p.rstd && t == 0) p.rstd[b] = rstd * pre;
  auto norm = [&](int c, const float (&s)[kVec], float (&v)[kVec]) {
    load8(p.weight + c, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = s[j] * pre * (rstd * v[j]);
  };
  float scale = 0.0f;
  if (p.y_dtype == PKM_FP8_E4M3) {
    float amax = 0.0f;
    for (int c = t * kVec; c < p.dim; c += per) {
      float s[kVec], v[kVec];
      load(c, s);
      norm(c, s, v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
    scale = scale_of(join_group<Max>(amax, p.warps, g, scratch[1][g]));
    if (t == 0) reinterpret_cast<float*>(static_cast<uint8_t*>(p.y) + (int64_t)p.B * p.dim)[b] = scale;
  }
  for (int c = t * kVec; c < p.dim; c += per) {  // (a place is read before it is written: sum and y in place)
    float s[kVec], v[kVec];
    load(c, s);
    norm(c, s, v);
    if (p.sum) store8(p.sum, p.sum_dtype, row + c, s);
    if (p.y_dtype == PKM_FP8_E4M3)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row + c) = codes_of(v, scale);
    else
      store8(p.y, p.y_dtype, row + c, v);
  }
}

// Rows of 16 bits are bound by what is on its way: three blocks of an SM (40 registers; 16384 x 2048 40.6 us, two
// blocks 45.6), two of the longest (64; 4096 x 16384 79.5 us, one block 106).  0: as they come.
template <typename X, typename R, int kN>
constexpr int kNormBlocks = sizeof(X) + sizeof(R) > 4 ? 0 : kN == 2 ? 3 : 2;

template <typename X, typename R, int kN>
__global__ void __launch_bounds__(kNormThreads, (kNormBlocks<X, R, kN>))
add_norm_kernel(const X* x, const R* r, const float* __restrict__ weight, float eps, int B, int dim,
                int warps, void* sum, int sum_dtype, void* y, int y_dtype, float* rstd_out) {
  __shared__ float scratch[2][kNormMaxWarps][kNormMaxWarps];
  const int g = (threadIdx.x >> 5) / warps, groups = (blockDim.x >> 5) / warps;
  const int t = threadIdx.x - g * 32 * warps, per = 32 * warps * kVec;
  const int64_t b = (int64_t)blockIdx.x * groups + g;
  wait_for_launch_ahead();
  if (b >= B) return;
  const int64_t row = b * dim;
  Raw<X> xs[kN];
  Raw<R> rs[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = i * per + t * kVec;
    if (c < dim) {
      xs[i].load(x + row + c);
      if (r) rs[i].load(r + row + c);
    }
  }
  float s[kN][kVec];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = i * per + t * kVec;
    if (c < dim) {
      xs[i].get(s[i]);
      if (r) {
        float v[kVec];
        rs[i].get(v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[i][j] += v[j];
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) ss = fmaf(s[i][j], s[i][j], ss);
    }
  }
  ss = join_group<Sum>(ss, warps, g, scratch[0][g]);
  const float mean = __fdiv_rn(ss, (float)dim) + eps;
  if (!(mean >= kLeastMean && mean < INFINITY)) {  // (the same in all of a row's threads)
    scaled_norm_row(x, r, NormArgs{weight, eps, B, dim, warps, sum, sum_dtype, y, y_dtype, rstd_out}, b, g,
                    scratch);
    return;
  }
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(mean));
  if (rstd_out && t == 0) rstd_out[b] = rstd;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = i * per + t * kVec;
    if (c < dim) {
      if (sum) store8(sum, sum_dtype, row + c, s[i]);
      float w[kVec];
      load8(weight + c, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        s[i][j] *= rstd * w[j];
        amax = fmaxf(amax, fabsf(s[i][j]));
      }
      if (y_dtype != PKM_FP8_E4M3) store8(y, y_dtype, row + c, s[i]);
    }
  }
  if (y_dtype != PKM_FP8_E4M3) return;
  amax = join_group<Max>(amax, warps, g, scratch[1][g]);
  const float scale = scale_of(amax);
  uint8_t* codes = static_cast<uint8_t*>(y);
  if (t == 0) reinterpret_cast<float*>(codes + (int64_t)B * dim)[b] = scale;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = i * per + t * kVec;
    if (c < dim) *reinterpret_cast<uint2*>(codes + row + c) = codes_of(s[i], scale);
  }
}

// Group after group of rows; a thread keeps its columns' part of dweight in registers.  A block's
// part goes to parts[block][dim], which norm_join_kernel adds in the order of the blocks.
template <typename S, typename Y, int kN>
__global__ void __launch_bounds__(kNormThreads)
add_norm_backward_kernel(const S* s_in, const float* __restrict__ weight,
                         const float* __restrict__ rstd_in, const Y* dy_in, const S* ds_in, int B,
                         int dim, int warps, void* d_out, int d_dtype, void* dx_out, int dx_dtype,
                         float* parts) {
  extern __shared__ float rows[];  // [groups][dim]
  __shared__ float scratch[2][kNormMaxWarps][kNormMaxWarps];
  const int g = (threadIdx.x >> 5) / warps, groups = (blockDim.x >> 5) / warps;
  const int t = threadIdx.x - g * 32 * warps, per = 32 * warps * kVec;
  float dw[kN][kVec] = {};
  wait_for_launch_ahead();
  const bool d = d_out || dx_out;
  const int64_t step = (int64_t)gridDim.x * groups;
  struct Row {
    Raw<S> s[kN], ds[kN];
    Raw<Y> dy[kN];
    float rstd;
  };
  auto load_row = [&](Row& r, int64_t b) {
    if (b >= B) return;
    const int64_t row = b * dim;
    r.rstd = rstd_in[b];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = i * per + t * kVec;
      if (c < dim) {
        r.s[i].load(s_in + row + c);
        r.dy[i].load(dy_in + row + c);
        if (ds_in && d) r.ds[i].load(ds_in + row + c);
      }
    }
  };
  // u = s * rstd and gy = dy * weight of vector i (twice, rather than kept)
  auto both = [&](const Row& r, int i, int c, float (&u)[kVec], float (&dy)[kVec], float (&gy)[kVec]) {
    load8(weight + c, gy);
    r.s[i].get(u);
    r.dy[i].get(dy);
#pragma unroll
    for (int j = 0; j < kVec; ++j) u[j] *= r.rstd, gy[j] *= dy[j];
  };
  int turn = 0;
  int64_t b = (int64_t)blockIdx.x * groups + g;
  Row next;
  load_row(next, b);
  for (; b < B; b += step) {
    const Row r = next;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = i * per + t * kVec;
      if (c < dim) {
        float u[kVec], dy[kVec], gy[kVec];
        both(r, i, c, u, dy, gy);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          dw[i][j] = fmaf(dy[j], u[j], dw[i][j]);
          dot = fmaf(gy[j], u[j], dot);
        }
      }
    }
    load_row(next, b + step);  // on its way while this row is joined
    if (!d) continue;
    const float mean = join_group<Sum>(dot, warps, g, scratch[turn][g]) / (float)dim;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = i * per + t * kVec;
      if (c < dim) {
        float u[kVec], dy[kVec], gy[kVec], v[kVec] = {};
        both(r, i, c, u, dy, gy);
        if (ds_in) r.ds[i].get(v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = fmaf(r.rstd, gy[j] - u[j] * mean, v[j]);
        if (d_out) store8(d_out, d_dtype, b * dim + c, v);
        if (dx_out) store8(dx_out, dx_dtype, b * dim + c, v);
      }
    }
  }
  if (!parts) return;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = i * per + t * kVec;
    if (c < dim) store8(rows + g * dim + c, dw[i]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < dim; c += blockDim.x) {
    float v = 0.0f;
    for (int i = 0; i < groups; ++i) v += rows[i * dim + c];
    parts[(int64_t)blockIdx.x * dim + c] = v;
  }
}

// out[c] = sum over the parts, 32 columns a block, its 32 warps each a share of the parts
__global__ void __launch_bounds__(1024)
norm_join_kernel(const float* __restrict__ parts, int count, int dim, float* out) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  wait_for_launch_ahead();
  float v = 0.0f;
  if (c < dim)
    for (int i = w; i < count; i += 32) v += parts[(int64_t)i * dim + c];
  sums[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < dim) {
    v = 0.0f;
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    out[c] = v;
  }
}

// A row's warps (a power of two) and vectors a thread: two, or four where a row is longer than 512 threads
// take so.  One vector (256 threads, 2048 columns) left too little on its way: 16384 x 2048 with an fp8
// result 88 us (two 69), bf16 59 (44); four 79 and 41, and too many registers in the backward pass, which rows
// above 8192 columns pay for.
// Blocks of 512 threads suit rows of 16 bits (bf16 44 -> 41 us, 97 % of the copy; fp32 69 -> 73), as
// the GPU starts only so many blocks a microsecond (of 128 threads: 62 and 95).
struct Shape {
  int warps, vectors, threads, groups;
};
Shape shape_of(int dim, int threads) {
  Shape s;
  s.vectors = dim <= 8192 ? 2 : 4;
  const int need = (dim + 32 * kVec * s.vectors - 1) / (32 * kVec * s.vectors);
  s.warps = 1;
  while (s.warps < need) s.warps *= 2;
  s.threads = 32 * s.warps < threads ? threads : 32 * s.warps;
  s.groups = s.threads / (32 * s.warps);
  return s;
}
// Blocks of the backward pass, and their parts of dweight: one to an SM (two of 256 threads 50 us at
// 16384 x 2048, three 61, this 48).
constexpr int kBackThreads = 512, kMaxParts = 152;
constexpr int kMostRowBytes = PKM_NORM_MAX_DIM * 4;  // of its dynamic shared memory

template <typename F>
cudaError_t with_type(int dtype, F&& f) {
  return dtype == PKM_BF16 ? f((__nv_bfloat16*)nullptr) : f((float*)nullptr);
}
template <int kValue>
struct Int {
  static constexpr int value = kValue;
};
template <typename F>
cudaError_t with_vectors(int n, F&& f) {
  return n == 2 ? f(Int<2>()) : f(Int<4>());
}

}  // namespace

size_t add_rms_norm_backward_workspace_bytes(int B, int dim) {
  return (size_t)(B < kMaxParts ? B : kMaxParts) * dim * 4;
}

cudaError_t launch_add_rms_norm(const void* x, int x_dtype, const void* r, int r_dtype,
                                const float* weight, float eps, int B, int dim, void* sum,
                                int sum_dtype, void* y, int y_dtype, float* rstd,
                                cudaStream_t stream) {
  const Shape s = shape_of(dim, x_dtype == PKM_BF16 && r_dtype == PKM_BF16 ? 512 : 256);
  const int blocks = (int)(((int64_t)B + s.groups - 1) / s.groups);
  return with_type(x_dtype, [&](auto* xt) {
    return with_type(r_dtype, [&](auto* rt) {
      return with_vectors(s.vectors, [&](auto n) {
        using X = std::remove_pointer_t<decltype(xt)>;
        using R = std::remove_pointer_t<decltype(rt)>;
        return launch_early(add_norm_kernel<X, R, decltype(n)::value>, dim3((unsigned)blocks), s.threads, 0, stream,
                            static_cast<const X*>(x), static_cast<const R*>(r), weight, eps, B, dim,
                            s.warps, sum, sum_dtype, y, y_dtype, rstd);
      });
    });
  });
}

cudaError_t launch_add_rms_norm_backward(const void* sum, int sum_dtype, const float* weight,
                                         const float* rstd, const void* dy, int dy_dtype,
                                         const void* ds, int B, int dim, void* workspace, void* d,
                                         int d_dtype, void* dx, int x_dtype, float* dweight,
                                         cudaStream_t stream) {
  const Shape s = shape_of(dim, kBackThreads);
  int blocks = (int)(((int64_t)B + s.groups - 1) / s.groups);
  if (blocks > kMaxParts) blocks = kMaxParts;
  const size_t smem = dweight ? (size_t)s.groups * dim * 4 : 0;
  cudaError_t e = with_type(sum_dtype, [&](auto* st) {
    return with_type(dy_dtype, [&](auto* yt) {
      return with_vectors(s.vectors, [&](auto n) {
        using S = std::remove_pointer_t<decltype(st)>;
        using Y = std::remove_pointer_t<decltype(yt)>;
        auto kernel = add_norm_backward_kernel<S, Y, decltype(n)::value>;
        if (smem > kSharedUnasked) {
          // (the most of any width: what is granted is the kernel's, not this call's, and a narrower call on
          // another host thread may come between here and the launch)
          cudaError_t e2 = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                kMostRowBytes);
          if (e2 != cudaSuccess) return e2;
        }
        return launch_early(kernel, dim3((unsigned)blocks), s.threads, smem, stream, static_cast<const S*>(sum), weight,
                            rstd, static_cast<const Y*>(dy), static_cast<const S*>(ds), B, dim, s.warps,
                            d, d_dtype, dx, x_dtype, dweight ? static_cast<float*>(workspace) : nullptr);
      });
    });
  });
  if (e != cudaSuccess || !dweight) return e;
  return launch_early(norm_join_kernel, dim3((unsigned)(dim + 31) / 32), 1024, 0, stream,
                      static_cast<const float*>(workspace), blocks, dim, dweight);
}

}  // namespace pkm

namespace {

bool norm_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool norm_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool norm_type(int dtype) { return dtype == PKM_F32 || dtype == PKM_BF16; }

int norm_rc(cudaError_t e) { return e == cudaSuccess ? PKM_OK : PKM_ERR_CUDA; }

}  // namespace

extern "C" int pkm_add_rms_norm(const void* x, int x_dtype, const void* residual, int res_dtype,
                                const float* weight, float eps, int B, int dim, void* sum,
                                int sum_dtype, void* y, int y_dtype, float* rstd, void* stream) {
  if (B < 0 || dim < 1 || !(eps >= 0.0f) || isinf(eps)) return PKM_ERR_INVALID;
  if (!norm_type(x_dtype) || !norm_type(res_dtype) || !norm_type(sum_dtype) ||
      (!norm_type(y_dtype) && y_dtype != PKM_FP8_E4M3))
    return PKM_ERR_UNSUPPORTED;
  if (dim % (y_dtype == PKM_FP8_E4M3 ? 16 : 8) || dim > PKM_NORM_MAX_DIM) return PKM_ERR_UNSUPPORTED;
  if (B == 0) return PKM_OK;
  if (!x || !weight || !y) return PKM_ERR_INVALID;
  for (const void* p : {x, residual, (const void*)weight, (const void*)sum, (const void*)y})
    if (!norm_aligned16(p)) return PKM_ERR_ALIGN;
  if (!norm_aligned4(rstd)) return PKM_ERR_ALIGN;
  return norm_rc(pkm::launch_add_rms_norm(x, x_dtype, residual, res_dtype, weight, eps, B, dim, sum,
                                          sum_dtype, y, y_dtype, rstd,
                                          static_cast<cudaStream_t>(stream)));
}

extern "C" size_t pkm_add_rms_norm_backward_workspace_bytes(int B, int dim) {
  return B < 0 || dim < 1 ? 0 : pkm::add_rms_norm_backward_workspace_bytes(B, dim);
}

extern "C" int pkm_add_rms_norm_backward(const void* sum, int sum_dtype, const float* weight,
                                         const float* rstd, const void* dy, int dy_dtype,
                                         const void* dsum, int B, int dim, void* workspace, void* dres,
                                         int res_dtype, void* dx, int x_dtype, float* dweight,
                                         void* stream) {
  if (B < 0 || dim < 1) return PKM_ERR_INVALID;
  if (!norm_type(sum_dtype) || !norm_type(dy_dtype) || !norm_type(res_dtype) || !norm_type(x_dtype) ||
      dim % 8 || dim > PKM_NORM_MAX_DIM)
    return PKM_ERR_UNSUPPORTED;
  if (B == 0) {  // no row: dweight is zero
    if (!norm_aligned16(dweight)) return PKM_ERR_ALIGN;
    return dweight ? norm_rc(cudaMemsetAsync(dweight, 0, (size_t)dim * 4,
                                             static_cast<cudaStream_t>(stream)))
                   : PKM_OK;
  }
  if (!dres && !dx && !dweight) return PKM_OK;
  if (!sum || !weight || !rstd || !dy || (dweight && !workspace)) return PKM_ERR_INVALID;
  for (const void* p : {sum, (const void*)weight, dy, dsum, (const void*)workspace, (const void*)dres,
                        (const void*)dx, (const void*)dweight})
    if (!norm_aligned16(p)) return PKM_ERR_ALIGN;
  if (!norm_aligned4(rstd)) return PKM_ERR_ALIGN;
  return norm_rc(pkm::launch_add_rms_norm_backward(sum, sum_dtype, weight, rstd, dy, dy_dtype, dsum, B,
                                                   dim, workspace, dres, res_dtype, dx, x_dtype, dweight,
                                                   static_cast<cudaStream_t>(stream)));
}
