// Distillation from a teacher's top logits: the loss and its gradient.
//
// Per row b of student logits z [V], with the teacher's list (idx_j, t_j),
// j < k, and a temperature T:
//   p = softmax(t / T) over the list, q = softmax(z / T) over all V,
//   loss = T^2 sum_j p_j (log p_j - log q[idx_j])
//   dz   = dloss * T * (P q - sum_j p_j [idx_j])      P = sum_j p_j (1, or 0
//                                                     for an empty list)
// An entry with a negative idx, or a t of -inf, is absent.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "pkm_internal.cuh"

namespace pkm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int DTHREADS = 512;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// log of a positive s as a double good to about 1e-8: the exponent's part
// exactly, the mantissa's (a value in [0.75, 1.5)) by logf.
__device__ __forceinline__ double log_split(float s) {
  int e;
  float f = frexpf(s, &e);  // [0.5, 1)
  if (f < 0.75f) {
    f *= 2.0f;
    --e;
  }
  return (double)e * 0.6931471805599453 + (double)logf(f);
}

struct ListStats {
  float tm;     // largest t of the present entries, -inf if none is present
  float total;  // sum of exp((t - tm) / T)
};

// By one whole warp.  An idx >= V counts as absent and is reported.
__device__ ListStats list_stats(const int64_t* __restrict__ idx, const float* __restrict__ t,
                                int k, int V, float c, int lane, int* status) {
  float tm = -INFINITY;
  for (int j = lane; j < k; j += 32) {
    const int64_t i = idx[j];
    if (i >= V) atomicExch(status, PKM_ERR_BAD_INDEX);
    const float v = t[j];
    if (i >= 0 && i < V) tm = v > tm || isnan(v) ? v : tm;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, tm, o);
    tm = v > tm || isnan(v) ? v : tm;
  }
  float total = 0.0f;
  if (tm != -INFINITY)
    for (int j = lane; j < k; j += 32)
      if (idx[j] >= 0 && idx[j] < V) total += exp2f((t[j] - tm) * c);
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  return ListStats{tm, total};
}

// loss and lse: one CTA per row.
template <typename E>
__global__ void __launch_bounds__(DTHREADS)
distill_forward_kernel(const E* __restrict__ z, int64_t ld, int V, const int64_t* __restrict__ idx,
                       const float* __restrict__ teacher, int k, float T, float* __restrict__ loss,
                       float* __restrict__ lse, int* __restrict__ status) {
  __shared__ float s_m[DTHREADS / 32], s_s[DTHREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x;
  const float c = kLog2e / T;
  const E* row = z + b * ld;
  float m = -INFINITY, s = 0.0f;
  for (int v = threadIdx.x; v < V; v += DTHREADS) {
    const float x = to_f(row[v]);
    if (x > m) {
      s *= exp2f((m - x) * c);
      m = x;
    }
    s += x == -INFINITY ? 0.0f : exp2f((x - m) * c);
  }
  auto join = [&](float m2, float s2) {
    const float mm = fmaxf(m, m2);
    if (mm != -INFINITY) {
      s = s * exp2f((m - mm) * c) + s2 * exp2f((m2 - mm) * c);
      m = mm;
    } else {
      s += s2;
    }
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m2, s2);
  }
  if (lane == 0) s_m[warp] = m, s_s[warp] = s;
  __syncthreads();
  if (warp) return;
  m = lane < DTHREADS / 32 ? s_m[lane] : -INFINITY;
  s = lane < DTHREADS / 32 ? s_s[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m2, s2);
  }
  const double inv_t = 1.0 / (double)T;
  const double L = s == 0.0f ? -INFINITY : m * inv_t + log_split(s);
  idx += b * k, teacher += b * k;
  const ListStats st = list_stats(idx, teacher, k, V, c, lane, status);
  double sum = 0.0;
  if (st.tm != -INFINITY) {
    const double off = L - st.tm * inv_t - log_split(st.total);
    for (int j = lane; j < k; j += 32) {
      const int64_t i = idx[j];
      if (i < 0 || i >= V) continue;
      const float p = exp2f((teacher[j] - st.tm) * c) / st.total;
      const float x = to_f(row[i]);
      if (p != 0.0f)
        sum += x == -INFINITY ? INFINITY : p * (((double)teacher[j] - x) * inv_t + off);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    loss[b] = (float)(sum * (double)T * T);
    if (lse) lse[b] = (float)L;
  }
}

// dz: one CTA per row.
template <typename E>
__global__ void __launch_bounds__(DTHREADS)
distill_backward_kernel(const E* z, int64_t ld, int V, const int64_t* __restrict__ idx,
                        const float* __restrict__ teacher, int k, float T,
                        const float* __restrict__ lse, const float* __restrict__ dloss, E* dz,
                        int64_t ld_d, int* __restrict__ status) {
  __shared__ ListStats s_st;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x;
  const float c = kLog2e / T, g = dloss[b] * T;
  const E* row = z + b * ld;
  E* out = dz + b * ld_d;
  idx += b * k, teacher += b * k;
  if (warp == 0) {
    const ListStats st = list_stats(idx, teacher, k, V, c, lane, status);
    if (lane == 0) s_st = st;
  }
  __syncthreads();
  const ListStats st = s_st;
  if (g == 0.0f || st.tm == -INFINITY) {
    for (int v = threadIdx.x; v < V; v += DTHREADS) put(out + v, 0.0f);
    return;
  }
  const float L = lse[b] * kLog2e;
  auto q = [&](float x) { return x == -INFINITY ? 0.0f : exp2f(fmaf(x, c, -L)); };
  // the listed columns, kept until every thread is done with the row (dz may be z)
  float keep = 0.0f;
  for (int j0 = 0; j0 < k; j0 += DTHREADS) {
    // (k <= DTHREADS: one round)
    const int j = j0 + threadIdx.x;
    if (j < k && idx[j] >= 0 && idx[j] < V) {
      float p = 0.0f;  // every entry of this column
      for (int l = 0; l < k; ++l)
        if (idx[l] == idx[j]) p += exp2f((teacher[l] - st.tm) * c);
      keep = g * (q(to_f(row[idx[j]])) - p / st.total);
    }
  }
  __syncthreads();
  for (int v = threadIdx.x; v < V; v += DTHREADS) put(out + v, g * q(to_f(row[v])));
  __syncthreads();
  if (threadIdx.x < k && idx[threadIdx.x] >= 0 && idx[threadIdx.x] < V)
    put(out + idx[threadIdx.x], keep);
}

}  // namespace

cudaError_t launch_distill(const void* z, int dtype, int64_t ld, int B, int V, const int64_t* idx,
                           const float* teacher, int k, float T, float* loss, float* lse,
                           int* status, cudaStream_t stream) {
  if (dtype == PKM_BF16)
    distill_forward_kernel<<<B, DTHREADS, 0, stream>>>(static_cast<const __nv_bfloat16*>(z), ld, V,
                                                       idx, teacher, k, T, loss, lse, status);
  else
    distill_forward_kernel<<<B, DTHREADS, 0, stream>>>(static_cast<const float*>(z), ld, V, idx,
                                                       teacher, k, T, loss, lse, status);
  return cudaGetLastError();
}

cudaError_t launch_distill_backward(const void* z, int dtype, int64_t ld, int B, int V,
                                    const int64_t* idx, const float* teacher, int k, float T,
                                    const float* lse, const float* dloss, void* dz, int64_t ld_d,
                                    int* status, cudaStream_t stream) {
  if (dtype == PKM_BF16)
    distill_backward_kernel<<<B, DTHREADS, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(z), ld, V, idx, teacher, k, T, lse, dloss,
        static_cast<__nv_bfloat16*>(dz), ld_d, status);
  else
    distill_backward_kernel<<<B, DTHREADS, 0, stream>>>(static_cast<const float*>(z), ld, V, idx,
                                                        teacher, k, T, lse, dloss,
                                                        static_cast<float*>(dz), ld_d, status);
  return cudaGetLastError();
}

}  // namespace pkm

namespace {

__device__ int g_distill_status;  // for calls that pass none

int distill_check(int dtype, int64_t ld, int B, int V, int k, float T) {
  if (B < 0 || V < 1 || k < 1 || !(T > 0.0f) || isinf(T)) return PKM_ERR_INVALID;
  if (dtype != PKM_F32 && dtype != PKM_BF16) return PKM_ERR_UNSUPPORTED;
  if (k > PKM_DISTILL_MAX_K) return PKM_ERR_UNSUPPORTED;
  if (ld < V) return PKM_ERR_RANGE;
  return PKM_OK;
}

// Pointers to whole elements: what CUDA's own types ask for.
bool distill_aligned(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == PKM_BF16 ? 1u : 3u)) == 0;
}

int distill_status(int* status, int** out) {
  *out = status;
  if (status) return PKM_OK;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_distill_status) != cudaSuccess) return PKM_ERR_CUDA;
  *out = static_cast<int*>(p);
  return PKM_OK;
}

}  // namespace

extern "C" int pkm_distill(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                           const int64_t* idx, const float* teacher, int k, float temperature,
                           float* loss, float* lse, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc || B == 0) return rc;
  if (!logits || !idx || !teacher || !loss) return PKM_ERR_INVALID;
  if (!distill_aligned(logits, logit_dtype)) return PKM_ERR_ALIGN;
  int* st;
  if ((rc = distill_status(status, &st))) return rc;
  return pkm::launch_distill(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature, loss,
                             lse, st, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

extern "C" int pkm_distill_backward(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                                    const int64_t* idx, const float* teacher, int k,
                                    float temperature, const float* lse, const float* dloss,
                                    void* dlogits, int64_t ld_d, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc) return rc;
  if (ld_d < V || (logits == dlogits && ld != ld_d)) return PKM_ERR_RANGE;
  if (B == 0) return PKM_OK;
  if (!logits || !idx || !teacher || !lse || !dloss || !dlogits) return PKM_ERR_INVALID;
  if (!distill_aligned(logits, logit_dtype) || !distill_aligned(dlogits, logit_dtype))
    return PKM_ERR_ALIGN;
  int* st;
  if ((rc = distill_status(status, &st))) return rc;
  return pkm::launch_distill_backward(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature,
                                      lse, dloss, dlogits, ld_d, st,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

extern "C" int pkm_distill_train(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                                 const int64_t* idx, const float* teacher, int k,
                                 float temperature, const float* dloss, float* loss, float* lse,
                                 void* dlogits, int64_t ld_d, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc) return rc;
  if (ld_d < V || (logits == dlogits && ld != ld_d)) return PKM_ERR_RANGE;
  if (B == 0) return PKM_OK;
  if (!logits || !idx || !teacher || !dloss || !loss || !lse || !dlogits) return PKM_ERR_INVALID;
  if (!distill_aligned(logits, logit_dtype) || !distill_aligned(dlogits, logit_dtype))
    return PKM_ERR_ALIGN;
  int* st;
  if ((rc = distill_status(status, &st))) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pkm::launch_distill(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature, loss, lse,
                          st, s) != cudaSuccess ||
      pkm::launch_distill_backward(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature,
                                   lse, dloss, dlogits, ld_d, st, s) != cudaSuccess)
    return PKM_ERR_CUDA;
  return PKM_OK;
}
