// Activations of the gated feed-forward block, its matrices as TMA takes them: shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/pkm.h"
#include "num_common.cuh"
#include "tc_common.cuh"

namespace pkm {

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + exp(-x)), with x log2(e) given
__device__ __forceinline__ float sigmoid2(float x2) { return rcp(1.0f + ex2(-x2)); }

constexpr float kTanh = 1.5957691216057308f;  // 2 sqrt(2 / pi): (1 + tanh v) / 2 = sigmoid(2 v)

// What calls without a status word report into (looked up by the kernels: the address costs the
// host 0.3 us a call).
static __device__ int g_ffn_status;
__device__ __forceinline__ int* status_of(int* status) { return status ? status : &g_ffn_status; }

// act(g) and act'(g)
template <int kAct>
__device__ __forceinline__ float2 act_both(float g) {
  if constexpr (kAct == PKM_ACT_SILU) {
    const float s = sigmoid2(g * kLog2e), a = g * s;
    return make_float2(a, fmaf(a, 1.0f - s, s));
  } else if constexpr (kAct == PKM_ACT_GELU) {
    // The normal distribution's cdf, good relative to itself in the negative tail, where
    // (1 + erf) / 2 cancels (at g = -5 it is 3e-7): exp(-g^2 / 2), which the slope needs anyway,
    // times a polynomial in 1 / (1 + 0.3625 |g|), fitted over |g| < 13.5 for the least largest
    // relative error (2^-20; 2^-17 with the exponent's rounding).  Forward 16384 x 1024 x 4096: 229 us
    // with erff, 270 with erfcf, 225 so.
    const float e = ex2(g * g * (-0.5f * kLog2e)), t = rcp(fmaf(0.3625f, fabsf(g), 1.0f));
    float r = fmaf(t, 0.0480628908f, -0.179742411f);
    r = fmaf(t, r, 0.175103992f);
    r = fmaf(t, r, 0.0296824165f);
    r = fmaf(t, r, 0.139256716f);
    r = fmaf(t, r, 0.142936394f);
    r = fmaf(t, r, 0.144700378f);
    const float tail = e * (t * r), cdf = g < 0.0f ? tail : 1.0f - tail;
    return make_float2(g * cdf, fmaf(g * 0.39894228f, e, cdf));
  } else if constexpr (kAct == PKM_ACT_GELU_TANH) {
    const float g2 = g * g;
    const float s = sigmoid2(kTanh * kLog2e * g * fmaf(0.044715f, g2, 1.0f)), a = g * s;
    return make_float2(a, fmaf(a * (1.0f - s), kTanh * fmaf(0.134145f, g2, 1.0f), s));
  } else {
    // (a NaN stays one, as in the other activations)
    return g <= 0.0f ? make_float2(0.0f, 0.0f) : make_float2(g, g > 0.0f ? 1.0f : g);
  }
}
template <int kAct>
__device__ __forceinline__ float act_fwd(float g) {
  return act_both<kAct>(g).x;
}
// f(tag) with the activation of a launch as the tag's value
template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == PKM_ACT_SILU)
    f(ActTag<PKM_ACT_SILU>());
  else if (act == PKM_ACT_GELU)
    f(ActTag<PKM_ACT_GELU>());
  else if (act == PKM_ACT_GELU_TANH)
    f(ActTag<PKM_ACT_GELU_TANH>());
  else
    f(ActTag<PKM_ACT_RELU>());
}

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// A [rows, cols] bf16 matrix in boxes of box_cols x box_rows, 128-byte swizzle.
inline bool encode_matrix(CUtensorMap* m, const void* ptr, int rows, int cols, int box_cols,
                          int box_rows) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pkm
