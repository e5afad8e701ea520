// Arithmetic shared by kernels: powers of two and bf16 packing.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace pkm {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&w);
}

}  // namespace pkm
