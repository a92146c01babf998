// The element-wise tail of a product: y = act(v + bias[n]) * mul[m][n] + residual[m][n],
// in float32, before the one rounding to binary16. The product kernels take it as an
// optional last argument (a parameter pack: none for the plain products, whose code and
// arguments it leaves as they are) and apply it where they would round their sums.
#pragma once

#include "../../include/awq_block.h"
#include "awq_internal.hpp"

namespace awq {

struct Epilogue {
  const uint16_t* bias;      // [N] or NULL
  const uint16_t* mul;       // [M][N] or NULL
  const uint16_t* residual;  // [M][N] or NULL
  int act;                   // AWQ_ACT_*
};

__device__ __forceinline__ float f16_to_f32(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case AWQ_ACT_RELU: return v < 0.0f ? 0.0f : v;  // NaN stays
    case AWQ_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case AWQ_ACT_GELU_TANH:  // 0.5 (1 + tanh u) = sigmoid(2 u)
      return v * sigmoid(1.5957691216057308f * (v + 0.044715f * v * v * v));
    case AWQ_ACT_SILU: return v * sigmoid(v);
    default: return v;
  }
}

// output n of a row, at element o of the [M][N] arrays
__device__ __forceinline__ float apply_epilogue(float v, int n, int64_t o, const Epilogue& e) {
  if (e.bias != nullptr) v += f16_to_f32(e.bias[n]);
  v = activate(v, e.act);
  if (e.mul != nullptr) v *= f16_to_f32(e.mul[o]);
  if (e.residual != nullptr) v += f16_to_f32(e.residual[o]);
  return v;
}
__device__ __forceinline__ float apply_epilogue(float v, int, int64_t) { return v; }

// the same for eight consecutive outputs of a row, with 16-byte accesses (n a multiple of 8)
__device__ __forceinline__ void add8(float v[8], uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] += static_cast<float>(as_h2(u[i]).x);
    v[2 * i + 1] += static_cast<float>(as_h2(u[i]).y);
  }
}
__device__ __forceinline__ void apply_epilogue8(float v[8], int n, int64_t o, const Epilogue& e, uint16_t* y) {
  if (e.bias != nullptr) add8(v, *reinterpret_cast<const uint4*>(e.bias + n));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate(v[i], e.act);
  if (e.mul != nullptr) {
    const uint4 w = *reinterpret_cast<const uint4*>(e.mul + o);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] *= static_cast<float>(as_h2(u[i]).x);
      v[2 * i + 1] *= static_cast<float>(as_h2(u[i]).y);
    }
  }
  if (e.residual != nullptr) add8(v, *reinterpret_cast<const uint4*>(e.residual + o));
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = as_u32(half2_t{static_cast<_Float16>(v[2 * i]), static_cast<_Float16>(v[2 * i + 1])});
  *reinterpret_cast<uint4*>(y + o) = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void apply_epilogue8(float*, int, int64_t, uint16_t*) {}

// Orders one wavefront's LDS accesses for the compiler (the hardware executes them in order):
// what some lanes store, other lanes read.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

hipError_t launch_gemv_fused(const uint16_t* x, const uint16_t* inv_s_c, const void* packed, int64_t M,
                             int64_t N, int64_t K, int32_t group, int32_t fmt, const Epilogue& e,
                             uint16_t* y, hipStream_t st);
hipError_t launch_splitk_reduce_fused(const float* part, int splits, int64_t mn, int64_t N,
                                      const Epilogue& e, uint16_t* y, hipStream_t st);
hipError_t launch_gemm_wide_fused(const uint16_t* x, const uint16_t* inv_s_c, const void* packed,
                                  int64_t M, int64_t N, int64_t K, int32_t group, int32_t fmt,
                                  const Epilogue& e, uint16_t* y, void* ws, size_t ws_bytes, hipStream_t st);
hipError_t launch_gemm_fused(const uint16_t* x, const uint16_t* inv_s_c, const void* packed, int64_t M,
                             int64_t N, int64_t K, int32_t group, int32_t fmt, const Epilogue& e,
                             uint16_t* y, void* ws, size_t ws_bytes, hipStream_t st);

}  // namespace awq
