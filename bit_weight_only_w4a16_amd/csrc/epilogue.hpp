// The element-wise tail of a product: y = act(v + bias[n]) * mul[m][n] + residual[m][n],
// in float32, before the one rounding to binary16. The product kernels take it as an
// optional last argument (a parameter pack: none for the plain products, whose code and
// arguments it leaves as they are) and apply it where they would round their sums, so that
// the tail costs its operands' bytes and no launch: 4096 -> 4096 of one token with a residual
// 4.1 us (without 4.0), 4096 -> 11008 of 16 tokens with silu and a factor 9.1 us, 4096 -> 14336
// of 2048 with bias, gelu and residual 228-236 us, 1.0 PFLOP/s (the product alone 221: the
// residual's 59 MB and the exponentials run while no products do, at the end of a tile).
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

// Orders one wavefront's LDS accesses for the compiler (the hardware executes them in order):
// what some lanes store, other lanes read.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// the same for eight consecutive outputs of a row, whose factors and residuals are in m and r
typedef float float8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ float8_t widen8(uint4 w) {
  const half8_t h = __builtin_bit_cast(half8_t, w);
  return __builtin_convertvector(h, float8_t);
}
template <int ACT>
__device__ __forceinline__ float8_t activate8(float8_t v) {
  return float8_t{activate(v[0], ACT), activate(v[1], ACT), activate(v[2], ACT), activate(v[3], ACT),
                  activate(v[4], ACT), activate(v[5], ACT), activate(v[6], ACT), activate(v[7], ACT)};
}
__device__ __forceinline__ uint4 apply_epilogue8(float8_t v, int n, uint4 m, uint4 r, const Epilogue& e) {
  if (e.bias != nullptr) v += widen8(*reinterpret_cast<const uint4*>(e.bias + n));
  switch (e.act) {  // once for the eight
    case AWQ_ACT_RELU: v = activate8<AWQ_ACT_RELU>(v); break;
    case AWQ_ACT_GELU: v = activate8<AWQ_ACT_GELU>(v); break;
    case AWQ_ACT_GELU_TANH: v = activate8<AWQ_ACT_GELU_TANH>(v); break;
    case AWQ_ACT_SILU: v = activate8<AWQ_ACT_SILU>(v); break;
    default: break;
  }
  if (e.mul != nullptr) v *= widen8(m);
  if (e.residual != nullptr) v += widen8(r);
  return __builtin_bit_cast(uint4, __builtin_convertvector(v, half8_t));
}

// A wavefront's MS x WN matrix-core tiles of sums (element q of lane l of a tile is row
// 4 (l / 16) + q, column l % 16) through its own LDS, 1 KiB per tile at tile(ms, j), so that
// a lane gets eight consecutive outputs of a row and the tail's operands and y move in
// 16-byte accesses; the operands of four such runs are on their way at a time (y may be one
// of the operands, so the compiler moves no load past a store by itself). sums(ms, j) is
// called once per tile, before its LDS is written. Rows from m0, columns from n0.
template <int MS, int WN, typename Tile, typename Sums>
__device__ __forceinline__ void store_tiles(Tile tile, Sums sums, int m0, int n0, int M, int N, const Epilogue& e,
                                            uint16_t* y) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const float4_t v = sums(ms, j);
      wave_lds_fence();  // sums may have read the tile's place
#pragma unroll
      for (int q = 0; q < 4; ++q) tile(ms, j)[(4 * (lane >> 4) + q) * 16 + (lane & 15)] = v[q];
    }
  wave_lds_fence();
  constexpr int RUNS = MS * 32 * WN, AHEAD = RUNS >= 256 ? 4 : (RUNS + 63) / 64;
#pragma unroll 1
  for (int at0 = lane; at0 < RUNS; at0 += 64 * AHEAD) {
    int64_t o[AHEAD];  // -1: past the output
    uint4 m[AHEAD], r[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int at = at0 + 64 * i, row = m0 + at / (2 * WN), n = n0 + 8 * (at % (2 * WN));
      o[i] = at < RUNS && row < M && n < N ? static_cast<int64_t>(row) * N + n : -1;
      m[i] = r[i] = make_uint4(0, 0, 0, 0);
      if (e.mul != nullptr && o[i] >= 0) m[i] = *reinterpret_cast<const uint4*>(e.mul + o[i]);
      if (e.residual != nullptr && o[i] >= 0) r[i] = *reinterpret_cast<const uint4*>(e.residual + o[i]);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (o[i] < 0) continue;
      const int at = at0 + 64 * i, ms = at / (32 * WN), oct = at % (2 * WN);
      const float* src = tile(ms, oct >> 1) + at / (2 * WN) % 16 * 16 + 8 * (oct & 1);
      const float4_t lo = *reinterpret_cast<const float4_t*>(src);
      const float4_t hi = *reinterpret_cast<const float4_t*>(src + 4);
      const float8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      *reinterpret_cast<uint4*>(y + o[i]) = apply_epilogue8(v, n0 + 8 * oct, m[i], r[i], e);
    }
  }
  wave_lds_fence();
}
template <int MS, int WN, typename Tile, typename Sums>
__device__ __forceinline__ void store_tiles(Tile, Sums, int, int, int, int, uint16_t*) {}

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
