// Internal declarations and device helpers of the feed-forward operators (awq_ffn.h).
#pragma once

#include "../../include/awq_ffn.h"
#include "block_internal.hpp"
#include "epilogue.hpp"

namespace awq {

hipError_t launch_rms_norm(const awq_rms_norm_args& a, hipStream_t st);
hipError_t launch_quant_i8(const awq_quant_i8_args& a, hipStream_t st);
hipError_t launch_pack_i8(const void* w, const void* s_c, int64_t N, int64_t K, int32_t dtype, void* packed,
                          hipStream_t st);
size_t gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_i8(const awq_gemm_i8_args& a, hipStream_t st);
size_t moe_route_workspace_bytes(int64_t tokens, int32_t hidden, int32_t experts);
hipError_t launch_moe_route(const awq_moe_route_args& a, hipStream_t st);
size_t moe_workspace_bytes(int64_t tokens, int32_t hidden, int32_t ffn, int32_t k);
hipError_t launch_moe(const awq_moe_args& a, hipStream_t st);

// The packed 8-bit layer: units of 16 rows x 64 channels.
constexpr int kI8Rows = 16, kI8Unit = 64;
struct I8Layout {
  int64_t tiles, units, scales_off, total_bytes;
};
inline I8Layout make_i8_layout(int64_t N, int64_t K) {
  I8Layout l;
  l.tiles = (N + kI8Rows - 1) / kI8Rows;
  l.units = (K + kI8Unit - 1) / kI8Unit;
  l.scales_off = l.tiles * l.units * 1024;
  l.total_bytes = (l.scales_off + l.tiles * kI8Rows * 4 + 255) / 256 * 256;
  return l;
}

// Rows whose largest value is not above this count as zeros: their scales' reciprocals stay finite.
constexpr float kLeastMax = 1e-30f;

// The scale of an 8-bit row and its reciprocal, from the largest bit pattern of the values'
// magnitudes (patterns of infinities and NaN lie above those of finite values). The scale is the product
// with 1 / 127, two roundings where a division has one: so does PyTorch divide by a constant on this
// device, and codes at halves come out as there.
struct RowScale {
  float scale, inv;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  const float most = __builtin_bit_cast(float, top);
  if (top >= 0x7F800000u) return {__builtin_nanf(""), 0.0f};
  if (!(most > kLeastMax)) return {0.0f, 0.0f};
  const float scale = most * (1.0f / 127.0f);
  return {scale, 1.0f / scale};
}
// rint(v / scale), at most 127 in magnitude; 0 where inv is 0, whatever v is. The product with inv is
// put right by what it leaves of v: products of short fractions are halves more often than chance has
// it, and there the product alone may fall on either side.
__device__ __forceinline__ int to_code(float v, const RowScale& s) {
  if (s.inv == 0.0f) return 0;
  const float t = v * s.inv;
  const float q = __builtin_rintf(__builtin_fmaf(__builtin_fmaf(-t, s.scale, v), s.inv, t));
  return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}
__device__ __forceinline__ uint32_t pack_codes(const float* v, const RowScale& s) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (static_cast<uint32_t>(to_code(v[i], s)) & 0xFFu) << (8 * i);
  return w;
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <typename T>
__device__ __forceinline__ void widen(uint4 w, float* v) {
  const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = T::to_float(static_cast<uint16_t>(p[i] & 0xFFFFu));
    v[2 * i + 1] = T::to_float(static_cast<uint16_t>(p[i] >> 16));
  }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float* v) {
  return make_uint4(T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7]));
}

}  // namespace awq
