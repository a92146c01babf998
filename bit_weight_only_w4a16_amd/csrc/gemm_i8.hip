// Product in 8-bit integers: y = act(s_x[m] s_w[n] sum_k q[m][k] w[n][k] + bias) * mul + residual.
//
// The sums are whole numbers below 2^31 (K <= 131056), so neither their order nor a split of K
// changes a result; float32 begins at the scales.
//
// Workgroups of eight wavefronts own 16 columns and up to 64 rows, the wavefronts taking units
// of 64 channels in turn; operands go from memory straight into the matrix instruction's
// registers, and the wavefronts' sums meet in LDS.
#include "ffn_internal.hpp"

namespace awq {
namespace {

typedef int int4_t __attribute__((ext_vector_type(4)));

struct I8Args {
  const uint8_t *q, *codes;
  const float *scale, *scales;
  const uint16_t *bias, *mul, *residual;
  uint16_t* y;
  int64_t M, N, q_stride;
  int K, units, act;
};

// outputs n, n + 1 of row m from their sums
template <typename T>
__device__ __forceinline__ void store2(const I8Args& a, int64_t m, int n, int s0, int s1) {
  const float sx = a.scale[m];
  float v[2] = {static_cast<float>(s0) * sx * a.scales[n], static_cast<float>(s1) * sx * a.scales[n + 1]};
  const int64_t o = m * a.N + n;
  auto both = [&](const uint16_t* p, int64_t at, float* f) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + at);
    f[0] = T::to_float(static_cast<uint16_t>(w & 0xFFFFu));
    f[1] = T::to_float(static_cast<uint16_t>(w >> 16));
  };
  float f[2];
  if (a.bias != nullptr) {
    both(a.bias, n, f);
    v[0] += f[0];
    v[1] += f[1];
  }
  v[0] = activate(v[0], a.act);
  v[1] = activate(v[1], a.act);
  if (a.mul != nullptr) {
    both(a.mul, o, f);
    v[0] *= f[0];
    v[1] *= f[1];
  }
  if (a.residual != nullptr) {
    both(a.residual, o, f);
    v[0] += f[0];
    v[1] += f[1];
  }
  *reinterpret_cast<uint32_t*>(a.y + o) = T::pack2(v[0], v[1]);
}

template <typename T, int RB>
__global__ void __launch_bounds__(512) i8_rows_kernel(I8Args a) {
  constexpr int WAVES = 8, AHEAD = 4, ROWS = 16 * RB;
  __shared__ int red[WAVES][ROWS][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, p = lane >> 4;
  const int64_t tile = blockIdx.x, m0 = static_cast<int64_t>(blockIdx.y) * ROWS;
  const int rows = static_cast<int>(a.M - m0 < ROWS ? a.M - m0 : ROWS);
  const uint32_t stride = static_cast<uint32_t>(a.q_stride);
  // rows past M and channels past K lie past the end: zeros
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q + m0 * a.q_stride, (rows - 1) * stride + a.K);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.codes + tile * a.units * 1024, a.units * 1024);
  int4_t acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = int4_t{0, 0, 0, 0};
  for (int u0 = wave; u0 < a.units; u0 += WAVES * AHEAD) {
    uint4 w[AHEAD], x[AHEAD][RB];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int u = u0 + WAVES * j;
      const uint32_t skip = u < a.units ? 0u : kNoLoad;
      w[j] = buf_load16_stream(rw, 16u * lane + skip, u * 1024u);
#pragma unroll
      for (int b = 0; b < RB; ++b) x[j][b] = buf_load16(rq, (16 * b + r) * stride + 16u * p + 64u * u + skip, 0);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(int4_t, x[j][b]),
                                                       __builtin_bit_cast(int4_t, w[j]), acc[b], 0, 0, 0);
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[wave][16 * b + 4 * p + j][r] = acc[b][j];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * ROWS; i += 512) {
    const int m = i / 8, c = 2 * (i % 8);
    const int n = static_cast<int>(tile) * 16 + c;
    if (m >= rows || n >= a.N) continue;
    int s0 = 0, s1 = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      s0 += red[w][m][c];
      s1 += red[w][m][c + 1];
    }
    store2<T>(a, m0 + m, n, s0, s1);
  }
}

template <typename T>
hipError_t launch_as(const I8Args& a, hipStream_t st) {
  const unsigned tiles = static_cast<unsigned>((a.N + 15) / 16);
  auto go = [&](auto kernel, int rows) {
    // blocks of rows beyond a launch's y extent go in launches of their own
    constexpr int64_t kMostY = 65535;
    I8Args part = a;
    for (int64_t m = 0; m < a.M; m += kMostY * rows) {
      part.M = a.M - m < kMostY * rows ? a.M - m : kMostY * rows;
      part.q = a.q + m * a.q_stride;
      part.scale = a.scale + m;
      part.mul = a.mul == nullptr ? nullptr : a.mul + m * a.N;
      part.residual = a.residual == nullptr ? nullptr : a.residual + m * a.N;
      part.y = a.y + m * a.N;
      hipLaunchKernelGGL(kernel, dim3(tiles, static_cast<unsigned>((part.M + rows - 1) / rows)), dim3(512), 0, st, part);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (a.M <= 16) return go(&i8_rows_kernel<T, 1>, 16);
  if (a.M <= 32) return go(&i8_rows_kernel<T, 2>, 32);
  return go(&i8_rows_kernel<T, 4>, 64);
}

}  // namespace

size_t gemm_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_i8(const awq_gemm_i8_args& p, hipStream_t st) {
  const I8Layout l = make_i8_layout(p.N, p.K);
  I8Args a;
  a.q = reinterpret_cast<const uint8_t*>(p.q);
  a.codes = static_cast<const uint8_t*>(p.packed);
  a.scale = p.scale;
  a.scales = reinterpret_cast<const float*>(a.codes + l.scales_off);
  a.bias = static_cast<const uint16_t*>(p.bias);
  a.mul = static_cast<const uint16_t*>(p.mul);
  a.residual = static_cast<const uint16_t*>(p.residual);
  a.y = static_cast<uint16_t*>(p.y);
  a.M = p.M;
  a.N = p.N;
  a.q_stride = p.q_stride;
  a.K = static_cast<int>(p.K);
  a.units = static_cast<int>(l.units);
  a.act = p.act;
  return p.dtype == AWQ_DT_F16 ? launch_as<F16>(a, st) : launch_as<BF16>(a, st);
}

}  // namespace awq
