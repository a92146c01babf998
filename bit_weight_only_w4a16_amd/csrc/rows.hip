// Rows of activations: root-mean-square norm with the residual's addition, 8-bit rows with a
// scale, and the packing of 8-bit weights.
//
//   h = T(x + residual);  v = h w r,  r = 1 / sqrt(mean(h^2) + eps);  s = max|v| / 127,
//   q = rint(v / s)
//
// A row is read once and stays in registers; its sum of squares, and for 8-bit rows max|v| after
// it, come from reductions over the row's threads, and every output is written from there. Memory
// is the only bound of long inputs: 16384 x 8192 bfloat16 with a residual 187 us (5.7 TB/s), 2048 x 14336
// to 8 bits 20.5 us one call behind the other and 23.2 by itself (4.3 and 3.8 TB/s); one row of 4096 2.9
// us, a launch, a trip to memory and a reduction.
#include "ffn_internal.hpp"

namespace awq {
namespace {

// Squares of rows past 2^63 overflow float32: such a row is summed times 2^-76 (the largest
// bfloat16 2^128 squared times 2^15 elements stays below 2^120), and eps times 2^-152 with it; so is one
// whose mean and eps pass it together.
constexpr float kDown = 0x1p-76f;

struct RowsArgs {
  const uint16_t *x, *residual, *weight;
  uint16_t *h, *y;
  uint8_t* q;
  float* scale;
  int64_t tokens, x_stride, residual_stride, h_stride, y_stride, q_stride;
  int width;
  float eps;
};

// `v` combined over a row's THREADS threads, left in all of them.
template <int THREADS, typename V, typename Op>
__device__ __forceinline__ V row_reduce(V v, V* shared, Op op) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v = op(v, __shfl_xor(v, s));
  if constexpr (THREADS > 64) {
    __syncthreads();  // an earlier reduction's values have been read
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = op(v, shared[w]);
  }
  return v;
}

// A value of which the compiler knows nothing from here on.
__device__ __forceinline__ void hide(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

// THREADS threads for each row, NV runs of eight elements for each thread.
template <typename T, int THREADS, int NV, bool NORM>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) rows_kernel(RowsArgs a) {
  constexpr int BLOCK = THREADS < 256 ? 256 : THREADS, ROWS = BLOCK / THREADS;
  __shared__ float sums[BLOCK / 64];
  __shared__ uint32_t tops[BLOCK / 64];
  const int t = threadIdx.x % THREADS;
  const int runs = a.width / 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / THREADS; row < a.tokens;
       row += static_cast<int64_t>(gridDim.x) * ROWS) {
    uint4 h[NV], w[NV];  // as elements: the sum is rounded to them
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = 8 * (t + THREADS * i);
      uint4 r = make_uint4(0, 0, 0, 0);
      h[i] = r;
      const uint32_t one = T::pack2(1.0f, 1.0f);
      w[i] = make_uint4(one, one, one, one);
      if (t + THREADS * i < runs) {
        h[i] = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + at);
        if (NORM && a.residual != nullptr)
          r = *reinterpret_cast<const uint4*>(a.residual + row * a.residual_stride + at);
        if (a.weight != nullptr) w[i] = *reinterpret_cast<const uint4*>(a.weight + at);
      }
      if (NORM && a.residual != nullptr) {
        float s[8], f[8];
        widen<T>(r, s);
        widen<T>(h[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += f[e];
        h[i] = narrow<T>(s);
        if (a.h != nullptr && t + THREADS * i < runs) *reinterpret_cast<uint4*>(a.h + row * a.h_stride + at) = h[i];
      }
    }
    // the compiler would keep all float32 values from one pass over the registers to the next:
    // twice the registers
    auto hide_all = [&] {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hide(h[i]);
        hide(w[i]);
      }
    };
    float down = 1.0f, r = 1.0f;
    if (NORM) {
      auto squares = [&] {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[8];
          widen<T>(h[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] *= down;
            sum = __builtin_fmaf(f[e], f[e], sum);
          }
        }
        hide_all();
        return row_reduce<THREADS>(sum, sums, [](float a, float b) { return a + b; });
      };
      const float width = static_cast<float>(a.width);
      float mean = squares() / width + a.eps;
      if (mean == __builtin_inff()) {
        down = kDown;
        mean = squares() / width + a.eps * kDown * kDown;  // 2^-152 itself is no float32
      }
      r = down / sqrtf(mean);
    }
    auto values = [&](int i, float* v) {
      float f[8];
      widen<T>(h[i], v);
      widen<T>(w[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (NORM ? v[e] * r : v[e]) * f[e];
    };
    RowScale s = {0.0f, 0.0f};
    if (a.q != nullptr) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[8];
        values(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = umax(top, magnitude(v[e]));
      }
      hide_all();
      s = row_scale(row_reduce<THREADS>(top, tops, [](uint32_t a, uint32_t b) { return umax(a, b); }));
      if (t == 0) a.scale[row] = s.scale;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const int at = 8 * (t + THREADS * i);
      if (t + THREADS * i >= runs) continue;
      float v[8];
      values(i, v);
      if (NORM && a.y != nullptr) *reinterpret_cast<uint4*>(a.y + row * a.y_stride + at) = narrow<T>(v);
      if (a.q != nullptr)
        *reinterpret_cast<uint2*>(a.q + row * a.q_stride + at) =
            make_uint2(pack_codes(v, s), pack_codes(v + 4, s));
    }
  }
}

template <typename T, int THREADS, int NV, bool NORM>
hipError_t launch_rows_as(const RowsArgs& a, hipStream_t st) {
  constexpr int BLOCK = THREADS < 256 ? 256 : THREADS, ROWS = BLOCK / THREADS;
  constexpr int64_t kMostBlocks = int64_t{1} << 20;  // a launch holds 2^32 threads; more rows go in turns
  int64_t blocks = (a.tokens + ROWS - 1) / ROWS;
  if (blocks > kMostBlocks) blocks = kMostBlocks;
  hipLaunchKernelGGL((rows_kernel<T, THREADS, NV, NORM>), dim3(static_cast<unsigned>(blocks)), dim3(BLOCK), 0, st, a);
  return hipGetLastError();
}

template <typename T, bool NORM>
hipError_t launch_rows(const RowsArgs& a, hipStream_t st) {
  const int runs = a.width / 8;
  if (runs <= 64) return launch_rows_as<T, 64, 1, NORM>(a, st);
  if (runs <= 128) return launch_rows_as<T, 64, 2, NORM>(a, st);
  if (runs <= 256) return launch_rows_as<T, 256, 1, NORM>(a, st);
  if (runs <= 512) return launch_rows_as<T, 256, 2, NORM>(a, st);
  if (runs <= 1024) return launch_rows_as<T, 256, 4, NORM>(a, st);
  if (runs <= 2048) return launch_rows_as<T, 512, 4, NORM>(a, st);
  return launch_rows_as<T, 1024, 4, NORM>(a, st);  // 32768 elements at most
}

// 16 rows of a packed 8-bit layer: 16 threads of a row find its largest value, then write its
// units' 16-byte pieces, for which they read it again: once for a layer's life, 14336 x 4096 in 61 us and
// 4096 x 14336, with a quarter of the workgroups, in 132 (read once, written once: 34).
template <typename T>
__global__ void __launch_bounds__(256)
    pack_i8_kernel(const uint16_t* w, const uint16_t* s_c, int64_t N, int64_t K, int64_t units, uint8_t* codes,
                   float* scales) {
  const int64_t tile = blockIdx.x;
  const int r = threadIdx.x / 16, t = threadIdx.x % 16;
  const int64_t n = tile * kI8Rows + r;
  auto value = [&](int64_t k, float* v) {  // eight channels of row n from k
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (n >= N || k >= K) return;
    widen<T>(*reinterpret_cast<const uint4*>(w + n * K + k), v);
    if (s_c == nullptr) return;
    float s[8];
    widen<T>(*reinterpret_cast<const uint4*>(s_c + k), s);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s[e];
  };
  uint32_t top = 0;
  for (int64_t k = 8 * t; k < K; k += 128) {
    float v[8];
    value(k, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = umax(top, magnitude(v[e]));
  }
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), s)));
  const RowScale s = row_scale(top);
  if (t == 0) scales[tile * kI8Rows + r] = s.scale;
  for (int64_t c = t; c < 4 * units; c += 16) {  // pieces of 16 channels
    float v[16];
    value(16 * c, v);
    value(16 * c + 8, v + 8);
    *reinterpret_cast<uint4*>(codes + (tile * units + c / 4) * 1024 + 16 * (16 * (c % 4) + r)) = make_uint4(
        pack_codes(v, s), pack_codes(v + 4, s), pack_codes(v + 8, s), pack_codes(v + 12, s));
  }
}

}  // namespace

hipError_t launch_rms_norm(const awq_rms_norm_args& p, hipStream_t st) {
  RowsArgs a{};
  a.x = static_cast<const uint16_t*>(p.x);
  a.residual = static_cast<const uint16_t*>(p.residual);
  a.weight = static_cast<const uint16_t*>(p.weight);
  a.h = static_cast<uint16_t*>(p.h_out);
  a.y = static_cast<uint16_t*>(p.y);
  a.q = reinterpret_cast<uint8_t*>(p.q);
  a.scale = p.scale;
  a.tokens = p.tokens;
  a.x_stride = p.x_stride;
  a.residual_stride = p.residual_stride;
  a.h_stride = p.h_stride;
  a.y_stride = p.y_stride;
  a.q_stride = p.q_stride;
  a.width = p.width;
  a.eps = p.eps;
  return p.dtype == AWQ_DT_F16 ? launch_rows<F16, true>(a, st) : launch_rows<BF16, true>(a, st);
}

hipError_t launch_quant_i8(const awq_quant_i8_args& p, hipStream_t st) {
  RowsArgs a{};
  a.x = static_cast<const uint16_t*>(p.x);
  a.weight = static_cast<const uint16_t*>(p.inv_s_c);
  a.q = reinterpret_cast<uint8_t*>(p.q);
  a.scale = p.scale;
  a.tokens = p.tokens;
  a.x_stride = p.x_stride;
  a.q_stride = p.q_stride;
  a.width = p.width;
  return p.dtype == AWQ_DT_F16 ? launch_rows<F16, false>(a, st) : launch_rows<BF16, false>(a, st);
}

hipError_t launch_pack_i8(const void* w, const void* s_c, int64_t N, int64_t K, int32_t dtype, void* packed,
                          hipStream_t st) {
  const I8Layout l = make_i8_layout(N, K);
  const auto kernel = dtype == AWQ_DT_F16 ? &pack_i8_kernel<F16> : &pack_i8_kernel<BF16>;
  uint8_t* base = static_cast<uint8_t*>(packed);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(l.tiles)), dim3(256), 0, st, static_cast<const uint16_t*>(w),
                     static_cast<const uint16_t*>(s_c), N, K, l.units, base,
                     reinterpret_cast<float*>(base + l.scales_off));
  return hipGetLastError();
}

}  // namespace awq
