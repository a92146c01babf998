// The router of a mixture of experts: logits = x w^T, scores, the k best and their weights.
//
// Which expert comes k-th is a border: two sums in another order of float32 would now and then
// choose differently. Products of two elements are exact in float64, and so are the sums to
// about 1e-16, so the choice is the definition's. The matrix cores' float64 instruction forms
// 16 tokens x 16 experts from four channels, one element of each operand in a lane, so every
// element is widened once.
//
// Two launches: partial sums of 16 x 16 logits over slices of the channels (a token alone
// would otherwise leave the card to a few wavefronts), then one wavefront or workgroup per
// token that adds them and ranks the experts: an expert's place is the number of experts in
// front of it, which all are counted at once, without a chain of k maxima. A few tokens with a small
// router take one launch.
#include "ffn_internal.hpp"

namespace awq {
namespace {

typedef double double4_t __attribute__((ext_vector_type(4)));

constexpr int kSliceWaves = 4, kRouteAhead = 2;

// Slices of the channels, one per workgroup of four wavefronts, so that about four workgroups per
// CU run; a wavefront has at least 32 channels. (One workgroup per CU left each float64
// instruction waiting for its operands: 517 tokens x 128 experts x 4096 31 us instead of 19;
// independent float64 matrix instructions alone would take 12.)
int route_wide(int64_t tokens) { return tokens > 16 ? 2 : 1; }  // tiles of 16 tokens for a wavefront
int route_slices(int64_t tokens, int hidden, int experts) {
  const int rows = 16 * route_wide(tokens);
  const int64_t tiles = (tokens + rows - 1) / rows * ((experts + 15) / 16);
  int64_t slices = (1024 + tiles / 2) / tiles;
  const int64_t most = (hidden + 32 * kSliceWaves - 1) / (32 * kSliceWaves);
  if (slices > most) slices = most;
  if (slices > 32) slices = 32;
  return slices < 1 ? 1 : static_cast<int>(slices);
}

struct RouteArgs {
  const uint16_t *x, *w;
  const float* bias;
  int32_t* ids;
  float* weights;
  double* part;  // [slices][tokens][experts]
  int64_t tokens, x_stride;
  int hidden, experts, k, slices, score, renormalize;
  float scale;
};

// grid: token tiles, expert tiles, slices. A wavefront's WIDE token tiles share an expert's operands,
// and their sums are chains of their own.
template <typename T, int WIDE>
__global__ void __launch_bounds__(64 * kSliceWaves) route_logits_kernel(RouteArgs a) {
  __shared__ double red[kSliceWaves][16 * WIDE][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, p = lane >> 4;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * (16 * WIDE);
  const int expert = blockIdx.y * 16 + r;
  const uint16_t* w = a.w + static_cast<int64_t>(expert < a.experts ? expert : 0) * a.hidden;
  const bool has_w = expert < a.experts;
  const uint16_t* x[WIDE];
  bool has_x[WIDE];
#pragma unroll
  for (int t = 0; t < WIDE; ++t) {
    const int64_t token = token0 + 16 * t + r;
    has_x[t] = token < a.tokens;
    x[t] = a.x + (has_x[t] ? token : 0) * a.x_stride;
  }
  // steps of 32 channels dealt to all slices' wavefronts in turn
  const int steps = (a.hidden + 31) / 32, waves = kSliceWaves * a.slices;
  double4_t acc[WIDE];
#pragma unroll
  for (int t = 0; t < WIDE; ++t) acc[t] = double4_t{0.0, 0.0, 0.0, 0.0};
  uint4 xv[kRouteAhead][WIDE], wv[kRouteAhead];
  auto load = [&](int i, int s) {  // zeros behind the last channel
    const int c = 32 * s + 8 * p;
    wv[i] = make_uint4(0, 0, 0, 0);
    if (c < a.hidden && has_w) wv[i] = *reinterpret_cast<const uint4*>(w + c);
#pragma unroll
    for (int t = 0; t < WIDE; ++t) {
      xv[i][t] = make_uint4(0, 0, 0, 0);
      if (c < a.hidden && has_x[t]) xv[i][t] = *reinterpret_cast<const uint4*>(x[t] + c);
    }
  };
  const int s0 = static_cast<int>(blockIdx.z) * kSliceWaves + wave;
#pragma unroll
  for (int i = 0; i < kRouteAhead; ++i) load(i, s0 + i * waves);
  for (int s = s0; s < steps; s += kRouteAhead * waves) {
#pragma unroll
    for (int i = 0; i < kRouteAhead; ++i) {
      float xf[WIDE][8], wf[8];
      widen<T>(wv[i], wf);
#pragma unroll
      for (int t = 0; t < WIDE; ++t) widen<T>(xv[i][t], xf[t]);
      load(i, s + (i + kRouteAhead) * waves);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double we = static_cast<double>(wf[e]);
#pragma unroll
        for (int t = 0; t < WIDE; ++t)
          acc[t] = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(xf[t][e]), we, acc[t], 0, 0, 0);
      }
    }
  }
  // element i of lane l is row 4 i + l / 16, column l % 16
#pragma unroll
  for (int t = 0; t < WIDE; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][16 * t + 4 * i + p][r] = acc[t][i];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < WIDE; ++t) {
    const int m = 16 * t + threadIdx.x / 16, n = threadIdx.x % 16;
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < kSliceWaves; ++v) sum += red[v][m][n];
    const int64_t token = token0 + m;
    const int e = blockIdx.y * 16 + n;
    if (token < a.tokens && e < a.experts) a.part[(blockIdx.z * a.tokens + token) * a.experts + e] = sum;
  }
}

// An order of choices as whole numbers: larger is better, NaN stands behind -infinity.
__device__ __forceinline__ uint64_t order(double v) {
  if (v != v) return 1;
  const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);  // one zero
  return static_cast<uint64_t>(b < 0 ? ~b : b | INT64_MIN);
}

// THREADS threads for each of a workgroup's TOKENS tokens, NE experts each (t, t + THREADS, ..), whose
// logits logit(e) gives. All threads of the workgroup call it.
template <int THREADS, int NE, int TOKENS, typename Logit>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t token, Logit logit) {
  constexpr int WAVES = THREADS / 64, MOST = THREADS * NE;
  __shared__ uint64_t keys[TOKENS][MOST];
  __shared__ double picked[TOKENS][AWQ_MOE_MAX_K];
  __shared__ double wave_top[TOKENS][WAVES], wave_add[TOKENS][WAVES];
  const int mine = threadIdx.x / THREADS, t = threadIdx.x % THREADS;
  const bool live = token < a.tokens;
  double p[NE];
  double top = -__builtin_inf();
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = t + THREADS * i;
    double l = 0.0;
    if (live && e < a.experts) {
      l = logit(e);
      const double bias = a.bias == nullptr ? 0.0 : static_cast<double>(a.bias[e]);
      if (a.score == AWQ_SCORE_SIGMOID) l = 1.0 / (1.0 + exp(-l));
      keys[mine][e] = order(l + bias);
      top = fmax(top, l);
    }
    p[i] = l;
  }
  if (a.score == AWQ_SCORE_SOFTMAX) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) top = fmax(top, __shfl_xor(top, s));
    if (WAVES > 1) {
      if ((t & 63) == 0) wave_top[mine][t >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmax(top, wave_top[mine][w]);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (t + THREADS * i >= a.experts) continue;
      p[i] = exp(p[i] - top);
      sum += p[i];
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
    if (WAVES > 1) {
      if ((t & 63) == 0) wave_add[mine][t >> 6] = sum;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += wave_add[mine][w];
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] /= sum;
  }
  __syncthreads();  // all keys
  if (live) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = t + THREADS * i;
      if (e >= a.experts) continue;
      const uint64_t key = keys[mine][e];
      int place = 0;
#pragma unroll 4
      for (int o = 0; o < a.experts; ++o) {
        const uint64_t other = keys[mine][o];
        place += other > key || (other == key && o < e);
      }
      if (place < a.k) {
        a.ids[token * a.k + place] = e;
        picked[mine][place] = p[i];
      }
    }
  }
  __syncthreads();
  if (!live || t >= a.k) return;
  double sum = 1.0;
  if (a.renormalize != 0) {
    sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += picked[mine][j];
  }
  const double v = picked[mine][t] * static_cast<double>(a.scale);
  a.weights[token * a.k + t] = sum == 0.0 ? 0.0f : static_cast<float>(v / sum);
}

template <int THREADS, int NE>
__global__ void __launch_bounds__(256) route_choose_kernel(RouteArgs a) {
  constexpr int TOKENS = 256 / THREADS;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * TOKENS + threadIdx.x / THREADS;
  choose<THREADS, NE, TOKENS>(a, token, [&](int e) {
    const double* part = a.part + token * a.experts + e;
    const int64_t slice = a.tokens * a.experts;
    double l = 0.0;
    for (int s = 0; s < a.slices; s += 8) {  // eight at a time on their way
      double v[8];
#pragma unroll
      for (int o = 0; o < 8; ++o) v[o] = part[min(s + o, a.slices - 1) * slice];
#pragma unroll
      for (int o = 0; o < 8; ++o) l += s + o < a.slices ? v[o] : 0.0;
    }
    return l;
  });
}

// A token or a few with a small router: everything in one workgroup and one launch. A wavefront takes
// a run of the channels of one expert (wavefronts share experts while there are fewer of them), one
// channel of each token in a lane's sums; the matrix cores' chains of dependent float64 products
// would take longer here (90 ns each).
constexpr int kSmallTokens = 4, kSmallExperts = 64, kSmallWaves = 16;
bool is_small(int64_t tokens, int hidden, int experts) {
  return tokens <= kSmallTokens && experts <= kSmallExperts && static_cast<int64_t>(experts) * hidden <= 65536;
}
template <typename T>
__global__ void __launch_bounds__(64 * kSmallWaves) route_small_kernel(RouteArgs a) {
  __shared__ double part[kSmallTokens][kSmallExperts][kSmallWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int share = a.experts >= kSmallWaves ? 1 : kSmallWaves / a.experts;  // wavefronts of an expert
  const int tokens = static_cast<int>(a.tokens);
  for (int e = wave / share; e < a.experts; e += kSmallWaves / share) {
    double sum[kSmallTokens] = {0.0, 0.0, 0.0, 0.0};
    for (int c = 8 * (64 * (wave % share) + lane); c < a.hidden; c += 512 * share) {
      float w[8];
      widen<T>(*reinterpret_cast<const uint4*>(a.w + static_cast<int64_t>(e) * a.hidden + c), w);
#pragma unroll
      for (int t = 0; t < kSmallTokens; ++t) {
        if (t >= tokens) break;
        float x[8];
        widen<T>(*reinterpret_cast<const uint4*>(a.x + t * a.x_stride + c), x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sum[t] = __builtin_fma(static_cast<double>(x[i]), static_cast<double>(w[i]), sum[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < kSmallTokens; ++t) {
      if (t >= tokens) break;
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) sum[t] += __shfl_xor(sum[t], s);
      if (lane == 0) part[t][e][wave % share] = sum[t];
    }
  }
  __syncthreads();
  choose<64, 1, kSmallWaves>(a, wave, [&](int e) {
    double l = 0.0;
    for (int s = 0; s < share; ++s) l += part[wave][e][s];
    return l;
  });
}

template <int THREADS, int NE>
hipError_t launch_choose(const RouteArgs& a, hipStream_t st) {
  constexpr int TOKENS = 256 / THREADS;
  hipLaunchKernelGGL((route_choose_kernel<THREADS, NE>), dim3(static_cast<unsigned>((a.tokens + TOKENS - 1) / TOKENS)),
                     dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t tokens, int32_t hidden, int32_t experts) {
  if (is_small(tokens, hidden, experts)) return 0;
  return static_cast<size_t>(8) * route_slices(tokens, hidden, experts) * tokens * experts;
}

hipError_t launch_moe_route(const awq_moe_route_args& p, hipStream_t st) {
  RouteArgs a;
  a.x = static_cast<const uint16_t*>(p.x);
  a.w = static_cast<const uint16_t*>(p.w);
  a.bias = p.bias;
  a.ids = p.ids;
  a.weights = p.weights;
  a.part = static_cast<double*>(p.ws);
  a.tokens = p.tokens;
  a.x_stride = p.x_stride;
  a.hidden = p.hidden;
  a.experts = p.experts;
  a.k = p.k;
  a.slices = route_slices(p.tokens, p.hidden, p.experts);
  a.score = p.score;
  a.renormalize = p.renormalize;
  a.scale = p.scale;
  if (is_small(p.tokens, p.hidden, p.experts)) {
    hipLaunchKernelGGL((p.dtype == AWQ_DT_F16 ? &route_small_kernel<F16> : &route_small_kernel<BF16>), dim3(1),
                       dim3(64 * kSmallWaves), 0, st, a);
    return hipGetLastError();
  }
  const int wide = route_wide(p.tokens);
  const dim3 grid(static_cast<unsigned>((p.tokens + 16 * wide - 1) / (16 * wide)), (p.experts + 15) / 16, a.slices);
  const bool f16 = p.dtype == AWQ_DT_F16;
  const auto logits = wide == 1 ? f16 ? &route_logits_kernel<F16, 1> : &route_logits_kernel<BF16, 1>
                                : f16 ? &route_logits_kernel<F16, 2> : &route_logits_kernel<BF16, 2>;
  hipLaunchKernelGGL(logits, grid, dim3(64 * kSliceWaves), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.experts <= 64) return launch_choose<64, 1>(a, st);
  if (p.experts <= 128) return launch_choose<128, 1>(a, st);
  if (p.experts <= 256) return launch_choose<256, 1>(a, st);
  return launch_choose<256, 4>(a, st);
}

}  // namespace awq
