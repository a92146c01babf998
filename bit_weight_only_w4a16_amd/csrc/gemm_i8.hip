// Product in 8-bit integers: y = act(s_x[m] s_w[n] sum_k q[m][k] w[n][k] + bias) * mul + residual.
//
// The sums are whole numbers below 2^31 (K <= 131056), so neither their order nor a split of K
// changes a result; float32 begins at the scales.
//
// Few rows: workgroups of eight wavefronts own 16 columns and up to 64 rows, the wavefronts taking
// units of 64 channels in turn; operands go from memory straight into the matrix instruction's
// registers, and the wavefronts' sums meet in LDS. Bound by memory: 4096 -> 14336 of one row 10.8 us
// (5.4 TB/s), 4096 -> 4096 4.6. More rows: tiles (below).
#include "ffn_internal.hpp"

#include <math.h>
#include <stdio.h>

namespace awq {
namespace {

typedef int int4_t __attribute__((ext_vector_type(4)));

struct I8Args {
  const uint8_t *q, *codes;
  const float *scale, *scales;
  const uint16_t *bias, *mul, *residual;
  uint16_t* y;
  int64_t M, N, q_stride;
  int32_t* part;  // [splits][M][N]: the sums of a split of the channels
  int K, units, act;
};

// A sum times both scales, in range wherever the result is: rows' scales reach 2^121 (bfloat16's largest
// by 127) and sums 2^31, so the row's scale goes first with 2^-24 and the channel's with 2^24 after it.
// (Powers of two: ordinary values have the bits that they have without them.)
__device__ __forceinline__ float row_factor(float s) { return s * 0x1p-24f; }
__device__ __forceinline__ float channel_factor(float s) { return s * 0x1p24f; }

// outputs n, n + 1 of row m from their sums
template <typename T>
__device__ __forceinline__ void store2(const I8Args& a, int64_t m, int n, int s0, int s1) {
  const float sx = row_factor(a.scale[m]);
  float v[2] = {static_cast<float>(s0) * sx * channel_factor(a.scales[n]),
                static_cast<float>(s1) * sx * channel_factor(a.scales[n + 1])};
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

// ------------------------------------------------------------------------------- tiles
//
// Four wavefronts own BM x BN outputs, a wavefront a quarter of them, in steps of 64 channels; with
// TEAMS = 2 a workgroup has two such teams, which take turns with the steps and add up their sums
// at the end (few tiles leave a SIMD one wavefront, whose every step waits for LDS and the barrier).
// Operands go from memory straight into LDS, W's into a ring of three or four steps, the rows' into one
// of two or three pairs of steps: a pair is a whole line of 128 bytes of each row (steps of 64 bytes by
// themselves: 142 us instead of 134 at 2048 x 14336 x 4096, 81 instead of 68 at 1000 x 11000 x 4080).
// The only barrier of a step stands before its second half, whose operands are in registers already.
// v_mfma_i32_32x32x32_i8 takes W's fragment as its first operand, so that a lane's results are
// runs of four outputs of one row. 2048 x 14336 x 4096 with silu and a factor 129-140 us by the card (1.7 to
// 1.9 POPS), of which the products alone take 64, the loads alone 61.

typedef int int16_t_ __attribute__((ext_vector_type(16)));

template <typename T>
__device__ __forceinline__ float8_t load8(const uint16_t* p) {
  float f[8];
  widen<T>(*reinterpret_cast<const uint4*>(p), f);
  return float8_t{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
}
// the tail of eight consecutive outputs, v scaled and with its bias, f and r the factors and residuals
template <typename T>
__device__ __forceinline__ uint4 tail8(const I8Args& a, float8_t v, uint4 f, uint4 r) {
  switch (a.act) {
    case AWQ_ACT_RELU: v = activate8<AWQ_ACT_RELU>(v); break;
    case AWQ_ACT_GELU: v = activate8<AWQ_ACT_GELU>(v); break;
    case AWQ_ACT_GELU_TANH: v = activate8<AWQ_ACT_GELU_TANH>(v); break;
    case AWQ_ACT_SILU: v = activate8<AWQ_ACT_SILU>(v); break;
    default: break;
  }
  float w[8];
  if (a.mul != nullptr) {
    widen<T>(f, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= w[e];
  }
  if (a.residual != nullptr) {
    widen<T>(r, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = v[e];
  return narrow<T>(w);
}

constexpr int kStep = 64;  // channels of a step
// W's steps in LDS. Three steps of 128 x 256 outputs leave room for two workgroups on a CU, one of
// which multiplies while the other stores (four steps: 149 us instead of 135 at 2048 x 14336 x
// 4096; tiles of 256 x 256, which have a CU to themselves: 155). Smaller tiles have less to do in a
// step and take four (64 x 128 at 333 x 4096 x 11008: 41 us with three, 32 with four, 33 with six),
// and three of the rows' pairs (there 38 us with two, 32 with three).
constexpr int ring(int bm, int bn) { return bm * bn > 16384 ? 3 : 4; }
constexpr int pairs(int bm, int bn) { return bm * bn > 16384 ? 2 : 3; }
constexpr int stages(int bm, int bn) { return ring(bm, bn) * bn * kStep + pairs(bm, bn) * 2 * bm * kStep; }

template <typename T, int BM, int BN, int TEAMS, bool SPLIT>
__global__ void __launch_bounds__(256 * TEAMS, 2) i8_tile_kernel(I8Args a) {
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 32, FN = TN / 32;
  constexpr int RING = ring(BM, BN), PAIRS = pairs(BM, BN), STAGE_W = BN * kStep, PAIR = 2 * BM * kStep;
  constexpr int PIECES_Q = BM / 32, PIECES_W = BN / 64;  // a wavefront's loads of a pair of steps, and of one
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int number = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wave = number & 3, team = number >> 2;
  const int wm = wave & 1, wn = wave >> 1, half = lane >> 5, l32 = lane & 31;

  // blocks of an XCD are neighbours: bands of eight row tiles, down the rows first
  const int mt = static_cast<int>((a.M + BM - 1) / BM), nt = static_cast<int>((a.N + BN - 1) / BN);
  const int id = xcd_block(blockIdx.x, mt * nt);
  const int band = id / (8 * nt), band_rows = min(8, mt - 8 * band), in_band = id - band * 8 * nt;
  const int tile_m = 8 * band + in_band % band_rows, tile_n = in_band / band_rows;
  const int64_t m0 = static_cast<int64_t>(tile_m) * BM;
  const int n0 = tile_n * BN;
  const int rows = static_cast<int>(min(a.M - m0, static_cast<int64_t>(BM)));
  const uint32_t stride = static_cast<uint32_t>(a.q_stride);
  const u32x4 rq = rsrc_words(a.q + m0 * a.q_stride, (rows - 1) * stride + a.K);
  const int tiles = static_cast<int>((a.N + 15) / 16);
  const u32x4 rw = rsrc_words(a.codes, static_cast<uint32_t>(tiles) * a.units * 1024u);
  const unsigned char* mine_lds = lds + team * stages(BM, BN);  // W's steps, then the rows' pairs of steps
  const uint32_t base = lds_offset(mine_lds);

  // units of this workgroup's share of the channels; a team's last step may lie past them (zeros)
  int first = 0, end = a.units;
  if (SPLIT) {
    first = static_cast<int>(static_cast<int64_t>(a.units) * blockIdx.y / gridDim.y);
    end = static_cast<int>(static_cast<int64_t>(a.units) * (blockIdx.y + 1) / gridDim.y);
  }
  const int steps = (end - first + TEAMS - 1) / TEAMS;
  first += team * steps;

  // Rows are read two steps at a time, whole lines of 128 bytes; in LDS a line's 16-byte pieces are
  // exchanged by the row's number (p ^ row / 2 % 8), so that sixteen rows' equal pieces lie in
  // different banks; the exchange is made where a lane loads.
  // All but a lane's own part of an offset is scalar (333 x 4096 x 11008 32.3 us -> 30.5).
  const uint32_t lane_col = 16u * ((lane & 7) ^ (lane >> 4));
  const uint32_t lane_q[2] = {(lane >> 3) * stride + lane_col, (lane >> 3) * stride + (lane_col ^ 64u)};
  auto issue_rows = [&](int slot, int pair, int i) {  // 1 KiB: eight rows
    const uint32_t piece = wave * PIECES_Q + i;
    const uint32_t unit = first + 2 * pair;
    const uint32_t at = 2 * pair < steps ? piece * 8u * stride + unit * kStep : kNoLoad;
    load_to_lds(rq, at + lane_q[i & 1], base + RING * STAGE_W + slot * PAIR + piece * 1024u);
  };
  auto issue_w = [&](int slot, int step, int i) {  // 1 KiB: a unit
    const int piece = wave * PIECES_W + i, t = n0 / 16 + piece, unit = first + step;
    const uint32_t at = t < tiles && step < steps && (TEAMS == 1 || unit < end)
                            ? (static_cast<uint32_t>(t) * a.units + unit) * 1024u
                            : kNoLoad;
    load_to_lds(rw, at + 16u * lane, base + slot * STAGE_W + piece * 1024u);
  };
  // operands of half s of a step, in the order of their use: W's, then the rows'
  int4_t fq[2][FM], fw[2][FN];
  auto read_one = [&](int step, int s, int i) {  // step: its number modulo UNROLL
    if (i < FN) {
      const unsigned char* w = mine_lds + step % RING * STAGE_W + (wn * TN / 16 + (l32 >> 4)) * 1024 +
                               16 * ((lane & 15) + 16 * (2 * s + half));
      fw[s][i] = *reinterpret_cast<const int4_t*>(w + i * 2048);
    } else {
      const unsigned char* q = mine_lds + RING * STAGE_W + step / 2 % PAIRS * PAIR + (wm * TM + l32) * 2 * kStep +
                               16 * ((4 * (step % 2) + 2 * s + half) ^ ((lane >> 1) & 7));
      fq[s][i - FN] = *reinterpret_cast<const int4_t*>(q + (i - FN) * 64 * kStep);
    }
  };
  int16_t_ acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  // A half's products in runs of FN, and between the runs an equal part of the next half's LDS
  // reads and of the loads of a step to come: a wavefront may have its SIMD to itself, and nothing
  // else would fill the matrix cores' pauses. (Left to the compiler, both stand in front.)
  // A step's loads go out in its second half: W's of step + RING, and from an odd step before them the
  // rows' of the pair that takes its own pair's place, which it was the last to read.
  auto products = [&](int s, int read_step, bool loads, int n, int step) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[s][j], fq[s][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int r = (FM + FN) * i / FM; r < (FM + FN) * (i + 1) / FM; ++r) read_one(read_step, s ^ 1, r);
      if (loads) {
        const int rows = n % 2 * PIECES_Q, all = rows + PIECES_W;
#pragma unroll
        for (int l = 0; l < PIECES_Q + PIECES_W; ++l) {
          if (l < all * i / FM || l >= all * (i + 1) / FM) continue;
          if (l < rows) {
            issue_rows(n / 2 % PAIRS, step / 2 + PAIRS, l);
          } else {
            issue_w(n % RING, step + RING, l - rows);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // in front of the first step the same loads in the same order; those past the end write zeros
#pragma unroll
  for (int n = 1 - 2 * PAIRS < -RING ? 1 - 2 * PAIRS : -RING; n < 0; ++n) {
    if (n % 2 != 0 && n >= 1 - 2 * PAIRS) {
#pragma unroll
      for (int l = 0; l < PIECES_Q; ++l) issue_rows((n + 2 * PAIRS) / 2, (n + 2 * PAIRS) / 2, l);
    }
    if (n >= -RING) {
#pragma unroll
      for (int l = 0; l < PIECES_W; ++l) issue_w(n + RING, n + RING, l);
    }
  }
  constexpr int AHEAD = (RING - 2) * PIECES_W;
  wait_loads<AHEAD + PIECES_W + (PAIRS - 1) * PIECES_Q>();
  lds_barrier();
#pragma unroll
  for (int r = 0; r < FM + FN; ++r) read_one(0, 0, r);
  constexpr int UNROLL = 12;
  for (int i0 = 0; i0 < steps; i0 += UNROLL) {
#pragma unroll
    for (int n = 0; n < UNROLL; ++n) {  // the steps' places in the rings are constants
      if (i0 + n >= steps) break;
      products(0, n, false, 0, 0);
      // This step's operands are read, and the next step's have landed when no more are on their way
      // than went out behind them: W's of RING - 2 steps and a pair of the rows'. (With two pairs
      // the rows' themselves are the last but AHEAD where the next step begins a pair.)
      if (PAIRS > 2 || n % 2 == 0) {
        wait_loads<AHEAD + PIECES_Q>();
      } else {
        wait_loads<AHEAD>();
      }
      lds_barrier();
      products(1, (n + 1) % UNROLL, true, n, i0 + n);
    }
  }
  wait_loads<0>();  // none may land in what follows

  constexpr int PITCH = TN + 4;
  if constexpr (TEAMS > 1) {  // behind the place of the output's transposition
    int16_t_* sums = reinterpret_cast<int16_t_*>(lds + 4 * 32 * PITCH * 4) + wave * FM * FN * 64 + lane;
    __syncthreads();  // all wavefronts have read their last operands
    if (team == 1) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) sums[(i * FN + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (team == 1) return;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] += sums[(i * FN + j) * 64];
  }
  // element e of lane l: output 8 (e / 4) + 4 (l / 32) + e % 4 of row l % 32
  if constexpr (SPLIT) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t m = m0 + wm * TM + 32 * i + l32;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int n = n0 + wn * TN + 32 * j + 8 * g + 4 * half;
          if (m < a.M && n < a.N)
            *reinterpret_cast<int4_t*>(a.part + (blockIdx.y * a.M + m) * a.N + n) =
                int4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        }
    }
    return;
  }
  // 32 rows at a time through the wavefront's own LDS, so that a lane gets eight outputs of a row
  // and sixteen (or eight, or four) lanes a whole line; rows are 4 floats apart from the banks'
  // period. A lane's columns stay the same: their scales and biases are read once, and the
  // factors and residuals of all 32 rows are on their way while the sums go through LDS.
  constexpr int LANES = TN / 8, RUNS = LANES / 2;
  float* mine = reinterpret_cast<float*>(lds) + wave * 32 * PITCH;
  const int c = 8 * (lane % LANES), n = n0 + wn * TN + c;
  const bool in = n < a.N;
  float8_t sw = {}, bias = {};
  if (in) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[e] = channel_factor(a.scales[n + e]);
    if (a.bias != nullptr) bias = load8<T>(a.bias + n);
  }
  float sx[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm * TM + 32 * i + l32;
    sx[i] = m < a.M ? row_factor(a.scale[m]) : 0.0f;
  }
  if constexpr (TEAMS == 1) __syncthreads();  // all wavefronts have read their last operands
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t top = m0 + wm * TM + 32 * i + lane / LANES;
    uint4 f[RUNS], r[RUNS];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t m = top + k * (64 / LANES), o = m * a.N + n;
      f[k] = r[k] = make_uint4(0, 0, 0, 0);
      if (a.mul != nullptr && in && m < a.M) f[k] = *reinterpret_cast<const uint4*>(a.mul + o);
      if (a.residual != nullptr && in && m < a.M) r[k] = *reinterpret_cast<const uint4*>(a.residual + o);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[i][j][4 * g + e]) * sx[i];
        *reinterpret_cast<float4_t*>(mine + l32 * PITCH + 32 * j + 8 * g + 4 * half) = v;
      }
    wave_lds_fence();
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const float* from = mine + (k * (64 / LANES) + lane / LANES) * PITCH + c;
      const float4_t lo = *reinterpret_cast<const float4_t*>(from), hi = *reinterpret_cast<const float4_t*>(from + 4);
      const int64_t m = top + k * (64 / LANES);
      if (in && m < a.M)
        *reinterpret_cast<uint4*>(a.y + m * a.N + n) =
            tail8<T>(a, float8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]} * sw + bias, f[k], r[k]);
    }
    wave_lds_fence();
  }
}

// the sums of a split of the channels, eight outputs for each thread
template <typename T>
__global__ void __launch_bounds__(256) i8_sum_kernel(I8Args a, int splits) {
  const int64_t runs = a.M * a.N / 8, all = a.M * a.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < runs; i += static_cast<int64_t>(gridDim.x) * 256) {
    int4_t lo = {0, 0, 0, 0}, hi = lo;
    for (int s = 0; s < splits; s += 4) {  // four at a time on their way
      int4_t v[4][2];
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const int4_t* p = reinterpret_cast<const int4_t*>(a.part + min(s + o, splits - 1) * all + 8 * i);
        v[o][0] = p[0];
        v[o][1] = p[1];
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        lo += s + o < splits ? v[o][0] : int4_t{0, 0, 0, 0};
        hi += s + o < splits ? v[o][1] : int4_t{0, 0, 0, 0};
      }
    }
    const int64_t m = 8 * i / a.N, n = 8 * i - m * a.N;
    const float sx = row_factor(a.scale[m]);
    float8_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = static_cast<float>(lo[e]) * sx * channel_factor(a.scales[n + e]);
      v[e + 4] = static_cast<float>(hi[e]) * sx * channel_factor(a.scales[n + 4 + e]);
    }
    if (a.bias != nullptr) v += load8<T>(a.bias + n);
    uint4 f = make_uint4(0, 0, 0, 0), r = f;
    if (a.mul != nullptr) f = *reinterpret_cast<const uint4*>(a.mul + 8 * i);
    if (a.residual != nullptr) r = *reinterpret_cast<const uint4*>(a.residual + 8 * i);
    *reinterpret_cast<uint4*>(a.y + 8 * i) = tail8<T>(a, v, f, r);
  }
}

// Which kernel a product takes: the one with the least time by an estimate in microseconds, whose
// constants were fitted (by least squares of the logarithms, 10 % rms) to 2400 timings of all
// kernels and splits at M = 17 .. 4096 and seven layers from 512 x 2048 to 14336 x 4096. Only the order of
// its times matters: they lie 3 to 26 % below what the kernels take now (2048 x 14336 x 4096 104 us for 122
// to 130, 4096 x 4096 x 14336 164 for 207, 64 x 14336 x 4096 10.1 for 13.7, 333 x 4096 x 11008 30.2 for 31.2). Over
// those sizes the choice costs 2.6 % more than the best one on average, 33 % at worst (33 x 8192 x
// 1024: 6.5 us, 4.9); a fit of its own to the 1765 timings that say so would cost 2.5 %.
// A CU's blocks share its matrix cores (`work` each and step) and pass their steps not faster than
// memory answers (`wait`, `fit` of them at a time). Two teams win where 64 x 64 tiles leave CUs to
// spare (200 x 4096 x 4096: 10.9 us, one team 12.9); with larger tiles they gained 2 % at most.
struct Tile {
  int bm, bn, teams, fit;
  float work, wait, once;
};
constexpr Tile kTiles[] = {{64, 64, 1, 5, 0.106f, 0.131f, 0.52f},
                           {64, 128, 1, 3, 0.153f, 0.143f, 0.97f},
                           {128, 128, 1, 2, 0.215f, 0.231f, 1.69f},
                           {128, 256, 1, 2, 0.345f, 0.370f, 3.12f},
                           {64, 64, 2, 2, 0.191f, 0.178f, 1.11f}};
constexpr int kKinds = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 16};
struct Choice {
  int tile, splits;  // tile -1: i8_rows_kernel
};
Choice choose(int64_t M, int64_t N, int64_t K) {
  if (const char* env = tuning_env("AWQ_I8_CFG")) {
    int bm = 0, bn = 0, splits = 0, teams = 1;
    if (sscanf(env, "%d,%d,%d,%d", &bm, &bn, &splits, &teams) >= 3) {
      for (int t = 0; t < kKinds; ++t)
        if (kTiles[t].bm == bm && kTiles[t].bn == bn && kTiles[t].teams == teams) return {t, splits};
      return {-1, 1};
    }
  }
  // few rows: 14336 x 4096 of one row 10.8 us, the best tiles 12.5; 8192 x 14336 of four 19.4 and 24.6
  if (M <= 8) return {-1, 1};
  constexpr float kCus = 256.0f;
  const float units = static_cast<float>((K + kI8Unit - 1) / kI8Unit), m = static_cast<float>(M), n = static_cast<float>(N);
  auto blocks = [](int64_t v, int64_t b) { return static_cast<float>((v + b - 1) / b); };
  const int row_blocks = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const float rounds = blocks(N, 16) * blocks(M, 16 * row_blocks) / kCus;
  Choice best = {-1, 1};
  float least = 2.4f + units / 8.0f * (rounds > 1.0f ? rounds : 1.0f) *
                           (0.31f + 0.19f * (m / 16.0f < row_blocks ? m / 16.0f : static_cast<float>(row_blocks)));
  for (int t = 0; t < kKinds; ++t)
    for (int splits : kSplits) {
      const Tile& k = kTiles[t];
      if (splits > 1 && units < 2.0f * splits * k.teams) break;
      const float per_cu = ceilf(blocks(M, k.bm) * blocks(N, k.bn) * splits / kCus), steps = ceilf(units / (splits * k.teams));
      const float waits = k.wait * ceilf(per_cu / k.fit), works = k.work * per_cu;
      float time = 2.87f + steps * (waits > works ? waits : works) + k.once * per_cu;
      if (splits > 1) time += 1.86f + 0.11f * splits + (8.0f * splits + 2.0f) * m * n / 5.4e6f;
      if (time < least) {
        least = time;
        best = {t, splits};
      }
    }
  return best;
}

template <typename T, int BM, int BN, int TEAMS>
hipError_t launch_tiles(const I8Args& a, int splits, hipStream_t st) {
  constexpr int STAGES = TEAMS * stages(BM, BN);
  constexpr int TAIL = 4 * 32 * (BN / 2 + 4) * 4 + (TEAMS > 1 ? BM * BN * 4 : 0), LDS = STAGES > TAIL ? STAGES : TAIL;
  static_assert(LDS <= 163840, "a CU's LDS");
  const unsigned blocks = static_cast<unsigned>((a.M + BM - 1) / BM * ((a.N + BN - 1) / BN));
  auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
    const hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kernel), LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(blocks, splits), dim3(256 * TEAMS), LDS, st, a);
    return hipGetLastError();
  };
  static std::atomic<uint64_t> whole{0}, split{0};
  if (splits == 1) return go(&i8_tile_kernel<T, BM, BN, TEAMS, false>, whole);
  hipError_t e = go(&i8_tile_kernel<T, BM, BN, TEAMS, true>, split);
  if (e != hipSuccess) return e;
  int64_t sums = (a.M * a.N / 8 + 255) / 256;
  if (sums > 65536) sums = 65536;
  hipLaunchKernelGGL((i8_sum_kernel<T>), dim3(static_cast<unsigned>(sums)), dim3(256), 0, st, a, splits);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_as(const I8Args& a, hipStream_t st) {
  const Choice c = choose(a.M, a.N, a.K);
  switch (c.tile) {
    case 0: return launch_tiles<T, 64, 64, 1>(a, c.splits, st);
    case 1: return launch_tiles<T, 64, 128, 1>(a, c.splits, st);
    case 2: return launch_tiles<T, 128, 128, 1>(a, c.splits, st);
    case 3: return launch_tiles<T, 128, 256, 1>(a, c.splits, st);
    case 4: return launch_tiles<T, 64, 64, 2>(a, c.splits, st);
    default: break;
  }
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

size_t gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const Choice c = choose(M, N, K);
  return c.splits == 1 ? 0 : static_cast<size_t>(4) * c.splits * M * N;
}

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
  a.part = static_cast<int32_t*>(p.ws);
  a.M = p.M;
  a.N = p.N;
  a.q_stride = p.q_stride;
  a.K = static_cast<int>(p.K);
  a.units = static_cast<int>(l.units);
  a.act = p.act;
  return p.dtype == AWQ_DT_F16 ? launch_as<F16>(a, st) : launch_as<BF16>(a, st);
}

}  // namespace awq
