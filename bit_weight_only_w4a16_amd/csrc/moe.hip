// A layer of gated W4A16 experts for a few tokens:
//
//   a[t, j] = binary16(act(Wg[e] x_t) * (Wu[e] x_t) * inv_down[e]),  e = ids[t][j]
//   y[t]    = residual[t] + sum_j weights[t][j] Wd[e] a[t, j]
//
// Bound by memory: each expert that some token names is read once. Which experts those are is
// known on the device alone, so the first launch has workgroups for as many experts as the
// ids could name (those past the last named one end at once), and each finds its expert as the
// n-th set bit of the bits that the ids set. In the second a workgroup owns 16 outputs of all
// tokens and walks over the named experts' rows, its wavefronts taking equal runs of units, so
// that its load does not depend on how many experts there are.
//
// Weights go from memory to registers, 1 KiB per load (awq_repack's units), are dequantized
// exactly to binary16 and meet up to 16 tokens' rows in one matrix instruction. A wavefront keeps
// its own sums; they are added in the wavefronts' order, so results do not vary.
#include "ffn_internal.hpp"

namespace awq {
namespace {

constexpr int kMostExperts = 1024, kMoeWaves = 8;

struct Layers {  // a stack of packed layers
  const uint8_t* base;
  int64_t bytes, scales_off, zeros_off;  // zeros_off -1: symmetric
};

struct MoeArgs {
  const uint16_t *x, *inv_in, *inv_down, *residual;
  const int32_t* ids;
  const float* weights;
  Layers gate, up, down;
  uint16_t* mid;  // [tokens * k][ffn]
  uint16_t* y;
  int64_t x_stride, residual_stride, y_stride, inv_in_stride, inv_down_stride;
  int tokens, hidden, ffn, experts, k, sets, act;
};

// The experts that the ids name, as bits in LDS; all threads of a workgroup take part.
__device__ __forceinline__ void find_named(const MoeArgs& a, uint32_t* bits) {
  for (int i = threadIdx.x; i < kMostExperts / 32; i += blockDim.x) bits[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * a.k; i += blockDim.x) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// This lane's word of the bits (lanes 0 .. 31), and how many bits lie in lanes before it.
struct Named {
  uint32_t word;
  int before, total;
};
__device__ __forceinline__ Named count_named(const uint32_t* bits) {
  const int lane = threadIdx.x & 63;
  Named n;
  n.word = lane < kMostExperts / 32 ? bits[lane] : 0u;
  const int mine = __popc(n.word);
  int upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int other = __shfl_up(upto, s);
    if (lane >= s) upto += other;
  }
  n.total = __shfl(upto, 31);
  n.before = upto - mine;
  return n;
}

// The tokens that name expert e, as bits (token t is lane t's); for lane t, the first j with
// ids[t][j] == e and the sum of the weights of all such j.
struct Rows {
  uint64_t tokens;
  int pair;
  float weight;
};
__device__ __forceinline__ Rows rows_of(const MoeArgs& a, int e) {
  const int t = threadIdx.x & 63;
  Rows r = {0, -1, 0.0f};
  if (t < a.tokens) {
    for (int j = a.k - 1; j >= 0; --j) {
      if (a.ids[t * a.k + j] != e) continue;
      r.pair = t * a.k + j;
      r.weight += a.weights[t * a.k + j];
    }
  }
  r.tokens = __ballot(r.pair >= 0);
  return r;
}

// One unit's words, scale and zero word of this lane.
struct Piece {
  uint4 c;
  uint16_t s;
  uint32_t z;
};
template <bool ASYM>
__device__ __forceinline__ Piece load_piece(const Layers& l, int64_t layer, int64_t unit, int sets, int lane) {
  const int r = lane & 15, set = lane_set(lane >> 4, sets);
  const uint8_t* base = l.base + layer * l.bytes;
  Piece p;
  typedef unsigned int u4 __attribute__((ext_vector_type(4)));
  const u4 c = __builtin_nontemporal_load(reinterpret_cast<const u4*>(base + unit * kUnitBytes) + lane);
  p.c = make_uint4(c[0], c[1], c[2], c[3]);
  p.s = reinterpret_cast<const uint16_t*>(base + l.scales_off)[(unit * sets + set) * kTileN + r];
  p.z = ASYM ? reinterpret_cast<const uint32_t*>(base + l.zeros_off)[(unit * sets + set) * 2 + (r >> 3)] : 0u;
  return p;
}

// acc += rows (four operands of 8 channels each) . the unit's weights
struct Dequant {
  half2_t scale;
  uint32_t nz1024, nz64;
};
template <bool ASYM>
__device__ __forceinline__ Dequant constants(const Piece& p, int lane) {
  const uint32_t z = ASYM ? (p.z >> (4 * (lane & 7))) & 15u : 8u;
  return {as_h2(p.s | static_cast<uint32_t>(p.s) << 16), neg_off1024(z), neg_off64(z)};
}
__device__ __forceinline__ half8_t weights8(const Piece& p, int i, const Dequant& d) {
  half2_t q[4];
  dequant_word(i == 0 ? p.c.x : i == 1 ? p.c.y : i == 2 ? p.c.z : p.c.w, d.nz1024, d.nz64, d.scale, q);
  return half8_t{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
}

// grid: tiles of 16 ffn outputs, experts that may be named
template <bool ASYM>
__global__ void __launch_bounds__(64 * kMoeWaves) moe_up_kernel(MoeArgs a) {
  __shared__ uint32_t bits[kMostExperts / 32];
  __shared__ int row_pair[64];
  __shared__ float red[kMoeWaves][2][16][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, p = lane >> 4;
  find_named(a, bits);
  const Named named = count_named(bits);
  const int slot = blockIdx.y;
  if (slot >= named.total) return;
  const uint64_t holds = __ballot(named.before <= slot && slot < named.before + __popc(named.word));
  const int word_at = __builtin_ctzll(holds);
  uint32_t word = __shfl(named.word, word_at);
  for (int skip = slot - __shfl(named.before, word_at); skip > 0; --skip) word &= word - 1;
  const int e = __builtin_amdgcn_readfirstlane(32 * word_at + __builtin_ctz(word));
  const Rows rows = rows_of(a, e);
  const int count = __popcll(rows.tokens);
  if (wave == 0 && rows.pair >= 0) row_pair[__popcll(rows.tokens & ((uint64_t{1} << lane) - 1))] = rows.pair;
  __syncthreads();

  const int64_t tile = blockIdx.x;
  const int units = a.hidden / kGroup;
  const uint16_t* inv = a.inv_in == nullptr ? nullptr : a.inv_in + e * a.inv_in_stride + 32 * p;
  for (int m0 = 0; m0 < count; m0 += 16) {
    const bool live = m0 + r < count;
    const uint16_t* x = a.x + (live ? row_pair[m0 + r] / a.k : 0) * a.x_stride + 32 * p;
    float4_t g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
    if (wave < units) {
      Piece pg = load_piece<ASYM>(a.gate, e, tile * units + wave, a.sets, lane);
      Piece pu = load_piece<ASYM>(a.up, e, tile * units + wave, a.sets, lane);
      for (int at = wave; at < units; at += kMoeWaves) {
        const Piece cg = pg, cu = pu;
        if (at + kMoeWaves < units) {
          pg = load_piece<ASYM>(a.gate, e, tile * units + at + kMoeWaves, a.sets, lane);
          pu = load_piece<ASYM>(a.up, e, tile * units + at + kMoeWaves, a.sets, lane);
        }
        uint4 xv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xv[i] = make_uint4(0, 0, 0, 0);
          if (live) xv[i] = *reinterpret_cast<const uint4*>(x + at * kGroup + 8 * i);
        }
        if (inv != nullptr) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xv[i] = scale_x8(xv[i], *reinterpret_cast<const uint4*>(inv + at * kGroup + 8 * i));
        }
        const Dequant dg = constants<ASYM>(cg, lane), du = constants<ASYM>(cu, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const half8_t xf = __builtin_bit_cast(half8_t, xv[i]);
          g = __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, weights8(cg, i, dg), g, 0, 0, 0);
          u = __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, weights8(cu, i, du), u, 0, 0, 0);
        }
      }
    }
    __syncthreads();  // the sums of the rows before these have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[wave][0][4 * p + j][r] = g[j];
      red[wave][1][4 * p + j][r] = u[j];
    }
    __syncthreads();
    const int m = threadIdx.x / 16, n = threadIdx.x % 16;
    if (m < 16 && m0 + m < count) {
      float sg = 0.0f, su = 0.0f;
#pragma unroll
      for (int w = 0; w < kMoeWaves; ++w) {
        sg += red[w][0][m][n];
        su += red[w][1][m][n];
      }
      const int f = static_cast<int>(tile) * kTileN + n;
      float v = activate(sg, a.act) * su;
      if (a.inv_down != nullptr) v *= f16_to_f32(a.inv_down[e * a.inv_down_stride + f]);
      a.mid[static_cast<int64_t>(row_pair[m0 + m]) * a.ffn + f] =
          __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
  }
}

// grid: tiles of 16 hidden outputs. Dynamic LDS: [waves][tokens][16] float32.
template <bool ASYM>
__global__ void __launch_bounds__(64 * kMoeWaves) moe_down_kernel(MoeArgs a) {
  __shared__ uint32_t bits[kMostExperts / 32];
  __shared__ uint16_t named_list[kMostExperts];
  __shared__ int row_pair[kMoeWaves][64];
  __shared__ float row_weight[kMoeWaves][64];
  extern __shared__ float sums[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, p = lane >> 4;
  float* mine = sums + wave * a.tokens * 16;
  for (int i = lane; i < a.tokens * 16; i += 64) mine[i] = 0.0f;
  find_named(a, bits);
  const Named named = count_named(bits);
  if (wave == 0) {
    uint32_t word = named.word;
    for (int at = named.before; word != 0; ++at, word &= word - 1)
      named_list[at] = static_cast<uint16_t>(32 * lane + __builtin_ctz(word));
  }
  __syncthreads();

  const int64_t tile = blockIdx.x;
  const int units = a.ffn / kGroup, all = __builtin_amdgcn_readfirstlane(named.total) * units;
  int at = static_cast<int>(static_cast<int64_t>(all) * wave / kMoeWaves);
  const int end = static_cast<int>(static_cast<int64_t>(all) * (wave + 1) / kMoeWaves);
  while (at < end) {
    const int slot = at / units, e = __builtin_amdgcn_readfirstlane(named_list[slot]);
    const int first = at - slot * units, last = min(units, end - slot * units);
    at = slot * units + last;
    const Rows rows = rows_of(a, e);
    const int count = __popcll(rows.tokens);
    wave_lds_fence();  // the rows of the expert before have been read
    if (rows.pair >= 0) {
      const int row = __popcll(rows.tokens & ((uint64_t{1} << lane) - 1));
      row_pair[wave][row] = rows.pair;
      row_weight[wave][row] = rows.weight;
    }
    wave_lds_fence();
    for (int m0 = 0; m0 < count; m0 += 16) {
      const bool live = m0 + r < count;
      const uint16_t* x = a.mid + static_cast<int64_t>(live ? row_pair[wave][m0 + r] : 0) * a.ffn + 32 * p;
      float4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
      Piece next = load_piece<ASYM>(a.down, e, tile * units + first, a.sets, lane);
      for (int u = first; u < last; ++u) {
        const Piece c = next;
        if (u + 1 < last) next = load_piece<ASYM>(a.down, e, tile * units + u + 1, a.sets, lane);
        const Dequant dq = constants<ASYM>(c, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 xv = make_uint4(0, 0, 0, 0);
          if (live) xv = *reinterpret_cast<const uint4*>(x + u * kGroup + 8 * i);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, xv), weights8(c, i, dq), d, 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + 4 * p + j;
        if (m < count) mine[row_pair[wave][m] / a.k * 16 + r] += row_weight[wave][m] * d[j];
      }
      wave_lds_fence();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * 16; i += 64 * kMoeWaves) {
    const int t = i / 16, n = static_cast<int>(tile) * 16 + i % 16;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) v += sums[w * a.tokens * 16 + i];
    if (a.residual != nullptr) v += f16_to_f32(a.residual[t * a.residual_stride + n]);
    a.y[t * a.y_stride + n] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
}

Layers make_layers(const void* base, int64_t N, int64_t K, int32_t group, int32_t fmt) {
  const PackedLayout l = make_layout(N, K, group, fmt);
  return {static_cast<const uint8_t*>(base), l.total_bytes, l.scales_off, l.zeros_off};
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int32_t, int32_t ffn, int32_t k) {
  return static_cast<size_t>(2) * tokens * k * ffn;
}

hipError_t launch_moe(const awq_moe_args& p, hipStream_t st) {
  MoeArgs a;
  a.x = p.x;
  a.inv_in = p.inv_in;
  a.inv_down = p.inv_down;
  a.residual = p.residual;
  a.ids = p.ids;
  a.weights = p.weights;
  a.gate = make_layers(p.gate, p.ffn, p.hidden, p.group, p.fmt);
  a.up = make_layers(p.up, p.ffn, p.hidden, p.group, p.fmt);
  a.down = make_layers(p.down, p.hidden, p.ffn, p.group, p.fmt);
  a.mid = static_cast<uint16_t*>(p.ws);
  a.y = p.y;
  a.x_stride = p.x_stride;
  a.residual_stride = p.residual_stride;
  a.y_stride = p.y_stride;
  a.inv_in_stride = p.inv_in_stride;
  a.inv_down_stride = p.inv_down_stride;
  a.tokens = static_cast<int>(p.tokens);
  a.hidden = p.hidden;
  a.ffn = p.ffn;
  a.experts = p.experts;
  a.k = p.k;
  a.sets = p.group < kGroup ? kGroup / p.group : 1;
  a.act = p.act;
  const int64_t pairs = p.tokens * p.k;
  const int slots = static_cast<int>(pairs < p.experts ? pairs : p.experts);
  const bool asym = p.fmt == AWQ_FMT_ASYM;
  hipLaunchKernelGGL((asym ? &moe_up_kernel<true> : &moe_up_kernel<false>), dim3(p.ffn / kTileN, slots),
                     dim3(64 * kMoeWaves), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((asym ? &moe_down_kernel<true> : &moe_down_kernel<false>), dim3(p.hidden / kTileN),
                     dim3(64 * kMoeWaves), static_cast<size_t>(4) * kMoeWaves * a.tokens * 16, st, a);
  return hipGetLastError();
}

}  // namespace awq
