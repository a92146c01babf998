// A layer of gated W4A16 experts for a few tokens:
//
//   a[t, j] = binary16(act(Wg[e] x_t) * (Wu[e] x_t) * inv_down[e]),  e = ids[t][j]
//   y[t]    = residual[t] + sum_j weights[t][j] Wd[e] a[t, j]
//
// Bound by memory: each expert that some token names is read once. Which experts those are is
// known on the device alone, so the first launch has workgroups for as many experts as the
// ids could name (those past the last named one end at once), and each finds its expert as the
// n-th set bit of the bits that the ids set. One workgroup of that launch writes the plan of the
// second: the named experts and their tokens in order. There a workgroup owns 32 outputs of all
// tokens and walks over the named experts, its wavefronts taking equal shares of their units, so
// that its load does not depend on how many experts there are; with few outputs, several
// workgroups share them, and the one that ends last adds their sums.
//
// Weights go from memory to registers, 1 KiB per load (awq_repack's units), ahead of their use; they
// are dequantized exactly to binary16 and meet up to 16 tokens' rows in one matrix instruction. Every
// sum has its place and order: results do not vary. Measured: one token through two of eight experts
// of 4096 x 14336 44.5 us (183 MB, 4.1 TB/s), 48 tokens over 64 experts of 4096 x 1536 138 us (628 MB,
// 4.5 TB/s); beside memory, dequantization issues vector instructions 30 to 50 % of the time.
#include "ffn_internal.hpp"

#include <type_traits>

namespace awq {
namespace {

constexpr int kMostExperts = 1024, kMostPairs = AWQ_MOE_MAX_TOKENS * AWQ_MOE_MAX_K;
constexpr int kUpWaves = 4, kDownWaves = 16, kDownWide = 2, kAheadW = 2;
// Rows of an expert that a wavefront has sums for at a time: chunks of 16, one for up to 16 tokens,
// else two (four, for 64 tokens, left two wavefronts on a SIMD); an expert of more tokens is read
// again for them.
constexpr int kChunks = 2;
constexpr int kMostRuns = kMostExperts + kMostPairs / (16 * kChunks);

struct Layers {  // a stack of packed layers
  const uint8_t* base;
  int64_t bytes;
  uint32_t scales_off, zeros_off;
};

// What the first launch tells the second (in the workspace).
struct Plan {
  int32_t* total;    // runs: a named expert with up to 16 CHUNKS of its tokens
  int32_t* experts;  // [pairs]: a run's expert, ascending
  int32_t* first;    // [pairs + 1]: where a run's tokens begin in the next two
  int32_t* pair;     // [pairs]: token * k + j
  float* weight;     // [pairs]
  int32_t* ended;    // [tiles]: workgroups that have written their sums
  float* part;       // [splits][tiles][tokens * 16]
};

struct MoeArgs {
  const uint16_t *x, *inv_in, *inv_down, *residual;
  const int32_t* ids;
  const float* weights;
  Layers gate, up, down;
  uint16_t* mid;  // [tokens * k][ffn]
  Plan plan;
  uint16_t* y;
  int64_t x_stride, residual_stride, y_stride, inv_in_stride, inv_down_stride;
  int tokens, hidden, ffn, experts, k, sets, act;
};

// The ids in LDS (-1 where they name no expert), and the experts that they name as bits; all
// threads of a workgroup take part.
__device__ __forceinline__ void find_named(const MoeArgs& a, int* ids, uint32_t* bits) {
  if (threadIdx.x < kMostExperts / 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * a.k; i += blockDim.x) {
    const int e = a.ids[i];
    const bool named = e >= 0 && e < a.experts;
    ids[i] = named ? e : -1;
    if (named) atomicOr(&bits[e >> 5], 1u << (e & 31));
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
// ids[t][j] == e.
struct Rows {
  uint64_t tokens;
  int pair;
};
__device__ __forceinline__ Rows rows_of(const MoeArgs& a, const int* ids, int e) {
  const int t = threadIdx.x & 63;
  Rows r = {0, -1};
  if (t < a.tokens)
    for (int j = a.k - 1; j >= 0; --j)
      if (ids[t * a.k + j] == e) r.pair = t * a.k + j;
  r.tokens = __ballot(r.pair >= 0);
  return r;
}

// One unit's words, scale and zero word of this lane; nothing is read where `skip` is kNoLoad.
struct Piece {
  uint4 c;
  uint32_t s, z;
};
struct Reader {  // a layer's regions of one tile of 16 outputs
  __amdgpu_buffer_rsrc_t all;
  uint32_t codes, scales, zeros;  // offsets of unit 0
};
__device__ __forceinline__ Reader reader(const Layers& l, int e, int tile, int units, int sets) {
  const uint32_t first = static_cast<uint32_t>(tile) * units;
  return {make_rsrc(l.base + e * l.bytes, static_cast<uint32_t>(l.bytes)), first * kUnitBytes,
          l.scales_off + first * (2 * kTileN * sets), l.zeros_off + first * (8 * sets)};
}
template <bool ASYM>
__device__ __forceinline__ Piece load_piece(const Reader& r, int unit, int sets, int lane, uint32_t skip) {
  const uint32_t set = lane_set(lane >> 4, sets), u = static_cast<uint32_t>(unit);
  Piece p;
  p.c = buf_load16_stream(r.all, 16u * lane + skip, r.codes + u * kUnitBytes);
  p.s = buf_load2(r.all, 2u * (kTileN * set + (lane & 15)) + skip, r.scales + u * (2 * kTileN * sets));
  p.z = ASYM ? buf_load4(r.all, 4u * (2 * set + ((lane & 15) >> 3)) + skip, r.zeros + u * (8 * sets)) : 0u;
  return p;
}
struct Dequant {
  half2_t scale;
  uint32_t nz1024, nz64;
};
template <bool ASYM>
__device__ __forceinline__ Dequant constants(const Piece& p, int lane) {
  const uint32_t z = ASYM ? (p.z >> (4 * (lane & 7))) & 15u : 8u;
  return {as_h2(p.s | p.s << 16), neg_off1024(z), neg_off64(z)};
}
__device__ __forceinline__ half8_t weights8(const Piece& p, int i, const Dequant& d) {
  half2_t q[4];
  dequant_word(i == 0 ? p.c.x : i == 1 ? p.c.y : i == 2 ? p.c.z : p.c.w, d.nz1024, d.nz64, d.scale, q);
  return half8_t{q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
}
__device__ __forceinline__ half8_t load_half8(const uint16_t* p) {
  return __builtin_bit_cast(half8_t, *reinterpret_cast<const uint4*>(p));
}

// The plan, by one workgroup. An expert's tokens stand in their own order: which of more than 16 CHUNKS
// are a run decides where their sums are cut. (Their LDS leaves room for four workgroups on a CU.)
__device__ __forceinline__ void write_plan(const MoeArgs& a, const int* ids, const uint32_t* bits, const Named& named,
                                           int tiles, int most_rows) {
  static_assert(kMostExperts <= 65536 && kMostPairs <= 65536, "16 bits each");
  __shared__ int before[kMostExperts / 32];
  __shared__ uint16_t who[kMostExperts], begin[kMostExperts];
  __shared__ unsigned long long tokens[kMostExperts];  // those that name the expert, as bits
  const int lane = threadIdx.x & 63, pairs = a.tokens * a.k;
  if (threadIdx.x < kMostExperts / 32) {
    before[lane] = named.before;
    uint32_t word = named.word;
    for (int at = named.before; word != 0; ++at, word &= word - 1)
      who[at] = static_cast<uint16_t>(32 * lane + __builtin_ctz(word));
  }
  for (int i = threadIdx.x; i < named.total; i += blockDim.x) tokens[i] = 0;
  for (int i = threadIdx.x; i < tiles; i += blockDim.x) a.plan.ended[i] = 0;
  __syncthreads();
  // an expert's place among the named ones
  auto place = [&](int e) {
    return before[e >> 5] + static_cast<int>(__popc(bits[e >> 5] & ((1u << (e & 31)) - 1)));
  };
  for (int i = threadIdx.x; i < pairs; i += blockDim.x)
    if (ids[i] >= 0) atomicOr(&tokens[place(ids[i])], 1ull << (i / a.k));
  __syncthreads();
  if (threadIdx.x < 64) {  // sums over the experts before one: of tokens (low half) and of runs
    int base = 0;
    for (int i0 = 0; i0 < named.total; i0 += 64) {
      const int rows = i0 + lane < named.total ? __popcll(tokens[i0 + lane]) : 0;
      const int runs = (rows + most_rows - 1) / most_rows, mine = rows | runs << 16;
      int upto = mine;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const int other = __shfl_up(upto, s);
        if (lane >= s) upto += other;
      }
      const int from = base + upto - mine;
      if (i0 + lane < named.total) {
        begin[i0 + lane] = static_cast<uint16_t>(from);
        for (int n = 0; n < runs; ++n) {
          a.plan.experts[(from >> 16) + n] = who[i0 + lane];
          a.plan.first[(from >> 16) + n] = (from & 0xFFFF) + n * most_rows;
        }
      }
      base += __shfl(upto, 63);
    }
    if (lane == 0) {
      a.plan.first[base >> 16] = base & 0xFFFF;
      *a.plan.total = base >> 16;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = ids[i], t = i / a.k;
    bool again = e < 0;  // an earlier j of the token names the expert
    for (int j = t * a.k; j < i; ++j) again |= ids[j] == e;
    if (again) continue;
    const int at = place(e), to = begin[at] + __popcll(tokens[at] & ((1ull << t) - 1));
    float weight = a.weights[i];
    for (int j = i + 1; j < (t + 1) * a.k; ++j)
      if (ids[j] == e) weight += a.weights[j];
    a.plan.pair[to] = i;
    a.plan.weight[to] = weight;
  }
}

// A workgroup owns WIDE tiles of 16 ffn outputs of one expert; its four wavefronts take every fourth
// unit each, and a unit's rows serve all tiles (with one tile each, the rows' loads took a fifth to a
// quarter of the time). grid: the outputs' workgroups and one for the plan, experts that may be named
template <bool ASYM, int WIDE, int CHUNKS>
__global__ void __launch_bounds__(64 * kUpWaves) moe_up_kernel(MoeArgs a) {
  __shared__ uint32_t bits[kMostExperts / 32];
  __shared__ int ids[kMostPairs];
  __shared__ int row_pair[64];
  __shared__ float4_t red[kUpWaves][WIDE][2][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, p = lane >> 4;
  const int slot = blockIdx.y;
  const bool plans = blockIdx.x == gridDim.x - 1;
  if (plans && slot != 0) return;
  find_named(a, ids, bits);
  const Named named = count_named(bits);
  if (plans) {
    write_plan(a, ids, bits, named, a.hidden / kTileN, 16 * CHUNKS);
    return;
  }
  if (slot >= named.total) return;
  const uint64_t holds = __ballot(named.before <= slot && slot < named.before + __popc(named.word));
  const int word_at = __builtin_ctzll(holds);
  uint32_t word = __shfl(named.word, word_at);
  for (int skip = slot - __shfl(named.before, word_at); skip > 0; --skip) word &= word - 1;
  const int e = __builtin_amdgcn_readfirstlane(32 * word_at + __builtin_ctz(word));

  const int units = a.hidden / kGroup, tile0 = blockIdx.x * WIDE;
  Reader rg[WIDE], ru[WIDE];
#pragma unroll
  for (int t = 0; t < WIDE; ++t) {
    rg[t] = reader(a.gate, e, tile0 + t, units, a.sets);
    ru[t] = reader(a.up, e, tile0 + t, units, a.sets);
  }
  Piece pg[WIDE], pu[WIDE];
  auto load = [&](int unit) {
    const uint32_t skip = unit < units ? 0u : kNoLoad;
#pragma unroll
    for (int t = 0; t < WIDE; ++t) {
      pg[t] = load_piece<ASYM>(rg[t], unit, a.sets, lane, skip);
      pu[t] = load_piece<ASYM>(ru[t], unit, a.sets, lane, skip);
    }
  };
  load(wave);

  const Rows rows = rows_of(a, ids, e);
  const int all_rows = __popcll(rows.tokens);
  if (wave == 0 && rows.pair >= 0) row_pair[__popcll(rows.tokens & ((uint64_t{1} << lane) - 1))] = rows.pair;
  __syncthreads();
  const uint16_t* inv = a.inv_in == nullptr ? nullptr : a.inv_in + e * a.inv_in_stride + 32 * p;
  auto load_x = [&](const uint16_t* from, int unit, half8_t (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = load_half8(from + unit * kGroup + 8 * i);
      if (inv != nullptr) f[i] *= load_half8(inv + unit * kGroup + 8 * i);
    }
  };
  for (int row0 = 0; row0 < all_rows; row0 += 16 * CHUNKS) {
    if (row0 > 0) load(wave);
    // rows past the last repeat it; their results are dropped
    const int count = min(all_rows - row0, 16 * CHUNKS), chunks = (count + 15) / 16;
    const uint16_t* x[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) x[c] = a.x + row_pair[row0 + min(16 * c + r, count - 1)] / a.k * a.x_stride + 32 * p;
    float4_t g[CHUNKS][WIDE], u[CHUNKS][WIDE];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int t = 0; t < WIDE; ++t) g[c][t] = u[c][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

    // One unit ahead: four wavefronts on a SIMD hide more than two whose registers hold more units
    // (one token through two of eight experts, this launch: 25 us, with two units ahead 27, three 32).
    for (int at = wave; at < units; at += kUpWaves) {
      half8_t f[CHUNKS][4];
      load_x(x[0], at, f[0]);
#pragma unroll
      for (int c = 1; c < CHUNKS; ++c)
        if (c < chunks) load_x(x[c], at, f[c]);
#pragma unroll
      for (int t = 0; t < WIDE; ++t) {
        const Dequant dg = constants<ASYM>(pg[t], lane), du = constants<ASYM>(pu[t], lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const half8_t wg = weights8(pg[t], i, dg), wu = weights8(pu[t], i, du);
          g[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[0][i], wg, g[0][t], 0, 0, 0);
          u[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[0][i], wu, u[0][t], 0, 0, 0);
#pragma unroll
          for (int c = 1; c < CHUNKS; ++c) {
            if (c >= chunks) break;
            g[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[c][i], wg, g[c][t], 0, 0, 0);
            u[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[c][i], wu, u[c][t], 0, 0, 0);
          }
        }
      }
      load(at + kUpWaves);
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (c >= chunks) break;
      if (c > 0 || row0 > 0) __syncthreads();  // the sums of the rows before these have been read
#pragma unroll
      for (int t = 0; t < WIDE; ++t) {
        red[wave][t][0][lane] = g[c][t];
        red[wave][t][1][lane] = u[c][t];
      }
      __syncthreads();
      if (wave < WIDE) {  // a wavefront for each tile
        const int t = wave;
        float4_t sg = red[0][t][0][lane], su = red[0][t][1][lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
          sg += red[w][t][0][lane];
          su += red[w][t][1][lane];
        }
        const int out = (tile0 + t) * kTileN + r;
        const float scale = a.inv_down == nullptr ? 1.0f : f16_to_f32(a.inv_down[e * a.inv_down_stride + out]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = 16 * c + 4 * p + j;
          if (m >= count) continue;
          const float v = activate(sg[j], a.act) * su[j] * scale;
          a.mid[static_cast<int64_t>(row_pair[row0 + m]) * a.ffn + out] =
              __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
        }
      }
    }
  }
}

// Workgroups own two tiles of 16 hidden outputs; a wavefront asks for weights two units ahead and for
// rows one. grid: the outputs' workgroups, splits of the runs' units.
// Dynamic LDS: [waves][tokens][16 WIDE] float32.
template <bool ASYM, int CHUNKS>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeArgs a) {
  constexpr int WIDE = kDownWide, WAVES = kDownWaves, OUT = 16 * WIDE;
  __shared__ int experts[kMostRuns], first[kMostRuns + 1];
  __shared__ int row_pair[kMostPairs];
  __shared__ float row_weight[kMostPairs];
  __shared__ int last_one;
  extern __shared__ float sums[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, p = lane >> 4;
  const int group = blockIdx.x, groups = gridDim.x, pairs = a.tokens * a.k;
  float* mine = sums + wave * a.tokens * OUT;
  for (int i = lane; i < a.tokens * OUT; i += 64) mine[i] = 0.0f;
  const int total = *a.plan.total;
  for (int i = threadIdx.x; i <= pairs; i += 64 * WAVES) {
    // what lies behind the last run (of kMostRuns at most) is not used
    if (i <= kMostRuns) first[i] = a.plan.first[i];
    if (i < kMostRuns && i < pairs) experts[i] = a.plan.experts[i];
    if (i < pairs) {
      row_pair[i] = a.plan.pair[i];
      row_weight[i] = a.plan.weight[i];
    }
  }
  __syncthreads();

  // this wavefront's share of the runs' units
  const int units = a.ffn / kGroup, all = total * units, waves = WAVES * gridDim.y;
  const int number = blockIdx.y * WAVES + wave;
  const int begin = static_cast<int>(static_cast<int64_t>(all) * number / waves);
  const int end = static_cast<int>(static_cast<int64_t>(all) * (number + 1) / waves);
  struct Cursor {
    int slot, unit;
  };
  auto next = [&](Cursor& c) {
    if (++c.unit == units) {
      c.unit = 0;
      ++c.slot;
    }
  };
  Piece pw[kAheadW][WIDE];
  half8_t px[4];  // of a run's first 16 rows
  auto load_w = [&](Piece (&w)[WIDE], const Cursor& c, int at) {
    const bool real = at < end;
    const int e = __builtin_amdgcn_readfirstlane(experts[real ? c.slot : 0]);
#pragma unroll
    for (int t = 0; t < WIDE; ++t)
      w[t] = load_piece<ASYM>(reader(a.down, e, WIDE * group + t, units, a.sets), real ? c.unit : 0, a.sets, lane,
                              real ? 0u : kNoLoad);
  };
  auto load_x = [&](half8_t (&x)[4], const Cursor& c, int at) {
    const bool real = at < end;
    const int slot = real ? c.slot : 0, row = min(first[slot] + r, first[slot + 1] - 1);
    const uint16_t* from = a.mid + static_cast<int64_t>(row_pair[row]) * a.ffn + (real ? c.unit : 0) * kGroup + 32 * p;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = load_half8(from + 8 * i);
  };
  if (begin < end) {
    Cursor now = {begin / units, begin % units}, ahead_w = now, ahead_x = now;
#pragma unroll
    for (int i = 0; i < kAheadW; ++i) {
      load_w(pw[i], ahead_w, begin + i);
      next(ahead_w);
    }
    load_x(px, ahead_x, begin);
    next(ahead_x);
    float4_t d[CHUNKS][WIDE];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int t = 0; t < WIDE; ++t) d[c][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int at0 = begin; at0 < end; at0 += kAheadW) {
#pragma unroll
      for (int n = 0; n < kAheadW; ++n) {
        const int at = at0 + n;
        if (at >= end) break;
        const int row0 = first[now.slot], count = __builtin_amdgcn_readfirstlane(first[now.slot + 1] - row0);
        half8_t w[WIDE][4];
#pragma unroll
        for (int t = 0; t < WIDE; ++t) {
          const Dequant dq = constants<ASYM>(pw[n][t], lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[t][i] = weights8(pw[n][t], i, dq);
            d[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(px[i], w[t][i], d[0][t], 0, 0, 0);
          }
        }
        load_w(pw[n], ahead_w, at + kAheadW);
        next(ahead_w);
        load_x(px, ahead_x, at + 1);
        next(ahead_x);
#pragma unroll
        for (int c = 1; c < CHUNKS; ++c) {
          if (16 * c >= count) break;
          const uint16_t* x = a.mid + static_cast<int64_t>(row_pair[row0 + min(16 * c + r, count - 1)]) * a.ffn +
                              now.unit * kGroup + 32 * p;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const half8_t f = load_half8(x + 8 * i);
#pragma unroll
            for (int t = 0; t < WIDE; ++t) d[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, w[t][i], d[c][t], 0, 0, 0);
          }
        }
        if (now.unit == units - 1 || at + 1 == end) {  // this wavefront's share of the run is complete
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            if (16 * c >= count) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int m = 16 * c + 4 * p + j;
              if (m >= count) continue;
              float* to = mine + row_pair[row0 + m] / a.k * OUT + r;
#pragma unroll
              for (int t = 0; t < WIDE; ++t) to[16 * t] += row_weight[row0 + m] * d[c][t][j];
            }
#pragma unroll
            for (int t = 0; t < WIDE; ++t) d[c][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
          }
          wave_lds_fence();
        }
        next(now);
      }
    }
  }
  __syncthreads();
  const int outputs = a.tokens * OUT;
  auto store = [&](int i, float v) {
    const int t = i / OUT, n = group * OUT + i % OUT;
    if (a.residual != nullptr) v += f16_to_f32(a.residual[t * a.residual_stride + n]);
    a.y[t * a.y_stride + n] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  };
  auto sum = [&](int i) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sums[w * outputs + i];
    return v;
  };
  if (gridDim.y == 1) {
    for (int i = threadIdx.x; i < outputs; i += 64 * WAVES) store(i, sum(i));
    return;
  }
  // The last workgroup of a group of outputs adds all parts, in their order. They go through the memory that
  // all XCDs see, one by one: an exchange has been seen by all when its result is there, and the
  // barrier waits for it (a fence writes back all that an XCD's cache holds, in every workgroup:
  // 57 us instead of 9 for 23 MB of weights).
  uint32_t seen = 0;
  for (int i = threadIdx.x; i < outputs; i += 64 * WAVES)
    seen |= __hip_atomic_exchange(reinterpret_cast<uint32_t*>(a.plan.part) +
                                      (static_cast<int64_t>(blockIdx.y) * groups + group) * outputs + i,
                                  __builtin_bit_cast(uint32_t, sum(i)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("" : : "v"(seen) : "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last_one = __hip_atomic_fetch_add(&a.plan.ended[group], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               static_cast<int>(gridDim.y) - 1;
  __syncthreads();
  if (!last_one) return;
  for (int i = threadIdx.x; i < outputs; i += 64 * WAVES) {
    float v = 0.0f;
    for (int s = 0; s < static_cast<int>(gridDim.y); ++s)
      v += __hip_atomic_load(a.plan.part + (static_cast<int64_t>(s) * groups + group) * outputs + i, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
    store(i, v);
  }
}

// Workgroups that share outputs in the second launch, so that at least one runs on each CU. (One
// token through two of eight experts, that launch: 18.6 us; with one tile 20, with eight wavefronts
// and eight units ahead 24. 48 tokens over 64 experts: 60, 72 and 76.)
int down_splits(int hidden) {
  const int groups = hidden / (kTileN * kDownWide), splits = (256 + groups - 1) / groups;
  return splits > 16 ? 16 : splits;
}

Layers make_layers(const void* base, int64_t N, int64_t K, int32_t group, int32_t fmt) {
  const PackedLayout l = make_layout(N, K, group, fmt);
  return {static_cast<const uint8_t*>(base), l.total_bytes, static_cast<uint32_t>(l.scales_off),
          static_cast<uint32_t>(l.zeros_off < 0 ? 0 : l.zeros_off)};
}

// The workspace: mid, then the plan. Returns its size.
size_t lay_out(int64_t tokens, int hidden, int ffn, int k, void* ws, uint16_t** mid, Plan* plan) {
  const size_t pairs = static_cast<size_t>(tokens) * k, tiles = hidden / kTileN;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 15) / 16 * 16;
    return static_cast<char*>(ws) + here;
  };
  uint16_t* m = reinterpret_cast<uint16_t*>(take(2 * pairs * ffn));
  Plan p;
  p.total = reinterpret_cast<int32_t*>(take(4));
  p.experts = reinterpret_cast<int32_t*>(take(4 * pairs));
  p.first = reinterpret_cast<int32_t*>(take(4 * (pairs + 1)));
  p.pair = reinterpret_cast<int32_t*>(take(4 * pairs));
  p.weight = reinterpret_cast<float*>(take(4 * pairs));
  p.ended = reinterpret_cast<int32_t*>(take(4 * tiles));
  const int splits = down_splits(hidden);
  p.part = reinterpret_cast<float*>(take(splits == 1 ? 0 : 4 * splits * tiles * tokens * 16));
  if (mid != nullptr) *mid = m;
  if (plan != nullptr) *plan = p;
  return at;
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int32_t hidden, int32_t ffn, int32_t k) {
  return lay_out(tokens, hidden, ffn, k, nullptr, nullptr, nullptr);
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
  lay_out(p.tokens, p.hidden, p.ffn, p.k, p.ws, &a.mid, &a.plan);
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
  const int tiles = p.ffn / kTileN;  // a multiple of eight
  auto up = [&](auto kernel, int wide) {
    hipLaunchKernelGGL(kernel, dim3(tiles / wide + 1, slots), dim3(64 * kUpWaves), 0, st, a);
  };
  auto up_fmt = [&](auto fmt) {
    constexpr bool ASYM = decltype(fmt)::value;
    const bool two = tiles * slots >= 512;  // one tile where workgroups would not reach all CUs
    if (a.tokens <= 16) return two ? up(&moe_up_kernel<ASYM, 2, 1>, 2) : up(&moe_up_kernel<ASYM, 1, 1>, 1);
    return two ? up(&moe_up_kernel<ASYM, 2, kChunks>, 2) : up(&moe_up_kernel<ASYM, 1, kChunks>, 1);
  };
  asym ? up_fmt(std::true_type{}) : up_fmt(std::false_type{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kSums = 4 * kDownWaves * 16 * kDownWide;  // bytes for each token
  auto down = [&](auto kernel, std::atomic<uint64_t>& done) {
    const hipError_t limit = ensure_lds_limit(reinterpret_cast<const void*>(kernel), kSums * AWQ_MOE_MAX_TOKENS, done);
    if (limit != hipSuccess) return limit;
    hipLaunchKernelGGL(kernel, dim3(p.hidden / (kTileN * kDownWide), down_splits(p.hidden)), dim3(64 * kDownWaves),
                       static_cast<size_t>(kSums) * a.tokens, st, a);
    return hipGetLastError();
  };
  static std::atomic<uint64_t> done[4];
  if (a.tokens <= 16) return asym ? down(&moe_down_kernel<true, 1>, done[0]) : down(&moe_down_kernel<false, 1>, done[1]);
  return asym ? down(&moe_down_kernel<true, kChunks>, done[2]) : down(&moe_down_kernel<false, kChunks>, done[3]);
}

}  // namespace awq
