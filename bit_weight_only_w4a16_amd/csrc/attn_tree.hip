// Attention of the last (new or drafted) tokens of each sequence over its paged cache
// (awq_attn_tree in awq_block.h). A handful of query rows read every cached key and value
// once: large calls are bound by streaming the cache from memory (16 sequences of up to 32768
// positions, 64 heads on 8, D = 128, single tokens: 1.33 GB in 236 us, 5.6 TB/s, more than a
// copy's reads and writes reach), small ones by the chain of a launch, the sequence, its pages
// and its first step (one token over 517 positions, 32 heads: 9.0 us; over 16 to 128
// positions 5.0 us).
//
// The query rows that share a key / value head (tokens x heads of the group) are handled
// together, so the cache is read once for all of them: up to 16 rows in one workgroup of
// the kernel described here, more in workgroups of 64 (attn_tree_rows_kernel). The
// context is split over workgroups, and inside a workgroup over its four wavefronts: each
// takes every fourth step of 32 positions, from the last to the first, and runs alone, with a running maximum and sum of
// its own, its own LDS ring and no barriers, until the four results are merged through LDS.
// With more than one split the merged result is a partial one (float32 maximum, sum and
// unnormalised row) in the workspace, and a second launch adds the splits in their order.
//
// A step's keys and values go from memory straight into LDS (16 bytes per lane, no
// registers), one step ahead (every load instruction of a step counts in wait_loads: each
// row's lanes cover all its chunks, so with D < DP some lane takes part in each). Both
// products are formed transposed, S^T = K Q^T and O^T = V^T P^T (16 x 16 x 32 matrix
// instruction): lane l holds the scores of one query (column l % 16), the positions it holds
// after S^T are the contraction slots it feeds to O^T, and V^T is read from LDS in that order
// with the transposing 16-bit read.
#include "block_internal.hpp"

#include <limits.h>
#include <math.h>
#include <stdlib.h>

#include <type_traits>

namespace awq {
namespace {

constexpr int kStep = 32;        // positions per wavefront and step
constexpr int kWaves = 4;
constexpr int kStages = 2;       // of a wavefront's ring: one in use, one on its way
constexpr int kMinChunk = kStep * kWaves;  // positions per split: at least this many
constexpr int kTableEntries = 1024;        // page numbers of a split staged in LDS
constexpr int kMaxSplits = 64;
// P carries a factor 2^shift, and the maximum in use is at most kSlack below the true one. In
// binary16 that is 2^7: P stays below 2^15, and down to 2^-21 of the maximum keeps its digits.
// bfloat16 has float32's exponents, and there it is small enough (2^-8 / the longest length) that
// a row's P add up to less than 1: no sum of values of any size passes float32's largest.
constexpr float kShift = 7.0f, kSlack = 8.0f;  // (binary16's shift)

struct TreeArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t *table, *ctx, *cu;
  const uint64_t* mask;
  float* part;  // [tokens * q_heads][splits][head_dim], then [..][splits][2]; NULL: one split
  int64_t q_token, q_head, o_token, o_head, cache_page, cache_head, cache_slot;
  int64_t max_len;  // table_width * page_size
  int32_t tokens, seqs, table_width, pages, page_size, max_q, q_heads, kv_heads, group, head_dim;
  int32_t splits, row_blocks;
  uint32_t page_mul, page_shift;  // pos / page_size = pos * page_mul >> page_shift
  float c;  // scale * log2(e)
  float shift;
};

// pos / page_size for 0 <= pos < 2^31 (page_mul = floor(2^page_shift / page_size) + 1 with
// page_shift = 31 + ceil(log2 page_size): the excess stays below one part in 2^31).
__device__ __forceinline__ int page_of(const TreeArgs& a, int pos) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * a.page_mul) >> a.page_shift);
}

// A sequence's tokens, context and length, clamped to what the buffers hold
struct Seq {
  int first, count, ctx, len;
};
__device__ __forceinline__ Seq sequence(const TreeArgs& a, int b) {
  Seq s;
  s.first = min(max(a.cu[b], 0), a.tokens);
  s.count = min(max(min(a.cu[b + 1], a.tokens) - s.first, 0), a.max_q);
  const int64_t ctx = max(a.ctx[b], 0);
  s.ctx = static_cast<int>(ctx < a.max_len ? ctx : a.max_len);
  const int64_t len = ctx + s.count;
  s.len = static_cast<int>(len < a.max_len ? len : a.max_len);
  return s;
}
// Positions per split of a sequence: the same for every workgroup of it, a multiple of what a
// step of the kernels takes
__device__ __forceinline__ int chunk_of(int len, int splits) {
  const int per = (len + splits - 1) / splits;
  return max((per + 63) / 64 * 64, kMinChunk);
}

// Which of a step's 32 positions a row sees, as bits: `back` is the step's first position less
// the context (bit j of `mask` is new token j), `left` the positions up to the split's end.
__device__ __forceinline__ uint32_t visible(uint64_t mask, int back, int left) {
  const int k = min(max(-back, 0), 31);  // positions of the step that are context (< 32 here)
  const uint32_t bits = (static_cast<uint32_t>(mask >> (max(back, 0) & 63)) << k) | ((1u << k) - 1u);
  return left < 32 ? bits & ((1u << left) - 1u) : bits;
}

// The factor that brings a partial result with maximum m and sum l to the maximum top (sums
// and rows of every part carry 2^shift). A
// part that saw no finite score (m = -inf) has l = 0, or NaN if it saw a NaN, and passes
// that on.
__device__ __forceinline__ float scale_of(float m, float l, float top) {
  return m == kNegInf ? l : __builtin_amdgcn_exp2f(m - top);
}

template <int DP>
__device__ __forceinline__ int k_pos(int r, int c) {
  return DP == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int v_pos(int r, int c) {
  return DP == 128 ? c ^ ((r & 7) << 1) : c ^ (((r >> 1) & 3) << 1);
}

// One wavefront writes a row's result (lane i has d = 2 i, 2 i + 1): the output, or the
// split's partial result.
template <typename T>
__device__ __forceinline__ void store_row(const TreeArgs& a, int token, int hq, int split, float m, float l,
                                          float2_t o) {
  const int lane = threadIdx.x & 63;
  if (2 * lane >= a.head_dim) return;
  if (a.part != nullptr) {
    const int64_t at = (static_cast<int64_t>(token) * a.q_heads + hq) * a.splits + split;
    *reinterpret_cast<float2_t*>(a.part + at * a.head_dim + 2 * lane) = o;
    if (lane == 0) {
      float* ml = a.part + static_cast<int64_t>(a.tokens) * a.q_heads * a.splits * a.head_dim;
      *reinterpret_cast<float2_t*>(ml + 2 * at) = float2_t{m, l};
    }
  } else {
    const float inv = inv_sum(l);
    *reinterpret_cast<uint32_t*>(a.out + token * a.o_token + hq * a.o_head + 2 * lane) =
        T::pack2(o.x * inv, o.y * inv);
  }
}

// LDS bytes of a workgroup: the rings (later the four float32 results), Q, the page numbers
template <int DP>
struct Lds {
  static constexpr int kRow = DP * 2;
  static constexpr int kTile = kStep * kRow;
  static constexpr int kRing = kWaves * kStages * 2 * kTile;
  static constexpr int kSumStride = DP + 4;  // floats: rows 4 banks apart
  static constexpr int kSums = kWaves * 16 * kSumStride * 4;
  static constexpr int kBig = kRing > kSums ? kRing : kSums;
  static constexpr int kQ = 16 * kRow;
  static constexpr int kStats = kWaves * 16 * 2 * 4;
  static constexpr int kTotal = kBig + kQ + kStats + kTableEntries * 4;
};

// PAD: head_dim < DP
template <typename T, int DP, bool PAD>
__global__ void __launch_bounds__(256, 1) attn_tree_kernel(TreeArgs a) {
  typedef typename T::v8 v8;
  typedef Lds<DP> L;
  constexpr int RB = L::kRow, RC = DP / 8, TILE = L::kTile;
  constexpr int ROWS = 1024 / RB;        // positions one load instruction fills
  constexpr int LOADS = kStep / ROWS;
  constexpr int NC = DP / 32, ND = DP / 16;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  unsigned char* q_lds = smem + L::kBig;
  float* stats = reinterpret_cast<float*>(q_lds + L::kQ);
  int* pages = reinterpret_cast<int*>(q_lds + L::kQ + L::kStats);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, kv_head = blockIdx.y, b = blockIdx.z;
  const Seq s = sequence(a, b);
  const int rows = s.count * a.group;
  if (rows == 0) return;
  const int chunk = chunk_of(s.len, a.splits);
  const int p0 = split * chunk, p1 = min(s.len, p0 + chunk);
  if (p0 >= p1 && a.part != nullptr) return;  // the second launch knows that it is empty

  // page numbers of the split, clamped to the cache
  const int t0 = page_of(a, p0);
  const int n_pages = p1 > p0 ? page_of(a, p1 - 1) - t0 + 1 : 0;
  for (int i = threadIdx.x; i < n_pages; i += 256)
    pages[i] = min(max(a.table[static_cast<int64_t>(b) * a.table_width + t0 + i], 0), a.pages - 1);
  // Q rows (row r: token r / group, head r % group of the key head), 0 past the last
  for (int i = threadIdx.x; i < 16 * RC; i += 256) {
    const int r = i / RC, ch = i % RC;
    u32x4 x = {0, 0, 0, 0};
    if (r < rows && 8 * ch < a.head_dim) {
      const int t = r / a.group, hq = kv_head * a.group + r % a.group;
      x = *reinterpret_cast<const u32x4*>(a.q + (s.first + t) * a.q_token + hq * a.q_head + 8 * ch);
    }
    *reinterpret_cast<u32x4*>(q_lds + r * RB + 16 * k_pos<DP>(r, ch)) = x;
  }
  unsigned char* ring = smem + wave * kStages * 2 * TILE;
  const uint32_t ring_at = lds_offset(smem) + wave * kStages * 2 * TILE;
  if constexpr (PAD) {  // chunks past D are never loaded: they stay 0
    for (int i = lane; i < kStages * 2 * TILE / 16; i += 64)
      *reinterpret_cast<u32x4*>(ring + 16 * i) = u32x4{0, 0, 0, 0};
    __builtin_amdgcn_s_waitcnt(0);
  }
  // this lane's row's mask over the new tokens
  const int own = min(col / a.group, s.count - 1);
  const uint64_t sees = a.mask != nullptr ? a.mask[s.first + own] : (2ull << own) - 1;
  __syncthreads();

  const uint16_t* kbase = a.k + kv_head * a.cache_head;
  const uint16_t* vbase = a.v + kv_head * a.cache_head;
  auto offset_of = [&](int pos) -> int64_t {
    const int page = page_of(a, pos);
    return pages[page - t0] * a.cache_page + (pos - page * a.page_size) * a.cache_slot;
  };
  // where this lane loads from in the step at position s0: load j takes position ROWS j + l / RC
  // (positions past the split repeat its last one: their scores are masked and their V rows
  // cleared below)
  auto find_step = [&](int s0, int64_t at[LOADS]) {
    const int64_t off = offset_of(min(s0 + (lane & 31), p1 - 1));
    const int off_lo = static_cast<int>(off), off_hi = static_cast<int>(off >> 32);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const uint32_t lo = __shfl(off_lo, ROWS * j + lane / RC), hi = __shfl(off_hi, ROWS * j + lane / RC);
      at[j] = static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
    }
  };
  auto load_step = [&](const int64_t at[LOADS], int stage) {
    const uint32_t dst = ring_at + stage * 2 * TILE;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int r = ROWS * j + lane / RC;
      const int ck = 8 * k_pos<DP>(r, lane % RC), cv = 8 * v_pos<DP>(r, lane % RC);
      if (!PAD || ck < a.head_dim) load_to_lds(kbase + at[j] + ck, dst + j * 1024);
      if (!PAD || cv < a.head_dim) load_to_lds(vbase + at[j] + cv, dst + TILE + j * 1024);
    }
  };

  float4_t acc[ND];
  float m = kNegInf, l = 0.0f;
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // One step is used while the next is on its way, and the addresses of the one after that
  // are found meanwhile. The last step, which may hold new tokens, comes first: where the sums
  // are NaN after it, they start again from zero without its values (see add_keys).
  const int first = p0 + kStep * wave;
  constexpr int kStride = kStep * kWaves;
  const int last = first < p1 ? first + (p1 - 1 - first) / kStride * kStride : first - 1;
  bool left_out = false;  // the last step's values are missing in acc
  int64_t at[LOADS];
  if (last >= first) {
    find_step(last, at);
    load_step(at, 0);
    if (last - kStride >= first) find_step(last - kStride, at);
  }
  // (the stage is a compile-time value: the LDS addresses then differ by constants)
  auto step = [&](auto stage_, int s0) {
    constexpr int stage = decltype(stage_)::value;
    if (s0 - kStride >= first) {
      wait_lds();  // the step before's reads of this stage are done
      load_step(at, stage ^ 1);
      wait_loads<2 * LOADS>();  // the step has landed
      if (s0 - 2 * kStride >= first) find_step(s0 - 2 * kStride, at);
    } else {
      wait_loads<0>();
    }
    const unsigned char* ks = ring + stage * 2 * TILE;
    unsigned char* vs = ring + stage * 2 * TILE + TILE;
    if (s0 + kStep > p1) {  // V rows past the split: 0
      for (int i = lane; i < (s0 + kStep - p1) * RC; i += 64)
        *reinterpret_cast<u32x4*>(vs + (p1 - s0) * RB + 16 * i) = u32x4{0, 0, 0, 0};
    }
    v8 kf[2][NC];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int r = 16 * t + col;
        kf[t][c] = *reinterpret_cast<const v8*>(ks + r * RB + 16 * k_pos<DP>(r, 4 * c + g));
      }
    float4_t sc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const v8 qf = *reinterpret_cast<const v8*>(q_lds + col * RB + 16 * k_pos<DP>(col, 4 * c + g));
      sc[0] = T::mfma16(kf[0][c], qf, sc[0]);
      sc[1] = T::mfma16(kf[1][c], qf, sc[1]);
    }
    // new tokens (or the end) in the step: one bit per position. (At most 16 tokens: a
    // wavefront meets one such step, its last.)
    const bool masked = s0 + kStep > s.ctx;
    if (masked) {
      const uint32_t bits = visible(sees, s0 - s.ctx, p1 - s0) >> (4 * g);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[t][i] = (bits & (1u << (16 * t + i))) != 0 ? sc[t][i] : kNegInf;
    }
    float top = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                      fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3]))) * a.c;
    if (__ballot(top > m + kSlack) != 0) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float m_new = fmaxf(m, top);
      const float keep = m_new == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= keep;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] *= keep;
    }
    const float off = m == kNegInf ? 0.0f : a.shift - m;
    u32x4 p;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint32_t pair = T::pack2(__builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i], a.c, off)),
                                       __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i + 1], a.c, off)));
        l = T::add2(pair, l);  // what is multiplied, as it was rounded
        p[2 * t + (i >> 1)] = pair;
      }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const int ra = 4 * g + (col >> 2), rb = ra + 16;
      const int ch = 2 * d + ((col & 3) >> 1), byte = 8 * (col & 1);
      const short4_t lo = lds_read_tr(vs + ra * RB + 16 * v_pos<DP>(ra, ch) + byte);
      const short4_t hi = lds_read_tr(vs + rb * RB + 16 * v_pos<DP>(rb, ch) + byte);
      acc[d] = T::mfma16(join8<v8>(lo, hi), __builtin_bit_cast(v8, p), acc[d]);
    }
    if (masked) {
      bool nan = false;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= acc[d][i] != acc[d][i];
      if (__ballot(nan) != 0) {
        left_out = true;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    asm volatile("" ::: "memory");
  };
  for (int s0 = last; s0 >= first; s0 -= 2 * kStride) {
    step(std::integral_constant<int, 0>{}, s0);
    if (s0 - kStride >= first) step(std::integral_constant<int, 1>{}, s0 - kStride);
  }
  if (left_out && col < rows) {
    const int t = col / a.group, hq = kv_head * a.group + col % a.group;
    add_keys<T, ND>(
        a.q + (s.first + t) * a.q_token + hq * a.q_head, a.head_dim, a.c, m == kNegInf ? 0.0f : a.shift - m, last,
        min(last + kStep, p1), 4 * g, 16,
        [&](int j, const uint16_t*& kr, const uint16_t*& vr) {
          const int64_t off = offset_of(j);
          kr = kbase + off;
          vr = vbase + off;
          return j < s.ctx || ((sees >> ((j - s.ctx) & 63)) & 1) != 0;
        },
        [&](int r, int i, float p, float x) { acc[r][i] = __builtin_fmaf(p, x, acc[r][i]); });
  }

  // merge the four wavefronts: maxima, then the rows brought to the common maximum
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    stats[(wave * 16 + col) * 2] = m;
    stats[(wave * 16 + col) * 2 + 1] = l;
  }
  __syncthreads();  // also: every ring is done with
  float* sums = reinterpret_cast<float*>(smem);
  {
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[(w * 16 + col) * 2]);
    const float f = scale_of(m, l, top);
#pragma unroll
    for (int d = 0; d < ND; ++d)
      *reinterpret_cast<float4_t*>(sums + (wave * 16 + col) * L::kSumStride + 16 * d + 4 * g) = acc[d] * f;
  }
  __syncthreads();
  // one wavefront per row: lane i has d = 2 i, 2 i + 1
  for (int r = wave; r < rows; r += kWaves) {
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[(w * 16 + r) * 2]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = stats[(w * 16 + r) * 2], lw = stats[(w * 16 + r) * 2 + 1];
      sum += lw * scale_of(mw, lw, top);
    }
    float2_t o = {0.0f, 0.0f};
    if (2 * lane < DP) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        o += *reinterpret_cast<const float2_t*>(sums + (w * 16 + r) * L::kSumStride + 2 * lane);
    }
    const int t = r / a.group, hq = kv_head * a.group + r % a.group;
    store_row<T>(a, s.first + t, hq, split, top, sum, o);
  }
}

// The same for more query rows, or more workgroups than run at once: 64 rows per workgroup,
// 64 positions per step, in LDS for all four wavefronts; each takes 32 of the rows and 32 of
// the positions, so that a fragment of K or V read from LDS serves two row tiles. The
// wavefronts keep their Q operands in registers and the two halves of the positions meet at
// the end; 64 KiB of LDS let two workgroups share a CU. Eight sequences of 0 to 4096 positions
// and 1 to 32 drafted tokens, 32 heads on 8 (58 MB of cache): 21.7 us and 5 us for the second
// launch; 64 sequences of 512 positions with 16 tokens each 27.5 us, 5.0 TB/s. (A
// wavefront on 16 rows and all positions, with loads that the compiler waited for, took 35 and
// 112 us where this takes 24 and 45: 8 and 32 sequences of 2048 positions, 16 tokens each.)
constexpr int kRowStep = 64;
constexpr int kRowTiles = 2;  // of 16 rows, per wavefront

// (D up to 64: 128 registers and 36 KiB of LDS, four workgroups per CU)
template <typename T, int DP, bool PAD>
__global__ void __launch_bounds__(256, DP == 64 ? 4 : 2) attn_tree_rows_kernel(TreeArgs a) {
  typedef typename T::v8 v8;
  constexpr int RB = DP * 2, RC = DP / 8, TILE = kRowStep * RB;
  constexpr int ROWS = 1024 / RB;               // positions one load instruction fills
  constexpr int OWN = kRowStep / kWaves;        // positions a wavefront loads
  constexpr int LOADS = OWN / ROWS;
  constexpr int NC = DP / 32, ND = DP / 16, NT = kRowTiles;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];  // [2][K tile, V tile], pages
  int* pages = reinterpret_cast<int*>(smem + 4 * TILE);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave >> 1;  // of a step's positions
  const int lane = threadIdx.x & 63;
  const int col = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % a.splits, rb = blockIdx.x / a.splits;
  const int kv_head = blockIdx.y, b = blockIdx.z;
  const Seq s = sequence(a, b);
  const int rows = s.count * a.group;
  if (rb * 64 >= rows) return;
  const int chunk = chunk_of(s.len, a.splits);
  const int p0 = split * chunk, p1 = min(s.len, p0 + chunk);
  if (p0 >= p1 && a.part != nullptr) return;  // the second launch knows that it is empty

  const int t0 = page_of(a, p0);
  const int n_pages = p1 > p0 ? page_of(a, p1 - 1) - t0 + 1 : 0;
  for (int i = threadIdx.x; i < n_pages; i += 256)
    pages[i] = min(max(a.table[static_cast<int64_t>(b) * a.table_width + t0 + i], 0), a.pages - 1);
  if constexpr (PAD) {  // chunks past D are never loaded: they stay 0
    for (int i = threadIdx.x; i < 4 * TILE / 16; i += 256)
      *reinterpret_cast<u32x4*>(smem + 16 * i) = u32x4{0, 0, 0, 0};
  }
  // this lane's rows, their masks and their Q operands (rows past the last repeat it)
  const int row0 = rb * 64 + 32 * (wave & 1) + col;
  int token[NT], head[NT];
  uint64_t sees[NT];
  v8 qf[NT][NC];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = min(row0 + 16 * n, rows - 1);
    const int t = r / a.group;
    token[n] = s.first + t;
    head[n] = kv_head * a.group + r - t * a.group;
    sees[n] = a.mask != nullptr ? a.mask[token[n]] : (2ull << t) - 1;
    const uint16_t* q = a.q + token[n] * a.q_token + head[n] * a.q_head;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 32 * c + 8 * g;
      u32x4 x = {0, 0, 0, 0};
      if (!PAD || d < a.head_dim) x = *reinterpret_cast<const u32x4*>(q + d);
      qf[n][c] = __builtin_bit_cast(v8, x);
    }
  }
  __syncthreads();

  const uint16_t* kbase = a.k + kv_head * a.cache_head;
  const uint16_t* vbase = a.v + kv_head * a.cache_head;
  auto offset_of = [&](int pos) -> int64_t {
    const int page = page_of(a, pos);
    return pages[page - t0] * a.cache_page + (pos - page * a.page_size) * a.cache_slot;
  };
  auto find_step = [&](int s0, int64_t at[LOADS]) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) at[j] = offset_of(min(s0 + OWN * wave + ROWS * j + lane / RC, p1 - 1));
  };
  auto load_step = [&](const int64_t at[LOADS], int stage) {
    const uint32_t dst = lds_offset(smem) + stage * 2 * TILE + OWN * wave * RB;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int r = ROWS * j + lane / RC;  // (of this wavefront's 16, a multiple of the patterns' period)
      const int ck = 8 * k_pos<DP>(r, lane % RC), cv = 8 * v_pos<DP>(r, lane % RC);
      if (!PAD || ck < a.head_dim) load_to_lds(kbase + at[j] + ck, dst + j * 1024);
      if (!PAD || cv < a.head_dim) load_to_lds(vbase + at[j] + cv, dst + TILE + j * 1024);
    }
  };

  float4_t acc[NT][ND];
  float m[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[n][d] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // The last steps, which may hold new tokens, come first: where the sums are NaN after one,
  // they start again from zero without the values so far (see add_keys).
  const int last = p0 < p1 ? p0 + (p1 - 1 - p0) / kRowStep * kRowStep : p0 - 1;
  int left_out = INT_MAX;  // the values from this step of the wavefront's on are missing in acc
  int64_t at[LOADS];
  if (last >= p0) {
    find_step(last, at);
    load_step(at, 0);
    if (last - kRowStep >= p0) find_step(last - kRowStep, at);
  }
  auto step = [&](auto stage_, int s0) {
    constexpr int stage = decltype(stage_)::value;
    const unsigned char* ks = smem + stage * 2 * TILE + 32 * half * RB;
    unsigned char* vs = smem + stage * 2 * TILE + TILE;
    wait_loads<0>();  // this wavefront's loads of the step have landed
    // V rows past the split: 0, each wavefront among those it loaded
    const int own = s0 + OWN * wave;
    if (own + OWN > p1) {
      const int from = max(p1 - own, 0);
      for (int j = lane; j < (OWN - from) * RC; j += 64)
        *reinterpret_cast<u32x4*>(vs + (OWN * wave + from) * RB + 16 * j) = u32x4{0, 0, 0, 0};
    }
    lds_barrier();  // the step is whole, and the other stage is done with
    if (s0 - kRowStep >= p0) load_step(at, stage ^ 1);
    if (s0 - 2 * kRowStep >= p0) find_step(s0 - 2 * kRowStep, at);
    const int mine = s0 + 32 * half;  // this wavefront's positions
    if (mine >= p1) return;
    vs += 32 * half * RB;

    float4_t sc[NT][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int r = 16 * j + col;
        const v8 kf = *reinterpret_cast<const v8*>(ks + r * RB + 16 * k_pos<DP>(r, 4 * c + g));
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][j] = T::mfma16(kf, qf[n][c], sc[n][j]);
      }
    }
    const bool masked = mine + 32 > s.ctx;  // new tokens (or the end) among them: one bit per position
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t bits = visible(sees[n], mine - s.ctx, p1 - mine) >> (4 * g);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][j][e] = (bits & (1u << (16 * j + e))) != 0 ? sc[n][j][e] : kNegInf;
      }
    }
    float top[NT];
    bool grown = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n] = fmaxf(fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3])),
                     fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3]))) * a.c;
      grown |= top[n] > m[n] + kSlack;
    }
    if (__ballot(grown) != 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
        const float m_new = fmaxf(m[n], top[n]);
        const float keep = m_new == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[n] - m_new);
        m[n] = m_new;
        l[n] *= keep;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[n][d] *= keep;
      }
    }
    u32x4 p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float off = m[n] == kNegInf ? 0.0f : a.shift - m[n];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const uint32_t pair = T::pack2(__builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j][e], a.c, off)),
                                         __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][j][e + 1], a.c, off)));
          l[n] = T::add2(pair, l[n]);
          p[n][2 * j + (e >> 1)] = pair;
        }
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const int ra = 4 * g + (col >> 2), rb2 = ra + 16;
      const int ch = 2 * d + ((col & 3) >> 1), byte = 8 * (col & 1);
      const short4_t lo = lds_read_tr(vs + ra * RB + 16 * v_pos<DP>(ra, ch) + byte);
      const short4_t hi = lds_read_tr(vs + rb2 * RB + 16 * v_pos<DP>(rb2, ch) + byte);
      const v8 vf = join8<v8>(lo, hi);
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][d] = T::mfma16(vf, __builtin_bit_cast(v8, p[n]), acc[n][d]);
    }
    if (masked) {
      bool nan = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) nan |= acc[n][d][e] != acc[n][d][e];
      if (__ballot(nan) != 0) {
        left_out = mine;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[n][d] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  };
  for (int s0 = last; s0 >= p0; s0 -= 2 * kRowStep) {
    step(std::integral_constant<int, 0>{}, s0);
    if (s0 - kRowStep >= p0) step(std::integral_constant<int, 1>{}, s0 - kRowStep);
  }
  for (int s0 = left_out; s0 < p1; s0 += kRowStep) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int x = opaque(lane), r = min(rb * 64 + 32 * (wave & 1) + 16 * n + (x & 15), rows - 1);
      const int t = r / a.group, own = s.first + t;
      const uint64_t bits = a.mask != nullptr ? a.mask[own] : (2ull << t) - 1;
      add_keys<T, ND>(
          a.q + own * a.q_token + (kv_head * a.group + r - t * a.group) * a.q_head, a.head_dim, a.c,
          m[n] == kNegInf ? 0.0f : a.shift - m[n], s0, min(s0 + 32, p1), 4 * (x >> 4), 16,
          [&](int j, const uint16_t*& kr, const uint16_t*& vr) {
            const int64_t off = offset_of(j);
            kr = kbase + off;
            vr = vbase + off;
            return j < s.ctx || ((bits >> ((j - s.ctx) & 63)) & 1) != 0;
          },
          [&](int r, int i, float p, float x) { acc[n][r][i] = __builtin_fmaf(p, x, acc[n][r][i]); });
    }
  }

  // the second half's results through LDS to the first (lane by lane, the same rows)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += __shfl_xor(l[n], 16);
    l[n] += __shfl_xor(l[n], 32);
  }
  lds_barrier();  // the stages are done with
  float4_t* sums = reinterpret_cast<float4_t*>(smem) + (wave & 1) * NT * ND * 64 + lane;
  float2_t* stats = reinterpret_cast<float2_t*>(smem + 2 * NT * ND * 64 * 16) + (wave & 1) * NT * 64 + lane;
  if (half == 1) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      stats[n * 64] = float2_t{m[n], l[n]};
#pragma unroll
      for (int d = 0; d < ND; ++d) sums[(n * ND + d) * 64] = acc[n][d];
    }
  }
  lds_barrier();
  if (half == 1) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2_t other = stats[n * 64];
    const float top = fmaxf(m[n], other.x);
    const float f0 = scale_of(m[n], l[n], top), f1 = scale_of(other.x, other.y, top);
    m[n] = top;
    l[n] = l[n] * f0 + other.y * f1;
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[n][d] = acc[n][d] * f0 + sums[(n * ND + d) * 64] * f1;
    if (row0 + 16 * n >= rows) continue;
    const int64_t at_row = (static_cast<int64_t>(token[n]) * a.q_heads + head[n]) * a.splits + split;
    const float inv = inv_sum(l[n]);
    uint16_t* o = a.out + token[n] * a.o_token + head[n] * a.o_head;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const int e = 16 * d + 4 * g;
      if (PAD && e >= a.head_dim) continue;
      if (a.part != nullptr) {
        *reinterpret_cast<float4_t*>(a.part + at_row * a.head_dim + e) = acc[n][d];
      } else {
        *reinterpret_cast<uint2*>(o + e) = make_uint2(T::pack2(acc[n][d][0] * inv, acc[n][d][1] * inv),
                                                      T::pack2(acc[n][d][2] * inv, acc[n][d][3] * inv));
      }
    }
    if (a.part != nullptr && g == 0) {
      float* ml = a.part + static_cast<int64_t>(a.tokens) * a.q_heads * a.splits * a.head_dim;
      *reinterpret_cast<float2_t*>(ml + 2 * at_row) = float2_t{m[n], l[n]};
    }
  }
}

// Adds the splits of a row in their order: one wavefront per token and head, lane i has
// d = 2 i, 2 i + 1. The launch is a few microseconds long and made of waiting, so everything
// the first eight splits need is asked for at once: their maxima, sums and rows, which are
// found from the token alone, and the sequences, 64 of them, that say how many splits count.
constexpr int kMergeLoads = 8;

// The sequence of a token: the last that starts at or before it. 64 lanes search 64 ways.
__device__ __forceinline__ bool sequence_of(const TreeArgs& a, int token, Seq& s) {
  const int lane = threadIdx.x & 63;
  int b0 = 0, count = a.seqs;
  while (true) {
    const int stride = (count + 63) >> 6, at = lane * stride;
    Seq mine = {INT_MAX, 0, 0, 0};
    if (at < count) mine = sequence(a, b0 + at);
    const uint64_t before = __ballot(mine.first <= token);
    if (before == 0) return false;
    const int w = 63 - __builtin_clzll(before);
    if (stride == 1) {
      s.first = __builtin_amdgcn_readlane(mine.first, w);
      s.count = __builtin_amdgcn_readlane(mine.count, w);
      s.len = __builtin_amdgcn_readlane(mine.len, w);
      return token - s.first < s.count;
    }
    b0 += w * stride;
    count = min(stride, count - w * stride);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) attn_tree_merge_kernel(TreeArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (row >= static_cast<int64_t>(a.tokens) * a.q_heads) return;
  const int token = static_cast<int>(row / a.q_heads), hq = static_cast<int>(row - static_cast<int64_t>(token) * a.q_heads);
  const int64_t at = row * a.splits;
  const float* ml = a.part + static_cast<int64_t>(a.tokens) * a.q_heads * a.splits * a.head_dim + 2 * at;
  const float* part = a.part + at * a.head_dim + min(2 * lane, a.head_dim - 2);
  // (splits past the sequence's hold anything: they are read and not used)
  auto load = [&](int first, float2_t x[kMergeLoads]) {
#pragma unroll
    for (int j = 0; j < kMergeLoads; ++j)
      x[j] = *reinterpret_cast<const float2_t*>(part + static_cast<int64_t>(min(first + j, a.splits - 1)) * a.head_dim);
  };
  float2_t x[kMergeLoads], own = *reinterpret_cast<const float2_t*>(ml + 2 * min(lane, a.splits - 1));
  load(0, x);
  Seq s;
  if (!sequence_of(a, token, s)) return;
  const int chunk = chunk_of(s.len, a.splits);
  const int n = (s.len + chunk - 1) / chunk;
  float top = lane < n ? own.x : kNegInf;
  for (int w = lane + 64; w < n; w += 64) top = fmaxf(top, ml[2 * w]);
  top = wave_max(top);
  float sum = 0.0f;
  float2_t o = {0.0f, 0.0f};
  for (int w0 = 0; w0 < n; w0 += 64) {  // 64 splits' factors, one per lane
    if (w0 > 0) own = *reinterpret_cast<const float2_t*>(ml + 2 * min(w0 + lane, n - 1));
    const float f = w0 + lane < n ? scale_of(own.x, own.y, top) : 0.0f;
    sum += wave_sum(w0 + lane < n ? own.y * f : 0.0f);
    const int here = min(64, n - w0);
    for (int i = 0; i < here; i += kMergeLoads) {  // that many rows in flight
      if (w0 + i > 0) load(w0 + i, x);
#pragma unroll
      for (int j = 0; j < kMergeLoads; ++j) {
        const float fj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), (i + j) & 63));
        if (i + j < here) o += x[j] * fj;
      }
    }
  }
  const float inv = inv_sum(sum);
  if (2 * lane < a.head_dim)
    *reinterpret_cast<uint32_t*>(a.out + token * a.o_token + hq * a.o_head + 2 * lane) =
        T::pack2(o.x * inv, o.y * inv);
}

// Which of the two kernels: 64 rows per workgroup for more than 16 rows (24 and 32 rows, 512
// positions, 64 sequences, 8 key heads: 26, 27 us; two tiles of 16 in the other kernel 34, 36), and
// for fewer where the other's workgroups, one per CU (two up to D = 64), would not all run at
// once (4 and 16 rows: 256 sequences of 16 positions 22, 24 us, the other 31, 40; 64 of 512 25,
// 25 and 26, 28; 16 of 2048, which do, 27, 29 either way).
bool by_rows(int64_t max_rows, int64_t seqs, int32_t kv_heads, int32_t head_dim) {
  return max_rows > 16 || seqs * kv_heads > (head_dim <= 64 ? 512 : 256);
}

// Splits that keep the pages of each within what a workgroup stages
int64_t least_splits(int64_t max_len, int32_t page_size) {
  const int64_t limit = static_cast<int64_t>(kTableEntries - 1) * page_size / kMinChunk * kMinChunk;
  return (max_len + limit - 1) / limit;
}

// Splits of the longest context the table holds, by what a call is expected to take (us, from
// timelines on MI355X): a workgroup's fixed time (finding its sequence, its pages and the
// first step, and its result), its positions, the longest last workgroup, and with more
// than one split the second launch and the traffic of the partial results. Lengths are not
// known here: sequences are taken to be 0.6 of the longest on average.
int pick_splits(int64_t tokens, int64_t seqs, int64_t max_len, int32_t page_size, int64_t max_rows, int32_t q_heads,
                int32_t kv_heads, int32_t head_dim) {
  const bool many = by_rows(max_rows, seqs, kv_heads, head_dim);
  const double slots = many ? 512.0 : 256.0;  // workgroups that run at once
  const double fixed = 4.0, per = (many ? 1.1 / 64 : 0.9 / 128) * (head_dim <= 64 ? 0.6 : 1.0);
  // workgroups per split: sequences of few rows need one row block, long ones several
  const double blocks = many ? static_cast<double>(tokens) * (q_heads / kv_heads) / 64 + 0.5 * seqs : seqs;
  const double groups = kv_heads * (blocks > seqs ? blocks : seqs);
  const double merged = static_cast<double>(tokens) * q_heads * head_dim * 8;  // bytes per split, both ways
  const int64_t least = least_splits(max_len, page_size);
  const int64_t most = (max_len + kMinChunk - 1) / kMinChunk;
  int64_t best = 1;
  double best_time = 0.0;
  for (int64_t s = 1; s <= kMaxSplits && s <= most; ++s) {
    const double longest = fixed + per * max_len / s, mean = fixed + per * 0.6 * max_len / s;
    double time = groups * s <= slots ? longest : groups * s * mean / slots + 0.5 * longest;
    if (s > 1) time += 4.0 + merged * s / 4e6;
    if (s == 1 || time < best_time) {
      best = s;
      best_time = time;
    }
  }
  if (const char* env = tuning_env("AWQ_TREE_SPLITS")) best = atoi(env) < most ? atoi(env) : most;
  return static_cast<int>(best > least ? best : least);
}

template <typename Kernel>
hipError_t launch_kernel(Kernel kernel, std::atomic<uint64_t>& lds_done, int lds, const TreeArgs& a, hipStream_t st) {
  const hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kernel), lds, lds_done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(a.row_blocks) * a.splits, a.kv_heads, a.seqs), dim3(256),
                     lds, st, a);
  return hipGetLastError();
}

template <typename T, int DP, bool PAD>
hipError_t launch_pad(const TreeArgs& a, bool many, hipStream_t st) {
  if (!many) {
    static std::atomic<uint64_t> done{0};
    return launch_kernel(&attn_tree_kernel<T, DP, PAD>, done, Lds<DP>::kTotal, a, st);
  }
  static std::atomic<uint64_t> done{0};
  return launch_kernel(&attn_tree_rows_kernel<T, DP, PAD>, done, 4 * kRowStep * DP * 2 + kTableEntries * 4, a, st);
}

template <typename T>
hipError_t launch_t(const TreeArgs& a, bool many, hipStream_t st) {
  const int d = a.head_dim;
  const hipError_t e = d == 64    ? launch_pad<T, 64, false>(a, many, st)
                       : d < 64   ? launch_pad<T, 64, true>(a, many, st)
                       : d == 128 ? launch_pad<T, 128, false>(a, many, st)
                                  : launch_pad<T, 128, true>(a, many, st);
  if (e != hipSuccess || a.part == nullptr) return e;
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
  hipLaunchKernelGGL(attn_tree_merge_kernel<T>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

// workgroups of 64 rows that a sequence's new tokens may need (1 in the kernel of 16 rows)
int64_t row_blocks(int64_t max_rows, int64_t seqs, int32_t kv_heads, int32_t head_dim) {
  return by_rows(max_rows, seqs, kv_heads, head_dim) ? (max_rows + 63) / 64 : 1;
}

int attn_tree_splits(int64_t tokens, int64_t seqs, int64_t table_width, int32_t page_size, int32_t max_q,
                     int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  return pick_splits(tokens, seqs, table_width * page_size, page_size,
                     static_cast<int64_t>(max_q) * (q_heads / kv_heads), q_heads, kv_heads, head_dim);
}

}  // namespace

size_t attn_tree_workspace_bytes(int64_t tokens, int64_t seqs, int64_t table_width, int32_t page_size,
                                 int32_t max_q, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  const int s = attn_tree_splits(tokens, seqs, table_width, page_size, max_q, q_heads, kv_heads, head_dim);
  return s > 1 ? static_cast<size_t>(tokens) * q_heads * s * (head_dim + 2) * 4 : 0;
}

int64_t attn_tree_blocks(int64_t seqs, int64_t table_width, int32_t page_size, int32_t max_q, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim) {
  const int64_t least = least_splits(table_width * page_size, page_size);
  return row_blocks(static_cast<int64_t>(max_q) * (q_heads / kv_heads), seqs, kv_heads, head_dim) *
         (least > kMaxSplits ? least : kMaxSplits);
}

hipError_t launch_attn_tree(const awq_attn_tree_args& g, hipStream_t st) {
  TreeArgs a;
  a.q = static_cast<const uint16_t*>(g.q);
  a.k = static_cast<const uint16_t*>(g.k_cache);
  a.v = static_cast<const uint16_t*>(g.v_cache);
  a.out = static_cast<uint16_t*>(g.out);
  a.table = g.block_table;
  a.ctx = g.ctx_lens;
  a.cu = g.cu_q;
  a.mask = g.mask;
  a.q_token = g.q_token;
  a.q_head = g.q_head;
  a.o_token = g.o_token;
  a.o_head = g.o_head;
  a.cache_page = g.cache_page;
  a.cache_head = g.cache_head;
  a.cache_slot = g.cache_slot;
  a.max_len = g.table_width * g.page_size;
  a.tokens = static_cast<int32_t>(g.tokens);
  a.seqs = static_cast<int32_t>(g.seqs);
  a.table_width = static_cast<int32_t>(g.table_width);
  a.pages = static_cast<int32_t>(g.pages);
  a.page_size = g.page_size;
  a.page_shift = 31;
  while ((int64_t{1} << (a.page_shift - 31)) < g.page_size) ++a.page_shift;
  a.page_mul = static_cast<uint32_t>((uint64_t{1} << a.page_shift) / static_cast<uint32_t>(g.page_size) + 1);
  a.max_q = g.max_q;
  a.q_heads = g.q_heads;
  a.kv_heads = g.kv_heads;
  a.group = g.q_heads / g.kv_heads;
  a.head_dim = g.head_dim;
  a.c = g.scale * kLog2e;
  a.shift = g.dtype == AWQ_DT_F16 ? kShift : -kSlack - log2_up(a.max_len);
  const int64_t rows = static_cast<int64_t>(g.max_q) * a.group;
  const bool many = by_rows(rows, g.seqs, g.kv_heads, g.head_dim);
  a.row_blocks = static_cast<int32_t>(row_blocks(rows, g.seqs, g.kv_heads, g.head_dim));
  a.splits = attn_tree_splits(g.tokens, g.seqs, g.table_width, g.page_size, g.max_q, g.q_heads, g.kv_heads,
                              g.head_dim);
  a.part = a.splits > 1 ? static_cast<float*>(g.ws) : nullptr;
  return g.dtype == AWQ_DT_F16 ? launch_t<F16>(a, many, st) : launch_t<BF16>(a, many, st);
}

}  // namespace awq
