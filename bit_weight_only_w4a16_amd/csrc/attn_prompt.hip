// Causal attention over packed prompts (awq_attn_prompt in awq_block.h).
//
// One pass over the keys with a running maximum and sum per row (float32, base 2; the maximum
// is brought up to date only when a tile needs it, see tile_step). A workgroup owns 128 query
// rows of one key / value head, four wavefronts of 32 tokens of a query head, and walks over
// the keys in tiles of 64 that all four share through LDS. The wavefronts take one query head
// at 128 tokens, or 2 or 4 heads of the group at the same 64 or 32 tokens, which leaves fewer
// rows empty in short sequences (pick_heads).
//
// Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, with the 32 x 32 x 16
// matrix instruction: lane l then holds scores of one query (column l % 32) for 16 keys per
// tile, so the softmax statistics are per lane (one exchange with lane l ^ 32), the factor
// that rescales O is one register, and P never changes lanes: the keys a lane holds after
// S^T, in order, are the contraction slots it feeds to O^T, and the V^T operand is read
// from LDS in that order with the transposing 16-bit read.
//
// The K and V tiles go from memory straight into LDS (16 bytes per lane, no registers), two
// tiles deep, one barrier per tile. Rows are 2 D bytes without padding; the 16-byte chunks
// of a row are permuted (below) so that the rows one LDS access touches fall into different
// banks. Elements past D and rows past the sequence read as 0.
//
// Bound by the matrix instructions and the exponentials together: a tile's 16 + 16 products
// and its 64 exponentials per lane take turns in a wavefront and overlap only between the two
// wavefronts of a SIMD. One sequence of 8192 tokens, 32 heads on 8, D = 128: 541-563 us, 1.0
// PFLOP/s of the triangle's products (a large matrix product reaches 1.3); six ragged
// prompts of 1 to 2048 tokens (bfloat16) 107-110 us, 0.76-0.78 PFLOP/s (the last tiles and the
// diagonals; both a quarter longer right after a pause); five of 1 to 120 tokens 8.0 us, of
// which the launch and the first tile's way from memory are most. 64 keys and 128 rows leave 104 registers and 64 KiB of LDS, two workgroups per CU;
// 256 rows were 1.5 % faster on the long sequence and 10 % slower on the ragged ones.
#include "block_internal.hpp"

#include <math.h>

#include <type_traits>

namespace awq {
namespace {

constexpr int kBK = 64;  // keys per tile

struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t* cu;
  int64_t q_token, k_token, v_token, o_token, q_head, k_head, v_head, o_head;
  int32_t tokens, seqs, tiles, q_heads, group, head_dim;
  int32_t heads_log2;  // of a workgroup's query heads; its tokens are 128 >> heads_log2
  float c;  // scale * log2(e)
  float shift, most;  // see tile_step
};

// chunk position of chunk c of row r in LDS. K is read 16 rows at one chunk, V 4 rows x 64
// bytes; with 128-byte rows (DP = 64) two rows share a 256-byte line.
template <int DP>
__device__ __forceinline__ int k_pos(int r, int c) {
  return DP == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int v_pos(int r, int c) {
  return DP == 128 ? c ^ ((r & 3) << 2) : c ^ (((r >> 1) & 1) << 2);
}

// Finds the sequence of query tile `tile` and which of its tiles that is. Sequence b's tiles
// are numbered from cu[b] / size + b, which leaves each its ceil(length / size) numbers and
// few unused ones, and needs no sum over the sequences before: 64 lanes search 64 ways.
// Returns false where the number is unused.
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int tile, int& start, int& len, int& q0) {
  const int lane = threadIdx.x & 63, shift = 7 - a.heads_log2;
  int b0 = 0, count = a.seqs;
  while (true) {  // the last of the sequences [b0, b0 + count) that starts at or before the tile
    const int stride = (count + 63) >> 6, mine = lane * stride, b = b0 + mine;
    int s = 0, e = 0;
    if (mine < count) {
      s = min(max(a.cu[b], 0), a.tokens);
      e = min(max(a.cu[b + 1], 0), a.tokens);
    }
    const uint64_t before = __ballot(mine < count && (s >> shift) + b <= tile);
    if (before == 0) return false;
    const int w = 63 - __builtin_clzll(before);
    if (stride == 1) {
      start = __builtin_amdgcn_readlane(s, w);
      len = __builtin_amdgcn_readlane(e, w) - start;
      q0 = (tile - (start >> shift) - b0 - w) << shift;
      return q0 < len;
    }
    b0 += w * stride;
    count = min(stride, count - w * stride);
  }
}

// Which query heads (from `head` on) and tile a workgroup takes. Workgroups go round the 8
// XCDs, and each XCD's L2 should see as few key / value heads as possible: XCD x takes head
// x, x + 8, .. one after the other where the heads are a multiple of 8, and an equal share of
// the tiles of head x % kv_heads where they divide 8. On an XCD the parts of the group come
// first (they read the same keys together), then the tiles, a sequence's last (longest) first.
__device__ __forceinline__ void work_item(const PromptArgs& a, int& head, int& tile) {
  const int kv_heads = a.q_heads / a.group, parts = a.group >> a.heads_log2, i = blockIdx.x;
  int kv, at;  // key head, number among its tiles x parts of the group
  if (kv_heads % 8 == 0) {
    const int per = a.tiles * parts, slot = i >> 3;
    kv = (i & 7) + 8 * (slot / per);
    at = slot % per;
  } else if (8 % kv_heads == 0) {
    kv = (i & 7) % kv_heads;
    at = (i >> 3) * (8 / kv_heads) + (i & 7) / kv_heads;
  } else {
    kv = i / parts % kv_heads;
    at = i / (kv_heads * parts) * parts + i % parts;
  }
  head = kv * a.group + (at % parts << a.heads_log2);
  tile = a.tiles - 1 - at / parts;  // < 0 past the last of an uneven share
}

template <typename T, int DP>
__global__ void __launch_bounds__(256, 2) attn_prompt_kernel(PromptArgs a) {
  constexpr int RB = DP * 2;            // bytes of a row in LDS
  constexpr int RC = DP / 8;            // 16-byte chunks of a row
  constexpr int TILE = kBK * RB;        // bytes of a K or V tile
  constexpr int ROWS = 1024 / RB;       // rows one load instruction of a wavefront fills
  constexpr int LOADS = kBK / ROWS / 4;  // load instructions per wavefront and tile
  constexpr int NC = DP / 16, ND = DP / 32;
  typedef typename T::v8 v8;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];  // [2][K tile, V tile]

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int col = lane & 31, h = lane >> 5;

  int head, tile;
  work_item(a, head, tile);
  int start, len, q0;
  if (!find_tile(a, tile, start, len, q0)) return;
  start = __builtin_amdgcn_readfirstlane(start);
  len = __builtin_amdgcn_readfirstlane(len);
  q0 = __builtin_amdgcn_readfirstlane(q0);
  const int kv_head = head / a.group, size = 128 >> a.heads_log2;
  const int sub = wave & ((4 >> a.heads_log2) - 1);  // which 32 of the tile's tokens
  head += wave >> (2 - a.heads_log2);
  const int wq0 = q0 + 32 * sub;  // this wavefront's first row
  const int row = wq0 + col;      // this lane's row

  const uint16_t* kbase = a.k + start * a.k_token + kv_head * a.k_head;
  const uint16_t* vbase = a.v + start * a.v_token + kv_head * a.v_head;

  // tile loads: instruction j of wavefront w fills rows ROWS (LOADS w + j).., lane l row
  // l / RC of them, chunk position l % RC
  uint32_t k_off[LOADS], v_off[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int r = ROWS * (LOADS * wave + j) + lane / RC;
    const int ck = k_pos<DP>(r, lane % RC), cv = v_pos<DP>(r, lane % RC);
    k_off[j] = 8 * ck < a.head_dim ? static_cast<uint32_t>(r * a.k_token + 8 * ck) * 2 : kNoLoad;
    v_off[j] = 8 * cv < a.head_dim ? static_cast<uint32_t>(r * a.v_token + 8 * cv) * 2 : kNoLoad;
  }
  auto load_tile = [&](int j) {
    const int kv0 = j * kBK, rows = min(kBK, len - kv0);
    const u32x4 rk =
        rsrc_words(kbase + kv0 * a.k_token, static_cast<uint32_t>((rows - 1) * a.k_token + a.head_dim) * 2);
    const u32x4 rv =
        rsrc_words(vbase + kv0 * a.v_token, static_cast<uint32_t>((rows - 1) * a.v_token + a.head_dim) * 2);
    const uint32_t dst = lds_offset(smem) + (j & 1) * 2 * TILE + LOADS * wave * 1024;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(rk, k_off[i], dst + i * 1024);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(rv, v_off[i], dst + TILE + i * 1024);
  };

  // key tiles this workgroup needs, and this wavefront (none where its rows are past the end)
  const int tiles = (min(len, q0 + size) + kBK - 1) / kBK;
  const int mine = wq0 < len ? min(tiles, (wq0 + 31) / kBK + 1) : 0;

  // Q^T operand: column l % 32, channels 16 c + 8 h .. + 7 (rows past the sequence: 0)
  v8 qf[NC];
  {
    const int rows = min(size, len - q0);
    const __amdgpu_buffer_rsrc_t rq =
        make_rsrc(a.q + (start + q0) * a.q_token + head * a.q_head,
                  static_cast<uint32_t>((rows - 1) * a.q_token + a.head_dim) * 2);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 16 * c + 8 * h;
      const uint32_t off =
          d < a.head_dim ? static_cast<uint32_t>((32 * sub + col) * a.q_token + d) * 2 : kNoLoad;
      qf[c] = __builtin_bit_cast(v8, buf_load16(rq, off, 0));
    }
  }

  float16_t acc[ND];
#pragma unroll
  for (int t = 0; t < ND; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.0f;
  float m = kNegInf;  // maximum in use (see below), in units of scores * c
  float l = 0.0f;     // this lane's part of the sum
  float off = -kNegInf;  // a.shift - m

  // LDS read positions
  const int tr_row = 4 * h + ((lane & 15) >> 2);                       // + 16 cc + 32 s (+ 8)
  const int tr_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);      // + 4 dt
  const int tr_byte = 8 * (lane & 1);

  // Tile j (from buffer `buf`). The probabilities are first formed with the maximum in use,
  // whatever the tile's own is, and added up as they were rounded: two ALU instructions per
  // pair and none for a maximum. Where the sum ran past `most` = 2^(shift + 10) (or is NaN: an
  // infinite one in binary16), the maximum and what was summed so far are brought up to date
  // and the tile's probabilities formed again. P carries 2^shift. In binary16 that is 2^12,
  // which keeps what is far below the maximum out of the subnormals; a maximum in use up to
  // 2^4 too low only makes P larger. bfloat16 has float32's exponents, and there it is small
  // enough (2^-6 / tokens) that all of a row's P add up to less than 1 (32 keys of a lane and
  // tile to at most `most`): no sum of values of any size passes float32's largest.
  auto tile_step = [&](auto buf_, int j) {
    const unsigned char* ks = smem + decltype(buf_)::value * 2 * TILE;
    const unsigned char* vs = ks + TILE;
    auto k_frag = [&](int t, int c) {
      const int r = 32 * t + col;
      return *reinterpret_cast<const v8*>(ks + r * RB + 16 * k_pos<DP>(r, 2 * c + h));
    };
    // all K fragments are read before the first product (left to itself the compiler reads
    // each right before its use and waits for LDS sixteen times)
    float16_t s[2];
    v8 kf[2][NC];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < NC; ++c) kf[t][c] = k_frag(t, c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) s[t] = T::mfma32(kf[t][c], qf[c], s[t]);
    }
    if (j * kBK + kBK - 1 > wq0) {  // the tile reaches past some row of the wavefront
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = j * kBK + 32 * t + 8 * (i >> 2) + 4 * h + (i & 3);
          s[t][i] = key <= row ? s[t][i] : kNegInf;
        }
    }
    u32x4 p[4];  // P^T operands of the four 16-key steps
    auto probabilities = [&]() {
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const uint32_t pair = T::pack2(__builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], a.c, off)),
                                         __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i + 1], a.c, off)));
          sum = T::add2(pair, sum);
          p[2 * t + (i >> 3)][(i >> 1) & 3] = pair;
        }
      return sum;
    };
    float sum = probabilities();
    if (__ballot(!(sum < a.most)) != 0) {
      float top = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
      top = fmaxf(m, xor32_max(top) * a.c);
      // a row that has seen only scores of -inf: they give 0 with off = 0, and the next tile
      // comes here again
      const bool none = top == kNegInf;
      const float keep = none ? 1.0f : __builtin_amdgcn_exp2f(m - top);
      m = top;
      off = none ? 0.0f : a.shift - m;
      l *= keep;
#pragma unroll
      for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] *= keep;
      sum = probabilities();
      off = a.shift - m;
    }
    l += sum;
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      const v8 pf = __builtin_bit_cast(v8, p[cc]);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        const int r0 = 16 * cc + tr_row, r1 = r0 + 8;
        const int ch = 4 * dt + tr_chunk;
        const short4_t lo = lds_read_tr(vs + r0 * RB + 16 * v_pos<DP>(r0, ch) + tr_byte);
        const short4_t hi = lds_read_tr(vs + r1 * RB + 16 * v_pos<DP>(r1, ch) + tr_byte);
        acc[dt] = T::mfma32(join8<v8>(lo, hi), pf, acc[dt]);
      }
    }
  };

  load_tile(0);
  auto pass = [&](auto buf, int j) {
    wait_loads<0>();  // this wavefront's loads of the tile have landed
    lds_barrier();    // everyone's have, and the other buffer is free
    if (j + 1 < tiles) load_tile(j + 1);
    if (j < mine) tile_step(buf, j);
  };
  for (int j = 0; j < tiles; j += 2) {
    pass(std::integral_constant<int, 0>{}, j);
    if (j + 1 < tiles) pass(std::integral_constant<int, 1>{}, j + 1);
  }

  l = xor32_add(l);
  const float inv = inv_sum(l);
  bool broken = false;
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) broken |= acc[dt][i] != acc[dt][i];
  // Rows that came out NaN though their probabilities' sum is not (masked ones add exactly 0),
  // and an infinity or NaN among the values of the diagonal's tile, which some rows do not see:
  // the products once more without that tile, whose values each row gets key by key. (Here and
  // not in the loop: a look at the tile's values there cost every call 1 to 9 %.) 4096 tokens, 32
  // heads, one NaN in the first value 0.4 ms, without it 0.17.
  if (__ballot(broken && row < len && l == l) != 0) {
    const int diagonal = (mine - 1) * kBK;
    bool finite = true;
    if (diagonal + lane < len)
      for (int d = 0; d < a.head_dim; d += 8)
        finite = finite && T::finite8(*reinterpret_cast<const u32x4*>(vbase + (diagonal + lane) * a.v_token + d));
    if (__ballot(!finite) != 0) {
      const float shift = m == kNegInf ? 0.0f : a.shift - m;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
#pragma unroll 1
      for (int kv0 = 0; kv0 < diagonal; kv0 += 32) {
        float16_t s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = 16 * c + 8 * h;
          u32x4 k = {0, 0, 0, 0};
          if (d < a.head_dim) k = *reinterpret_cast<const u32x4*>(kbase + (kv0 + col) * a.k_token + d);
          s = T::mfma32(__builtin_bit_cast(v8, k), qf[c], s);
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          u32x4 p;
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            p[i >> 1] = T::pack2(__builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * cc + i], a.c, shift)),
                                 __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * cc + i + 1], a.c, shift)));
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) {
            typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
            u16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
            if (32 * dt + col < a.head_dim) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                v[i] = vbase[(kv0 + 16 * cc + 8 * (i >> 2) + 4 * h + (i & 3)) * a.v_token + 32 * dt + col];
            }
            acc[dt] = T::mfma32(__builtin_bit_cast(v8, v), __builtin_bit_cast(v8, p), acc[dt]);
          }
        }
      }
      if (row < len)
        add_keys<T, 4 * ND>(
            a.q + (start + row) * a.q_token + head * a.q_head, a.head_dim, a.c, shift, diagonal, min(len, wq0 + 32),
            4 * h, 8,
            [&](int j, const uint16_t*& kr, const uint16_t*& vr) {
              kr = kbase + j * a.k_token;
              vr = vbase + j * a.v_token;
              return j <= row;
            },
            [&](int r, int i, float p, float x) {
              acc[r >> 2][4 * (r & 3) + i] = __builtin_fmaf(p, x, acc[r >> 2][4 * (r & 3) + i]);
            });
    }
  }
  if (row < len) {
    uint16_t* o = a.out + (start + row) * a.o_token + head * a.o_head;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * dt + 2 * i + 4 * h;
        if (d < a.head_dim)
          *reinterpret_cast<uint2*>(o + d) = make_uint2(T::pack2(acc[dt][i] * inv, acc[dt][i + 1] * inv),
                                                        T::pack2(acc[dt][i + 2] * inv, acc[dt][i + 3] * inv));
      }
  }
}

template <typename T, int DP>
hipError_t launch_dp(const PromptArgs& a, int64_t blocks, hipStream_t st) {
  constexpr int lds = 4 * kBK * DP * 2;
  static std::atomic<uint64_t> lds_done{0};
  const hipError_t e =
      ensure_lds_limit(reinterpret_cast<const void*>(&attn_prompt_kernel<T, DP>), lds, lds_done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_prompt_kernel<T, DP>), dim3(static_cast<unsigned>(blocks)), dim3(256), lds, st, a);
  return hipGetLastError();
}

// Heads of a workgroup (log2). Many short sequences: as many as divide the group, for each
// workgroup then fills its rows and a group's keys are read once (32 query heads on 8, D =
// 128, 16 tokens each: 64, 256, 1024 sequences take 13, 35, 135 us; one head at a time 23, 83,
// 332). From 256 tokens on, and where one head at a time leaves workgroups' slots empty, one:
// the batches measured then take the same within 1 % (1 x 16 tokens 5.9 us, with four heads
// 6.7; 6 ragged prompts of 993 tokens on average 121, 123; 8192 tokens 548, 552).
int pick_heads(int64_t tokens, int64_t seqs, int q_heads, int group) {
  if (tokens >= 256 * seqs || seqs * q_heads <= 512) return 0;
  return group % 4 == 0 ? 2 : group % 2 == 0 ? 1 : 0;
}

}  // namespace

hipError_t launch_attn_prompt(const awq_attn_prompt_args& g, hipStream_t st) {
  PromptArgs a;
  a.q = static_cast<const uint16_t*>(g.q);
  a.k = static_cast<const uint16_t*>(g.k);
  a.v = static_cast<const uint16_t*>(g.v);
  a.out = static_cast<uint16_t*>(g.out);
  a.cu = g.cu;
  a.q_token = g.q_token;
  a.k_token = g.k_token;
  a.v_token = g.v_token;
  a.o_token = g.o_token;
  a.q_head = g.q_head;
  a.k_head = g.k_head;
  a.v_head = g.v_head;
  a.o_head = g.o_head;
  a.tokens = static_cast<int32_t>(g.tokens);
  a.seqs = static_cast<int32_t>(g.seqs);
  a.q_heads = g.q_heads;
  a.group = g.q_heads / g.kv_heads;
  a.head_dim = g.head_dim;
  a.heads_log2 = pick_heads(g.tokens, g.seqs, g.q_heads, a.group);
  const int64_t tiles = (g.tokens >> (7 - a.heads_log2)) + g.seqs;  // (the numbers, see find_tile)
  a.tiles = static_cast<int32_t>(tiles);
  a.c = g.scale * kLog2e;
  a.shift = g.dtype == AWQ_DT_F16 ? 12.0f : -6.0f - log2_up(g.tokens);
  a.most = exp2f(a.shift + 10.0f);
  const int64_t blocks = ((tiles * g.q_heads >> a.heads_log2) + 7) / 8 * 8;  // (an uneven share leaves some idle)
  if (g.dtype == AWQ_DT_F16)
    return g.head_dim <= 64 ? launch_dp<F16, 64>(a, blocks, st) : launch_dp<F16, 128>(a, blocks, st);
  return g.head_dim <= 64 ? launch_dp<BF16, 64>(a, blocks, st) : launch_dp<BF16, 128>(a, blocks, st);
}

}  // namespace awq
