// Rotary positions for q and k with the write of k and v into the paged cache
// (awq_rope in awq_block.h).
//
// Three multiply-adds per element: the kernel is bound by reading and writing each element
// once (671 MB of 16384 tokens x 72 heads in 146 us, 4.6 TB/s; 50 MB of 2048 tokens x 48
// heads in 10.6 us, 4.7 TB/s; a large copy moves 4.95 TB/s; one token of 96 heads 3.6 us, the
// launch and two memory round trips). A thread owns one chunk position of the head (V first elements and V second
// elements of V pairs: 16 + 16 bytes) of one token, forms the V cosines and sines once, and
// walks over a share of the heads with them, so the trigonometry is paid once per token
// and share and not per head.
//
// The angle in turns, positions * inv_freq / (2 pi), is formed and reduced to [-1/2, 1/2] in
// float64: at position 10^5 a float32 product would be off by up to 0.004 rad. The hardware
// sine and cosine take turns; at most 8 of them per thread, they hide behind the loads.
#include "block_internal.hpp"

namespace awq {
namespace {

constexpr double kInvTwoPi = 0.15915494309189533577;

// V elements as one access
template <int V>
struct Vec;
template <>
struct Vec<8> {
  typedef uint4 type;
};
template <>
struct Vec<2> {
  typedef uint32_t type;
};
template <>
struct Vec<1> {
  typedef uint16_t type;
};

template <int V>
union Elems {
  typename Vec<V>::type vec;
  uint16_t e[V];
};

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(awq_rope_args a, int heads_per_thread) {
  typedef typename Vec<V>::type vec;
  const int rot_chunks = a.rot_dim / (2 * V), chunks = rot_chunks + (a.head_dim - a.rot_dim) / V;
  // (a launch holds 2^32 threads along x)
  const int64_t i = (static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= a.tokens) return;
  const int c = static_cast<int>(i - t * chunks);
  const bool turns = c < rot_chunks;
  // the chunk's first and second elements; past rot_dim one run of V elements to copy
  int at0, at1;
  if (!turns) {
    at0 = at1 = a.rot_dim + (c - rot_chunks) * V;
  } else if (INTERLEAVED) {
    at0 = 2 * V * c;
    at1 = at0 + V;
  } else {
    at0 = V * c;
    at1 = at0 + a.rot_dim / 2;
  }
  float cs[V], sn[V];
  if (turns) {
    const double pos = static_cast<double>(a.positions[t]) * kInvTwoPi;
    const float sign = a.inverse ? -a.scale : a.scale;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const double turn = pos * static_cast<double>(a.inv_freq[V * c + e]);
      const float f = static_cast<float>(turn - __builtin_rint(turn));
      cs[e] = a.scale * __builtin_amdgcn_cosf(f);
      sn[e] = sign * __builtin_amdgcn_sinf(f);
    }
  }
  int64_t cache_at = -1;
  if (a.slots != nullptr) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < a.pages * a.page_size) {
      const int64_t page = slot / a.page_size;
      cache_at = page * a.cache_page + (slot - page * a.page_size) * a.cache_slot;
    }
  }
  const int rows = a.q_heads + 2 * a.kv_heads;
  const int h0 = blockIdx.y * heads_per_thread, h1 = min(rows, h0 + heads_per_thread);
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
    const int hk = is_q ? h : is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
    const uint16_t* src;
    uint16_t *dst, *dst2 = nullptr;
    if (is_q) {
      src = static_cast<const uint16_t*>(a.q) + t * a.q_token + hk * a.q_head;
      dst = static_cast<uint16_t*>(a.q_out) + t * a.qo_token + hk * a.qo_head;
    } else {
      void* cache = is_v ? a.v_cache : a.k_cache;
      src = is_v ? static_cast<const uint16_t*>(a.v) + t * a.v_token + hk * a.v_head
                 : static_cast<const uint16_t*>(a.k) + t * a.k_token + hk * a.k_head;
      dst = cache != nullptr && cache_at >= 0
                ? static_cast<uint16_t*>(cache) + cache_at + hk * a.cache_head
                : nullptr;
      if (!is_v && a.k_out != nullptr)
        dst2 = static_cast<uint16_t*>(a.k_out) + t * a.ko_token + hk * a.ko_head;
    }
    if (dst == nullptr && dst2 == nullptr) continue;
    Elems<V> x, y;
    x.vec = *reinterpret_cast<const vec*>(src + at0);
    y.vec = *reinterpret_cast<const vec*>(src + at1);
    if (turns && !is_v) {
      if (INTERLEAVED) {
        // elements of x, then of y, in pairs
        Elems<V> rx = x, ry = y;
        if constexpr (V >= 2) {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float p = T::to_float(x.e[2 * e]), q = T::to_float(x.e[2 * e + 1]);
            rx.e[2 * e] = T::bits(p * cs[e] - q * sn[e]);
            rx.e[2 * e + 1] = T::bits(q * cs[e] + p * sn[e]);
            const float u = T::to_float(y.e[2 * e]), w = T::to_float(y.e[2 * e + 1]);
            ry.e[2 * e] = T::bits(u * cs[V / 2 + e] - w * sn[V / 2 + e]);
            ry.e[2 * e + 1] = T::bits(w * cs[V / 2 + e] + u * sn[V / 2 + e]);
          }
        } else {
          const float p = T::to_float(x.e[0]), q = T::to_float(y.e[0]);
          rx.e[0] = T::bits(p * cs[0] - q * sn[0]);
          ry.e[0] = T::bits(q * cs[0] + p * sn[0]);
        }
        x = rx;
        y = ry;
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float p = T::to_float(x.e[e]), q = T::to_float(y.e[e]);
          x.e[e] = T::bits(p * cs[e] - q * sn[e]);
          y.e[e] = T::bits(q * cs[e] + p * sn[e]);
        }
      }
    }
    if (dst != nullptr) {
      *reinterpret_cast<vec*>(dst + at0) = x.vec;
      if (turns) *reinterpret_cast<vec*>(dst + at1) = y.vec;
    }
    if (dst2 != nullptr) {
      *reinterpret_cast<vec*>(dst2 + at0) = x.vec;
      if (turns) *reinterpret_cast<vec*>(dst2 + at1) = y.vec;
    }
  }
}

template <typename T, int V>
hipError_t launch_v(const awq_rope_args& a, hipStream_t st) {
  const int chunks = a.rot_dim / (2 * V) + (a.head_dim - a.rot_dim) / V;
  const int64_t blocks = (a.tokens * chunks + 255) / 256;
  const int rows = a.q_heads + 2 * a.kv_heads;
  // heads per thread: enough threads to fill the chip first, then up to 8 for one set of
  // cosines (1, 4, 8, 16 heads: one token 4.1, 4.8, 6.7, 10.5 us; 2048 tokens x 48 heads 12.7,
  // 10.7, 12.3, 17.4; 16384 tokens x 72 heads 157, 149, 145, 167)
  const int64_t share = blocks * rows / 2048;
  const int per = share < 1 ? 1 : share > 8 ? 8 : static_cast<int>(share);
  const int64_t z = (blocks + (1 << 23) - 1) >> 23;
  const dim3 grid(static_cast<unsigned>((blocks + z - 1) / z), static_cast<unsigned>((rows + per - 1) / per),
                  static_cast<unsigned>(z));
  if (a.interleaved) {
    hipLaunchKernelGGL((rope_kernel<T, V, true>), grid, dim3(256), 0, st, a, per);
  } else {
    hipLaunchKernelGGL((rope_kernel<T, V, false>), grid, dim3(256), 0, st, a, per);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const awq_rope_args& a, hipStream_t st) {
  // 16-byte accesses where the pairs' halves start on them, else 4 or 2 bytes
  if (a.rot_dim % 16 == 0) return launch_v<T, 8>(a, st);
  if (a.rot_dim % 4 == 0) return launch_v<T, 2>(a, st);
  return launch_v<T, 1>(a, st);
}

}  // namespace

hipError_t launch_rope(const awq_rope_args& args, hipStream_t st) {
  awq_rope_args a = args;
  if (a.q == nullptr) a.q_heads = 0;
  if (a.k == nullptr) a.kv_heads = 0;
  return a.dtype == AWQ_DT_F16 ? launch_t<F16>(a, st) : launch_t<BF16>(a, st);
}

}  // namespace awq
