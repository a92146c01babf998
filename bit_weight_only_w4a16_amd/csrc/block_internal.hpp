// Internal declarations and device helpers of the decoder-block operators (awq_block.h).
#pragma once

#include "../../include/awq_block.h"
#include "awq_internal.hpp"

namespace awq {

hipError_t launch_rope(const awq_rope_args& a, hipStream_t st);
hipError_t launch_attn_prompt(const awq_attn_prompt_args& a, hipStream_t st);
size_t attn_tree_workspace_bytes(int64_t tokens, int64_t seqs, int64_t table_width, int32_t page_size,
                                 int32_t max_q, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
// most workgroups of a call along x: row blocks times splits
int64_t attn_tree_blocks(int64_t seqs, int64_t table_width, int32_t page_size, int32_t max_q, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim);
hipError_t launch_attn_tree(const awq_attn_tree_args& a, hipStream_t st);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

// the least n with 2^n >= v, for v >= 1
inline float log2_up(int64_t v) {
  int n = 0;
  while ((int64_t{1} << n) < v) ++n;
  return static_cast<float>(n);
}

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The two element types: conversions round to nearest even.
struct F16 {
  typedef half8_t v8;
  static __device__ __forceinline__ float to_float(uint16_t b) {
    return static_cast<float>(__builtin_bit_cast(_Float16, b));
  }
  static __device__ __forceinline__ uint16_t bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, half2_t));
  }
  // sum + the two elements of a pair, in float32
  static __device__ __forceinline__ float add2(uint32_t pair, float sum) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2_t, pair), half2_t{1.0f, 1.0f}, sum, false);
  }
  // whether eight elements are neither infinities nor NaN
  static __device__ __forceinline__ bool finite8(u32x4 x) {
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      finite = finite && (x[i] & 0x7C00u) != 0x7C00u && (x[i] & 0x7C000000u) != 0x7C000000u;
    return finite;
  }
  static __device__ __forceinline__ float16_t mfma32(v8 a, v8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float4_t mfma16(v8 a, v8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
struct BF16 {
  typedef bf8_t v8;
  static __device__ __forceinline__ float to_float(uint16_t b) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16);
  }
  static __device__ __forceinline__ uint16_t bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, bf2_t));
  }
  static __device__ __forceinline__ float add2(uint32_t pair, float sum) {
    const bf2_t ones = {static_cast<__bf16>(1.0f), static_cast<__bf16>(1.0f)};
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2_t, pair), ones, sum, false);
  }
  // whether eight elements are neither infinities nor NaN
  static __device__ __forceinline__ bool finite8(u32x4 x) {
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      finite = finite && (x[i] & 0x7F80u) != 0x7F80u && (x[i] & 0x7F800000u) != 0x7F800000u;
    return finite;
  }
  static __device__ __forceinline__ float16_t mfma32(v8 a, v8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float4_t mfma16(v8 a, v8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// Loads from memory straight into LDS: lane l's 16 bytes go to LDS byte `dst` + 16 l (dst the
// same in all lanes). Written as assembly because the compiler, which cannot tell the
// stages of a ring apart, waits for every such load of its own before each transposing LDS
// read (the prefetched step would be waited for in the middle of the one before it). The
// instructions have no register result; the kernels wait with wait_loads, and a wait that
// the compiler counts for a load of its own only gets longer by these.
__device__ __forceinline__ uint32_t lds_offset(const void* shared) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const unsigned char*)(shared)));
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}
__device__ __forceinline__ void load_to_lds(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(uniform(dst)), "v"(src)
               : "m0", "memory");
}
// the same from a buffer resource: an offset past its end writes zeros
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t offset, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(uniform(dst)), "v"(offset), "s"(rsrc)
               : "m0", "memory");
}
// the words of make_rsrc's resource, in scalar registers
__device__ __forceinline__ u32x4 rsrc_words(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{uniform(static_cast<uint32_t>(a)), uniform(static_cast<uint32_t>(a >> 32) & 0xFFFFu), uniform(bytes),
               0x00020000u};
}
// Waits until at most N of this wavefront's memory loads are on their way (they land in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  // vmcnt in bits 0..3 and 14..15, the other counters at their largest: not waited for
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  asm volatile("" ::: "memory");
}
// Waits for this wavefront's LDS accesses.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) only
  asm volatile("" ::: "memory");
}
// A barrier for LDS alone: loads into LDS that are on their way stay so.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) short4_t lds_short4;

// Transposed LDS read of 16-bit elements: lane i of each group of 16 lanes gets element
// i % 4 of the 8 bytes that lane 4 r + i / 4 of its group points at, for r = 0 .. 3. With
// lane j pointing at row j / 4, columns 4 (j % 4).. of a 4 x 16 block, lane i gets column i.
__device__ __forceinline__ short4_t lds_read_tr(const unsigned char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(p));
}
template <typename V8>
__device__ __forceinline__ V8 join8(short4_t a, short4_t b) {
  typedef short short8_t __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(V8, short8_t{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
}

// v combined with that of the lane 32 lanes away, by maximum / sum. The swap instruction
// exchanges one operand's upper half with the other's lower: of v and a copy of it, the
// results are the lower halves twice and the upper halves twice. (The copy is opaque to
// the compiler, which otherwise takes the two results for one value.)
__device__ __forceinline__ float2_t halves(float v) {
  unsigned int a = __builtin_bit_cast(unsigned int, v), b = a;
  asm("" : "+v"(b));
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  const unsigned int lo = r[0], hi = r[1];
  return float2_t{__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float xor32_max(float v) {
  const float2_t h = halves(v);
  return fmaxf(h.x, h.y);
}
__device__ __forceinline__ float xor32_add(float v) {
  const float2_t h = halves(v);
  return h.x + h.y;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

// 1 / sum of a row's probabilities; 0 for a row that saw nothing
__device__ __forceinline__ float inv_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// Values that a row does not see have probability 0, and the matrix instruction multiplies them
// with it: an infinity or NaN among them makes the row NaN. That can only happen in the steps
// that hold values which not every row sees (a causal tile's diagonal, the new tokens). Where it
// may have, a kernel forms its sums without such a step, and add_keys adds what each row
// sees of it, key by key. What is NaN after that is NaN by its definition, in its own channel.

// v, of which the compiler knows nothing: what is computed from it is computed there, and not kept
// in registers over a loop for code that hardly ever runs.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// p_j v_j of keys first .. end - 1 that this lane's row sees, in float32, with the probabilities
// rounded as the matrix instruction takes them: channels at + step r .. + 3 by add(r, i, p, v)
// for r < RUNS, i < 4. key(j, k, v) gives key j's rows and whether the row sees it.
template <typename T, int RUNS, typename Key, typename Add>
__device__ __forceinline__ void add_keys(const uint16_t* q, int head_dim, float c, float off, int first, int end, int at,
                                         int step, Key key, Add add) {
#pragma unroll 1
  for (int j = first; j < end; ++j) {
    const uint16_t *k, *v;
    if (!key(j, k, v)) continue;
    float dot = 0.0f;
#pragma unroll 1
    for (int d = 0; d < head_dim; d += 8) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(q + d), b = *reinterpret_cast<const u32x4*>(k + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dot = __builtin_fmaf(T::to_float(a[i] & 0xFFFFu), T::to_float(b[i] & 0xFFFFu), dot);
        dot = __builtin_fmaf(T::to_float(a[i] >> 16), T::to_float(b[i] >> 16), dot);
      }
    }
    const float p = T::to_float(T::bits(__builtin_amdgcn_exp2f(__builtin_fmaf(dot, c, off))));
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if (at + step * r >= head_dim) continue;
      const uint2 x = *reinterpret_cast<const uint2*>(v + at + step * r);
      add(r, 0, p, T::to_float(x.x & 0xFFFFu));
      add(r, 1, p, T::to_float(x.x >> 16));
      add(r, 2, p, T::to_float(x.y & 0xFFFFu));
      add(r, 3, p, T::to_float(x.y >> 16));
    }
  }
}

}  // namespace awq
