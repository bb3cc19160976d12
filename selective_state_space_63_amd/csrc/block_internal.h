// block_internal.h -- device and host helpers of the block operators (the C
// ABI is include/s6_block.h): the multi-head scan (heads_*.hip) and the norms
// (norm.hip).
#ifndef S6_BLOCK_INTERNAL_H_
#define S6_BLOCK_INTERNAL_H_

#include "s6_block.h"
#include "s6_internal.h"

namespace s6i {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two floats as packed bf16 (round to nearest even).
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf_low(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf_high(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return v;
}

// V consecutive elements as floats (V = 4 or 8: vector loads of an address
// aligned to min(16, V * sizeof(T)) bytes; V = 1: one element).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = to_f32(*p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else if constexpr (V == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = bf_low(v.x); f[1] = bf_high(v.x); f[2] = bf_low(v.y); f[3] = bf_high(v.y);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    f[0] = bf_low(v.x); f[1] = bf_high(v.x); f[2] = bf_low(v.y); f[3] = bf_high(v.y);
    f[4] = bf_low(v.z); f[5] = bf_high(v.z); f[6] = bf_low(v.w); f[7] = bf_high(v.w);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]));
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]), bf_pack(f[4], f[5]), bf_pack(f[6], f[7]));
  }
}

// Sum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dpp_f<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dpp_f<0x141>(v);  // row_half_mirror
  v += dpp_f<0x140>(v);  // row_mirror
  return v;
}
// Sum over lanes l and l ^ 16 (rows 2i and 2i + 1), in every lane.
__device__ __forceinline__ float pair_row_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sum over lanes l and l ^ 32, in every lane.
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float wave_sum(float v) { return half_sum(pair_row_sum(row_sum(v))); }

// A decay's exponent in log2 units, held above -150: 2^-150 is 0 in fp32, and
// sums of a chunk stay finite where a step or A is infinite (a NaN passes).
constexpr float kMinLog2 = -150.0f;
__device__ __forceinline__ float clamp_log2(float v) { return v < kMinLog2 ? kMinLog2 : v; }

// ------------------------------------------------------------ host helpers --
constexpr int kMaxHeadState = 128;  // largest dstate of the heads entry points

// Sizes, types, flags and strides of a heads call (seqlen and token strides
// only where tokens is set).
int check_heads(const s6_heads_dims* d, int in_dtype, int flags, bool has_delta, bool has_bias, bool tokens);

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace s6i

#endif  // S6_BLOCK_INTERNAL_H_
