// Loads and stores of values whose storage type is chosen at run time or by template (bf16, binary16,
// fp32), always as fp32 in registers.
#pragma once
#include "common.hpp"

namespace moe {

template <int DT>
struct Val;  // storage type of a moe_dtype
template <>
struct Val<MOE_DT_BF16> {
  typedef uint16_t S;
  static __device__ __forceinline__ float get(S v) { return bf16_bits_to_f32(v); }
};
template <>
struct Val<MOE_DT_FP16> {
  typedef uint16_t S;
  static __device__ __forceinline__ float get(S v) { return (float)bitcast<_Float16>(v); }
};
template <>
struct Val<MOE_DT_FP32> {
  typedef float S;
  static __device__ __forceinline__ float get(S v) { return v; }
};

// Eight consecutive values as they are stored (16 or 32 bytes), and their fp32 values.  The addresses need a
// value's alignment only: gfx950 takes 16-byte global accesses at any address.
template <int DT>
struct Raw8 {
  u32x4 q[DT == MOE_DT_FP32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> ld_raw8(const void* p, int64_t i) {  // i: index of the first value
  Raw8<DT> r;
  __builtin_memcpy(&r, reinterpret_cast<const typename Val<DT>::S*>(p) + i, sizeof(r));
  return r;
}
template <int DT>
__device__ __forceinline__ void raw8_to_f32(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (DT == MOE_DT_FP32)
      v[j] = __uint_as_float(r.q[j >> 2][j & 3]);
    else
      v[j] = Val<DT>::get((uint16_t)(r.q[0][j >> 1] >> (16 * (j & 1))));
  }
}

// Run-time storage type: one value, or eight consecutive ones.
__device__ __forceinline__ float ld_value(const void* p, int dt, int64_t i) {
  if (dt == MOE_DT_FP32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
  return dt == MOE_DT_BF16 ? Val<MOE_DT_BF16>::get(b) : Val<MOE_DT_FP16>::get(b);
}
__device__ __forceinline__ uint16_t f32_to_16(float v, int dt) {  // round to nearest even
  return dt == MOE_DT_BF16 ? bitcast<uint16_t>((__bf16)v) : bitcast<uint16_t>((_Float16)v);
}
__device__ __forceinline__ void st_value(void* p, int dt, int64_t i, float v) {
  if (dt == MOE_DT_FP32)
    reinterpret_cast<float*>(p)[i] = v;
  else
    reinterpret_cast<uint16_t*>(p)[i] = f32_to_16(v, dt);
}
template <int DT>
__device__ __forceinline__ void st8_as(void* p, int64_t i, const float (&v)[8]) {
  typename Val<DT>::S* d = reinterpret_cast<typename Val<DT>::S*>(p) + i;
  if constexpr (DT == MOE_DT_FP32) {
    __builtin_memcpy(d, v, 32);
  } else {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = (uint32_t)f32_to_16(v[2 * j], DT) | ((uint32_t)f32_to_16(v[2 * j + 1], DT) << 16);
    __builtin_memcpy(d, &q, 16);
  }
}
__device__ __forceinline__ void st8(void* p, int dt, int64_t i, const float (&v)[8]) {
  if (dt == MOE_DT_FP32)
    st8_as<MOE_DT_FP32>(p, i, v);
  else if (dt == MOE_DT_BF16)
    st8_as<MOE_DT_BF16>(p, i, v);
  else
    st8_as<MOE_DT_FP16>(p, i, v);
}
__device__ __forceinline__ void ld8(const void* p, int dt, int64_t i, float (&v)[8]) {
  if (dt == MOE_DT_FP32)
    raw8_to_f32(ld_raw8<MOE_DT_FP32>(p, i), v);
  else if (dt == MOE_DT_BF16)
    raw8_to_f32(ld_raw8<MOE_DT_BF16>(p, i), v);
  else
    raw8_to_f32(ld_raw8<MOE_DT_FP16>(p, i), v);
}

}  // namespace moe
