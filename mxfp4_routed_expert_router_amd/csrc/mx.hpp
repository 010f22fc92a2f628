// MX block quantisation on the device: element formats, the E8M0 scale of a 32-value block, and the
// encoders of whole blocks and quarter blocks.  Shared by the MX expert FFN (activations x and h) and the
// RMS norm's 8-, 6- and 4-bit output.
#pragma once
#include "common.hpp"

namespace moe {

// Element formats: code bits, MFMA operand format code, exponent/fraction bits, bias, exponent of
// the largest normal, largest code and value.
template <int F>
struct Mx;
template <>
struct Mx<MOE_MX_FP8_E4M3> {
  static constexpr int kBits = 8, kMfma = 0, kMBits = 3, kBias = 7, kEmax = 8;
  static constexpr uint32_t kMaxCode = 0x7E;  // 448 (0x7F is NaN)
  static constexpr float kMax = 448.0f;
};
template <>
struct Mx<MOE_MX_FP4_E2M1> {
  static constexpr int kBits = 4, kMfma = 4, kMBits = 1, kBias = 1, kEmax = 2;
  static constexpr uint32_t kMaxCode = 0x7;  // 6
  static constexpr float kMax = 6.0f;
};
template <>
struct Mx<MOE_MX_FP6_E2M3> {
  static constexpr int kBits = 6, kMfma = 2, kMBits = 3, kBias = 1, kEmax = 2;
  static constexpr uint32_t kMaxCode = 0x1F;  // 7.5
  static constexpr float kMax = 7.5f;
};
// E8M0 code of a block whose largest magnitude is amax (finite, >= 0):
// floor(log2 amax) - emax + 127 clamped to [0, 254]; 0 for an all-zero block.  floor(log2) comes
// from the binary32 exponent field, or from the leading fraction bit for a subnormal amax.
template <int F>
__device__ __forceinline__ uint32_t mx_scale_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 0;
  const uint32_t ef = u >> 23;
  const int e = ef ? (int)ef - 127 : (31 - (int)__builtin_clz(u)) - 149;
  const int c = e - Mx<F>::kEmax + 127;
  return (uint32_t)(c < 0 ? 0 : (c > 254 ? 254 : c));
}
// 2^(127 - c), the reciprocal of the block scale, as a binary32 value (exact).
__device__ __forceinline__ float mx_inv_scale(uint32_t c) {
  return __uint_as_float(c <= 253 ? (254u - c) << 23 : 0x00400000u);
}

// Nearest element code to q (ties to the even code), saturating at the largest value, with q's
// sign.  Subnormal range: q / 2^(1 - bias - m_bits) rounded to an integer (which reaches the
// smallest normal code exactly when it rounds up to 2^m_bits).  Normal range: the fraction of q
// rounded to m_bits; a carry out of the fraction lands on the next exponent's code.
template <int F>
__device__ __forceinline__ uint32_t mx_encode(float q) {
  typedef Mx<F> M;
  const uint32_t u = __float_as_uint(q);
  const float a = fabsf(q);
  uint32_t c;
  if (a >= M::kMax) {
    c = M::kMaxCode;
  } else if (a < __uint_as_float((uint32_t)(127 + 1 - M::kBias) << 23)) {
    c = (uint32_t)__builtin_rintf(a * __uint_as_float((uint32_t)(127 + M::kBias - 1 + M::kMBits) << 23));
  } else {
    const int e = (int)((u >> 23) & 0xFF) - 127;
    const float r = __uint_as_float((u & 0x007FFFFFu) | 0x3F800000u);
    const uint32_t m = (uint32_t)__builtin_rintf((r - 1.0f) * (float)(1 << M::kMBits));
    c = ((uint32_t)(e + M::kBias) << M::kMBits) + m;
  }
  return c | ((u >> 31) << (M::kBits - 1));
}

// Codes of 2 * NP values q (already divided by the block scale), packed as in the block layout,
// with the hardware conversions at scale 1: over every code's value, every midpoint between
// neighbouring codes and the floats next to them, signed zeros and a million log-spread values,
// they give the codes of mx_encode exactly -- FP6 and FP4 everywhere, FP8 once the input is
// clamped to the largest value (past it the conversion returns the NaN code).  The FP6
// conversion takes 32 values as two halves and interleaves them (field 2i from the first half,
// 2i + 1 from the second), so the halves are the even and the odd values.
typedef short v2s __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
template <int F, int NP>
__device__ __forceinline__ void mx_hw_pack(const float* q, uint32_t* dw) {
  static_assert(NP == 4 || NP == 16, "a quarter block or a whole block");
  static_assert(NP == 16 || Mx<F>::kBits != 6, "FP6 quarters take the software encoder");
  if constexpr (Mx<F>::kBits == 4) {
#pragma unroll
    for (int w = 0; w < NP / 4; ++w) {
      const float* p = q + 8 * w;  // byte i of the dword from values 2i, 2i + 1
      uint32_t d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, p[0], p[1], 1.0f, 0);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, p[2], p[3], 1.0f, 1);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, p[4], p[5], 1.0f, 2);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, p[6], p[7], 1.0f, 3);
      dw[w] = d;
    }
  } else if constexpr (Mx<F>::kBits == 8) {
    auto cl = [](float x) { return fminf(fmaxf(x, -Mx<F>::kMax), Mx<F>::kMax); };
#pragma unroll
    for (int w = 0; w < NP / 2; ++w) {
      v2s d = {0, 0};
      d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, cl(q[4 * w]), cl(q[4 * w + 1]), 1.0f, false);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(d, cl(q[4 * w + 2]), cl(q[4 * w + 3]), 1.0f, true);
      dw[w] = __builtin_bit_cast(uint32_t, d);
    }
  } else {
    v16f a = {}, b = {};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      a[i] = q[2 * i];
      b[i] = q[2 * i + 1];
    }
    const auto r = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(a, b, 1.0f);
#pragma unroll
    for (int w = 0; w < (NP == 16 ? 6 : 2); ++w) dw[w] = (uint32_t)r[w];
    if constexpr (NP == 4) dw[1] &= 0xFFFFu;  // fields 8 .. 31 are codes of zero anyway
  }
}

// One 32-value block: E8M0 code and the packed element codes (4 * bits bytes in dw[0 .. bits/2)).
template <int F>
__device__ __forceinline__ uint32_t mx_pack_block(const float (&v)[32], uint32_t (&dw)[8]) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(v[j]));
  const uint32_t sc = mx_scale_code<F>(amax);
  const float inv = mx_inv_scale(sc);
  float q[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) q[j] = v[j] * inv;
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0;
  mx_hw_pack<F, 16>(q, dw);
  return sc;
}

// Stores the 4 * bits bytes of a packed block (dst aligned to 8 bytes, and to 16 for FP8/FP4).
template <int F>
__device__ __forceinline__ void mx_store_block(uint8_t* dst, const uint32_t (&dw)[8]) {
  if constexpr (Mx<F>::kBits == 6) {
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x2*>(dst + 8 * i) = u32x2{dw[2 * i], dw[2 * i + 1]};
  } else {
#pragma unroll
    for (int i = 0; i < Mx<F>::kBits / 4; ++i) st16(dst + 16 * i, u32x4{dw[4 * i], dw[4 * i + 1], dw[4 * i + 2], dw[4 * i + 3]});
  }
}

// Codes of 8 consecutive values (a quarter block) packed as in the block layout: bits bytes, in
// dw[0] and (FP6, FP8) dw[1].
template <int F>
// (FP6 quarters take the software encoder: the 32-value FP6 conversion's two 16-register halves
// made the gate/up kernel spill inside its main loop, 3.75 -> 3.79 ms; FP4 with the hardware
// conversion 3.58 -> 3.49 ms.)
__device__ __forceinline__ void mx_pack_quarter(const float (&v)[8], float inv, uint32_t (&dw)[2]) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = v[j] * inv;
  dw[0] = 0;
  dw[1] = 0;
  if constexpr (Mx<F>::kBits == 6) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = mx_encode<F>(q[j]);
      const int bit = 6 * j, w = bit >> 5, o = bit & 31;
      dw[w] |= c << o;
      if (o + 6 > 32) dw[w + 1] |= c >> (32 - o);
    }
  } else {
    mx_hw_pack<F, 4>(q, dw);
  }
}

}  // namespace moe
