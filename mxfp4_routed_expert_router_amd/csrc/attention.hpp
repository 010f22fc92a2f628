// What the prompt and the decode attention share: 16-bit MFMA operands, base-2 exponentials, and the partial results of
// key ranges that several workgroups share.
//
// A row (one query head of one token) over keys j: s_j = c q.k_j with c = scale * log2(e), l = sum 2^(s_j - m),
// O = sum 2^(s_j - m) v_j for a reference m (struct Reference); then y = O / l and lse = (m + log2 l) ln 2.  Parts of a
// row's keys join by M = max m, l = sum l_p 2^(m_p - M), O likewise.
#pragma once
#include "launch.hpp"
#include "values.hpp"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr float kLn2 = 0.6931471805599453f;

template <bool F16>
__device__ __forceinline__ f32x16 mfma_32x32x16(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16) return __builtin_amdgcn_mfma_f32_32x32x16_f16(bitcast<f16x8>(a), bitcast<f16x8>(b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bitcast<bf16x8>(a), bitcast<bf16x8>(b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ f32x4 mfma_16x16x32(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(bitcast<f16x8>(a), bitcast<f16x8>(b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bitcast<bf16x8>(a), bitcast<bf16x8>(b), c, 0, 0, 0);
}
// Two fp32 values as a dword of 16-bit ones, rounded to nearest even.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16) return bitcast<uint32_t>(f16x2{(_Float16)a, (_Float16)b});
  else return bitcast<uint32_t>(bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ float unpack16(uint32_t w, int half, bool f16) {
  const uint16_t b = (uint16_t)(half ? w >> 16 : w);
  return f16 ? Val<MOE_DT_FP16>::get(b) : Val<MOE_DT_BF16>::get(b);
}

typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;
// LDS at a byte address.
__device__ __forceinline__ uint32_t lds_address(const u32x4* p) {
  return (uint32_t)(uintptr_t)(lds_u32x4*)p;
}
__device__ __forceinline__ u32x4 lds_16(uint32_t at) { return *(lds_u32x4*)(uintptr_t)at; }
// Four keys of a 16-bit [key][d] tile for one d per lane: sixteen lanes give the addresses of four keys' rows of sixteen
// values (lane i: row i / 4, values 4 (i % 4) ..), lane i gets value i of the four rows.
__device__ __forceinline__ u32x2 lds_tr(uint32_t at) {
  return bitcast<u32x2>(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)at));
}

// Swizzles (in 16-byte chunks) of the rows of DP values of a tile in LDS.  K: sixteen consecutive rows' chunks of one column fall
// into different banks.  V: so do the 32-byte pieces of four consecutive rows that a transposing read takes.  Each stays
// inside aligned spans of 256, 128 or 64 bytes, of which a row is a multiple.
template <int DP>
constexpr int kSpanOf = DP % 128 == 0 ? 256 : (DP % 64 == 0 ? 128 : 64);
template <int DP>
__device__ __forceinline__ int swizzle_k(int row) {
  return kSpanOf<DP> == 256 ? row & 15 : (kSpanOf<DP> == 128 ? (row >> 1) & 7 : (row >> 2) & 3);
}
template <int DP>
__device__ __forceinline__ int swizzle_v(int row) {
  return kSpanOf<DP> == 256 ? (row & 3) << 2 : (kSpanOf<DP> == 128 ? ((row >> 1) & 1) << 2 : 0);
}

// (a ballot is uniform to the compiler, __any() is not: its branches would keep both sides' values in registers)
__device__ __forceinline__ bool wave_any(bool v) { return __builtin_amdgcn_ballot_w64(v) != 0; }

// The reference m of a row's exponentials 2^(s - m), which are rounded to 16 bits, while l and O stay fp32.
//   bf16 has fp32's exponents: m is the first tile's maximum and rises only when a later one passes it by more than 2^8, so
// that factors are rare.
//   fp16 ends at 2^-24, and with m at the maximum a weight 2^-20 of it kept four bits, one of 2^-25 none: a row whose largest
// weight meets a value near zero came out percents off.  So m follows the tiles both ways: a tile's largest exponential
// stands between 2^0 and 2^15.5 (65504 is the type's end), and a move, by a power of two that O and l take exactly, puts it
// at 2^7.5, half way.  Then a weight of 2^-14 of its tile's largest or more has all its bits, and a smaller one is off by
// 2^-25 of that largest at most; in the tile of the row's largest, which never stands below 2^7, it is 2^-21 and 2^-32.  m
// falls no further than 40 below where it last rose, so that O stays inside fp32.  Each row moves by itself, whatever
// its neighbours in the wave hold.  8192 tokens, 32 heads of 128 on 8: 551 us, with m at the maximum 545; a narrower range
// (2^6 to 2^15.5, moved to 2^11) costs a move in many tiles: 587.
template <bool F16>
struct Reference {
  static constexpr float kMost = F16 ? 15.5f : 8.0f, kLeast = 0.0f, kAt = F16 ? 7.5f : 0.0f, kFall = 40.0f;
  float m = -INFINITY, floor = -INFINITY;
  // top: the largest s - m of a tile (m still -inf: the largest s)
  __device__ __forceinline__ bool moves(float top) const {
    bool r = (top > kMost) | ((m == -INFINITY) & (top > -INFINITY));
    if constexpr (F16) r |= (top < kLeast) & (top > -INFINITY);
    return r;
  }
  // How far m goes up; before the first key O and l are zero.
  __device__ __forceinline__ float way(float top) const {
    if (m == -INFINITY) return top == -INFINITY ? 0.0f : top - kAt;
    if constexpr (F16) return moves(top) ? fmaxf(__builtin_rintf(top - kAt), floor - m) : 0.0f;
    else return fmaxf(top, 0.0f);
  }
  __device__ __forceinline__ float factor(float up) const { return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(-up); }
  __device__ __forceinline__ void move(float top, float up) {
    m = m == -INFINITY ? top - kAt : m + up;
    if constexpr (F16) floor = fmaxf(floor, m - kFall);
  }
};

// Partial results in a workspace: (m, l) of every row and part, then O.
struct AttnParts {
  float* ml;  // [rows][parts][2]
  float* o;   // [rows][parts][D], 16-byte aligned
  int parts;
};
inline size_t attn_parts_bytes(int64_t rows, int parts, int D) {
  return parts > 1 ? (size_t)rows * parts * (size_t)(D + 2) * 4 + 8 : 0;
}
inline AttnParts attn_parts(void* ws, int64_t rows, int parts) {
  AttnParts p;
  p.ml = (float*)ws;
  p.o = parts > 1 ? (float*)ws + (2 * rows * parts + 3) / 4 * 4 : nullptr;
  p.parts = parts;
  return p;
}

__device__ __forceinline__ AttnParts attn_parts_dev(void* ws, int64_t rows, int parts) {
  AttnParts p;
  p.ml = (float*)ws;
  p.o = (float*)ws + (2 * rows * parts + 3) / 4 * 4;
  p.parts = parts;
  return p;
}
struct AttnJoin {
  AttnParts parts;
  int64_t rows;        // token * Hq + head
  int Hq, D, f16;
  uint16_t* y;
  int64_t y_ts, y_hs;
  float* lse;
  const int32_t* cu_q;  // prompts: rows outside cu_q[0] .. cu_q[n_seqs] are left alone; NULL: all rows
  int n_seqs;
};
hipError_t launch_attn_join(const AttnJoin& j, hipStream_t stream);

// n / d for 0 <= n < 2^31 by a multiplication: with 2^s < d <= 2^(s+1) and mul = ceil(2^(32+s) / d), mul d exceeds
// 2^(32+s) by less than d <= 2^(s+1), so the quotient is exact for n < 2^31.
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  if (d > 1) {
    while (((uint64_t)2 << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)((((uint64_t)1 << (32 + f.shift)) + d - 1) / d);
  }
  return f;
}
__device__ __forceinline__ uint32_t div_by(FastDiv f, uint32_t n) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

}  // namespace moe
