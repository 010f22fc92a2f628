// Products with 4-bit weights: y[t][n] = sum_k x[t][k] W[n][k] (+ bias[n]), W as MXFP4, INT4 group-32 or NVFP4
// (the formats of the expert weights), x bf16, fp32 sums.
//
// Weights are decoded in registers into bf16 MFMA operands whose values are exact: E2M1 times a power of two
// (MXFP4) or times an E4M3 scale (NVFP4, at most 6 significant bits) in one operand, (code - zero) * scale
// (INT4, at most 15 bits) as a high and a low operand.  Products are exact in fp32; the fp32 sums round.
#include "launch.hpp"
#include "values.hpp"

namespace moe {

namespace {

// One lane's 32-value block of a weight row and its scale data.
template <int FMT>
struct Blk {
  u32x4 q;
  float s0, s1;  // MXFP4: s0; NVFP4: the two 16-value scales; INT4: scale and -zero * scale
};

__device__ __forceinline__ float e4m3_value(uint32_t c) {  // bias 7, subnormals at exponent field 0
  const uint32_t ex = (c >> 3) & 15u, fr = c & 7u;
  const float mag = ex ? __uint_as_float(((ex + 120u) << 23) | (fr << 20)) : (float)fr * 0.001953125f;
  return (c & 0x80u) ? -mag : mag;
}

template <int FMT>
__device__ __forceinline__ Blk<FMT> load_block(const LinArgs& a, int n, int b, bool ok) {
  Blk<FMT> r;
  r.q = u32x4{0, 0, 0, 0};
  r.s0 = r.s1 = 0.0f;
  if (!ok) return r;  // a scale of zero: zero weights
  r.q = ld16(a.w.w + (int64_t)n * a.w.wr + 16 * (int64_t)b);
  const uint8_t* s = a.w.s + (int64_t)n * a.w.sr;
  if constexpr (FMT == MOE_W_MXFP4) {
    r.s0 = e8m0_to_f32(s[b]);
  } else if constexpr (FMT == MOE_W_INT4_G32) {
    r.s0 = (float)bitcast<_Float16>((uint16_t)(s[2 * b] | (s[2 * b + 1] << 8)));
    const uint32_t z = (a.w.z[(int64_t)n * a.w.zr + (b >> 1)] >> (4 * (b & 1))) & 15u;
    r.s1 = -(float)z * r.s0;
  } else {
    r.s0 = e4m3_value(s[2 * b]);
    r.s1 = e4m3_value(s[2 * b + 1]);
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_high(float a, float b) {  // the upper halves of two floats
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// MFMA operands of dword s (eight codes) of a block; INT4 also writes the low operand.
template <int FMT>
__device__ __forceinline__ bf16x8 decode(const Blk<FMT>& r, int s, bf16x8& lo) {
  if constexpr (FMT == MOE_W_MXFP4) {
    return decode8_bf16(r.q[s], r.s0);
  } else if constexpr (FMT == MOE_W_NVFP4) {
    const float sc = s < 2 ? r.s0 : r.s1;
    const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.q[s], 1.0f, 0);
    const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.q[s], 1.0f, 1);
    const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.q[s], 1.0f, 2);
    const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.q[s], 1.0f, 3);
    return bitcast<bf16x8>(u32x4{pack_high(v0[0] * sc, v0[1] * sc), pack_high(v1[0] * sc, v1[1] * sc),
                                 pack_high(v2[0] * sc, v2[1] * sc), pack_high(v3[0] * sc, v3[1] * sc)});
  } else {
    uint32_t hi[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = r.q[s] >> (8 * i);
      const float v0 = __builtin_fmaf((float)(c & 15u), r.s0, r.s1);  // exact: at most 15 bits
      const float v1 = __builtin_fmaf((float)((c >> 4) & 15u), r.s0, r.s1);
      hi[i] = pack_high(v0, v1);  // truncated; the rest has at most 7 bits
      l[i] = pack_high(v0 - __uint_as_float(hi[i] << 16), v1 - __uint_as_float(hi[i] & 0xFFFF0000u));
    }
    lo = bitcast<bf16x8>(u32x4{l[0], l[1], l[2], l[3]});
    return bitcast<bf16x8>(u32x4{hi[0], hi[1], hi[2], hi[3]});
  }
}

// 16 rows of W times 16 MT tokens per workgroup; its four waves take every fourth step of 128 values of K and
// their sums meet in LDS.  Lane (r = lane % 16, q = lane / 16) holds row r's block 4 step + q.
template <int FMT, int MT>
__global__ __launch_bounds__(256) void linear_rows_kernel(LinArgs a) {
  __shared__ float part[4][MT][16][17];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int n = blockIdx.x * 16 + l16, t0 = blockIdx.y * 16 * MT;
  const int blocks = a.K / 32;
  f32x4 acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int b0 = 4 * wave; b0 < blocks; b0 += 16) {
    const int b = b0 + q;
    const Blk<FMT> w = load_block<FMT>(a, n, b, n < a.N && b < blocks);
    bf16x8 x[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = t0 + 16 * m + l16;
      const bool ok = t < a.T && b < blocks;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[m][s] = bitcast<bf16x8>(ok ? ld16(a.x + (int64_t)t * a.x_stride + 32 * (int64_t)b + 8 * s) : u32x4{0, 0, 0, 0});
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 lo;
      const bf16x8 hi = decode<FMT>(w, s, lo);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, x[m][s], acc[m], 0, 0, 0);
        if constexpr (FMT == MOE_W_INT4_G32)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, x[m][s], acc[m], 0, 0, 0);
      }
    }
  }
  // lane holds rows 4q + i of token l16
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][m][l16][4 * q + i] = acc[m][i];
  __syncthreads();
  const float ts = FMT == MOE_W_NVFP4 ? *a.w.ts : 1.0f;
  for (int i = threadIdx.x; i < MT * 256; i += 256) {
    const int m = i >> 8, tl = (i >> 4) & 15, r = i & 15;
    const int t = t0 + 16 * m + tl, row = blockIdx.x * 16 + r;
    if (t >= a.T || row >= a.N) continue;
    float v = (part[0][m][tl][r] + part[1][m][tl][r]) + (part[2][m][tl][r] + part[3][m][tl][r]);
    if constexpr (FMT == MOE_W_NVFP4) v *= ts;
    if (a.bias) v += a.bias[row];
    st_value(a.y, a.y_dt, (int64_t)t * a.y_stride + row, v);
  }
}

template <int FMT>
void linear_fmt(const LinArgs& a, hipStream_t stream) {
  const unsigned gn = (unsigned)((a.N + 15) / 16);
  if (a.T <= 16)
    linear_rows_kernel<FMT, 1><<<dim3(gn, 1), 256, 0, stream>>>(a);
  else
    linear_rows_kernel<FMT, 4><<<dim3(gn, (unsigned)((a.T + 63) / 64)), 256, 0, stream>>>(a);
}

}  // namespace

size_t linear_workspace_bytes(int T, int fmt, int N, int K) {
  (void)T, (void)fmt, (void)N, (void)K;
  return 0;
}

hipError_t launch_linear(const LinArgs& a, hipStream_t stream) {
  if (a.fmt == MOE_W_MXFP4) linear_fmt<MOE_W_MXFP4>(a, stream);
  else if (a.fmt == MOE_W_INT4_G32) linear_fmt<MOE_W_INT4_G32>(a, stream);
  else linear_fmt<MOE_W_NVFP4>(a, stream);
  return hipGetLastError();
}

}  // namespace moe
