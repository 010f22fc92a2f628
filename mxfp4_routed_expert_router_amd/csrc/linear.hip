// Products with 4-bit weights: y[t][n] = sum_k x[t][k] W[n][k] (+ bias[n]), W as MXFP4, INT4 group-32 or NVFP4
// (the formats of the expert weights), x bf16, fp32 sums.
//
// Weights are decoded in registers into bf16 MFMA operands whose values are exact: E2M1 times a power of two
// (MXFP4) or times an E4M3 scale (NVFP4, at most 6 significant bits) in one operand, (code - zero) * scale
// (INT4, at most 15 bits) as a high and a low operand.  Products are exact in fp32; the fp32 sums round.
#include <algorithm>

#include "launch.hpp"
#include "tiles.hpp"
#include "values.hpp"

namespace moe {

namespace {

// One lane's 32-value block of a weight row and its scale data.
template <int FMT>
struct Blk {
  u32x4 q;
  float s0, s1;  // MXFP4: s0; NVFP4: the two 16-value scales; INT4: scale and -zero * scale
};

__device__ __forceinline__ float e4m3_value(uint32_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

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
    // a code c as an E4M3 byte is c 2^-9, for every c of four bits
    uint32_t hi[4], l[4];
    const uint32_t even = r.q[s] & 0x0F0F0F0Fu, odd = (r.q[s] >> 4) & 0x0F0F0F0Fu;
    const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, false);
    const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, true);
    const f32x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, false);
    const f32x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, true);
    const float ce[4] = {e0[0], e0[1], e1[0], e1[1]}, co[4] = {o0[0], o0[1], o1[0], o1[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = __builtin_fmaf(ce[i], r.s0, r.s1);  // exact: at most 15 bits
      const float v1 = __builtin_fmaf(co[i], r.s0, r.s1);
      const uint32_t h0 = __float_as_uint(v0) & 0xFFFF0000u, h1 = __float_as_uint(v1) & 0xFFFF0000u;
      hi[i] = pack_high(v0, v1);  // truncated; the rest has at most 7 bits
      l[i] = pack_high(v0 - __uint_as_float(h0), v1 - __uint_as_float(h1));
    }
    lo = bitcast<bf16x8>(u32x4{l[0], l[1], l[2], l[3]});
    return bitcast<bf16x8>(u32x4{hi[0], hi[1], hi[2], hi[3]});
  }
}

// Bytes at any address through a buffer descriptor (u8 or u16; offsets need no alignment).
template <int FMT>
__device__ __forceinline__ uint32_t bld_scale(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff) {
  if constexpr (FMT == MOE_W_MXFP4) return __builtin_amdgcn_raw_buffer_load_b8(r, off, soff, 0);
  return __builtin_amdgcn_raw_buffer_load_b16(r, off, soff, 0);
}
// A block's scale data in one word: the scale bytes, and for INT4 its zero point in bits 16 .. 19 (odd: the block's
// index is odd, its zero point is the high nibble of the byte z).
template <int FMT>
__device__ __forceinline__ uint32_t scale_word(uint32_t s, uint32_t z, int odd) {
  return FMT == MOE_W_INT4_G32 ? s | (((z >> (4 * odd)) & 15u) << 16) : s;
}
// in: the block lies inside K (MXFP4's scale code 0 is not 0).
template <int FMT>
__device__ __forceinline__ Blk<FMT> unpack_block(u32x4 codes, uint32_t w, bool in) {
  Blk<FMT> b;
  b.q = codes;
  if constexpr (FMT == MOE_W_MXFP4) {
    b.s0 = in ? e8m0_to_f32(w) : 0.0f;
    b.s1 = 0.0f;
  } else if constexpr (FMT == MOE_W_INT4_G32) {
    b.s0 = (float)bitcast<_Float16>((uint16_t)w);
    b.s1 = -(float)(w >> 16) * b.s0;
  } else {
    b.s0 = e4m3_value(w & 255u);
    b.s1 = e4m3_value(w >> 8);
  }
  return b;
}
// Four consecutive outputs n .. n+3 of token t from their sums.
template <int FMT>
__device__ __forceinline__ void store_out(const LinArgs& a, int t, int n, f32x4 v, float ts) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= a.N) break;
    float o = v[e];
    if constexpr (FMT == MOE_W_NVFP4) o *= ts;
    if (a.bias) o += a.bias[n + e];
    st_value(a.y, a.y_dt, (int64_t)t * a.y_stride + n + e, o);
  }
}

// ---- one to four tokens: dot products on the vector ALU ----
// 8 rows per workgroup, whose NW waves share K in spans of 256 values, two spans in flight each (four: the same or
// slower): a lane holds block lane % 8 of the span of row lane / 8, so a load instruction takes 8 whole 128-byte
// lines (nontemporal: used once).  A span of x (512 bytes a token) is loaded as it lies, two tokens per instruction,
// and passes through LDS of the wave's own to the lanes that need its blocks: loaded in the lanes' order (16 bytes
// every 64) it took four instructions a token and bound the kernel.  Codes are unpacked to bf16 pairs of small exact
// integers or E2M1 values, two products per v_dot2_f32_bf16; the block's sum D then takes its scale s in fp32:
// acc += s D.  INT4 codes have their zero point subtracted before the products: c - z is exact in bf16, while
// D - z sum(x) carries the roundings of c x into weights that are zero.  (A 4-bit code c as an E4M3 byte is c 2^-9
// for every c, so codes unpack by the 8-bit conversion.  7168 x 7168 INT4: 11.2 us with the subtraction and 10.5 with
// sum(x) for one token, 13.0 and 13.3 for two; 4 x 3200 x 4096 6.7 and 7.1.)
// Bound: one token x 7168 x 7168 MXFP4 reads its 27.3 MB in 7.8 us (3.5 TB/s; of which about 3 us are a launch and
// the first loads' latency); from three tokens on by the vector ALU (4 tokens of that size 13.7 us).
constexpr int kSpan = 256;

struct DotScale {
  uint32_t s, z;
};

// Eight codes of dword d as four bf16 pairs (k ascending), less z for INT4.
template <int FMT>
__device__ __forceinline__ void unpack_pairs(uint32_t d, float z, bf16x2 (&w)[4]) {
  if constexpr (FMT == MOE_W_INT4_G32) {
    const uint32_t even = d & 0x0F0F0F0Fu, odd = (d >> 4) & 0x0F0F0F0Fu;
    const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, false);
    const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, true);
    const f32x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, false);
    const f32x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, true);
    w[0] = bitcast<bf16x2>(pack_high(e0[0] - z, o0[0] - z));
    w[1] = bitcast<bf16x2>(pack_high(e0[1] - z, o0[1] - z));
    w[2] = bitcast<bf16x2>(pack_high(e1[0] - z, o1[0] - z));
    w[3] = bitcast<bf16x2>(pack_high(e1[1] - z, o1[1] - z));
  } else {
    w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0);
    w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1);
    w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2);
    w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3);
  }
}

template <int FMT, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void linear_dot_kernel(LinArgs a) {
  constexpr int DP = 2;             // spans in flight
  constexpr int XL = (TT + 1) / 2;  // x loads per span
  __shared__ float red[NW][8][TT];
  __shared__ __attribute__((aligned(16))) uint8_t xlds[NW][XL * 1024];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int lr = lane >> 3, lc = lane & 7;
  const int n0 = blockIdx.x * 8;
  const int blocks = a.K / 32, spans = (a.K + kSpan - 1) / kSpan;
  const int p0 = (int)((int64_t)spans * wave / NW), p1 = (int)((int64_t)spans * (wave + 1) / NW);
  const int rows = min(8, a.N - n0);
  // rows past N fall past the buffer's range and read zeros
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(a.w.w + (int64_t)n0 * a.w.wr, (int64_t)(rows - 1) * a.w.wr + a.K / 2);
  const uint32_t lbase = (uint32_t)(lr * a.w.wr) + 16u * lc;
  const int64_t nr = n0 + min(lr, rows - 1);
  const uint8_t* const srow = a.w.s + nr * a.w.sr;
  const uint8_t* const zrow = FMT == MOE_W_INT4_G32 ? a.w.z + nr * a.w.zr : nullptr;
  // this lane's part of x: 16-byte piece lane % 32 of the span of token 2 i + lane / 32 (tokens past the last
  // repeat it; not stored).  Piece i of block b lies at piece i ^ (b / 4) of the block: distinct banks.
  const int xp = lane & 31;
  const uint16_t* xrow[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) xrow[i] = a.x + (int64_t)min(2 * i + (lane >> 5), a.T - 1) * a.x_stride;
  uint8_t* const xw = xlds[wave] + 512 * (lane >> 5) + 64 * (xp >> 2) + 16 * ((xp & 3) ^ (xp >> 4));
  const uint8_t* const xr = xlds[wave] + 64 * lc;
  u32x4 codes[DP], x[DP][XL];
  DotScale sc[DP];
  auto load = [&](int p, u32x4& c, DotScale& s, u32x4 (&v)[XL]) {
    const bool in = p < p1 && 8 * p + lc < blocks;
    const int b = in ? 8 * p + lc : blocks - 1;  // past the wave's share or past K: codes of zero, the rest unused
    c = bld16nt(wr, in ? lbase + 128u * p : kOutOfRange);
    if constexpr (FMT == MOE_W_MXFP4) {
      s.s = srow[b];
    } else {
      uint16_t h;
      __builtin_memcpy(&h, srow + 2 * b, 2);
      s.s = h;
      if constexpr (FMT == MOE_W_INT4_G32) s.z = zrow[b >> 1];
    }
    const int k = min(kSpan * p + 8 * xp, a.K - 8);
#pragma unroll
    for (int i = 0; i < XL; ++i) v[i] = ld16(xrow[i] + k);
  };
#pragma unroll
  for (int d = 0; d < DP; ++d) load(p0 + d, codes[d], sc[d], x[d]);
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0f;
  auto fence = [] {  // LDS operations of one wave stay in program order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  auto span = [&](int p, const u32x4& c, const DotScale& s, const u32x4 (&xs)[XL]) {
    const bool in = p < p1 && 8 * p + lc < blocks;
#pragma unroll
    for (int i = 0; i < XL; ++i) st16(xw + 1024 * i, xs[i]);
    fence();
    u32x4 v[TT][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[t][i] = ld16(xr + 512 * t + 16 * (i ^ (lc >> 2)));
    fence();
    // zero point of block 8 p + lc, whose parity is lc's
    const float z = FMT == MOE_W_INT4_G32 ? (float)((s.z >> (4 * (lc & 1))) & 15u) : 0.0f;
    float D[2][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) D[0][t] = D[1][t] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x2 w[4];
      unpack_pairs<FMT>(c[i], z, w);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          D[i >> 1][t] = __builtin_amdgcn_fdot2_f32_bf16(w[k], bitcast<bf16x2>(v[t][i][k]), D[i >> 1][t], false);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float o;
      if constexpr (FMT == MOE_W_MXFP4) {
        o = e8m0_to_f32(s.s) * (D[0][t] + D[1][t]);
      } else if constexpr (FMT == MOE_W_INT4_G32) {
        o = (float)bitcast<_Float16>((uint16_t)s.s) * (D[0][t] + D[1][t]);
      } else {
        o = __builtin_fmaf(e4m3_value(s.s & 255u), D[0][t], e4m3_value(s.s >> 8) * D[1][t]);
      }
      acc[t] += in ? o : 0.0f;
    }
  };
  for (int pb = p0; pb < p1; pb += DP) {
#pragma unroll
    for (int d = 0; d < DP; ++d) {
      span(pb + d, codes[d], sc[d], x[d]);  // (past the wave's share: adds nothing)
      load(pb + d + DP, codes[d], sc[d], x[d]);
    }
  }
  // over the eight lanes of a row, then over the waves
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    float v = acc[t];
    v += __shfl_xor(v, 1, kWave);
    v += __shfl_xor(v, 2, kWave);
    v += __shfl_xor(v, 4, kWave);
    if (lc == 0) red[wave][lr][t] = v;
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i < 8 * TT) {
    const int t = i / 8, r = i % 8;
    if (t >= a.T || r >= rows) return;
    float v = red[0][r][t];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w][r][t];
    if constexpr (FMT == MOE_W_NVFP4) v *= *a.w.ts;
    if (a.bias) v += a.bias[n0 + r];
    st_value(a.y, a.y_dt, (int64_t)t * a.y_stride + n0 + r, v);
  }
}

// ---- few tokens: the weights stream, 16 RT rows x 16 MT tokens per workgroup, its NW waves share K in whole spans ----
// A span is 256 values of K: 128 bytes of codes per row, so a load instruction (8 rows x 128 bytes) takes whole
// lines, with the nontemporal hint (a line is used once; the lines of the 16-row x 64-byte shape that the MFMA
// layout would give read about 13% slower from HBM, and lanes that are neighbours in different rows cost the
// address unit a cycle each; scale bytes are loaded in the same order for that reason).  A wave keeps a span of
// codes and of x in registers and turns them (x by halves of a span, 256 bytes a token, four tokens per load) into
// MFMA layout through LDS of its own.  Half a span of x is loaded as soon as the one before it is in LDS (64 tokens,
// 7168 x 7168 MXFP4: 24.1 us with all loads after the products, 21.2 so), the codes after the span's products
// (earlier, or two spans ahead: the same or slower).  No load is conditional (registers of loads in flight would be
// merged, and waited for, at the end of each turn): lanes past K and past the wave's share read zeros.
// Bound: not by bandwidth (32 tokens, 16384 rows x 4096 NVFP4: 39 MB in 17 us, 2.3 TB/s; 16 tokens, 7168 x 7168
// MXFP4: 27 MB in 11.5 us).  Reading the weights (5.5 us of the 17), all of x once per workgroup through the L2,
// both through LDS, and decoding follow one another in each wave, and the registers leave two waves per SIMD.
template <int FMT, int RT, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void linear_stream_kernel(LinArgs a) {
  constexpr int kWave = RT * 2048 + RT * 512 + MT * 4096;  // a wave's LDS: its span of codes and scales, half span of x
  constexpr int kSlots = NW * kWave, kRed = NW * RT * MT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSlots > kRed ? kSlots : kRed];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l16 = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
  const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * MT;
  const int blocks = a.K / 32, spans = (a.K + kSpan - 1) / kSpan;
  const int p0 = (int)((int64_t)spans * wave / NW), p1 = (int)((int64_t)spans * (wave + 1) / NW);
  // Buffer descriptors end with the last row's last value.  Only a load's per-lane offset is checked against them,
  // so that offset holds the row (rows past N and tokens past T lie past the end: zeros) and is put out of range
  // for a lane past K or past the wave's share; the uniform offset adds the place in K, inside the row for the rest.
  constexpr int kPer = FMT == MOE_W_MXFP4 ? 1 : 2;  // scale bytes per block
  const int rows = min(16 * RT, a.N - n0), toks = min(16 * MT, a.T - t0);
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(a.w.w + (int64_t)n0 * a.w.wr, (int64_t)(rows - 1) * a.w.wr + a.K / 2);
  const __amdgpu_buffer_rsrc_t sr =
      make_rsrc(a.w.s + (int64_t)n0 * a.w.sr, (int64_t)(rows - 1) * a.w.sr + kPer * blocks);
  const __amdgpu_buffer_rsrc_t zr =
      FMT == MOE_W_INT4_G32 ? make_rsrc(a.w.z + (int64_t)n0 * a.w.zr, (int64_t)(rows - 1) * a.w.zr + (blocks + 1) / 2)
                            : sr;
  const __amdgpu_buffer_rsrc_t xr =
      make_rsrc(a.x + (int64_t)t0 * a.x_stride, ((int64_t)(toks - 1) * a.x_stride + a.K) * 2);
  const uint32_t woff = (uint32_t)(lr * a.w.wr) + 16u * lc;
  const uint32_t soff = (uint32_t)(lr * a.w.sr) + kPer * lc, zoff = (uint32_t)(lr * a.w.zr) + (lc >> 1);
  const uint32_t xoff = (uint32_t)(q * a.x_stride) * 2u + 16u * l16;  // token 4 i + q, piece l16 of a half span
  u32x4 codes[RT][2], x[2][MT][4];
  uint32_t sc[RT][2], zp[RT][2];
  auto load_w = [&](int p) {
    const uint32_t out = p < p1 && 8 * p + lc < blocks ? 0u : kOutOfRange;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int row = 16 * r + 8 * g;
        codes[r][g] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, (woff + (uint32_t)(row * a.w.wr)) | out, 128u * p, 2));
        sc[r][g] = bld_scale<FMT>(sr, (soff + (uint32_t)(row * a.w.sr)) | out, 8u * kPer * p);
        zp[r][g] = 0;
        if constexpr (FMT == MOE_W_INT4_G32)
          zp[r][g] = __builtin_amdgcn_raw_buffer_load_b8(zr, (zoff + (uint32_t)(row * a.w.zr)) | out, 4u * p, 0);
      }
  };
  auto load_x = [&](int p, int j) {
    const uint32_t out = p < p1 && kSpan * p + 128 * j + 8 * l16 < a.K ? 0u : kOutOfRange;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[j][m][i] = bld16s(xr, (xoff + (uint32_t)((16 * m + 4 * i) * a.x_stride) * 2u) | out, 512u * p + 256u * j);
  };
  load_w(p0);
  load_x(p0, 0);
  load_x(p0, 1);
  f32x4 acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* const slot = lds + wave * kWave;
  uint32_t* const sslot = reinterpret_cast<uint32_t*>(slot + RT * 2048);  // [16 RT rows][8]: a block's scale bytes
  uint8_t* const xslot = slot + RT * 2560;
  auto fence = [] {  // LDS operations of one wave stay in program order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  for (int p = p0; p < p1; ++p) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int w = 8 * g + lr;
        st16(slot + 2048 * r + 128 * w + 16 * (lc ^ (w >> 1)), codes[r][g]);
        sslot[(16 * r + w) * 8 + lc] = scale_word<FMT>(sc[r][g], zp[r][g], lc & 1);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = 8 * p + 4 * j + q < blocks;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st16(xslot + 4096 * m + 256 * (4 * i + q) + 16 * (l16 ^ (4 * i + q)), x[j][m][i]);
      load_x(p + 1, j);
      __builtin_amdgcn_sched_barrier(0);
      fence();
      Blk<FMT> b[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        b[r] = unpack_block<FMT>(ld16(slot + 2048 * r + 128 * l16 + 16 * ((4 * j + q) ^ (l16 >> 1))),
                                 sslot[(16 * r + l16) * 8 + 4 * j + q], in);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8 xf[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          xf[m] = bitcast<bf16x8>(ld16(xslot + 4096 * m + 256 * l16 + 16 * ((4 * q + k) ^ l16)));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          bf16x8 lo;
          const bf16x8 hi = decode<FMT>(b[r], k, lo);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, xf[m], acc[r][m], 0, 0, 0);
            if constexpr (FMT == MOE_W_INT4_G32)
              acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, xf[m], acc[r][m], 0, 0, 0);
          }
        }
        if (k == 1) __builtin_amdgcn_sched_barrier(0);  // (or the reads of all four k come first, and spill)
      }
      fence();
    }
    load_w(p + 1);
    __builtin_amdgcn_sched_barrier(0);  // (the next span's waits stay behind its loads)
  }
  // the waves' sums: [wave][r][m][lane] as four rows of one token
  __syncthreads();
  f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[((wave * RT + r) * MT + m) * 64 + lane] = acc[r][m];
  __syncthreads();
  const float ts = FMT == MOE_W_NVFP4 ? *a.w.ts : 1.0f;
  for (int i = threadIdx.x; i < RT * MT * 64; i += 64 * NW) {
    f32x4 v = red[i];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w * RT * MT * 64 + i];
    const int l = i & 63, m = (i >> 6) % MT, r = i / (64 * MT);
    const int t = 16 * m + (l & 15), n = n0 + 16 * r + 4 * (l >> 4);
    if (t < toks) store_out<FMT>(a, t0 + t, n, v, ts);
  }
}

// ---- many tokens: tiles of 128 rows of W x 32 MTW tokens, shared by four waves ----
// Two by two waves of 64 rows x 16 MTW tokens, so that two waves decode each weight; INT4, whose decoding takes the
// vector ALU about as long as its two MFMAs take the matrix core, has four waves of 32 rows x all tokens (WT = 1),
// which decodes each weight once and reads twice the x from LDS (2048 tokens x 4096 x 7168: 280 -> 201 us).
// K runs in spans of 256 values, each in four steps of 64.  Weights: the workgroup loads a span of codes (whole
// 128-byte lines, eight neighbouring lanes per row) and scale bytes into registers one span ahead, and passes them
// to the other of two LDS buffers a quarter per step; waves read them in MFMA layout and decode in registers.  x:
// 128 bytes per token and step, loaded XD steps ahead, through a two-stage LDS ring.  (Loading codes and scales
// straight in MFMA layout, 16 rows x 4 lanes, cost the address unit one cycle per lane: 2048 tokens x 4096 x 7168
// took 146 us, 118 us so.)  16-byte pieces are exchanged inside a row so that the rows of an MFMA operand read
// distinct banks.  With few tiles the workgroups of a tile share K (splits) and leave fp32 partial sums, which
// linear_join_kernel adds in order.
constexpr int kRowsT = 128;  // rows of a tile

// MFMA operands of two dwords (sixteen codes, half `h` of a 32-value block) and the block's scale word; INT4 also
// the low operands.  Codes and scale words past K are zero, and so are their weights.
template <int FMT>
__device__ __forceinline__ void decode_half(u32x2 c, uint32_t w, int h, bf16x8 (&hi)[2], bf16x8 (&lo)[2]) {
  Blk<FMT> b;
  b.q = u32x4{c[0], c[1], 0u, 0u};
  if constexpr (FMT == MOE_W_MXFP4) {
    b.s0 = e8m0_to_f32(w);
  } else if constexpr (FMT == MOE_W_INT4_G32) {
    b.s0 = (float)bitcast<_Float16>((uint16_t)w);
    b.s1 = -(float)(w >> 16) * b.s0;
  } else {
    b.s0 = e4m3_value((w >> (8 * h)) & 255u);
  }
  hi[0] = decode<FMT>(b, 0, lo[0]);
  hi[1] = decode<FMT>(b, 1, lo[1]);
}

template <int DT>
__device__ __forceinline__ void store4(const LinArgs& a, int t, int n, f32x4 v, bool vec) {
  typename Val<DT>::S* d = reinterpret_cast<typename Val<DT>::S*>(a.y) + (int64_t)t * a.y_stride + n;
  if (vec && n + 4 <= a.N) {
    if constexpr (DT == MOE_DT_FP32)
      *reinterpret_cast<f32x4*>(d) = v;
    else
      *reinterpret_cast<u32x2*>(d) = u32x2{(uint32_t)f32_to_16(v[0], DT) | ((uint32_t)f32_to_16(v[1], DT) << 16),
                                           (uint32_t)f32_to_16(v[2], DT) | ((uint32_t)f32_to_16(v[3], DT) << 16)};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.N) {
      if constexpr (DT == MOE_DT_FP32)
        d[e] = v[e];
      else
        d[e] = f32_to_16(v[e], DT);
    }
}

// A wave's outputs: rows n + 16 r + i of token t + 16 m from acc[r][m][i].
template <int FMT, int DT, int RW, int MW>
__device__ __forceinline__ void tile_out(const LinArgs& a, int t, int n, const f32x4 (&acc)[RW][MW],
                                         const f32x4 (&bias)[RW], float ts, bool vec) {
#pragma unroll
  for (int m = 0; m < MW; ++m)
    if (t + 16 * m < a.T) {
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        f32x4 v = acc[r][m];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = FMT == MOE_W_NVFP4 ? __builtin_fmaf(v[e], ts, bias[r][e]) : v[e] + bias[r][e];
        store4<DT>(a, t + 16 * m, n + 16 * r, v, vec);
      }
    }
}

template <int FMT, int MTW>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinArgs a, int t_tiles, int n_tiles, int splits) {
  constexpr int WT = FMT == MOE_W_INT4_G32 ? 1 : 2;               // waves along the tokens
  constexpr int RW = 2 * WT, MW = 2 * MTW / WT;                  // a wave's row and token tiles of 16
  constexpr int kTok = 32 * MTW, kX = kTok * 128, kW = kRowsT * 128, kS = kRowsT * 8;
  __shared__ __attribute__((aligned(16))) uint8_t xbuf[2][kX];
  __shared__ __attribute__((aligned(16))) uint8_t wbuf[2][kW];
  __shared__ uint32_t sbuf[2][kS];  // [row][8]: a block's scale word
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int l16 = lane & 15, q = lane >> 4;
  const int split = blockIdx.x / (t_tiles * n_tiles), tile = blockIdx.x % (t_tiles * n_tiles);
  const int t0 = (tile % t_tiles) * kTok, n0 = (tile / t_tiles) * kRowsT;
  const int wn = (wave / WT) * 16 * RW, wt = (wave % WT) * 16 * MW;  // the wave's first row and token in the tile
  const int blocks = a.K / 32, spans = (a.K + kSpan - 1) / kSpan;
  const int p0 = (int)((int64_t)spans * split / splits), n = (int)((int64_t)spans * (split + 1) / splits) - p0;
  // As in the streaming kernel, a load's per-lane offset holds the row and is checked (rows past N and tokens past
  // T read zeros; so do lanes past K), the uniform offset adds the place in K.  No load is conditional: the
  // registers of loads in flight would be merged, and waited for, at the end of each turn.
  constexpr int kPer = FMT == MOE_W_MXFP4 ? 1 : 2;  // scale bytes per block
  const int rows = min(kRowsT, a.N - n0), toks = min(kTok, a.T - t0);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w.w + (int64_t)n0 * a.w.wr, (int64_t)(rows - 1) * a.w.wr + a.K / 2);
  const __amdgpu_buffer_rsrc_t sr =
      make_rsrc(a.w.s + (int64_t)n0 * a.w.sr, (int64_t)(rows - 1) * a.w.sr + kPer * blocks);
  const __amdgpu_buffer_rsrc_t zr =
      FMT == MOE_W_INT4_G32 ? make_rsrc(a.w.z + (int64_t)n0 * a.w.zr, (int64_t)(rows - 1) * a.w.zr + (blocks + 1) / 2)
                            : sr;
  const __amdgpu_buffer_rsrc_t xr =
      make_rsrc(a.x + (int64_t)t0 * a.x_stride, ((int64_t)(toks - 1) * a.x_stride + a.K) * 2);
  const int pr = tid >> 3, pc = tid & 7;  // this thread's rows pr + 32 i and block (piece of x) pc of a row
  const uint32_t woff = (uint32_t)(pr * a.w.wr) + 16u * pc, soff = (uint32_t)(pr * a.w.sr) + kPer * pc;
  const uint32_t zoff = (uint32_t)(pr * a.w.zr) + (pc >> 1), xoff = (uint32_t)(pr * a.x_stride) * 2u + 16u * pc;
  constexpr int XD = 2;  // steps of x in flight (four: the same time, and spills in the INT4 kernel)
  u32x4 codes[4], x[XD][MTW];  // row group i of the next span; pieces i of the next steps
  uint32_t sc[4], zp[4];
  auto load_w = [&](int turn, int i) {
    const int p = p0 + turn;
    const uint32_t out = turn < n && 8 * p + pc < blocks ? 0u : kOutOfRange;
    codes[i] = bld16s(wr, (woff + (uint32_t)(32 * i * a.w.wr)) | out, 128u * p);
    sc[i] = bld_scale<FMT>(sr, (soff + (uint32_t)(32 * i * a.w.sr)) | out, 8u * kPer * p);
    if constexpr (FMT == MOE_W_INT4_G32)
      zp[i] = __builtin_amdgcn_raw_buffer_load_b8(zr, (zoff + (uint32_t)(32 * i * a.w.zr)) | out, 4u * p, 0);
  };
  auto put_w = [&](int buf, int i) {
    const int row = pr + 32 * i;
    st16(wbuf[buf] + 128 * row + 16 * (pc ^ ((row >> 1) & 7)), codes[i]);
    sbuf[buf][8 * row + pc] = scale_word<FMT>(sc[i], zp[i], pc & 1);
  };
  // set: step % XD, given apart so that it is a constant
  auto load_x = [&](int step, int set) {
    const int turn = step >> 2, k = kSpan * (p0 + turn) + 64 * (step & 3);
    const uint32_t out = turn < n && k + 8 * pc < a.K ? 0u : kOutOfRange;
#pragma unroll
    for (int i = 0; i < MTW; ++i)
      x[set][i] = bld16s(xr, (xoff + (uint32_t)(32 * i * a.x_stride) * 2u) | out, 2u * k);
  };
  auto put_x = [&](int stage, int set) {
#pragma unroll
    for (int i = 0; i < MTW; ++i) {
      const int t = pr + 32 * i;
      st16(xbuf[stage] + 128 * t + 16 * (pc ^ (t & 7)), x[set][i]);
    }
  };
  f32x4 acc[RW][MW];
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int m = 0; m < MW; ++m) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) load_w(0, i);
#pragma unroll
  for (int c = 0; c < XD; ++c) load_x(c, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    put_w(0, i);
    load_w(1, i);
  }
  put_x(0, 0);
  load_x(XD, 0);
  __syncthreads();
  for (int turn = 0; turn < n; ++turn) {
    const int buf = turn & 1;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int stage = c & 1, b = 2 * c + (q >> 1);  // this lane's block of the span
      bf16x8 xf[MW][2];
#pragma unroll
      for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          xf[m][s] = bitcast<bf16x8>(ld16(xbuf[stage] + 128 * (wt + 16 * m + l16) + 16 * ((2 * q + s) ^ (l16 & 7))));
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const int row = wn + 16 * r + l16;
        const u32x2 cd =
            *reinterpret_cast<const u32x2*>(wbuf[buf] + 128 * row + 16 * (b ^ ((l16 >> 1) & 7)) + 8 * (q & 1));
        bf16x8 hi[2], lo[2];
        decode_half<FMT>(cd, sbuf[buf][8 * row + b], q & 1, hi, lo);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < MW; ++m) {
            acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[s], xf[m][s], acc[r][m], 0, 0, 0);
            if constexpr (FMT == MOE_W_INT4_G32)
              acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[s], xf[m][s], acc[r][m], 0, 0, 0);
          }
      }
      __builtin_amdgcn_sched_barrier(0);  // the waits for the next step's data stay behind the products
      put_x(stage ^ 1, (c + 1) % XD);
      put_w(buf ^ 1, c);
      load_x(4 * turn + c + 1 + XD, (c + 1) % XD);
      load_w(turn + 2, c);
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const int tw = wt, nw = n0 + wn;
  // lane: rows 4q + i of row tile r, token l16 of token tile m
  f32x4 bias[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = nw + 16 * r + 4 * q + e;
      bias[r][e] = a.bias && splits == 1 && n < a.N ? a.bias[n] : 0.0f;
    }
  const float ts = FMT == MOE_W_NVFP4 && splits == 1 ? *a.w.ts : 1.0f;
  if (splits > 1) {
    LinArgs o = a;
    o.y = reinterpret_cast<float*>(a.ws) + (int64_t)split * a.T * a.N;
    o.y_stride = a.N;
    tile_out<FMT, MOE_DT_FP32>(o, t0 + tw + l16, nw + 4 * q, acc, bias, ts, a.N % 4 == 0);
    return;
  }
  const bool vec = a.y_stride % 4 == 0 && ((uintptr_t)a.y & (a.y_dt == MOE_DT_FP32 ? 15u : 7u)) == 0;
  if (a.y_dt == MOE_DT_FP32) tile_out<FMT, MOE_DT_FP32>(a, t0 + tw + l16, nw + 4 * q, acc, bias, ts, vec);
  else if (a.y_dt == MOE_DT_BF16) tile_out<FMT, MOE_DT_BF16>(a, t0 + tw + l16, nw + 4 * q, acc, bias, ts, vec);
  else tile_out<FMT, MOE_DT_FP16>(a, t0 + tw + l16, nw + 4 * q, acc, bias, ts, vec);
}

// y = the partial sums of the splits in order, with the tensor scale and the bias.  Eight loads of a thread are
// issued before the first addition (one after another they took 11 us for 128 tokens x 7168, eight splits).
constexpr int kMaxSplits = 32;
template <int FMT>
__global__ __launch_bounds__(256) void linear_join_kernel(LinArgs a, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int n4 = (a.N + 3) / 4;
  if (i >= (int64_t)a.T * n4) return;
  const int t = (int)(i / n4), n = (int)(i % n4) * 4;
  const float* p = reinterpret_cast<const float*>(a.ws) + (int64_t)t * a.N + min(n, max(a.N - 4, 0));
  const int64_t plane = (int64_t)a.T * a.N;
  const float ts = FMT == MOE_W_NVFP4 ? *a.w.ts : 1.0f;
  if (n + 4 <= a.N) {
    constexpr int kBatch = 8;
    f32x4 v[kBatch], sum = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += kBatch) {
#pragma unroll
      for (int s = 0; s < kBatch; ++s) __builtin_memcpy(&v[s], p + min(s0 + s, splits - 1) * plane, 16);
#pragma unroll
      for (int s = 0; s < kBatch; ++s)
        if (s0 + s < splits) sum += v[s];
    }
    store_out<FMT>(a, t, n, sum, ts);
  } else {  // the last columns of a row
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) sum[e] += reinterpret_cast<const float*>(a.ws)[s * plane + (int64_t)t * a.N + n + e];
    store_out<FMT>(a, t, n, sum, ts);
  }
}

// Eight rows per workgroup; eight waves where the rows give at most a workgroup per CU (one token, 1000 x 2080
// INT4 3.3 against 3.5 us with four waves, 512 x 7168 NVFP4 3.5 against 4.3), four beyond (7168 x 7168 MXFP4 7.9
// against 9.2).
template <int FMT, int TT>
void launch_dot_tokens(const LinArgs& a, hipStream_t stream) {
  const dim3 g((unsigned)((a.N + 7) / 8));
  if (a.N <= 2048) linear_dot_kernel<FMT, TT, 8><<<g, 512, 0, stream>>>(a);
  else linear_dot_kernel<FMT, TT, 4><<<g, 256, 0, stream>>>(a);
}

// Rows (16 rt) and tokens (16 mt) of a streaming workgroup.
// Up to 16 tokens two workgroups of 16 or 32 rows share a CU (53 and 74 KB of LDS), one of 64 has it alone.  16 rows
// while each workgroup has a CU of its own (INT4, whose decoding bounds it: to 12288 rows), 32 beyond; MXFP4 from six
// spans of K on takes 64 where they leave the last round of the card more than half full.  us for 16 tokens with 16, 32
// and 64 rows a workgroup:
//   MXFP4  K = 1024   8300 rows  6.1  4.9  5.8    NVFP4  K = 4096   4096 rows  6.2  7.6 11.3
//          K = 1536  16384       9.0  6.9  6.7                      6144       9.2  8.1 11.6
//          K = 4096   4096       6.2  7.0  9.8                     12800      16.0 12.7 12.6
//                     6144       9.0  7.3 10.1                     18432      19.0 17.1 22.2
//                     8300      11.8 11.2 10.5                     32768      29.8 24.0 25.2
//                    16384      16.0 12.7 12.6    INT4   K = 1024   9216       7.9  6.8  9.3
//                    18432      18.5 16.5 19.5           K = 4096   6144      10.7 10.9 17.1
//          K = 7168   8300      18.3 17.7 15.8                     12288      15.2 16.7 18.1
//                    18432      29.8 26.5 30.1                     12800      18.3 16.8 18.4
//                    32768      47.3 37.9 35.3                     18432      22.5 23.0 32.8
//                   129280     173.4 133.0 127.1         K = 7168   9216      23.0 25.6 29.5
// Beyond 16 tokens a workgroup has a CU alone: the fewest rows that leave at most one workgroup per CU, since those of
// a second round start when the first have ended (32 tokens x 4096 MXFP4: 4096 rows 8.0 us, 4500 rows 13.8 with 16
// rows a workgroup and 9.5 with 32; 8192 rows 10.2 with 32, 8838 rows 16.9, and 13.4 with 64).  More than 32
// tokens take a workgroup per 32 or 64 of them and rows, in place of tiles (mt 0), while one round holds them all and
// K is not long, since then a tile's steps and the join of its shares wait for their loads (us, streamed and tiles:
// 135 x 257 x 1728 INT4 5.6 and 15.1, 256 x 1024 x 2048 MXFP4 7.0 and 11.6, 128 x 4096 x 4096 13.3 and 18.9, 512 x
// 2048 x 7168 30.3 and 32.1; K = 9248 18.1 and 21.8, 16384 20.8 and 19.3).  64 rows x 64 tokens of INT4, four waves
// with two products per weight, only to K = 4096 (512 x 2048 x 1024 13.1 and 17.9, 100 x 6144 x 4096 30.8 and 29.6,
// 40 x 8838 x 7296 55 and 38).
constexpr int kCus = 256;
struct StreamPlan {
  int rt, mt;
};
StreamPlan stream_plan(int fmt, int T, int N, int K) {
  if (T <= 16) {
    if (N <= (fmt == MOE_W_INT4_G32 ? 48 : 16) * kCus) return {1, 1};
    const int last = (N + 63) / 64 % kCus;  // 64-row workgroups of the last round, 0: it is full
    return {fmt == MOE_W_MXFP4 && K > 5 * kSpan && (last == 0 || last > kCus / 2) ? 4 : 2, 1};
  }
  if (T > 32 && K > 12288) return {0, 0};
  constexpr StreamPlan sizes[] = {{1, 2}, {2, 2}, {4, 2}, {4, 4}};
  for (const StreamPlan& p : sizes) {
    const int64_t groups = (int64_t)((N + 16 * p.rt - 1) / (16 * p.rt)) * ((T + 16 * p.mt - 1) / (16 * p.mt));
    if (groups <= kCus && !(p.mt == 4 && fmt == MOE_W_INT4_G32 && K > 4096)) return p;
  }
  return T <= 32 ? StreamPlan{4, 2} : StreamPlan{0, 0};
}
// Eight waves, four where their LDS does not fit (64 rows and 64 tokens).
template <int FMT, int RT, int MT>
void launch_stream(const LinArgs& a, hipStream_t stream) {
  constexpr int NW = RT * MT == 16 ? 4 : 8;
  const dim3 g((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.T + 16 * MT - 1) / (16 * MT)));
  linear_stream_kernel<FMT, RT, MT, NW><<<g, 64 * NW, 0, stream>>>(a);
}

// Three and four tokens: dot products up to this many rows, 200 workgroups of the streaming kernel (4 tokens, 2048 x
// 7168 MXFP4: 6.0 us, streamed 7.5; 4096 x 4096: 5.9 and 5.6; 7168 x 7168: 13.7 and 10.2; 3200 x 4096 INT4 6.7 and
// 7.0).  Two tokens are faster by dot products at every size (7168 x 7168 MXFP4 9.1 us and 9.8, INT4 13.0 and 17.7).
constexpr int kDotRows = 16 * 200;

// Tiles and K shares of the tile kernel.  128-token tiles where they give a workgroup per CU (2048 tokens x 4096 x
// 7168 MXFP4: 118 us, 156 with 64), 64-token ones below.  K is shared over up to 32 workgroups, at least a span each,
// until there are up to two workgroups per CU (60 tokens x 65 x 13088 INT4: 19.8 us, 22.1 with 16, 29.1 with 8); at
// least five spans each from 128 tiles on (440 tokens x 2714 x 1024 NVFP4: 17.3 us, 24.5 with three shares; 512 x
// 2048 x 7168 INT4: 49 with four, 57 with three); not at all where the tiles alone come near one per CU (1024 tokens x
// 2048 x 2048: 20 us, 24 with two shares).
struct TilePlan {
  int mtw, t_tiles, n_tiles, splits;
};
TilePlan tile_plan(int T, int N, int K) {
  TilePlan p;
  p.n_tiles = (N + kRowsT - 1) / kRowsT;
  p.mtw = (int64_t)((T + 127) / 128) * p.n_tiles >= 256 ? 4 : 2;
  p.t_tiles = (T + 32 * p.mtw - 1) / (32 * p.mtw);
  const int64_t tiles = (int64_t)p.t_tiles * p.n_tiles;
  const int64_t most =
      tiles >= 192 ? 1 : std::min<int64_t>(kMaxSplits, std::max(1, K / (tiles >= 128 ? 5 * kSpan : kSpan)));
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, 512 / tiles));
  return p;
}

template <int FMT>
hipError_t linear_tiles(const LinArgs& a, hipStream_t stream) {
  const TilePlan p = tile_plan(a.T, a.N, a.K);
  const int64_t g = (int64_t)p.t_tiles * p.n_tiles * p.splits;
  if (g > 0x7FFFFF) return hipErrorInvalidConfiguration;  // (more than 2^31 threads)
  if (p.mtw == 2)
    linear_tile_kernel<FMT, 2><<<dim3((unsigned)g), 256, 0, stream>>>(a, p.t_tiles, p.n_tiles, p.splits);
  else
    linear_tile_kernel<FMT, 4><<<dim3((unsigned)g), 256, 0, stream>>>(a, p.t_tiles, p.n_tiles, p.splits);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.splits == 1) return err;
  const int64_t n = (int64_t)a.T * ((a.N + 3) / 4);
  linear_join_kernel<FMT><<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(a, p.splits);
  return hipGetLastError();
}

template <int FMT>
hipError_t linear_fmt(const LinArgs& a, hipStream_t stream) {
  const StreamPlan s = stream_plan(FMT, a.T, a.N, a.K);
  if (a.T == 1) launch_dot_tokens<FMT, 1>(a, stream);
  else if (a.T == 2) launch_dot_tokens<FMT, 2>(a, stream);
  else if (a.T <= 4 && a.N <= kDotRows) launch_dot_tokens<FMT, 4>(a, stream);
  else if (s.mt == 0) return linear_tiles<FMT>(a, stream);
  else if (s.mt == 4) launch_stream<FMT, 4, 4>(a, stream);
  else if (s.mt == 2 && s.rt == 4) launch_stream<FMT, 4, 2>(a, stream);
  else if (s.mt == 2 && s.rt == 2) launch_stream<FMT, 2, 2>(a, stream);
  else if (s.mt == 2) launch_stream<FMT, 1, 2>(a, stream);
  else if (s.rt == 4) launch_stream<FMT, 4, 1>(a, stream);
  else if (s.rt == 2) launch_stream<FMT, 2, 1>(a, stream);
  else launch_stream<FMT, 1, 1>(a, stream);
  return hipGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(int fmt, int T, int N, int K) {
  if (stream_plan(fmt, T, N, K).mt != 0) return 0;
  const TilePlan p = tile_plan(T, N, K);
  return p.splits > 1 ? sizeof(float) * (size_t)p.splits * (size_t)T * (size_t)N : 0;
}

hipError_t launch_linear(const LinArgs& a, hipStream_t stream) {
  if (a.fmt == MOE_W_MXFP4) return linear_fmt<MOE_W_MXFP4>(a, stream);
  if (a.fmt == MOE_W_INT4_G32) return linear_fmt<MOE_W_INT4_G32>(a, stream);
  return linear_fmt<MOE_W_NVFP4>(a, stream);
}

}  // namespace moe
