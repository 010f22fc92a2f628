// Rotary positions and the write into a paged key-value cache.  For a token at position p, with the angles' cosines and
// sines from a table, every head of q and k turns its first R values in pairs (a, b):
//   a' = a cos - b sin,  b' = b cos + a sin     (fp32, each product and sum rounded by itself)
// pairs (i, i + R/2) or (2i, 2i + 1); values from R on pass through, and so does v.  One rounding at each output; the
// MXFP8 codes come from the fp32 values, not from rounded ones.
//
// Bytes bound it: every value is read and written once.  A lane takes eight consecutive values of a head, a head's
// lanes sit in one wave (so q may be rotated in place: a wave has read a head before it writes it), the four lanes of an
// MX block share its largest magnitude by two moves.
#include "attention.hpp"
#include "mx.hpp"

namespace moe {

namespace {

#pragma clang fp contract(off)
__device__ __forceinline__ float turn_low(float a, float b, float c, float s) { return a * c - b * s; }
__device__ __forceinline__ float turn_high(float a, float b, float c, float s) { return b * c + a * s; }
#pragma clang fp contract(fast)

// The turned value d of a row, one value at a time (R/2 off the grid of eight).
template <int XD>
__device__ __forceinline__ float turned(const RopeArgs& a, const void* x, int64_t row, int d, int64_t angle) {
  const float v = ld_value(x, XD, row + d);
  if (d >= a.R) return v;
  const int half = a.R >> 1;
  const bool high = a.neighbours ? (d & 1) != 0 : d >= half;
  const int i = a.neighbours ? d >> 1 : (high ? d - half : d);
  const float o = ld_value(x, XD, row + (a.neighbours ? d ^ 1 : (high ? d - half : d + half)));
  const float c = a.cos[angle + i], s = a.sin[angle + i];
  return high ? turn_high(o, v, c, s) : turn_low(v, o, c, s);
}

// FAST: R/2 (halves) or R (neighbours) is a multiple of eight, so a run of eight has its partners in one other run, or
// in itself.
template <int XD, bool FAST>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  const int lane = threadIdx.x & 63;
  const int in_wave = lane / a.runs;             // head row of the wave
  const int d = 8 * (lane - in_wave * a.runs);
  // (T * n_rows is at most 2^27)
  const uint32_t unit = (blockIdx.x * 4 + (threadIdx.x >> 6)) * (uint32_t)a.rows_per_wave + (uint32_t)in_wave;
  const bool there = in_wave < a.rows_per_wave && unit < (uint32_t)a.T * a.n_rows.d;
  const int64_t t = there ? div_by(a.n_rows, unit) : 0;
  const int r = there ? (int)(unit - (uint32_t)t * a.n_rows.d) : 0;
  const int which = r < a.Hq ? 0 : (r < a.Hq + a.Hkv ? 1 : 2);
  const int h = which == 0 ? r : r - a.Hq - (which == 2 ? a.Hkv : 0);
  const HeadsDev& in = a.in[which];
  const int p = a.positions && there ? a.positions[t] : 0;
  const bool ok = there && in.p && (!a.positions || (uint32_t)p < (uint32_t)a.n_positions);
  const int64_t row = t * in.ts + h * in.hs;
  const int64_t angle = (int64_t)p * (a.R >> 1);
  float y[8];
  if (ok) {
    if constexpr (FAST) {
      raw8_to_f32(ld_raw8<XD>(in.p, row + d), y);
      if (which < 2 && d < a.R) {
        if (a.neighbours) {
          float c[4], s[4];
          __builtin_memcpy(c, a.cos + angle + (d >> 1), 16);
          __builtin_memcpy(s, a.sin + angle + (d >> 1), 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = y[2 * j], hi = y[2 * j + 1];
            y[2 * j] = turn_low(lo, hi, c[j], s[j]);
            y[2 * j + 1] = turn_high(lo, hi, c[j], s[j]);
          }
        } else {
          const int half = a.R >> 1;
          const bool high = d >= half;
          const int i = high ? d - half : d;
          float o[8], c[8], s[8];
          raw8_to_f32(ld_raw8<XD>(in.p, row + (high ? d - half : d + half)), o);
          raw8_to_f32(ld_raw8<MOE_DT_FP32>(a.cos, angle + i), c);
          raw8_to_f32(ld_raw8<MOE_DT_FP32>(a.sin, angle + i), s);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = high ? turn_high(o[j], y[j], c[j], s[j]) : turn_low(y[j], o[j], c[j], s[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = which < 2 ? turned<XD>(a, in.p, row, d + j, angle) : ld_value(in.p, XD, row + d + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = 0.0f;
  }
  const HeadsDev& out = a.out[which];
  if (ok && out.p) st8(out.p, out.dt, t * out.ts + h * out.hs + d, y);
  if (which == 0 && a.fmt != MOE_KV_MXFP8) return;  // (the MX blocks' moves below need every lane)
  const int slot = ok && which != 0 && a.slots ? a.slots[t] : -1;
  const bool keep = slot >= 0 && slot < a.n_slots;
  const int page = keep ? (int)div_by(a.page_size, (uint32_t)slot) : 0;
  const int at = keep ? slot - page * (int)a.page_size.d : 0;
  void* base = which == 2 ? a.cache_v : a.cache_k;
  const int64_t i = (int64_t)page * a.c_page + (int64_t)h * a.c_head + (int64_t)at * a.c_token + d;
  if (a.fmt != MOE_KV_MXFP8) {
    if (keep) st8(base, a.fmt, i, y);
    return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
  amax = fmaxf(amax, __shfl_xor(amax, 1, kWave));
  amax = fmaxf(amax, __shfl_xor(amax, 2, kWave));
  if (!keep) return;
  const uint32_t sc = mx_scale_code<MOE_MX_FP8_E4M3>(amax);
  uint32_t dw[2];
  mx_pack_quarter<MOE_MX_FP8_E4M3>(y, mx_inv_scale(sc), dw);
  *reinterpret_cast<u32x2*>((uint8_t*)base + i) = u32x2{dw[0], dw[1]};
  if ((d & 31) == 0) {
    uint8_t* scales = which == 2 ? a.scale_v : a.scale_k;
    scales[(int64_t)page * a.s_page + (int64_t)h * a.s_head + (int64_t)at * a.s_token + (d >> 5)] = (uint8_t)sc;
  }
}

template <int XD>
void launch_rope_x(const RopeArgs& a, dim3 g, hipStream_t stream) {
  if (a.R % (a.neighbours ? 8 : 16) == 0) rope_kernel<XD, true><<<g, 256, 0, stream>>>(a);
  else rope_kernel<XD, false><<<g, 256, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_rope(RopeArgs a, hipStream_t stream) {
  a.runs = a.D / 8;
  a.rows_per_wave = 64 / a.runs;
  const int64_t waves = ((int64_t)a.T * a.n_rows.d + a.rows_per_wave - 1) / a.rows_per_wave;
  const dim3 g((unsigned)((waves + 3) / 4));
  if (a.x_dt == MOE_DT_BF16) launch_rope_x<MOE_DT_BF16>(a, g, stream);
  else if (a.x_dt == MOE_DT_FP16) launch_rope_x<MOE_DT_FP16>(a, g, stream);
  else launch_rope_x<MOE_DT_FP32>(a, g, stream);
  return hipGetLastError();
}

}  // namespace moe
