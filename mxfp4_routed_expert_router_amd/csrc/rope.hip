// Rotary positions and the write into a paged key-value cache.  For a token at position p, with the angles' cosines and
// sines from a table, every head of q and k turns its first R values in pairs (a, b):
//   a' = a cos - b sin,  b' = b cos + a sin     (fp32, each product and sum rounded by itself)
// pairs (i, i + R/2) or (2i, 2i + 1); values from R on pass through, and so does v.  One rounding at each output; the
// MXFP8 codes come from the fp32 values, not from rounded ones.
//
// Bytes bound it: every value is read and written once.  A lane takes eight consecutive values of a head, a head's
// lanes sit in one wave (so q may be rotated in place: a wave has read a head before it writes it), the four lanes of an
// MX block share its largest magnitude by two moves.  A wave's heads are of one token and of one of q, k and v, so that
// position, slot, strides and table row are scalars: 8192 tokens of 64 + 16 heads of 128 in bf16 take 86 us (4.35 TB/s),
// with heads of several kinds in a wave 118; two or four rows to a lane 125 and 167 (fewer waves in flight).
#include <algorithm>

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
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int in_wave = lane / a.runs;             // head row of the wave
  const int d = 8 * (lane - in_wave * a.runs);
  // A wave's rows are heads of one token and of one of q, k and v: all of that is in scalar registers.
  const uint32_t unit = blockIdx.x * 4 + wave;
  if (unit >= (uint32_t)a.T * a.groups.d) return;
  const int64_t t = div_by(a.groups, unit);
  const int r = (int)(unit - (uint32_t)t * a.groups.d);
  const int which = r < a.q_groups ? 0 : (r < a.q_groups + a.kv_groups ? 1 : 2);
  const int h0 = (r - (which == 0 ? 0 : (which == 1 ? a.q_groups : a.q_groups + a.kv_groups))) * a.rows_per_wave;
  const int h = h0 + in_wave;
  const HeadsDev in = a.in[which], out = a.out[which];
  const int p = a.positions ? a.positions[t] : 0;
  const int slot = which != 0 && a.slots ? a.slots[t] : -1;
  if (!in.p || (a.positions && (uint32_t)p >= (uint32_t)a.n_positions)) return;
  const bool ok = in_wave < a.rows_per_wave && h < (which == 0 ? a.Hq : a.Hkv);
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
  if (ok && out.p) st8(out.p, out.dt, t * out.ts + h * out.hs + d, y);
  if (slot < 0 || slot >= a.n_slots) return;
  const int page = (int)div_by(a.page_size, (uint32_t)slot), at = slot - page * (int)a.page_size.d;
  void* base = which == 2 ? a.cache_v : a.cache_k;
  const int64_t i = (int64_t)page * a.c_page + (int64_t)h * a.c_head + (int64_t)at * a.c_token + d;
  if (a.fmt != MOE_KV_MXFP8) {
    if (ok) st8(base, a.fmt, i, y);
    return;
  }
  float amax = 0.0f;  // (every lane takes part in the moves)
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
  amax = fmaxf(amax, __shfl_xor(amax, 1, kWave));
  amax = fmaxf(amax, __shfl_xor(amax, 2, kWave));
  if (!ok) return;
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
  a.q_groups = (a.Hq + a.rows_per_wave - 1) / a.rows_per_wave;
  a.kv_groups = (a.Hkv + a.rows_per_wave - 1) / a.rows_per_wave;
  a.groups = fast_div((uint32_t)(a.q_groups + 2 * a.kv_groups));
  const int most = std::max(1, (1 << 25) / (int)a.groups.d);  // tokens of a launch: at most 2^31 threads
  for (int left = a.T; left > 0;) {
    a.T = std::min(left, most);
    const dim3 g((unsigned)(((int64_t)a.T * a.groups.d + 3) / 4));
    if (a.x_dt == MOE_DT_BF16) launch_rope_x<MOE_DT_BF16>(a, g, stream);
    else if (a.x_dt == MOE_DT_FP16) launch_rope_x<MOE_DT_FP16>(a, g, stream);
    else launch_rope_x<MOE_DT_FP32>(a, g, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    left -= a.T;
    for (HeadsDev* h : {a.in, a.out})
      for (int i = 0; i < 3; ++i)
        if (h[i].p) h[i].p = (char*)h[i].p + a.T * h[i].ts * (h[i].dt == MOE_DT_FP32 ? 4 : 2);
    if (a.positions) a.positions += a.T;
    if (a.slots) a.slots += a.T;
  }
  return hipSuccess;
}

}  // namespace moe
