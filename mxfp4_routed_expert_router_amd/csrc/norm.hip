// Residual addition and root-mean-square norm, with an optional MX output (8-, 6- or 4-bit codes with one E8M0
// scale per 32 values, the layout the MX expert FFN reads).  Per row of H values:
//   s = x + residual                      (fp32; residual_out = s rounded to the residual's type)
//   r = 1 / sqrt(sum(s^2) / H + eps)      (fp32 sums of a thread and of a wave; from there in 64 bits, rounded once)
//   y = s * r * weight                    (fp32; rounded once to y's type)
//   codes, scales = MX blocks of the fp32 y (not of the rounded one: one rounding, not two)
// It reads x and residual and writes residual_out, y and the codes once each, so the bytes bound it; the row
// stays in registers between the sum and the outputs.
#include <algorithm>

#include "launch.hpp"
#include "mx.hpp"
#include "values.hpp"

namespace moe {

namespace {

// 1 / sqrt(sum / H + eps) of the workgroup's v, the same value in every thread (fixed order: a wave's lanes by a
// tree, the waves in wave order).  red: one float per wave.  Joining the waves and the root in 64 bits leave about
// half an fp32 rounding in r, which every value of the row shares, and take less time than fp32's exact division
// and square root: the reciprocal root instruction (2^-24 or better) and one Newton step.
__device__ __forceinline__ float row_scale(const NormArgs& a, float v, float* red) {
  const int wave = threadIdx.x >> 6, n = (blockDim.x + 63) >> 6;
  v = wave_sum_dpp(v);
  double s = (double)v;
  if (n > 1) {
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < n; ++w) s += (double)red[w];
  }
  const double m = __builtin_fma(s, a.inv_h, (double)a.eps);
  const double r = __builtin_amdgcn_rsq(m);
  const double e = __builtin_fma(-m * r, r, 1.0);
  return (float)(m > 0.0 && m < (double)INFINITY ? __builtin_fma(0.5 * r, e, r) : r);  // (0 and infinity have no step)
}

// Codes and scale of a 32-value block held by four consecutive lanes, eight values each (element i of the
// row is the first of this lane's).
template <int F>
__device__ __forceinline__ void store_quarter(const float (&y)[8], uint8_t* __restrict__ codes_row,
                                              uint8_t* __restrict__ scales_row, int i, bool ok) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
  amax = fmaxf(amax, __shfl_xor(amax, 1, kWave));
  amax = fmaxf(amax, __shfl_xor(amax, 2, kWave));
  const uint32_t sc = mx_scale_code<F>(amax);
  uint32_t dw[2];
  mx_pack_quarter<F>(y, mx_inv_scale(sc), dw);
  const int q = (i >> 3) & 3;
  uint8_t* blk = codes_row + (int64_t)(i >> 5) * (4 * Mx<F>::kBits);
  if constexpr (Mx<F>::kBits == 6) {  // 6 bytes per lane: pairs of lanes write 12
    const uint32_t o0 = (uint32_t)__shfl_xor((int)dw[0], 1, kWave);
    const uint32_t o1 = (uint32_t)__shfl_xor((int)dw[1], 1, kWave);
    if (ok && (q & 1) == 0) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(blk + 6 * q);
      dst[0] = dw[0];
      dst[1] = (dw[1] & 0xFFFFu) | (o0 << 16);
      dst[2] = (o0 >> 16) | (o1 << 16);
    }
  } else if constexpr (Mx<F>::kBits == 8) {
    if (ok) *reinterpret_cast<u32x2*>(blk + 8 * q) = u32x2{dw[0], dw[1]};
  } else {
    if (ok) *reinterpret_cast<uint32_t*>(blk + 4 * q) = dw[0];
  }
  if (ok && q == 0) scales_row[i >> 5] = (uint8_t)sc;
}

// One row per workgroup; a thread holds NV runs of eight consecutive values (run v at 8 (v * threads + tid)).  The
// last run of a row ends with it, so it may overlap the one before (H not a multiple of eight): both compute the
// shared values, which count once in the sum.  Accesses are 16 bytes at any alignment.  RD: the residual's type, or
// -1 without one.  Rows of 16-byte aligned pointers and odd ones run alike: 333 rows of 4097 fp16 values 18.8 us one
// value per access, 7.1 us with all of a row's loads in flight, 4.7 us as here.
template <int XD, int RD, int NV>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ float red[16];
  const int64_t t = blockIdx.x;
  const int H = a.H;
  constexpr int RT = RD < 0 ? MOE_DT_BF16 : RD;
  Raw8<XD> xr[NV];
  Raw8<RT> rr[NV];
  int at[NV];  // first value of the run, and where it does not overlap the run before
#pragma unroll
  for (int v = 0; v < NV; ++v) {  // runs past the row read its last and are not used
    at[v] = min(8 * (v * (int)blockDim.x + (int)threadIdx.x), H - 8);
    xr[v] = ld_raw8<XD>(a.x, t * a.x_stride + at[v]);
    if constexpr (RD >= 0) rr[v] = ld_raw8<RT>(a.residual, t * a.r_stride + at[v]);
  }
  // residual_out may be residual, so with overlapping runs it is written behind the sum's barrier
  const bool overlap = H % 8 != 0;
  float s[NV][8], sum = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = 8 * (v * (int)blockDim.x + (int)threadIdx.x);
    raw8_to_f32(xr[v], s[v]);
    if constexpr (RD >= 0) {
      float r[8];
      raw8_to_f32(rr[v], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[v][j] += r[j];
      if (a.residual_out && !overlap && i < H) st8_as<RT>(a.residual_out, t * a.ro_stride + i, s[v]);
    }
    float p = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) p = at[v] + j >= i ? __builtin_fmaf(s[v][j], s[v][j], p) : p;
    sum += i < H ? p : 0.0f;
  }
  const float rstd = row_scale(a, sum, red);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = 8 * (v * (int)blockDim.x + (int)threadIdx.x);
    const bool ok = i < H;
    float w[8], y[8];
    ld8(a.weight, a.w_dt, at[v], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = s[v][j] * rstd * w[j];
    if constexpr (RD >= 0) {
      if (a.residual_out && overlap && ok) st8_as<RT>(a.residual_out, t * a.ro_stride + at[v], s[v]);
    }
    if (a.y && ok) st8(a.y, a.y_dt, t * H + at[v], y);
    if (a.mx) {  // the four lanes of a block are all inside the row or all outside (H % 32 == 0)
      uint8_t* cr = a.codes + t * a.code_row;
      uint8_t* sr = a.scales + t * (H >> 5);
      if (a.mx == MOE_MX_FP8_E4M3) store_quarter<MOE_MX_FP8_E4M3>(y, cr, sr, i, ok);
      else if (a.mx == MOE_MX_FP6_E2M3) store_quarter<MOE_MX_FP6_E2M3>(y, cr, sr, i, ok);
      else store_quarter<MOE_MX_FP4_E2M1>(y, cr, sr, i, ok);
    }
  }
}

// Rows shorter than eight or longer than 32768 values: two passes over the row, one value at a time (the second
// pass finds it in the caches).  residual_out may be residual itself, so the second pass reads a value before it
// writes it.
template <int F>
__device__ __forceinline__ void norm_block(const NormArgs& a, int64_t t, int b, float rstd) {
  float y[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int i = 32 * b + j;
    float s = ld_value(a.x, a.x_dt, t * a.x_stride + i);
    if (a.residual) s += ld_value(a.residual, a.r_dt, t * a.r_stride + i);
    y[j] = s * rstd * ld_value(a.weight, a.w_dt, i);
  }
  uint32_t dw[8];
  const uint32_t sc = mx_pack_block<F>(y, dw);
  mx_store_block<F>(a.codes + t * a.code_row + (int64_t)b * (4 * Mx<F>::kBits), dw);
  a.scales[t * (a.H >> 5) + b] = (uint8_t)sc;
}

__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs a) {
  __shared__ float red[16];
  const int64_t t = blockIdx.x;
  const int H = a.H;
  float sum = 0.0f;
  for (int i = threadIdx.x; i < H; i += 256) {
    float s = ld_value(a.x, a.x_dt, t * a.x_stride + i);
    if (a.residual) s += ld_value(a.residual, a.r_dt, t * a.r_stride + i);
    sum = __builtin_fmaf(s, s, sum);
  }
  const float rstd = row_scale(a, sum, red);
  if (a.mx) {  // before residual_out is written: it may be residual
    for (int b = threadIdx.x; b < (H >> 5); b += 256) {
      if (a.mx == MOE_MX_FP8_E4M3) norm_block<MOE_MX_FP8_E4M3>(a, t, b, rstd);
      else if (a.mx == MOE_MX_FP6_E2M3) norm_block<MOE_MX_FP6_E2M3>(a, t, b, rstd);
      else norm_block<MOE_MX_FP4_E2M1>(a, t, b, rstd);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < H; i += 256) {
    float s = ld_value(a.x, a.x_dt, t * a.x_stride + i);
    if (a.residual) s += ld_value(a.residual, a.r_dt, t * a.r_stride + i);
    if (a.residual_out) st_value(a.residual_out, a.r_dt, t * a.ro_stride + i, s);
    if (a.y) st_value(a.y, a.y_dt, t * H + i, s * rstd * ld_value(a.weight, a.w_dt, i));
  }
}

template <int XD, int RD>
void launch_norm_vec(const NormArgs& a, int threads, int nv, hipStream_t stream) {
  const dim3 g((unsigned)a.T);
  if (nv == 1) norm_kernel<XD, RD, 1><<<g, threads, 0, stream>>>(a);
  else if (nv == 2) norm_kernel<XD, RD, 2><<<g, threads, 0, stream>>>(a);
  else norm_kernel<XD, RD, 4><<<g, threads, 0, stream>>>(a);
}
template <int XD>
void launch_norm_x(const NormArgs& a, int threads, int nv, hipStream_t stream) {
  if (!a.residual) launch_norm_vec<XD, -1>(a, threads, nv, stream);
  else if (a.r_dt == MOE_DT_BF16) launch_norm_vec<XD, MOE_DT_BF16>(a, threads, nv, stream);
  else if (a.r_dt == MOE_DT_FP16) launch_norm_vec<XD, MOE_DT_FP16>(a, threads, nv, stream);
  else launch_norm_vec<XD, MOE_DT_FP32>(a, threads, nv, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int kMostRows = 1 << 20;  // of a launch: fewer than 2^32 threads
  if (a.T > kMostRows) {
    for (int64_t t = 0; t < a.T; t += kMostRows) {
      const auto row = [t](auto* p, int64_t values, int dt) {
        return p ? (decltype(p))((uintptr_t)p + t * values * (dt == MOE_DT_FP32 ? 4 : 2)) : p;
      };
      NormArgs b = a;
      b.x = row(a.x, a.x_stride, a.x_dt);
      b.residual = row(a.residual, a.r_stride, a.r_dt);
      b.residual_out = row(a.residual_out, a.ro_stride, a.r_dt);
      b.y = row(a.y, a.H, a.y_dt);
      if (a.mx) {
        b.codes = a.codes + t * a.code_row;
        b.scales = a.scales + t * (a.H / 32);
      }
      b.T = (int)std::min<int64_t>(kMostRows, a.T - t);
      const hipError_t err = launch_norm(b, stream);
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  }
  if (a.H < 8 || a.H > 8 * 1024 * 4) {
    norm_any_kernel<<<dim3((unsigned)a.T), 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  // As few values per thread as 1024 threads allow: at 7168 values one run per thread takes 3.1 us for one row (two
  // 3.4, four 4.1), 5.1 us for 176 (5.7, 7.0), and 8192 rows are bound by their bytes (95.8, 94.0, 96.5).
  const int runs = (a.H + 7) / 8;
  const int nv = runs <= 1024 ? 1 : (runs <= 2048 ? 2 : 4);
  const int threads = ((runs + nv - 1) / nv + 63) / 64 * 64;
  if (a.x_dt == MOE_DT_BF16) launch_norm_x<MOE_DT_BF16>(a, threads, nv, stream);
  else if (a.x_dt == MOE_DT_FP16) launch_norm_x<MOE_DT_FP16>(a, threads, nv, stream);
  else launch_norm_x<MOE_DT_FP32>(a, threads, nv, stream);
  return hipGetLastError();
}

}  // namespace moe
