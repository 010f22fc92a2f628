// Choice of experts from router logits: scores, balance bias, groups, top-k, weights (moe_select_experts), and
// the same choice on the partial sums of the router's logits kernel (moe_route_grouped).
//
// Per token, with L the logits and b the selection bias:
//   s = sigmoid(L) or softmax(L),  key = s + b;  an expert is available when L and b are finite;
//   a group's rank is the sum of its two largest available keys, or its largest; the topk_groups groups of the
//   largest ranks stay (lowest index first on ties), and of their experts the top_k largest keys (likewise);
//   weights = routed_scale * s / (sum of the selected s), or routed_scale * s.
//
// The choice is defined on the exact keys.  It is made on fp32 keys, whose distance from the exact ones is
// bounded (kSigmoidUlps and kSoftmaxUlps below).  Where two compared ranks or keys lie closer than their bounds, the
// groups are ranked again on keys in 64 bits, or the keys of the selected experts and of those that are too close to
// the last of them are computed in 64 bits, one per lane, and ordered.  Without a bias the scores rise with the
// logits, so the logits themselves are the keys and their comparison is exact.
//
// One wave per token.  Each group owns 64 / (n_groups rounded up to a power of two) consecutive lanes, a lane
// VPL consecutive experts of its group, so the lanes hold the experts in ascending order (which makes "the
// lowest lane, then the lowest register" the lowest index) and a group is reduced by butterflies inside its
// lanes.  Vector instructions bound it, not bytes.
#include <cfloat>

#include "launch.hpp"
#include "values.hpp"

namespace moe {

namespace {

constexpr int kSelWaves = 4;  // tokens per workgroup

// Bounds of a score's distance from its exact value, in 2^-24.  Sigmoid (s <= 1): exp 2 s (1 - s) <= 1/2, the
// addition 1, the reciprocal 2, and some to spare.  Softmax, relative to the largest score p_0 (the scores are
// p_0 e^-d): the rounded argument d at most d e^-d <= 0.37, exp 2, reciprocal and product 3, the denominator's VPL + 6 additions
// one each and its terms' 2, and some to spare.
constexpr float kSigmoidUlps = 4.0f, kSoftmaxUlps = 16.0f;  // softmax: plus VPL, times p_0
constexpr float kEps = 5.9604645e-8f;  // 2^-24

struct SelArgs {
  const void* logits;    // [T] rows, or the logits kernel's partial sums [splits][T][E]
  int64_t row_stride;    // in values
  int dt;
  int splits;            // 0: plain logits
  int vec;               // rows of logits and scores allow vector accesses of a lane's VPL values
  const float* bias;
  int T, E, top_k, n_shared, n_groups, per, lanes, lane_bits, topk_groups;
  int sigmoid, group_max, renorm;
  float scale, shared_weight;
  int32_t* ids;
  float* weights;
  float* scores;
};

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Maximum over the wave, uniform.  A source lane out of its row gives 0, the maximum's identity, which lets each
// step be one instruction (the moves of wave_max_u32_dpp keep the lane's own value there: three).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_step(uint32_t u) {
  return max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max_key(uint32_t u) {
  u = max_step<kDppRowShr1, 0xF>(u);
  u = max_step<kDppRowShr2, 0xF>(u);
  u = max_step<kDppRowShr4, 0xF>(u);
  u = max_step<kDppRowShr8, 0xF>(u);
  u = max_step<kDppRowBcast15, 0xA>(u);
  u = max_step<kDppRowBcast31, 0xC>(u);
  return __builtin_amdgcn_readlane(u, 63);
}
__device__ __forceinline__ float wave_max_f32(float v) { return f32_from_order_key(wave_max_key(f32_order_key(v))); }

// Largest and second largest of two such pairs.
template <typename V>
__device__ __forceinline__ void merge2(V& m1, V& m2, V o1, V o2) {
  const V lo = m1 < o1 ? m1 : o1;
  const V hi2 = m2 < o2 ? o2 : m2;
  m1 = m1 < o1 ? o1 : m1;
  m2 = hi2 < lo ? lo : hi2;
}

// One logit, as load_logits gives it.
__device__ __forceinline__ float load_logit(const SelArgs& a, int t, int e) {
  if (a.splits == 0) return ld_value(a.logits, a.dt, (int64_t)t * a.row_stride + e) + 0.0f;
  const float* p = reinterpret_cast<const float*>(a.logits) + (int64_t)t * a.E + e;
  float L = 0.0f;
  for (int q = 0; q < a.splits; ++q) L += p[(int64_t)q * a.T * a.E];
  return L + 0.0f;
}

// A value of another lane of the same group: lane ^ 1, ^ 2, then the mirror image in 8 and 16 lanes (whose halves
// agree by then), then lane ^ 16, ^ 32.
template <int STEP>
__device__ __forceinline__ float group_lane(float v) {
  // quad_perm 1,0,3,2 and 2,3,0,1, row_half_mirror, row_mirror
  if constexpr (STEP == 1) return __uint_as_float(dpp_u32<0xB1, 0xF>(0u, __float_as_uint(v)));
  else if constexpr (STEP == 2) return __uint_as_float(dpp_u32<0x4E, 0xF>(0u, __float_as_uint(v)));
  else if constexpr (STEP == 4) return __uint_as_float(dpp_u32<0x141, 0xF>(0u, __float_as_uint(v)));
  else if constexpr (STEP == 8) return __uint_as_float(dpp_u32<0x140, 0xF>(0u, __float_as_uint(v)));
  else return __shfl_xor(v, STEP, kWave);
}
template <int STEP>
__device__ __forceinline__ double group_lane(double v) {
  const uint64_t u = bitcast<uint64_t>(v);
  const uint32_t lo = __float_as_uint(group_lane<STEP>(__uint_as_float((uint32_t)u)));
  const uint32_t hi = __float_as_uint(group_lane<STEP>(__uint_as_float((uint32_t)(u >> 32))));
  return bitcast<double>((uint64_t)hi << 32 | lo);
}
// Largest two of a group's lanes, in all of them.
template <int STEP, typename V>
__device__ __forceinline__ void merge_step(V& m1, V& m2) {
  const V o1 = group_lane<STEP>(m1), o2 = group_lane<STEP>(m2);
  merge2(m1, m2, o1, o2);
}
template <typename V>
__device__ __forceinline__ void merge_group(V& m1, V& m2, int lanes) {  // lanes: uniform
  if (lanes > 1) merge_step<1>(m1, m2);
  if (lanes > 2) merge_step<2>(m1, m2);
  if (lanes > 4) merge_step<4>(m1, m2);
  if (lanes > 8) merge_step<8>(m1, m2);
  if (lanes > 16) merge_step<16>(m1, m2);
}
__device__ __forceinline__ double read_lane(double v, int lane) {  // lane: uniform
  const uint64_t u = bitcast<uint64_t>(v);
  return bitcast<double>((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)u, lane));
}
__device__ __forceinline__ uint64_t f64_order_key(double f) {
  const uint64_t b = bitcast<uint64_t>(f);
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  v += group_lane<1>(v);
  v += group_lane<2>(v);
  v += group_lane<4>(v);
  v += group_lane<8>(v);
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}
// A softmax numerator, or a sigmoid score.
__device__ __forceinline__ double exact_term(bool sigmoid, float L, float mx) {
  const double x = exp(sigmoid ? -(double)L : (double)L - (double)mx);
  return sigmoid ? 1.0 / (1.0 + x) : x;
}

// The choice on keys in 64 bits of all the available experts left (bits of avail): selected places (lane * VPL +
// register) in order; returns how many.
template <int VPL>
__device__ __forceinline__ int select_all64(const SelArgs& a, const float (&L)[VPL], const float (&bias)[VPL], float mx,
                                            uint32_t avail, uint16_t* sel) {
  const int lane = threadIdx.x & 63;
  double x[VPL], den = 0.0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    x[v] = finite(L[v]) ? exact_term(a.sigmoid, L[v], mx) : 0.0;
    den += x[v];
  }
  den = a.sigmoid ? 1.0 : wave_sum_f64(den);
  uint64_t ok[VPL];  // order keys, 0 for an expert that is not left
#pragma unroll
  for (int v = 0; v < VPL; ++v) ok[v] = (avail >> v) & 1u ? f64_order_key(x[v] / den + (double)bias[v]) : 0u;
  int n = 0;
  for (; n < a.top_k; ++n) {
    uint64_t best = ok[VPL - 1];
#pragma unroll
    for (int v = VPL - 2; v >= 0; --v) best = ok[v] > best ? ok[v] : best;
    const uint32_t hi = wave_max_key((uint32_t)(best >> 32));
    if (hi == 0u) break;
    const bool cand = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = wave_max_key(cand ? (uint32_t)best : 0u);
    const int wl = __builtin_ffsll((long long)__ballot(cand && (uint32_t)best == lo)) - 1;
    if (lane == wl) {
      bool found = false;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {  // the lowest index of the largest
        if (!found && ok[v] == best) {
          found = true;
          sel[n] = (uint16_t)(lane * VPL + v);
          ok[v] = 0u;
        }
      }
    }
  }
  return n;
}

// The logits of a lane's experts (e0 + v, v < n_mine; -inf past them).  Every load is issued before the first value
// is used, past the end the last expert's again: a load under a condition would be waited for on its own.
template <int VPL>
__device__ __forceinline__ void load_logits(const SelArgs& a, int t, int e0, int n_mine, float (&L)[VPL]) {
  const int64_t row = (int64_t)t * a.row_stride;
  if (a.splits == 0) {
    if (a.dt == MOE_DT_FP32) {
      const float* p = reinterpret_cast<const float*>(a.logits) + row;
      if (a.vec) {
        __builtin_memcpy(L, __builtin_assume_aligned(p + (n_mine ? e0 : 0), 4 * VPL > 16 ? 16 : 4 * VPL), 4 * VPL);
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) L[v] = p[min(e0 + v, a.E - 1)];
      }
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(a.logits) + row;
      uint16_t r[VPL];
      if (a.vec) {
        __builtin_memcpy(r, __builtin_assume_aligned(p + (n_mine ? e0 : 0), 2 * VPL > 16 ? 16 : 2 * VPL), 2 * VPL);
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) r[v] = p[min(e0 + v, a.E - 1)];
      }
      if (a.dt == MOE_DT_BF16) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) L[v] = Val<MOE_DT_BF16>::get(r[v]);
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) L[v] = Val<MOE_DT_FP16>::get(r[v]);
      }
    }
  } else {  // the logits kernel's partial sums, in slice order
    const float* p = reinterpret_cast<const float*>(a.logits) + (int64_t)t * a.E;
    constexpr int kBatch = VPL <= 4 ? 8 : 2;
#pragma unroll
    for (int v = 0; v < VPL; ++v) L[v] = 0.0f;
    for (int q0 = 0; q0 < a.splits; q0 += kBatch) {
      float r[kBatch][VPL];
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          r[q][v] = p[(int64_t)min(q0 + q, a.splits - 1) * a.T * a.E + min(e0 + v, a.E - 1)];
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
#pragma unroll
        for (int v = 0; v < VPL; ++v) L[v] += q0 + q < a.splits ? r[q][v] : 0.0f;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) L[v] = v < n_mine ? L[v] + 0.0f : -INFINITY;  // -0 counts as 0
}

template <int VPL>
__global__ __launch_bounds__(64 * kSelWaves) void select_kernel(SelArgs a) {
  __shared__ __attribute__((aligned(16))) float score_lds[kSelWaves][64 * VPL];  // by place: lane * VPL + register
  __shared__ uint16_t lds[kSelWaves][MOE_MAX_SLOTS_PER_TOKEN];                   // selected places
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * kSelWaves + wave;
  if (t >= a.T) return;  // the whole wave; no barrier follows
  uint16_t* const sel = lds[wave];
  float* const score = score_lds[wave];

  const int group = lane >> a.lane_bits, i0 = (lane & (a.lanes - 1)) * VPL;  // group, first expert inside it
  const int n_mine = group < a.n_groups ? min(max(a.per - i0, 0), VPL) : 0;
  const int e0 = group * a.per + i0;
  float L[VPL], bias[VPL];
  if (a.bias) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) bias[v] = a.bias[min(e0 + v, a.E - 1)];
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) bias[v] = 0.0f;
  }
  load_logits<VPL>(a, t, e0, n_mine, L);
  // scores, and the order keys (0: not available)
  float s[VPL];
  float mx = -INFINITY;
#pragma unroll
  for (int v = 0; v < VPL; ++v) mx = fmaxf(mx, finite(L[v]) ? L[v] : -INFINITY);
  float err = kSigmoidUlps * kEps;
  if (!a.sigmoid) {
    mx = wave_max_f32(mx);
    float den = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      s[v] = finite(L[v]) ? expf(L[v] - mx) : 0.0f;
      den += s[v];
    }
    den = wave_sum_dpp(den);
    const float rden = __builtin_amdgcn_rcpf(den);  // (den > 0 where any logit is finite; not used elsewhere)
    err = (kSoftmaxUlps + VPL) * kEps * rden;
#pragma unroll
    for (int v = 0; v < VPL; ++v) s[v] = finite(L[v]) ? s[v] * rden : 0.0f;
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) s[v] = finite(L[v]) ? __builtin_amdgcn_rcpf(1.0f + expf(-L[v])) : 0.0f;
  }
  if (a.scores) {
    float* out = a.scores + (int64_t)t * a.E + e0;
    if (a.vec) {
      if (n_mine) __builtin_memcpy(__builtin_assume_aligned(out, 4 * VPL > 16 ? 16 : 4 * VPL), s, 4 * VPL);
    } else {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (v < n_mine) out[v] = s[v];
    }
  }
  __builtin_memcpy(__builtin_assume_aligned(score + lane * VPL, 4 * VPL > 16 ? 16 : 4 * VPL), s, 4 * VPL);
  float key[VPL];
  uint32_t avail = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const bool ok = finite(L[v]) && finite(bias[v]);  // (L is -inf past the lane's experts)
    key[v] = ok ? s[v] + bias[v] : -INFINITY;
    avail |= ok ? 1u << v : 0u;
  }
  bool keep = true;
  if (a.topk_groups < a.n_groups) {
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      merge2(m1, m2, (a.group_max && !a.bias && key[v] != -INFINITY) ? L[v] : key[v], -INFINITY);
    merge_group(m1, m2, a.lanes);
    const bool one = a.group_max || m2 == -INFINITY, any = m1 != -INFINITY;  // any: an expert is available
    const float rank = one ? m1 : m1 + m2;
    int before = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const float r = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(rank), g * a.lanes));
      before += (r > rank || (r == rank && g < group)) ? 1 : 0;
    }
    keep = before < a.topk_groups;
    if (!(a.group_max && !a.bias)) {  // (the largest logit as the rank is exact)
      // distance of the rank from its exact value: two scores, two roundings of a key, one of the sum; infinite
      // where two finite keys sum beyond fp32, which leads to 64 bits whatever the other ranks are
      const float rerr = 2.0f * err + 2.0f * kEps * (fabsf(m1) + (one ? 0.0f : fabsf(m2)));
      const float lo = -wave_max_f32(keep && any ? rerr - fminf(rank, FLT_MAX) : -INFINITY);
      const float hi = wave_max_f32(!keep && any ? rerr + fmaxf(rank, -FLT_MAX) : -INFINITY);
      if (hi >= lo) {  // uniform; the ranks again, in 64 bits
        double x[VPL], sum = 0.0, d1 = -INFINITY, d2 = -INFINITY;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          x[v] = finite(L[v]) ? exact_term(a.sigmoid, L[v], mx) : 0.0;
          sum += x[v];
        }
        sum = a.sigmoid ? 1.0 : wave_sum_f64(sum);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          merge2(d1, d2, (avail >> v) & 1u ? x[v] / sum + (double)bias[v] : (double)-INFINITY, (double)-INFINITY);
        merge_group(d1, d2, a.lanes);
        const double exact = a.group_max || d2 == -INFINITY ? d1 : d1 + d2;
        before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
          const double r = read_lane(exact, g * a.lanes);
          before += (r > exact || (r == exact && g < group)) ? 1 : 0;
        }
        keep = before < a.topk_groups;
      }
    }
  }
  // keys of the kept groups in the order of unsigned integers; without a bias, of the logits
  uint32_t ok[VPL], best = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    ok[v] = keep && ((avail >> v) & 1u) ? f32_order_key(a.bias ? key[v] : L[v]) : 0u;
    best = max(best, ok[v]);
  }
  // A lane's keys are sorted once (neighbours change places only if out of order, so equal keys keep theirs) where
  // that is shorter than a search in every round: 8192 tokens x 256 experts, top-8 of 4 groups 14.1 -> 13.9 us, 2048 x
  // 512, top-16 of 8 groups 12.7 -> 11.8.
  constexpr bool kSorted = VPL <= 8;
  uint32_t places = 0;  // their registers, four bits each
  if constexpr (kSorted) {
    uint32_t at[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) at[v] = v;
#pragma unroll
    for (int last = VPL - 1; last > 0; --last)
#pragma unroll
      for (int v = 0; v < last; ++v) {
        const bool swap = ok[v] < ok[v + 1];
        const uint32_t k0 = ok[v], a0 = at[v];
        ok[v] = max(k0, ok[v + 1]);
        ok[v + 1] = min(k0, ok[v + 1]);
        at[v] = swap ? at[v + 1] : a0;
        at[v + 1] = swap ? a0 : at[v + 1];
      }
#pragma unroll
    for (int v = 0; v < VPL; ++v) places |= at[v] << (4 * v);
  }
  // Rounds of the largest key and the lowest index that has it.  Past top_k they go on while the next key is too
  // close to the last one to tell; more than one key per lane, or top_k beyond a wave, take all keys in 64 bits.
  const auto near = [&](uint32_t kx, uint32_t ky) {
    const float x = f32_from_order_key(kx), y = f32_from_order_key(ky);
    return x - y <= 2.0f * err + 2.0f * kEps * fmaxf(fabsf(x), fabsf(y));
  };
  bool all64 = a.bias && a.top_k >= kWave;
  int n = 0;
  uint32_t prev = 0, keys = 0;  // lane j keeps round j's key
  while (!all64) {
    const uint32_t m = wave_max_key(best);
    if (m == 0u) break;
    if (n >= a.top_k) {
      if (!a.bias || !near(prev, m)) break;
      if (n == kWave) {
        all64 = true;
        break;
      }
    }
    prev = m;
    keys = lane == n ? m : keys;
    const int wl = __builtin_ffsll((long long)__ballot(best == m)) - 1;
    if (lane == wl) {
      if constexpr (kSorted) {
        sel[n] = (uint16_t)(lane * VPL + (places & 15u));
        places >>= 4;
#pragma unroll
        for (int v = 0; v + 1 < VPL; ++v) ok[v] = ok[v + 1];
        ok[VPL - 1] = 0u;
        best = ok[0];
      } else {
        int at = VPL - 1;
#pragma unroll
        for (int v = VPL - 2; v >= 0; --v) at = ok[v] == m ? v : at;  // the lowest of the lane's that holds it
        sel[n] = (uint16_t)(lane * VPL + at);
        best = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          ok[v] = v == at ? 0u : ok[v];
          best = max(best, ok[v]);
        }
      }
    }
    ++n;
  }
  const auto fence = [] {  // the winners' LDS writes, read by other lanes
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  };
  if (all64) n = select_all64<VPL>(a, L, bias, mx, keep ? avail : 0u, sel);
  fence();
  const auto expert = [&](int place) {  // a.lanes = 1 << a.lane_bits
    const int l = place / VPL;
    return (l >> a.lane_bits) * a.per + (l & (a.lanes - 1)) * VPL + place % VPL;
  };
  const uint32_t next = (uint32_t)__shfl_down((int)keys, 1, kWave);
  if (a.bias && !all64 && __ballot(lane + 1 < n && near(keys, next))) {
    double den = 1.0;
    if (!a.sigmoid) {
      den = 0.0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) den += finite(L[v]) ? exact_term(false, L[v], mx) : 0.0;
      den = wave_sum_f64(den);
    }
    const int place = sel[lane < n ? lane : 0], id = expert(place);
    const double key = exact_term(a.sigmoid, load_logit(a, t, id), mx) / den + (double)a.bias[id];
    int before = 0;
    for (int i = 0; i < n; ++i) {
      const double r = read_lane(key, i);
      before += (r > key || (r == key && __builtin_amdgcn_readlane(id, i) < id)) ? 1 : 0;
    }
    fence();
    if (lane < n && before < a.top_k) sel[before] = (uint16_t)place;
    fence();
  }
  n = min(n, a.top_k);

  // slot lane of each token in registers, those past a wave in turn
  const int place0 = sel[lane < n ? lane : 0] & (64 * VPL - 1);  // (an empty choice has no slot 0)
  const float s0 = score[place0];
  float sum = lane < n ? s0 : 0.0f;
  for (int j = lane + kWave; j < n; j += kWave) sum += score[sel[j]];
  const float total = a.renorm ? wave_sum_dpp(sum) : 1.0f;
  const int k_total = a.top_k + a.n_shared;
  const auto put = [&](int j, int place, float sc) {
    int id = -1;
    float w = 0.0f;
    if (j >= a.top_k) {
      id = a.E + (j - a.top_k);
      w = a.shared_weight;
    } else if (j < n) {
      id = expert(place);
      w = total > 0.0f ? a.scale * (sc / total) : 0.0f;
    }
    a.ids[(int64_t)t * k_total + j] = id;
    a.weights[(int64_t)t * k_total + j] = w;
  };
  if (lane < k_total) put(lane, place0, s0);
  for (int j = lane + kWave; j < k_total; j += kWave) {
    const int place = j < n ? sel[j] : 0;
    put(j, place, score[place]);
  }
}

hipError_t run_select(SelArgs a, hipStream_t stream) {
  a.lane_bits = 6;
  while ((a.n_groups << a.lane_bits) > 64) --a.lane_bits;
  const int lanes = a.lanes = 1 << a.lane_bits;
  a.per = a.E / a.n_groups;
  const int vpl = (a.per + lanes - 1) / lanes;
  int v = 1;
  while (v < vpl) v *= 2;  // the kernel's VPL
  const int bytes = v * (a.splits || a.dt == MOE_DT_FP32 ? 4 : 2), al = bytes > 16 ? 16 : bytes;
  a.vec = a.per % v == 0 && (uintptr_t)a.logits % al == 0 && a.row_stride % v == 0 &&
          (!a.scores || ((uintptr_t)a.scores % (v > 4 ? 16 : 4 * v) == 0 && a.E % v == 0));
  const dim3 g((unsigned)((a.T + kSelWaves - 1) / kSelWaves));
  if (vpl <= 1) select_kernel<1><<<g, 64 * kSelWaves, 0, stream>>>(a);
  else if (vpl <= 2) select_kernel<2><<<g, 64 * kSelWaves, 0, stream>>>(a);
  else if (vpl <= 4) select_kernel<4><<<g, 64 * kSelWaves, 0, stream>>>(a);
  else if (vpl <= 8) select_kernel<8><<<g, 64 * kSelWaves, 0, stream>>>(a);
  else if (vpl <= 16) select_kernel<16><<<g, 64 * kSelWaves, 0, stream>>>(a);
  else select_kernel<32><<<g, 64 * kSelWaves, 0, stream>>>(a);
  return hipGetLastError();
}

SelArgs from_rule(const moe_route_rule& r, int T, int E, int32_t* ids, float* weights, float* scores) {
  SelArgs a{};
  a.bias = r.selection_bias;
  a.T = T;
  a.E = E;
  a.top_k = r.top_k;
  a.n_shared = r.n_shared;
  a.n_groups = r.n_groups;
  a.topk_groups = r.topk_groups;
  a.sigmoid = r.score == MOE_SCORE_SIGMOID;
  a.group_max = r.group_score == MOE_GROUP_MAX;
  a.renorm = r.renormalise != 0;
  a.scale = r.routed_scale;
  a.shared_weight = r.shared_weight;
  a.ids = ids;
  a.weights = weights;
  a.scores = scores;
  return a;
}

}  // namespace

hipError_t launch_select(const void* logits, int dt, int64_t row_stride, int T, int E, const moe_route_rule& rule,
                         int32_t* ids, float* weights, float* scores, hipStream_t stream) {
  SelArgs a = from_rule(rule, T, E, ids, weights, scores);
  a.logits = logits;
  a.dt = dt;
  a.row_stride = row_stride;
  return run_select(a, stream);
}

hipError_t launch_route_grouped(const void* x, int x_fp16, int T, int H, const float* w_router, int E,
                                const moe_route_rule& rule, int32_t* ids, float* weights, float* scores,
                                float* partial, hipStream_t stream) {
  const int splits = route_splits(T, H, E);
  const hipError_t err = launch_route_logits(x, x_fp16, T, H, w_router, E, partial, splits, stream);
  if (err != hipSuccess) return err;
  SelArgs a = from_rule(rule, T, E, ids, weights, scores);
  a.logits = partial;
  a.splits = splits;
  return run_select(a, stream);
}

}  // namespace moe
