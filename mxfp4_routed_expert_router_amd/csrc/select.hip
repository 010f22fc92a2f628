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
// bounded (kSigmoidUlps and kSoftmaxUlps below), and a token in which two compared keys or ranks lie closer than their bounds is decided
// again on keys in 64 bits.  Without a bias the scores rise with the logits, so the logits themselves are the
// keys and their comparison is exact.
//
// One wave per token.  Each group owns 64 / (n_groups rounded up to a power of two) consecutive lanes, a lane
// VPL consecutive experts of its group, so the lanes hold the experts in ascending order (which makes "the
// lowest lane, then the lowest register" the lowest index) and a group is reduced by butterflies inside its
// lanes.  Vector instructions bound it, not bytes.
#include "launch.hpp"
#include "values.hpp"

namespace moe {

namespace {

constexpr int kSelWaves = 4;  // tokens per workgroup

// Bounds of a score's distance from its exact value, in 2^-24.  Sigmoid (s <= 1): exp 2, the addition 1, the
// division 1, and some to spare.  Softmax, relative to the largest score p_0 (the scores are p_0 e^-d): the
// rounded argument d at most d e^-d <= 0.37, exp 2, division 1, the denominator's VPL + 6 additions one each
// and its terms' 2, and some to spare.
constexpr float kSigmoidUlps = 8.0f, kSoftmaxUlps = 16.0f;  // softmax: plus VPL, times p_0
constexpr float kEps = 5.9604645e-8f;  // 2^-24

struct SelArgs {
  const void* logits;    // [T] rows, or the logits kernel's partial sums [splits][T][E]
  int64_t row_stride;    // in values
  int dt;
  int splits;            // 0: plain logits
  const float* bias;
  int T, E, top_k, n_shared, n_groups, per, lanes, topk_groups;
  int sigmoid, group_max, renorm;
  float scale, shared_weight;
  int32_t* ids;
  float* weights;
  float* scores;
};

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Largest and second largest of two such pairs.
template <typename V>
__device__ __forceinline__ void merge2(V& m1, V& m2, V o1, V o2) {
  const V lo = m1 < o1 ? m1 : o1;
  const V hi2 = m2 < o2 ? o2 : m2;
  m1 = m1 < o1 ? o1 : m1;
  m2 = hi2 < lo ? lo : hi2;
}

// The token's choice on keys in 64 bits.  Lane-private inputs: L (the fp32 logits), ok (available).  Writes the
// selected ids and scores of slot j to sel_id / sel_s and returns how many were selected.
template <int VPL>
__device__ __noinline__ int select_exact(const SelArgs& a, const float (&L)[VPL], uint32_t avail, int e0, int group,
                                         int* sel_id, float* sel_s) {
  const int lane = threadIdx.x & 63;
  double s[VPL], key[VPL];
  double mx = -INFINITY;
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (finite(L[v])) mx = fmax(mx, (double)L[v]);
  for (int o = 32; o >= 1; o >>= 1) mx = fmax(mx, __shfl_xor(mx, o, kWave));
  double den = 0.0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    if (a.sigmoid) {
      s[v] = 1.0 / (1.0 + exp(-(double)L[v]));
    } else {
      s[v] = finite(L[v]) ? exp((double)L[v] - mx) : 0.0;
      den += s[v];
    }
  }
  for (int o = 32; o >= 1; o >>= 1) den += __shfl_xor(den, o, kWave);
  double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    if (!a.sigmoid) s[v] /= den;
    const bool ok = (avail >> v) & 1u;
    key[v] = ok ? s[v] + (a.bias ? (double)a.bias[e0 + v] : 0.0) : -INFINITY;
    merge2(m1, m2, key[v], (double)-INFINITY);
  }
  bool keep = true;
  if (a.topk_groups < a.n_groups) {
    for (int o = a.lanes >> 1; o >= 1; o >>= 1) {
      const double o1 = __shfl_xor(m1, o, kWave), o2 = __shfl_xor(m2, o, kWave);
      merge2(m1, m2, o1, o2);
    }
    const double rank = a.group_max || m2 == -INFINITY ? m1 : m1 + m2;
    int before = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const double r = __shfl(rank, g * a.lanes, kWave);
      before += (r > rank || (r == rank && g < group)) ? 1 : 0;
    }
    keep = before < a.topk_groups;
  }
  // without a bias the logits order the experts exactly (scores near 1 may be equal even in 64 bits)
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    if (!keep) key[v] = -INFINITY;
    else if (!a.bias && key[v] != -INFINITY) key[v] = (double)L[v];
  }
  int n = 0;
  for (; n < a.top_k; ++n) {
    double best = key[0];
    int at = 0;
    float bs = (float)s[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
        bs = (float)s[v];
      }
    double m = best;
    for (int o = 32; o >= 1; o >>= 1) m = fmax(m, __shfl_xor(m, o, kWave));
    if (m == -INFINITY) break;
    const int wl = __builtin_ffsll((long long)__ballot(best == m)) - 1;
    if (lane == wl) {
      sel_id[n] = e0 + at;
      sel_s[n] = bs;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (v == at) key[v] = -INFINITY;
    }
  }
  return n;
}

template <int VPL>
__global__ __launch_bounds__(64 * kSelWaves) void select_kernel(SelArgs a) {
  __shared__ int lds_id[kSelWaves][MOE_MAX_SLOTS_PER_TOKEN];
  __shared__ float lds_s[kSelWaves][MOE_MAX_SLOTS_PER_TOKEN];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * kSelWaves + wave;
  if (t >= a.T) return;  // the whole wave; no barrier follows
  int* sel_id = lds_id[wave];
  float* sel_s = lds_s[wave];

  const int group = lane / a.lanes, i0 = (lane % a.lanes) * VPL;  // group, first expert inside it
  const int n_mine = group < a.n_groups ? min(max(a.per - i0, 0), VPL) : 0;
  const int e0 = group * a.per + i0;
  float L[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) L[v] = -INFINITY;
  if (a.splits == 0) {
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (v < n_mine) L[v] = ld_value(a.logits, a.dt, (int64_t)t * a.row_stride + e0 + v) + 0.0f;  // -0 is 0
  } else {
    const float* p = reinterpret_cast<const float*>(a.logits) + (int64_t)t * a.E + e0;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (v < n_mine) {
        float sum = 0.0f;  // slices in slice order
        for (int q = 0; q < a.splits; ++q) sum += p[(int64_t)q * a.T * a.E + v];
        L[v] = sum;  // (never -0: the sum starts at 0)
      }
  }
  // scores, and the order keys (0: not available)
  float s[VPL];
  float mx = -INFINITY;
#pragma unroll
  for (int v = 0; v < VPL; ++v) mx = fmaxf(mx, finite(L[v]) ? L[v] : -INFINITY);
  float err = kSigmoidUlps * kEps;
  if (!a.sigmoid) {
    mx = wave_max_dpp(mx);
    float den = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      s[v] = finite(L[v]) ? expf(L[v] - mx) : 0.0f;
      den += s[v];
    }
    den = wave_sum_dpp(den);
    err = (kSoftmaxUlps + VPL) * kEps / den;  // (not used where nothing is finite)
#pragma unroll
    for (int v = 0; v < VPL; ++v) s[v] = finite(L[v]) ? s[v] / den : 0.0f;  // (den > 0 where any is finite)
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) s[v] = finite(L[v]) ? 1.0f / (1.0f + expf(-L[v])) : 0.0f;
  }
  if (a.scores) {
    float* out = a.scores + (int64_t)t * a.E + e0;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (v < n_mine) out[v] = s[v];
  }
  float key[VPL];
  uint32_t avail = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const float b = (a.bias && v < n_mine) ? a.bias[e0 + v] : 0.0f;
    const bool ok = v < n_mine && finite(L[v]) && finite(b);
    key[v] = ok ? s[v] + b : -INFINITY;
    avail |= ok ? 1u << v : 0u;
  }
  bool close = false, keep = true;
  if (a.topk_groups < a.n_groups) {
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v) merge2(m1, m2, (a.group_max && !a.bias && key[v] != -INFINITY) ? L[v] : key[v], -INFINITY);
    for (int o = a.lanes >> 1; o >= 1; o >>= 1) {
      const float o1 = __shfl_xor(m1, o, kWave), o2 = __shfl_xor(m2, o, kWave);
      merge2(m1, m2, o1, o2);
    }
    const bool one = a.group_max || m2 == -INFINITY;
    const float rank = one ? m1 : m1 + m2;
    int before = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const float r = __shfl(rank, g * a.lanes, kWave);
      before += (r > rank || (r == rank && g < group)) ? 1 : 0;
    }
    keep = before < a.topk_groups;
    if (!(a.group_max && !a.bias)) {  // (the largest logit as the rank is exact)
      // distance of the rank from its exact value: two scores, two roundings of a key, one of the sum
      const float rerr = 2.0f * err + 2.0f * kEps * (fabsf(m1) + (one ? 0.0f : fabsf(m2)));
      const float lo = -wave_max_dpp(keep && rank != -INFINITY ? rerr - rank : -INFINITY);
      const float hi = wave_max_dpp(!keep && rank != -INFINITY ? rerr + rank : -INFINITY);
      close = hi >= lo;
    }
  }
  // keys of the kept groups in the order of unsigned integers; without a bias, of the logits
  uint32_t ok[VPL], best = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    ok[v] = keep && ((avail >> v) & 1u) ? f32_order_key(a.bias ? key[v] : L[v]) : 0u;
    best = max(best, ok[v]);
  }
  int n = 0;
  uint32_t prev = 0;
  // one round more than top_k: the last pair compared is the last selected expert and the first left out
  for (int j = 0; j <= a.top_k; ++j) {
    const uint32_t m = wave_max_u32_dpp(best);
    if (a.bias && j > 0 && m) {
      const float x = f32_from_order_key(prev), y = f32_from_order_key(m);
      close |= x - y <= 2.0f * err + 2.0f * kEps * fmaxf(fabsf(x), fabsf(y));
    }
    if (m == 0u || j == a.top_k) break;
    prev = m;
    const int wl = __builtin_ffsll((long long)__ballot(best == m)) - 1;
    if (lane == wl) {
      bool found = false;
      best = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        if (!found && ok[v] == m) {
          found = true;
          ok[v] = 0u;
          sel_id[j] = e0 + v;
          sel_s[j] = s[v];
        }
        best = max(best, ok[v]);
      }
    }
    ++n;
  }
  if (__ballot(close)) n = select_exact<VPL>(a, L, avail, e0, group, sel_id, sel_s);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");  // the winners' LDS writes, read by other lanes below
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");

  float sum = 0.0f;
  for (int j = lane; j < n; j += kWave) sum += sel_s[j];
  const float total = a.renorm ? wave_sum_dpp(sum) : 1.0f;
  const int k_total = a.top_k + a.n_shared;
  for (int j = lane; j < k_total; j += kWave) {
    int id = -1;
    float w = 0.0f;
    if (j >= a.top_k) {
      id = a.E + (j - a.top_k);
      w = a.shared_weight;
    } else if (j < n) {
      id = sel_id[j];
      w = total > 0.0f ? a.scale * (sel_s[j] / total) : 0.0f;
    }
    a.ids[(int64_t)t * k_total + j] = id;
    a.weights[(int64_t)t * k_total + j] = w;
  }
}

hipError_t run_select(SelArgs a, hipStream_t stream) {
  int lanes = 64;
  while (lanes * a.n_groups > 64) lanes >>= 1;
  a.lanes = lanes;
  a.per = a.E / a.n_groups;
  const int vpl = (a.per + lanes - 1) / lanes;
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
