// Attention over packed prompts: softmax(scale q k^T, masked) v per head, sequences one after another, any number of
// query heads per key-value head.
//
// A workgroup takes rows of one sequence and key-value head, the group's query heads of a token next to each other, so
// that all of them share the keys' tiles in LDS, and walks over those tiles once with the running maximum and sum of
// each row.  A wave holds 32 rows: S^T = K Q^T puts a row into two lanes (column lane & 31, half the keys each), so
// maxima, sums and rescaling stay inside a lane but for one exchange, and the registers of S^T, rounded to 16 bits, are
// the operand of O^T = V^T P^T as they stand: its sum runs over keys in whatever order both operands share.
//
// Operations bound it: 4 D per row and key on the matrix cores, and about as much time on the vector ALU for the
// exponentials, which other waves hide.  P is rounded to 16 bits (half a step, as the output is; its errors are random
// and average out over the keys); maxima, sums and O are fp32.
#include <algorithm>

#include "attention.hpp"

namespace moe {

namespace {

constexpr int kTileKeys = 64, kPartKeys = 512;

// Swizzles (in 16-byte chunks) of a tile's rows of DP values.  K: sixteen consecutive rows' chunks of one column fall
// into different banks.  V: so do the 32-byte pieces of four consecutive rows that a transposing read takes.
template <int DP>
__device__ __forceinline__ int swizzle_k(int row) {
  return DP % 128 == 0 ? row & 15 : (row >> 1) & 7;
}
template <int DP>
__device__ __forceinline__ int swizzle_v(int row) {
  return DP % 128 == 0 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

__device__ __forceinline__ float other_half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

struct Piece {  // a workgroup's rows
  int q0, nq, k0, nk, tile;  // tile < 0: none
};

// Workgroup `slot` of a key-value head: sequences have ceil(nq G / rows) tiles each, the last (most keys) first.
__device__ __forceinline__ Piece find_piece(const PromptArgs& a, int slot, int rows) {
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < a.n_seqs; b0 += 64) {
    const int b = b0 + lane;
    int q0 = 0, q1 = 0;
    if (b < a.n_seqs) {
      q0 = min(max(a.cu_q[b], 0), a.Tq);
      q1 = min(max(a.cu_q[b + 1], q0), a.Tq);
    }
    const int tiles = (int)(((int64_t)(q1 - q0) * a.G.d + rows - 1) / rows);
    const int incl = (int)wave_incl_scan_dpp((uint32_t)tiles);
    const uint64_t past = __ballot(slot < incl);
    if (past) {
      const int s = __builtin_ctzll(past);
      Piece p;
      p.q0 = __builtin_amdgcn_readlane(q0, s);
      p.nq = __builtin_amdgcn_readlane(q1, s) - p.q0;
      p.tile = __builtin_amdgcn_readlane(incl, s) - 1 - slot;
      p.k0 = min(max(a.cu_k[b0 + s], 0), a.Tk);
      p.nk = min(max(a.cu_k[b0 + s + 1], p.k0), a.Tk) - p.k0;
      p.k0 = __builtin_amdgcn_readfirstlane(p.k0);
      p.nk = __builtin_amdgcn_readfirstlane(p.nk);
      return p;
    }
    slot -= __builtin_amdgcn_readlane(incl, 63);
  }
  return Piece{0, 0, 0, 0, -1};
}

// Whether a dword of two 16-bit values holds an infinity or NaN.
template <bool F16>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}

template <bool F16, int DP, bool EXACT, int NW, int PER_SIMD>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void prompt_kernel(PromptArgs a) {
  constexpr int CH = DP / 8;          // 16-byte chunks of a row
  constexpr int BN = kTileKeys, KT = BN / 32, DT = DP / 32, ST = DP / 16;
  constexpr int ROWS = 32 * NW;
  __shared__ __attribute__((aligned(1024))) u32x4 lds[2][2][BN * CH];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int kvh = blockIdx.x % a.Hkv;
  const Piece pc = find_piece(a, blockIdx.x / a.Hkv, ROWS);
  if (pc.tile < 0) return;
  const int G = (int)a.G.d;
  const int n_rows = pc.nq * G;

  // This lane's row: its token, head and keys [lo, hi)
  const int first = pc.tile * ROWS;
  const int my = first + 32 * wave + col;
  const int rr = min(my, n_rows - 1);
  const int tok = (int)div_by(a.G, (uint32_t)rr), g = rr - tok * G;
  const int shift = pc.nk - pc.nq;
  const auto range_hi = [&](int t) { return a.causal ? min(pc.nk, t + shift + 1) : pc.nk; };
  const auto range_lo = [&](int t) { return a.window ? max(0, t + shift + 1 - a.window) : 0; };
  int hi = range_hi(tok), lo = range_lo(tok);
  // of the wave's and the workgroup's rows (tokens rise with rows)
  const int w_t0 = (int)div_by(a.G, (uint32_t)min(first + 32 * wave, n_rows - 1));
  const int w_t1 = (int)div_by(a.G, (uint32_t)min(first + 32 * wave + 31, n_rows - 1));
  const int b_t0 = (int)div_by(a.G, (uint32_t)first);
  const int b_t1 = (int)div_by(a.G, (uint32_t)min(first + ROWS - 1, n_rows - 1));
  int w_hi_min = range_hi(w_t0), w_hi = range_hi(w_t1), w_lo = range_lo(w_t0), w_lo_max = range_lo(w_t1);
  int b_lo = range_lo(b_t0) / BN * BN, b_hi = range_hi(b_t1);
  if (a.parts > 1) {  // this workgroup's share of them
    const int from = b_lo + (int)blockIdx.y * a.part_keys;
    b_hi = min(b_hi, from + a.part_keys);
    b_lo = from;
    w_hi = min(w_hi, b_hi);
  }
  const int n_tiles = b_hi > b_lo ? (b_hi - b_lo + BN - 1) / BN : 0;

  // Q as the right operand: column = row of the tile, eight values of d per half and step
  u32x4 qf[ST];
  const uint16_t* qp = a.q + (int64_t)(pc.q0 + tok) * a.q_ts + (int64_t)(kvh * G + g) * a.q_hs;
#pragma unroll
  for (int st = 0; st < ST; ++st) {
    const int d = 16 * st + 8 * half;
    qf[st] = u32x4{0, 0, 0, 0};
    if (EXACT || d < a.D) qf[st] = ld16(qp + d);
  }

  const uint16_t* kp = a.k + (int64_t)pc.k0 * a.k_ts + (int64_t)kvh * a.k_hs;
  const uint16_t* vp = a.v + (int64_t)pc.k0 * a.v_ts + (int64_t)kvh * a.v_hs;
  if constexpr (!EXACT) {  // columns past D are never loaded: zeros, once
    for (int i = tid; i < 4 * BN * CH; i += 64 * NW) (&lds[0][0][0])[i] = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  const auto load_tile = [&](int buf, int j0) {
#pragma unroll
    for (int u = 0; u < BN * CH / (64 * NW); ++u) {
      const int p = u * 64 * NW + tid, row = p / CH, cc = p % CH;
      const int key = min(j0 + row, pc.nk - 1);  // rows past the last key repeat it, and are masked
      const int ck = cc ^ swizzle_k<DP>(row), cv = cc ^ swizzle_v<DP>(row);
      u32x4* dk = &lds[buf][0][u * 64 * NW + 64 * wave];
      u32x4* dv = &lds[buf][1][u * 64 * NW + 64 * wave];
      if (EXACT || 8 * ck < a.D)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(kp + (int64_t)key * a.k_ts + 8 * ck),
                                         (__attribute__((address_space(3))) void*)dk, 16, 0, 0);
      if (EXACT || 8 * cv < a.D)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(vp + (int64_t)key * a.v_ts + 8 * cv),
                                         (__attribute__((address_space(3))) void*)dv, 16, 0, 0);
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  float m = -INFINITY, l = 0.0f;  // m: reference of the exponents (at most 8 below the maximum), l: this lane's keys
  const float c = a.c, slack = 8.0f / c;

  if (n_tiles > 0) load_tile(0, b_lo);
  for (int it = 0; it < n_tiles; ++it) {
    const int j0 = b_lo + it * BN, buf = it & 1;
    __syncthreads();  // tile `it` is there, and nobody reads the other buffer any more
    if (it + 1 < n_tiles) load_tile(buf ^ 1, j0 + BN);
    if (j0 >= w_hi || j0 + BN <= w_lo) continue;  // nothing of the tile is the wave's

    f32x16 s[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const u32x4 kf = lds[buf][0][(32 * kt + col) * CH + ((2 * st + half) ^ swizzle_k<DP>(col))];
        s[kt] = mfma_32x32x16<F16>(kf, qf[st], s[kt]);
      }
    const bool masked = j0 + BN > w_hi_min || j0 < w_lo_max;
    if (masked) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = j0 + 32 * kt + 8 * (r >> 2) + 4 * half + (r & 3);
          s[kt][r] = j >= lo && j < hi ? s[kt][r] : -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kt][r]);
    top = other_half_max(top);
    // The reference rises only when some row's maximum passes it by more than 2^8: every exponential stays below that
    if (__any(top > m + slack || (m == -INFINITY && top > m))) {
      const float next = fmaxf(m, top);
      const float f = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - next) * c);
      m = next;
      l *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m * c;
    u32x4 pf[2 * KT];
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r], c, -base));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r + 1], c, -base));
        part[(r >> 1) & 3] += e0 + e1;
        pf[2 * kt + (r >> 3)][(r >> 1) & 3] = pack16<F16>(e0, e1);
      }
    l += (part[0] + part[1]) + (part[2] + part[3]);

    const char* vt = reinterpret_cast<const char*>(&lds[buf][1][0]);
    const int vi = lane & 15, vsub = 16 * ((lane >> 4) & 1);
    const auto v_frag = [&](int ks, int dt) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * ks + 8 * e + 4 * half + (vi >> 2), d = 32 * dt + vsub + 4 * (vi & 3);
        const u32x2 t = lds_read_tr(vt + row * (2 * DP) + (((d >> 3) ^ swizzle_v<DP>(row)) << 4) + ((d & 7) << 1));
        w[2 * e] = t[0];
        w[2 * e + 1] = t[1];
      }
      return w;
    };
    bool wild = false;
    if (masked) {  // 0 * infinity is no zero: a masked key's value must not reach a row
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const u32x4 w = v_frag(ks, dt);
          wild |= not_finite<F16>(w[0]) || not_finite<F16>(w[1]) || not_finite<F16>(w[2]) || not_finite<F16>(w[3]);
        }
      wild = __any(wild);
    }
    if (!wild) {
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = mfma_32x32x16<F16>(v_frag(ks, dt), pf[ks], o[dt]);
    } else {  // one key at a time, into the rows that see it
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks)
        for (int kk = 0; kk < 16; ++kk) {
          const int j = j0 + 16 * ks + kk;
          const bool seen = j >= lo && j < hi;
          u32x4 pm, vm;
          const int e = kk - 4 * half;  // element of this half's operand: 0-3, or 8-11 for its second four
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int at = 8 * (w >> 1) + 2 * (w & 1);
            pm[w] = (e == at ? 0xFFFFu : 0u) | (e == at + 1 ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) {
            vm = v_frag(ks, dt) & pm;
            const f32x16 n = mfma_32x32x16<F16>(vm, pf[ks] & pm, o[dt]);
#pragma unroll
            for (int r = 0; r < 16; ++r) o[dt][r] = seen ? n[r] : o[dt][r];
          }
        }
    }
  }

  l = other_half_sum(l);
  const bool mine = my < n_rows;
  const int64_t orow = (int64_t)(pc.q0 + tok) * a.Hq + kvh * G + g;
  if (a.parts > 1) {
    if (!mine) return;
    const AttnParts w = attn_parts_dev(a.ws, (int64_t)a.Tq * a.Hq, a.parts);
    const int64_t at = orow * a.parts + blockIdx.y;
    if (half == 0) {
      w.ml[2 * at] = m * c;
      w.ml[2 * at + 1] = l;
    }
    if (n_tiles == 0) return;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const int d = 32 * dt + 8 * q4 + 4 * half;
        const f32x4 v = {o[dt][4 * q4], o[dt][4 * q4 + 1], o[dt][4 * q4 + 2], o[dt][4 * q4 + 3]};
        if (EXACT || d < a.D) *reinterpret_cast<f32x4*>(w.o + at * a.D + d) = v;
      }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* yp = a.y + (int64_t)(pc.q0 + tok) * a.y_ts + (int64_t)(kvh * G + g) * a.y_hs;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int q4 = 0; q4 < 4; q4 += 2) {
      // values 8 q4 .. of both halves change places, so that each lane stores eight consecutive ones
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x0 = pack16<F16>(o[dt][4 * q4 + 2 * e] * inv, o[dt][4 * q4 + 2 * e + 1] * inv);
        const uint32_t x1 = pack16<F16>(o[dt][4 * q4 + 4 + 2 * e] * inv, o[dt][4 * q4 + 5 + 2 * e] * inv);
        const auto r = __builtin_amdgcn_permlane32_swap(x0, x1, false, false);
        w[e] = r[0];
        w[2 + e] = r[1];
      }
      const int d = 32 * dt + 8 * (q4 + half);
      if (mine && (EXACT || d < a.D)) st16(yp + d, w);
    }
  if (mine && half == 0 && a.lse) a.lse[orow] = l == 0.0f ? -INFINITY : (m * c + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool F16, int DP, int NW, int PER_SIMD>
void launch_exact(const PromptArgs& a, dim3 g, hipStream_t stream) {
  if (a.D == DP) prompt_kernel<F16, DP, true, NW, PER_SIMD><<<g, 64 * NW, 0, stream>>>(a);
  else prompt_kernel<F16, DP, false, NW, PER_SIMD><<<g, 64 * NW, 0, stream>>>(a);
}

struct PromptPlan {
  int waves;  // of a workgroup, 32 rows each
  int64_t slots;
  int parts, part_keys;
};
PromptPlan plan_prompt(int Tq, int Tk, int n_seqs, int Hq, int Hkv, int D) {
  PromptPlan p;
  p.waves = 4;
  const int rows = 32 * p.waves;
  p.slots = ((int64_t)Tq * (Hq / Hkv) + rows - 1) / rows + n_seqs;
  // Keys are shared where tiles are few: at least 512 keys a part, parts for 512 workgroups
  const int64_t blocks = p.slots * Hkv, most = (Tk + kPartKeys - 1) / kPartKeys;
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((512 + blocks - 1) / blocks, most));
  p.part_keys = std::max<int64_t>(1, ((Tk + parts - 1) / parts + kTileKeys - 1) / kTileKeys) * kTileKeys;
  p.parts = (int)std::max<int64_t>(1, ((int64_t)Tk + p.part_keys - 1) / p.part_keys);
  return p;
}

}  // namespace

size_t prompt_workspace_bytes(int Tq, int Tk, int n_seqs, int Hq, int Hkv, int D) {
  return attn_parts_bytes((int64_t)Tq * Hq, plan_prompt(Tq, Tk, n_seqs, Hq, Hkv, D).parts, D);
}

hipError_t launch_prompt(PromptArgs a, hipStream_t stream) {
  const PromptPlan p = plan_prompt(a.Tq, a.Tk, a.n_seqs, a.Hq, a.Hkv, a.D);
  a.parts = p.parts;
  a.part_keys = p.part_keys;
  const dim3 g((unsigned)(p.slots * a.Hkv), (unsigned)p.parts);
#define MOE_PROMPT(DP, NW, OCC) \
  (a.f16 ? launch_exact<true, DP, NW, OCC>(a, g, stream) : launch_exact<false, DP, NW, OCC>(a, g, stream))
  if (a.D <= 64) MOE_PROMPT(64, 4, 2);
  else if (a.D <= 128) MOE_PROMPT(128, 4, 2);
  else if (a.D <= 192) MOE_PROMPT(192, 4, 1);
  else MOE_PROMPT(256, 4, 1);
#undef MOE_PROMPT
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.parts == 1) return err;
  AttnJoin j{};
  j.parts = attn_parts(a.ws, (int64_t)a.Tq * a.Hq, p.parts);
  j.rows = (int64_t)a.Tq * a.Hq;
  j.Hq = a.Hq;
  j.D = a.D;
  j.f16 = a.f16;
  j.y = a.y;
  j.y_ts = a.y_ts;
  j.y_hs = a.y_hs;
  j.lse = a.lse;
  j.cu_q = a.cu_q;
  j.n_seqs = a.n_seqs;
  return launch_attn_join(j, stream);
}

}  // namespace moe
