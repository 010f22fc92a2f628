// Attention of one new token per sequence over a paged cache, split over the cache's length and joined.
//
// A workgroup takes a sequence's key-value head, up to sixteen of its query heads and a range of its keys; its waves
// take 32 keys at a time, each with a running maximum and sum of its own, and join at the end through LDS.  S^T = K Q^T
// puts a head into a column (lane & 15), so maxima, sums and rescaling stay in a lane but for two exchanges, and P^T is
// the right operand of O^T = V^T P^T as it stands, rounded to a high and a low 16-bit part: the cache's bytes bound the
// kernel, so the second product costs nothing and only the output is rounded (in fp16 as far as its exponents reach).
//
// Consecutive lanes read consecutive 16 bytes of a token's row, whole 128-byte lines a load and past the caches: in MFMA
// layout at once (64 bytes of sixteen rows a load) 176 sequences of up to 4096 tokens take 266 us, so 215 (5.6 TB/s; reading
// alone reaches 7.17; on pages of 16 tokens, with an address to a key, the same within 3%, in MXFP8 5% more).  The tile then
// turns through a part of LDS that is the wave's own.  The next tile's K and V are on their way meanwhile (MXFP8 from heads of
// 128 on: one of them).
//
// 16-bit caches are operands as they are, E4M3 codes times a power of two are exact in bf16.
#include <algorithm>

#include "attention.hpp"

namespace moe {

namespace {

constexpr int kDecodeWaves = 4, kWaveKeys = 32;

// A wave's tile of K or V on the way: load n has chunk (64 n + lane) of its rows' 16-byte chunks, one row behind another.
template <int FMT, int DP>
struct Rows {
  static constexpr int CH = FMT == MOE_KV_MXFP8 ? DP / 16 : DP / 8;  // chunks of a row as it is stored
  static constexpr int N = kWaveKeys * CH / 64;
  u32x4 q[N];
  static __device__ __forceinline__ int row(int n, int lane) {
    return 64 % CH == 0 ? n * (64 / CH) + lane / CH : (64 * n + lane) / CH;
  }
  static __device__ __forceinline__ int chunk(int n, int lane) { return 64 % CH == 0 ? lane % CH : (64 * n + lane) % CH; }
};
__device__ __forceinline__ int64_t from_lane(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, lane, kWave), hi = (uint32_t)__shfl((int)(v >> 32), lane, kWave);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// E8M0 codes of a row's 32-value blocks.
template <int DP>
struct RowScales {
  uint32_t w[(DP / 32 + 3) / 4];
};

// WHOLE: pages are multiples of a tile's 32 keys, so that a tile lies on one page and its addresses are scalars but for a
// lane's place in it; else each key has its own.
template <int FMT, int DP, bool EXACT, bool WHOLE, int PER_SIMD>
__global__ __launch_bounds__(64 * kDecodeWaves, PER_SIMD) void decode_kernel(DecodeArgs a) {
  constexpr bool F16 = FMT == MOE_KV_FP16, MX = FMT == MOE_KV_MXFP8;
  constexpr int ST = DP / 32, CT = DP / 16, W = kDecodeWaves;
  // V of a tile is asked for when its K is in LDS, and the next K when V is, so that one of them is in registers at a time.
  // In MXFP8 that is what lets two waves of heads of 256 share a SIMD (64 rows of up to 4096: 229 -> 132 us; of 160 148 ->
  // 140, of 128 the same within 1%); 16-bit rows lose by it (heads of 128: 215 -> 217).
  constexpr bool kLate = MX && DP >= 128;
  // Rows of a power of two: a lane's LDS addresses differ by exclusive-ors with constants and by constants.
  constexpr bool kXor = (DP & (DP - 1)) == 0;
  typedef Rows<FMT, DP> R;
  __shared__ __attribute__((aligned(512))) u32x4 tiles[W][kWaveKeys * DP / 8];  // K, then V, of 16 bits; in the end O
  __shared__ float stat[W][2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int m_tiles = (a.G + 15) >> 4, per_part = a.Hkv * m_tiles;
  const int unit = blockIdx.x / per_part, in = blockIdx.x - unit * per_part;
  const int b = unit / a.parts, part = unit - b * a.parts;
  const int kvh = in / m_tiles, head0 = (in - kvh * m_tiles) * 16, heads = min(16, a.G - head0);
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int lo = a.window > 0 ? max(0, len - a.window) : 0;
  // (tiles start at multiples of 32 keys; those in front of the window are masked)
  const int64_t from64 = lo / kWaveKeys * kWaveKeys + (int64_t)part * a.part_keys;
  const int from = (int)min(from64, (int64_t)len), to = (int)min(from64 + a.part_keys, (int64_t)len);
  const AttnParts parts = attn_parts_dev(a.ws, (int64_t)a.B * a.Hq, a.parts);
  if (a.parts > 1 && from >= to) {  // nothing here
    if (wave == 0 && g == 0 && r < heads) {
      const int64_t slot = ((int64_t)b * a.Hq + kvh * a.G + head0 + r) * a.parts + part;
      parts.ml[2 * slot] = -INFINITY;
      parts.ml[2 * slot + 1] = 0.0f;
    }
    return;
  }
  const int32_t* table = a.table + (int64_t)b * a.table_stride;

  u32x4 qf[ST];
  const uint16_t* qp = a.q + (int64_t)b * a.q_ts + (int64_t)(kvh * a.G + head0 + min(r, heads - 1)) * a.q_hs;
#pragma unroll
  for (int st = 0; st < ST; ++st) {
    const int d = 32 * st + 8 * g;
    qf[st] = u32x4{0, 0, 0, 0};
    if (EXACT || d < a.D) qf[st] = ld16(qp + d);
  }

  // Where a tile's rows are.  A key past the range or on a page that is none counts as masked; its row is read from the
  // cache's first page.
  //   WHOLE: 64 tiles' pages are loaded at once, one to a lane, and a tile's is read from its lane.
  //   Else a tile's keys are one to a lane (twice), with page and byte offset.  Loads return in order, so a tile's pages are
  // asked for before the K and V of the tile in front of it: their use then waits for neither.
  constexpr int kStep = W * kWaveKeys;
  const int start = from + wave * kWaveKeys;
  int page, key;
  const auto look_up = [&](int j0) {
    if constexpr (WHOLE) {
      if (((j0 - start) / kStep & 63) == 0)
        page = table[div_by(a.page_size, (uint32_t)min(j0 + lane * kStep, a.max_len - 1))];
    } else {
      key = j0 + (lane & 31);
      page = table[div_by(a.page_size, (uint32_t)min(key, a.max_len - 1))];
    }
  };
  int64_t at, sat;
  uint32_t seen;  // bit: key of the tile
  const auto place = [&](int j0) {
    if constexpr (WHOLE) {
      const int of = __builtin_amdgcn_readlane(page, (j0 - start) / kStep & 63);
      const bool ok = (uint32_t)of < (uint32_t)a.n_pages;
      const int64_t p = ok ? of : 0;
      const int off = j0 - (int)(div_by(a.page_size, (uint32_t)j0) * a.page_size.d);
      at = p * a.c_page + (int64_t)off * a.c_token + (int64_t)kvh * a.c_head;
      sat = p * a.s_page + (int64_t)off * a.s_token + (int64_t)kvh * a.s_head;
      seen = to - j0 >= 32 ? ~0u : (1u << (to - j0)) - 1;
      if (lo > j0) seen &= ~0u << (lo - j0);  // (lo < j0 + 32)
      if (!ok) seen = 0;
    } else {
      const bool ok = key < to && key >= lo && (uint32_t)page < (uint32_t)a.n_pages;
      const int64_t p = ok ? page : 0;
      const int off = ok ? key - (int)(div_by(a.page_size, (uint32_t)key) * a.page_size.d) : 0;
      at = p * a.c_page + (int64_t)off * a.c_token + (int64_t)kvh * a.c_head;
      sat = p * a.s_page + (int64_t)off * a.s_token + (int64_t)kvh * a.s_head;
      seen = (uint32_t)__builtin_amdgcn_ballot_w64(ok);
    }
    if (!MX) at *= 2;
  };
  const uint32_t token = (uint32_t)a.c_token * (MX ? 1 : 2);  // bytes (WHOLE: below 2^24 values)
  const auto load = [&](R& t, const void* base) {
#pragma unroll
    for (int n = 0; n < R::N; ++n) {
      const int c = R::chunk(n, lane);
      const char* p;
      if constexpr (WHOLE && 64 % R::CH == 0)
        p = (const char*)base + at + n * (64 / R::CH) * (int64_t)token + ((uint32_t)R::row(0, lane) * token + 16 * c);
      else if constexpr (WHOLE)
        p = (const char*)base + at + ((uint32_t)R::row(n, lane) * token + 16 * c);
      else
        p = (const char*)base + from_lane(at, R::row(n, lane)) + 16 * c;
      t.q[n] = u32x4{0, 0, 0, 0};
      if (EXACT || c * (MX ? 16 : 8) < a.D) t.q[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    }
  };
  RowScales<DP> sc;  // MXFP8: lanes 0-31 have those of K, lanes 32-63 of V
  const auto load_scales = [&]() {
    if constexpr (MX) {
      const uint8_t* p = (lane < 32 ? a.scale_k : a.scale_v) + sat + (WHOLE ? (int64_t)(lane & 31) * a.s_token : 0);
#pragma unroll
      for (uint32_t& w : sc.w) w = 0;
      if constexpr (EXACT) {
        __builtin_memcpy(sc.w, p, DP / 32);
      } else {
#pragma unroll
        for (int i = 0; i < DP / 32; ++i)
          if (32 * i < a.D) sc.w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
      }
    }
  };
  // A tile into LDS as 16-bit rows; rows of masked keys as zeros where those are asked for (0 * NaN is no zero).
  const uint32_t lds0 = lds_address(tiles[wave]);
  uint32_t put_k = 0, put_v = 0, get_k = 0, get_v = 0;
  if constexpr (kXor) {
    const int row = lane / R::CH, ch = lane % R::CH * (MX ? 2 : 1), v_row = 4 * g + (r >> 2);
    put_k = lds0 + row * (2 * DP) + ((ch ^ swizzle_k<DP>(row)) << 4);
    put_v = lds0 + row * (2 * DP) + ((ch ^ swizzle_v<DP>(row)) << 4);
    get_k = lds0 + r * (2 * DP) + ((g ^ swizzle_k<DP>(r)) << 4);
    get_v = lds0 + v_row * (2 * DP) + ((((r & 3) >> 1) ^ swizzle_v<DP>(v_row)) << 4) + ((r & 1) << 3);
  }
  const auto store = [&](const R& t, bool v, uint32_t keep) {
#pragma unroll
    for (int n = 0; n < R::N; ++n) {
      const int row = R::row(n, lane), c = R::chunk(n, lane);
      const int sw = v ? swizzle_v<DP>(row) : swizzle_k<DP>(row);
      u32x4 x = t.q[n];
      if (v && keep != ~0u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (keep >> row) & 1 ? x[i] : 0u;
      }
      const auto to = [&](int ch, u32x4 w) {  // (ch: the lane's 16-bit chunk, or the one behind it)
        if constexpr (kXor) {
          const int first = n * (64 / R::CH);
          const int turn = (v ? swizzle_v<DP>(first) : swizzle_k<DP>(first)) ^ (MX ? ch & 1 : 0);
          const uint32_t at = (v ? put_v : put_k) ^ (turn << 4);
          *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(at + first * (2 * DP)) = w;
        } else {
          tiles[wave][row * (DP / 8) + (ch ^ sw)] = w;
        }
      };
      if constexpr (MX) {
        uint32_t code = 0;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(sc.w) / 4); ++i) {
          const uint32_t w = (uint32_t)__shfl((int)sc.w[i], row + (v ? 32 : 0), kWave);
          code = (c >> 3) == i ? (w >> (8 * ((c >> 1) & 3))) & 0xFF : code;
        }
        const float s = e8m0_to_f32(v && keep != ~0u && !((keep >> row) & 1) ? 127u : code);
        u32x4 y[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i >> 1][2 * (i & 1)] = bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], s, false));
          y[i >> 1][2 * (i & 1) + 1] = bitcast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], s, true));
        }
        to(2 * c, y[0]);
        to(2 * c + 1, y[1]);
      } else {
        to(c, x);
      }
    }
  };

  f32x4 o[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) o[i] = f32x4{0, 0, 0, 0};
  Reference<F16> ref;
  float l = 0.0f;
  const float c = a.c;
  R k, v;
  RowScales<DP> sc_now;
  if (start < to) {
    look_up(start);
    place(start);
    look_up(start + kStep);
    load_scales();
    load(k, a.cache_k);
    if constexpr (!kLate) load(v, a.cache_v);
  }
  for (int j0 = start; j0 < to; j0 += kStep) {
    const uint32_t now = seen;
    const bool more = j0 + kStep < to;
    // (the addresses are made anew in each tile: kept, they would cost the registers that the second wave needs)
    if constexpr (kLate && kXor) asm volatile("" : "+v"(put_k), "+v"(put_v), "+v"(get_k), "+v"(get_v));
    store(k, false, now);
    const auto next = [&]() {
      place(j0 + kStep);
      look_up(j0 + 2 * kStep);
      load_scales();
      load(k, a.cache_k);
    };
    if constexpr (kLate) {
      load(v, a.cache_v);
    } else {
      if constexpr (MX) sc_now = sc;
      if (more) next();
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s[h] = mfma_16x16x32<F16>(
            lds_16(kXor ? (get_k ^ (st << 6)) + 16 * h * (2 * DP)
                        : lds0 + (16 * h + r) * (2 * DP) + (((4 * st + g) ^ swizzle_k<DP>(16 * h + r)) << 4)),
            qf[st], s[h]);
    const float base = ref.m == -INFINITY ? 0.0f : ref.m;
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[h][e] = __builtin_fmaf(s[h][e], c, -base);
        s[h][e] = (now >> (16 * h + 4 * g + e)) & 1 ? s[h][e] : -INFINITY;
        top = fmaxf(top, s[h][e]);
      }
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    top = fmaxf(top, __shfl_xor(top, 32, kWave));
    if (__builtin_expect(wave_any(ref.moves(top)), 0)) {
      float up = ref.way(top);
      asm volatile("" : "+v"(up));  // (nothing of this rare block ahead of its branch)
      const float f = ref.factor(up);
      ref.move(top, up);
      l *= f;
#pragma unroll
      for (int i = 0; i < CT; ++i) o[i] *= f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] -= up;
    }
    u32x4 ph, pl;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float e0 = __builtin_amdgcn_exp2f(s[h][e]), e1 = __builtin_amdgcn_exp2f(s[h][e + 1]);
        l += e0 + e1;
        const uint32_t hi = pack16<F16>(e0, e1);
        ph[2 * h + (e >> 1)] = hi;
        pl[2 * h + (e >> 1)] = pack16<F16>(e0 - unpack16(hi, 0, F16), e1 - unpack16(hi, 1, F16));
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if constexpr (MX && !kLate) {  // (the next tile's scales are on their way already)
      const RowScales<DP> next_sc = sc;
      sc = sc_now;
      store(v, true, now);
      sc = next_sc;
    } else {
      store(v, true, now);
    }
    if (more) {
      if constexpr (kLate) next();
      else load(v, a.cache_v);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * h + 4 * g + (r >> 2), d = 16 * i + 4 * (r & 3);
        const u32x2 t = lds_tr(kXor ? (get_v ^ (i << 5)) + 16 * h * (2 * DP)
                                    : lds0 + row * (2 * DP) + (((d >> 3) ^ swizzle_v<DP>(row)) << 4) + ((d & 7) << 1));
        w[2 * h] = t[0];
        w[2 * h + 1] = t[1];
      }
      o[i] = mfma_16x16x32<F16>(w, pl, o[i]);
      o[i] = mfma_16x16x32<F16>(w, ph, o[i]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // The waves' parts: reference and sum of each head, then O scaled to the common reference and added
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (g == 0) {
    stat[wave][0][r] = ref.m;
    stat[wave][1][r] = l;
  }
  __syncthreads();
  float all = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) all = fmaxf(all, stat[w][0][r]);
#pragma unroll
  for (int w = 0; w < W; ++w)
    sum += stat[w][0][r] == -INFINITY ? stat[w][1][r] : stat[w][1][r] * __builtin_amdgcn_exp2f(stat[w][0][r] - all);
  const float f = ref.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ref.m - all);
  // O of a wave as [16 heads][DP] fp32, in its tile's place: float 4-groups of a head's row take turns with the head
  float* ow = reinterpret_cast<float*>(tiles[wave]);
#pragma unroll
  for (int i = 0; i < CT; ++i)
    *reinterpret_cast<f32x4*>(ow + r * DP + ((4 * i + g) ^ (r & 7)) * 4) = o[i] * f;
  __syncthreads();
  // thread: head tid / 16, values in groups of four
  const int oh = tid >> 4;
  const float* o0 = reinterpret_cast<const float*>(&tiles[0][0]);
  const float total = __shfl(sum, oh & 15, kWave), top = __shfl(all, oh & 15, kWave);
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t orow = (int64_t)b * a.Hq + kvh * a.G + head0 + oh;
  if (oh < heads) {
#pragma unroll
    for (int u = 0; u < (DP + 63) / 64; ++u) {
      const int q4 = 16 * u + (tid & 15), d = 4 * q4;
      if (DP % 64 != 0 && d >= DP) continue;
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < W; ++w)
        x += *reinterpret_cast<const f32x4*>(o0 + w * (16 * DP) + oh * DP + ((q4 ^ (oh & 7)) << 2));
      if (!EXACT && d >= a.D) continue;
      if (a.parts > 1) {
        *reinterpret_cast<f32x4*>(parts.o + (orow * a.parts + part) * a.D + d) = x;
      } else {
        u32x2 y = {pack16<F16>(x[0] * inv, x[1] * inv), pack16<F16>(x[2] * inv, x[3] * inv)};
        *reinterpret_cast<u32x2*>(a.y + (int64_t)b * a.y_ts + (int64_t)(kvh * a.G + head0 + oh) * a.y_hs + d) = y;
      }
    }
    if ((tid & 15) == 0) {
      if (a.parts > 1) {
        parts.ml[2 * (orow * a.parts + part)] = top;
        parts.ml[2 * (orow * a.parts + part) + 1] = total;
      } else if (a.lse) {
        a.lse[orow] = total == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(total)) * kLn2;
      }
    }
  }
}

constexpr int kFewParts = 8;

// A workgroup per row joins its parts: the waves read all references and sums at once, then L lanes take a part's O and
// 256 / L groups of them the parts in turn, joined in order through LDS.
template <int L>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoin a) {
  constexpr int GROUPS = 256 / L;
  __shared__ f32x4 sum[GROUPS][L];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t row = blockIdx.x;
  const int64_t t = row / a.Hq;
  const int h = (int)(row - t * a.Hq);
  if (a.cu_q && (t < a.cu_q[0] || t >= a.cu_q[a.n_seqs])) return;
  const int P = a.parts.parts;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.parts.ml) + row * P;
  const f32x2 first = lane < P ? ml[lane] : f32x2{-INFINITY, 0.0f};
  float top = first[0];
  for (int p = lane + 64; p < P; p += 64) top = fmaxf(top, ml[p][0]);
  top = wave_max_dpp(top);
  // (a part without keys has the sum 0, whatever its reference)
  float total = first[1] == 0.0f ? 0.0f : first[1] * __builtin_amdgcn_exp2f(first[0] - top);
  for (int p = lane + 64; p < P; p += 64) total += ml[p][1] == 0.0f ? 0.0f : ml[p][1] * __builtin_amdgcn_exp2f(ml[p][0] - top);
  total = wave_sum_dpp(total);
  const int g = tid / L, d = 4 * (tid % L);
  f32x4 x = {0, 0, 0, 0};
  if (d < a.D) {
#pragma unroll 4
    for (int p = g; p < P; p += GROUPS) {
      const f32x2 w = ml[p];
      if (w[1] != 0.0f) x += *reinterpret_cast<const f32x4*>(a.parts.o + (row * P + p) * a.D + d) * __builtin_amdgcn_exp2f(w[0] - top);
    }
  }
  sum[g][tid % L] = x;
  __syncthreads();
  if (g == 0 && d < a.D) {
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) x += sum[i][tid];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const u32x2 y = {(uint32_t)f32_to_16(x[0] * inv, a.f16) | (uint32_t)f32_to_16(x[1] * inv, a.f16) << 16,
                     (uint32_t)f32_to_16(x[2] * inv, a.f16) | (uint32_t)f32_to_16(x[3] * inv, a.f16) << 16};
    *reinterpret_cast<u32x2*>(a.y + t * a.y_ts + (int64_t)h * a.y_hs + d) = y;
  }
  if (tid == 0 && a.lse) a.lse[row] = total == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(total)) * kLn2;
}

// Few parts: L lanes take a row and read all of its parts at once (38400 rows of two parts: 35 us by the kernel above).
template <int L>
__global__ __launch_bounds__(256) void attn_join_few_kernel(AttnJoin a) {
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= a.rows) return;
  const int64_t t = row / a.Hq;
  const int h = (int)(row - t * a.Hq), d = 4 * (threadIdx.x % L), P = a.parts.parts;
  if (a.cu_q && (t < a.cu_q[0] || t >= a.cu_q[a.n_seqs])) return;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.parts.ml) + row * P;
  const f32x4* o = reinterpret_cast<const f32x4*>(a.parts.o + row * P * a.D + d);
  f32x2 w[kFewParts];
  f32x4 v[kFewParts];
  float top = -INFINITY;
#pragma unroll
  for (int p = 0; p < kFewParts; ++p) {
    w[p] = p < P ? ml[p] : f32x2{-INFINITY, 0.0f};
    v[p] = f32x4{0, 0, 0, 0};
    if (p < P && d < a.D) v[p] = o[(int64_t)p * (a.D / 4)];  // (not written where the part's sum is 0)
    top = fmaxf(top, w[p][0]);
  }
  float total = 0.0f;
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < kFewParts; ++p) {
    const float f = w[p][1] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(w[p][0] - top);
    total += w[p][1] * f;
    x += f == 0.0f ? f32x4{0, 0, 0, 0} : v[p] * f;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  if (d < a.D) {
    const u32x2 y = {(uint32_t)f32_to_16(x[0] * inv, a.f16) | (uint32_t)f32_to_16(x[1] * inv, a.f16) << 16,
                     (uint32_t)f32_to_16(x[2] * inv, a.f16) | (uint32_t)f32_to_16(x[3] * inv, a.f16) << 16};
    *reinterpret_cast<u32x2*>(a.y + t * a.y_ts + (int64_t)h * a.y_hs + d) = y;
  }
  if (d == 0 && a.lse) a.lse[row] = total == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(total)) * kLn2;
}

struct DecodePlan {
  int parts, part_keys;
};
// Parts of a row of up to n keys (in a window: of what it can touch).  Few rows: two workgroups a CU, of one step of their
// waves at least (one sequence of 777 tokens: 8.7 us; two steps 9.6).  Up to four units of row and head a CU: twelve
// workgroups a CU, of two steps at least, up to 64 to a row (three rows of 131072 in MXFP8 join in 9.3 us from 128 parts, in
// 5 from 43), which evens out rows of different lengths (us with 4, 8, 12, 24 a CU: 64 sequences of up to 8192 245, 243,
// 220, 220; 16 of up to 16384 in MXFP8 82, 74, 74, 78; 8 of 4096 in steps of 128 29.6, of 256 27.7).  More units are even
// enough (176 sequences of up to 4096: one part 215, two 227, three 221) unless rows are very long; past 64 units a CU
// parts would only take workspace.
int64_t most_parts(int64_t units, int64_t n) {
  constexpr int kBlockKeys = kDecodeWaves * kWaveKeys, kCus = 256;
  const auto for_blocks = [&](int64_t blocks) { return (blocks + units - 1) / units; };
  const int64_t some = std::min(for_blocks(2 * kCus), (n + kBlockKeys - 1) / kBlockKeys);
  const int64_t more = units < 4 * kCus ? std::min(std::min<int64_t>(for_blocks(12 * kCus), 64), n / (2 * kBlockKeys))
                                        : (units < 64 * kCus ? std::min<int64_t>(16, n / 8192) : 1);
  return std::max<int64_t>(1, std::max(some, more));
}
int64_t decode_units(int B, int Hq, int Hkv) { return (int64_t)B * Hkv * ((Hq / Hkv + 15) / 16); }
DecodePlan plan_decode(const DecodeArgs& a) {
  constexpr int kBlockKeys = kDecodeWaves * kWaveKeys;
  const int64_t n = a.window > 0 ? std::min<int64_t>(a.max_len, (int64_t)a.window + kWaveKeys - 1) : a.max_len;
  const int64_t parts = most_parts(decode_units(a.B, a.Hq, a.Hkv), n);
  const int64_t keys = std::max<int64_t>(1, ((n + parts - 1) / parts + kBlockKeys - 1) / kBlockKeys) * kBlockKeys;
  return DecodePlan{(int)std::max<int64_t>(1, (n + keys - 1) / keys), (int)keys};
}

template <int FMT>
void launch_decode_fmt(const DecodeArgs& a, dim3 g, hipStream_t stream) {
#define MOE_DECODE_W(DP, WHOLE, OCC)                                                              \
  (a.D == DP ? decode_kernel<FMT, DP, true, WHOLE, OCC><<<g, 64 * kDecodeWaves, 0, stream>>>(a)   \
             : decode_kernel<FMT, DP, false, WHOLE, OCC><<<g, 64 * kDecodeWaves, 0, stream>>>(a))
#define MOE_DECODE(DP, OCC) (whole ? MOE_DECODE_W(DP, true, OCC) : MOE_DECODE_W(DP, false, OCC))
  const bool whole = a.page_size.d % kWaveKeys == 0 && a.c_token < 1 << 24;
  if (a.D <= 64) MOE_DECODE(64, 4);
  else if (a.D <= 96) MOE_DECODE(96, 2);
  else if (a.D <= 128) MOE_DECODE(128, 2);
  else if (a.D <= 192) MOE_DECODE(192, (FMT == MOE_KV_MXFP8 ? 2 : 1));  // (16 bits, 64 rows of up to 4096: 176 us, so 227)
  else MOE_DECODE(256, (FMT == MOE_KV_MXFP8 ? 2 : 1));  // (16 bits, 64 rows of up to 4096: 212-230 us, so 270)
#undef MOE_DECODE
#undef MOE_DECODE_W
}

}  // namespace

size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D, int max_len) {
  return attn_parts_bytes((int64_t)B * Hq, (int)most_parts(decode_units(B, Hq, Hkv), max_len), D);
}

hipError_t launch_attn_join(const AttnJoin& j, hipStream_t stream) {
  // (64 rows of seven parts: 2.6 us a workgroup each, 3.9 so)
  if (j.parts.parts <= kFewParts && j.rows > 2048) {
    const int rows = j.D <= 64 ? 16 : (j.D <= 128 ? 8 : 4);
    const dim3 g((unsigned)((j.rows + rows - 1) / rows));
    if (j.D <= 64) attn_join_few_kernel<16><<<g, 256, 0, stream>>>(j);
    else if (j.D <= 128) attn_join_few_kernel<32><<<g, 256, 0, stream>>>(j);
    else attn_join_few_kernel<64><<<g, 256, 0, stream>>>(j);
    return hipGetLastError();
  }
  const dim3 g((unsigned)j.rows);
  if (j.D <= 64) attn_join_kernel<16><<<g, 256, 0, stream>>>(j);
  else if (j.D <= 128) attn_join_kernel<32><<<g, 256, 0, stream>>>(j);
  else attn_join_kernel<64><<<g, 256, 0, stream>>>(j);
  return hipGetLastError();
}

hipError_t launch_decode(DecodeArgs a, hipStream_t stream) {
  const DecodePlan p = plan_decode(a);
  a.parts = p.parts;
  a.part_keys = p.part_keys;
  const dim3 g((unsigned)((int64_t)a.B * p.parts * a.Hkv * ((a.G + 15) / 16)));
  if (a.fmt == MOE_KV_BF16) launch_decode_fmt<MOE_KV_BF16>(a, g, stream);
  else if (a.fmt == MOE_KV_FP16) launch_decode_fmt<MOE_KV_FP16>(a, g, stream);
  else launch_decode_fmt<MOE_KV_MXFP8>(a, g, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.parts == 1) return err;
  AttnJoin j{};
  j.parts = attn_parts(a.ws, (int64_t)a.B * a.Hq, p.parts);
  j.rows = (int64_t)a.B * a.Hq;
  j.Hq = a.Hq;
  j.D = a.D;
  j.f16 = a.fmt == MOE_KV_FP16;
  j.y = a.y;
  j.y_ts = a.y_ts;
  j.y_hs = a.y_hs;
  j.lse = a.lse;
  return launch_attn_join(j, stream);
}

}  // namespace moe
