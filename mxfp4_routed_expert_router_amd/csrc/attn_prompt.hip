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
// exponentials, which run beside them.  16384 tokens, 64 heads of 128 on 8: 4.0 ms, 1.1 PFLOP/s, the matrix cores busy 61%
// of the cycles at 1.72 GHz; the card's power holds it there (with 50% the clock was 1.97 GHz).  P is rounded to 16 bits
// (half a step, as the output is); maxima, sums and O are fp32.  The sum is of the unrounded exponentials, which the log sum
// needs: errors that differ from key to key average out, but where many keys of one score carry a row they all err alike, and
// y by as much, up to that half step.  A second sum, of the rounded ones, would take that out for 5% more time (16384 tokens:
// 3835 -> 4035 us; heads of 256, which have no registers left for it, 186 -> 232).
#include <limits.h>

#include <algorithm>

#include "attention.hpp"

namespace moe {

namespace {

constexpr int kTileKeys = 64;

__device__ __forceinline__ float other_half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sixteen bytes a lane from base + off straight into LDS, consecutive lanes behind one another from `to` on.  The compiler
// waits for such loads of its own at the next LDS read that it cannot tell apart, in the middle of the tile that they
// should overlap; written out (FREE), only loads_done() waits for them, which stands in front of the barrier that publishes
// them either way.  Heads of 128: 4130 -> 4010 us for 16384 tokens.  With one wave on a SIMD (heads beyond 128) the
// compiler's own order of loads and arithmetic is worth more: 342 us for 4096 tokens of heads of 256, so 395.
// (The load has no registers to write; one instruction lies between a write of m0 and its use; nothing else in these
// kernels uses m0.)
template <bool FREE>
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, u32x4* to) {
  if constexpr (FREE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds_address(to))), "v"(off), "s"(base)
                 : "memory");
  else
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)((const char*)base + off),
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Next in a block's order: READS LDS reads; a matrix product with TRANS exponentials, VALU vector instructions and READS
// LDS reads behind it.
template <int READS>
__device__ __forceinline__ void then_read() {
  __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
}
template <int TRANS, int VALU, int READS>
__device__ __forceinline__ void then_multiply() {
  __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
  if constexpr (TRANS > 0) __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
  if constexpr (VALU > 0) __builtin_amdgcn_sched_group_barrier(0x2, VALU, 0);
  if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
}

struct Piece {  // a workgroup's rows
  int q0, nq, k0, nk, tile;  // tile < 0: none
};

// Workgroup `slot` of a key-value head.  Sequence b has the slots from floor(cu_q[b] G / rows) + b on, which leaves room for
// its ceil(nq G / rows) tiles (a spare slot ends at once), so its place is searched, 64 sequences a step, and not summed.  The
// last tile (most keys) comes first.  Two thousand sequences of 8: 210 us, summed 435.
__device__ __forceinline__ Piece find_piece(const PromptArgs& a, int slot, int rows) {
  const int lane = threadIdx.x & 63;
  int from = 0;
  for (int span = a.n_seqs; span > 64;) {
    const int step = (span + 63) / 64, b = from + lane * step;
    const bool before = b < from + span && (int)((int64_t)min(max(a.cu_q[min(b, a.n_seqs)], 0), a.Tq) * a.G.d / rows) + b <= slot;
    const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(before));
    const int at = max(n - 1, 0) * step;
    span = min(step, span - at);
    from += at;
  }
  const int b = from + lane;
  int q0 = 0, q1 = 0, k0 = 0, k1 = 0, first = INT_MAX;
  if (b < a.n_seqs) {
    q0 = min(max(a.cu_q[b], 0), a.Tq);
    q1 = min(max(a.cu_q[b + 1], q0), a.Tq);
    k0 = min(max(a.cu_k[b], 0), a.Tk);
    k1 = min(max(a.cu_k[b + 1], k0), a.Tk);
    first = (int)((int64_t)q0 * a.G.d / rows) + b;
  }
  const uint64_t before = __builtin_amdgcn_ballot_w64(first <= slot);
  if (before == 0) return Piece{0, 0, 0, 0, -1};
  const int s = __builtin_popcountll(before) - 1;  // (cu_q ascends)
  Piece p;
  p.q0 = __builtin_amdgcn_readlane(q0, s);
  p.nq = __builtin_amdgcn_readlane(q1, s) - p.q0;
  p.k0 = __builtin_amdgcn_readlane(k0, s);
  p.nk = __builtin_amdgcn_readlane(k1, s) - p.k0;
  const int tiles = (int)(((int64_t)p.nq * a.G.d + rows - 1) / rows);
  p.tile = tiles - 1 - (slot - __builtin_amdgcn_readlane(first, s));
  if (p.tile >= tiles) p.tile = -1;  // (a cu_q that descends)
  return p;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// The 16-bit values of a dword that are infinite or NaN, as a mask.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0xFFFFu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}

// DP: head size that the tiles are made for (EXACT: the head's own).  NW: waves.  PER_SIMD: waves of a SIMD that share its
// registers; two workgroups of four waves on a CU stand at different tiles, so that one's products run beside the other's
// vector work.
template <bool F16, int DP, bool EXACT, int NW, int PER_SIMD>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void prompt_kernel(PromptArgs a) {
  constexpr int CH = DP / 8;          // 16-byte chunks of a row
  constexpr int BN = kTileKeys, KT = BN / 32, DT = DP / 32, ST = DP / 16;
  // Whether the next tile's scores run between a tile's exponentials.  Heads of 128 gain by it (16384 tokens: 4340 -> 4130
  // us); heads of 64 have less to multiply, and the registers of the second set of scores cost them a third wave (33 -> 44).
  constexpr bool kAhead = DP > 64;
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
  // Tiles go from memory straight into LDS, a wave 1 KB a time.  A lane's place in a row repeats after KEEP rounds (where
  // those are sixteen rows), which are a scalar further; else each round has an offset of its own.
  constexpr int ROUNDS = BN * CH / (64 * NW), STEP = 64 * NW / CH;
  constexpr bool WHOLE = (64 * NW) % CH == 0 && (STEP % 16 == 0 || 16 % STEP == 0);
  constexpr int KEEP = !WHOLE ? ROUNDS : (STEP >= 16 ? 1 : 16 / STEP);
  const auto place = [&](int u, int64_t ts, bool v, int last) {  // byte offset of round u's 16 bytes from the tile's first row
    const int p = u * 64 * NW + tid, row = p / CH, cc = p % CH;
    const int c = cc ^ (v ? swizzle_v<DP>(row) : swizzle_k<DP>(row));
    return (EXACT || 8 * c < a.D) ? (uint32_t)min(row, last) * (uint32_t)(2 * ts) + 16 * c : ~0u;
  };
  uint32_t k_off[KEEP], v_off[KEEP];
#pragma unroll
  for (int u = 0; u < KEEP; ++u) {
    k_off[u] = place(u, a.k_ts, false, BN);
    v_off[u] = place(u, a.v_ts, true, BN);
  }
  const auto put = [&](const uint16_t* base, uint32_t off, u32x4* to) {
    if (EXACT || off != ~0u) load_to_lds<DP <= 128>(base, off, to);
  };
  const auto load_tile = [&](int buf, int v, const uint16_t* rows, int64_t ts, const uint32_t* off, int j0) {
    const uint16_t* from = rows + j0 * ts;
    u32x4* to = &lds[buf][v][64 * wave];
    if (DP <= 192 && j0 + BN <= pc.nk) {  // (kept offsets would not fit the registers of heads beyond 192: 345 -> 381 us)
#pragma unroll
      for (int u = 0; u < ROUNDS; ++u)
        put(from + u / KEEP * KEEP * STEP * ts, off[u % KEEP], to + u * 64 * NW);
    } else {  // rows past the last key repeat it, and are masked
#pragma unroll
      for (int u = 0; u < ROUNDS; ++u) put(from, place(u, ts, v != 0, pc.nk - 1 - j0), to + u * 64 * NW);
    }
  };
  const auto load_k = [&](int t) { load_tile(t & 1, 0, kp, a.k_ts, k_off, b_lo + t * BN); };
  const auto load_v = [&](int t) { load_tile(t & 1, 1, vp, a.v_ts, v_off, b_lo + t * BN); };

  // LDS addresses.  A step inside a span is an exclusive-or of a lane's address, one to another span an addition.
  constexpr int kSpan = kSpanOf<DP>, KS = kSpan / 32, VS = kSpan / 64;
  const uint32_t lds0 = lds_address(&lds[0][0][0]);
  constexpr uint32_t kTile = BN * CH * 16;
  const uint32_t k_at = lds0 + col * (2 * DP) + ((half ^ swizzle_k<DP>(col)) << 4);
  const int vi = lane & 15, v_row = 4 * half + (vi >> 2);
  const uint32_t v_at = lds0 + kTile + v_row * (2 * DP) +
                        (((2 * ((lane >> 4) & 1) + ((vi & 3) >> 1)) ^ swizzle_v<DP>(v_row)) << 4) + ((vi & 1) << 3);

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
  Reference<F16> ref;
  float l = 0.0f;  // sum over this lane's keys
  const float c = a.c;

  const auto v_frag = [&](uint32_t buf, int ks, int dt) {
    const uint32_t at = ((v_at + buf) ^ (uint32_t)((dt % VS) << 6)) + dt / VS * kSpan + ks * (16 * 2 * DP);
    const u32x2 x = lds_tr(at), y = lds_tr(at + 8 * 2 * DP);
    return u32x4{x[0], x[1], y[0], y[1]};
  };
  const auto scores = [&](f32x16 (&s)[KT], uint32_t buf) {
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const u32x4 kf = lds_16(((k_at + buf) ^ (uint32_t)((st % KS) << 5)) + st / KS * kSpan + kt * (32 * 2 * DP));
        f32x16 zero;
#pragma unroll
        for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
        s[kt] = mfma_32x32x16<F16>(kf, qf[st], st == 0 ? zero : s[kt]);
      }
  };
  // Tile t from its scores on (kAhead: with the scores of the tile after it, `after`, on the way).
  const auto tile = [&](f32x16 (&s)[KT], f32x16 (&after)[KT], int t) {
    const int j0 = b_lo + t * BN;
    const uint32_t buf = (t & 1) * 2 * kTile, buf_after = buf ^ (2 * kTile);
    // V of tile t is there, K too (kAhead: of tile t + 1), and nobody reads what the next loads replace any more
    loads_done();
    __syncthreads();
    if (t + 1 + kAhead < n_tiles) load_k(t + 1 + kAhead);
    if (t + 1 < n_tiles) load_v(t + 1);
    if (j0 >= w_hi || j0 + BN <= w_lo) {  // nothing of the tile is the wave's
      if constexpr (kAhead) scores(after, buf_after);
      return;
    }
    if constexpr (!kAhead) scores(s, buf);
    const bool masked = j0 + BN > w_hi_min || j0 < w_lo_max;
    // 0 * infinity is no zero: a masked key's value must not reach a row, so values that are not finite go by themselves
    bool wild = false;
    if (__builtin_expect(masked, 0)) {
      u16x2 most = {0, 0};  // of the values' bits without the sign
#pragma unroll
      for (int u = 0; u < BN * CH / 64; ++u) {
        const u32x4 w = lds_16(lds0 + buf + kTile + (64 * u + lane) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, bitcast<u16x2>(w[i] & 0x7FFF7FFFu));
      }
      wild = wave_any(std::max<uint16_t>(most[0], most[1]) >= (F16 ? 0x7C00 : 0x7F80));
    }
    const float base = ref.m == -INFINITY ? 0.0f : ref.m;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[kt][r] = __builtin_fmaf(s[kt][r], c, -base);
    if (__builtin_expect(masked, 0)) {
      int lo_j = lo - j0 - 4 * half, hi_j = hi - j0 - 4 * half;
      asm volatile("" : "+v"(lo_j), "+v"(hi_j));  // (nothing of this block ahead of its branch)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = 32 * kt + 8 * (r >> 2) + (r & 3);
          s[kt][r] = ((j >= lo_j) & (j < hi_j)) ? s[kt][r] : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kt][r]);
    top = other_half_max(top);
    if (__builtin_expect(wave_any(ref.moves(top)), 0)) {
      float up = ref.way(top);
      asm volatile("" : "+v"(up));  // (nothing of this rare block ahead of its branch)
      const float f = ref.factor(up);
      ref.move(top, up);
      l *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] *= f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[kt][r] -= up;
    }
    u32x4 pf[2 * KT], vf[DT];
    const auto exponentials = [&](int ks) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const int r = 8 * (ks & 1) + e;
        const float e0 = __builtin_amdgcn_exp2f(s[ks >> 1][r]), e1 = __builtin_amdgcn_exp2f(s[ks >> 1][r + 1]);
        s[ks >> 1][r] = e0;
        s[ks >> 1][r + 1] = e1;
        pf[ks][e >> 1] = pack16<F16>(e0, e1);
      }
    };
    if constexpr (kAhead) {
      scores(after, buf_after);
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks) exponentials(ks);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) vf[dt] = v_frag(buf, 0, dt);
    }
    if constexpr (kAhead) {  // products between the exponentials, operands four products before their use, then the first V
      constexpr int N = ST * KT;
      then_read<4>();
#pragma unroll
      for (int i = 0; i < N - 4; ++i) then_multiply<16 * KT / N, 8 * KT / N, 1>();
#pragma unroll
      for (int i = 0; i < 4; ++i) then_multiply<16 * KT / N, 8 * KT / N, (DT + 1) / 2>();
    }
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const auto add = [&](int ks) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[e & 3] += s[ks >> 1][8 * (ks & 1) + e];
    };
    if (__builtin_expect(!wild, 1)) {
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks) {
        if constexpr (!kAhead) exponentials(ks);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          if constexpr (!kAhead) vf[dt] = v_frag(buf, ks, dt);
          o[dt] = mfma_32x32x16<F16>(vf[dt], pf[ks], o[dt]);
          if (kAhead && ks + 1 < 2 * KT) vf[dt] = v_frag(buf, ks + 1, dt);
        }
        add(ks);
      }
      l += (part[0] + part[1]) + (part[2] + part[3]);
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < 2 * KT * DT; ++i) then_multiply<0, 2, 2>();
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 2 * KT; ++ks) {
        if constexpr (!kAhead) exponentials(ks);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          u32x4 w = v_frag(buf, ks, dt);
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] &= ~not_finite<F16>(w[x]);
          o[dt] = mfma_32x32x16<F16>(w, pf[ks], o[dt]);
        }
        add(ks);
      }
      l += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll 1
      for (int kk = 0; kk < BN; ++kk) {  // what was left out, into the rows that see it
        const bool seen = (j0 + kk >= lo) & (j0 + kk < hi);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          f32x16 more;
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const u32x2 w = *(lds_u32x2*)(uintptr_t)(lds0 + buf + kTile + kk * (2 * DP) +
                                          (((4 * dt + q4) ^ swizzle_v<DP>(kk)) << 4) + 8 * half);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t bad = not_finite<F16>(w[x >> 1]) & (x & 1 ? 0xFFFF0000u : 0xFFFFu);
              more[4 * q4 + x] = (seen & (bad != 0)) ? unpack16(w[x >> 1], x & 1, F16) : 0.0f;
            }
          }
          o[dt] += more;
        }
      }
    }
  };

  if (n_tiles > 0) {
    load_k(0);
    load_v(0);
    f32x16 s0[KT], s1[KT];
    if constexpr (kAhead) {
      if (n_tiles > 1) load_k(1);
      loads_done();
      __syncthreads();
      scores(s0, 0);
      // (behind the last tile the other buffer's scores are computed once more and not used)
      for (int t = 0; t < n_tiles; t += 2) {
        tile(s0, s1, t);
        if (t + 1 < n_tiles) tile(s1, s0, t + 1);
      }
    } else {
      for (int t = 0; t < n_tiles; ++t) tile(s0, s0, t);
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
      w.ml[2 * at] = ref.m;
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
  if (mine && half == 0 && a.lse) a.lse[orow] = l == 0.0f ? -INFINITY : (ref.m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <bool F16, int DP, int NW, int PER_SIMD>
void launch_exact(const PromptArgs& a, dim3 g, hipStream_t stream) {
  if (a.D == DP) prompt_kernel<F16, DP, true, NW, PER_SIMD><<<g, 64 * NW, 0, stream>>>(a);
  else prompt_kernel<F16, DP, false, NW, PER_SIMD><<<g, 64 * NW, 0, stream>>>(a);
}

// Keys are shared where a prompt's tiles are too few for the card.  The parts' results cost their bytes twice and a second
// launch, so the number is the one of least estimated time: rounds of workgroups, tiles of each, and the joining (us, at
// heads of 128: a tile takes 1.6 alone on its SIMDs and 1.9 with another, 4 for a workgroup's start and end, 4 for a launch;
// parts' bytes move at 4 TB/s).  A sequence's keys are not known here: twice the mean, at most all.
// Measured, parts of 1 / 8: 128 tokens behind 16000 (64 heads on 8) 340 / 86 us; 301 tokens 13.6 in one part, 35 in three.
struct PromptPlan {
  int waves;  // of a workgroup, 32 rows each
  int64_t slots;
  int parts, part_keys;
};
PromptPlan plan_prompt(int Tq, int Tk, int n_seqs, int Hq, int Hkv, int D) {
  PromptPlan p;
  p.waves = 4;
  const int rows = 32 * p.waves;
  const int64_t tiles = ((int64_t)Tq * (Hq / Hkv) + rows - 1) / rows, all_rows = (int64_t)Tq * Hq;
  p.slots = (int64_t)Tq * (Hq / Hkv) / rows + n_seqs;
  p.parts = 1;
  p.part_keys = std::max(1, (Tk + kTileKeys - 1) / kTileKeys) * kTileKeys;
  const int64_t blocks = std::max<int64_t>(tiles, std::min(n_seqs, Tq)) * Hkv;
  const int at_once = 256 * (D <= 64 ? 4 : (D <= 128 ? 2 : 1));
  if (blocks >= at_once / 2) return p;
  const double keys = std::min<double>(Tk, 2.0 * Tk / n_seqs);
  double best = 0.0;
  for (const int n : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
    const int64_t part = ((int64_t)(keys / n) + kTileKeys) / kTileKeys * kTileKeys;
    const int64_t parts = n == 1 ? 1 : (Tk + part - 1) / part;
    if (n > 1 && (parts < 2 || parts > 1024 || attn_parts_bytes(all_rows, (int)parts, D) > (size_t)256 << 20)) continue;
    const double rounds = (double)((blocks * n + at_once - 1) / at_once);
    const double tile = (blocks * n > 256 ? 1.9 : 1.6) * D / 128;
    const double us = rounds * ((double)part / kTileKeys * tile + 4) + (n > 1 ? 4 + (double)all_rows * n * (D + 2) * 8 / 4e6 : 0);
    if (n == 1 || us < 0.9 * best) {
      best = us;
      p.parts = (int)parts;
      if (n > 1) p.part_keys = (int)part;
    }
  }
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
  if (a.D <= 64) MOE_PROMPT(64, 4, 4);
  else if (a.D <= 96) MOE_PROMPT(96, 4, 2);
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
