// Host-side launchers of the gfx950 kernels (one per kernel family), called by the C ABI after it
// has validated every argument.  Each returns the launch status (hipGetLastError after enqueue).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// ---- router ----
int route_splits(int T, int H, int E);
// sigmoid: Cascadia's sigmoid router (bias on the selection only, weights routed_scale * s / sum s,
// shared slots shared_weight) instead of softmax -> top-k -> renormalise.
hipError_t launch_route(const void* x, int x_fp16, int T, int H, const float* w_router, const float* bias,
                        int E, int top_k, int n_shared, int32_t* ids, float* weights, float* probs,
                        float* partial, int splits, hipStream_t stream, bool sigmoid = false,
                        float routed_scale = 1.0f, float shared_weight = 1.0f);

// The router's logits alone: partial sums [splits][T][E].
hipError_t launch_route_logits(const void* x, int x_fp16, int T, int H, const float* w_router, int E, float* partial,
                               int splits, hipStream_t stream);

// ---- choice of experts by a rule (scores, bias, groups, top-k), from logits or from x ----
hipError_t launch_select(const void* logits, int dt, int64_t row_stride, int T, int E, const moe_route_rule& rule,
                         int32_t* ids, float* weights, float* scores, hipStream_t stream);
hipError_t launch_route_grouped(const void* x, int x_fp16, int T, int H, const float* w_router, int E,
                                const moe_route_rule& rule, int32_t* ids, float* weights, float* scores,
                                float* partial, hipStream_t stream);

// Router, bucketing and (table != NULL) the expert FFN's tile table in two launches (logits, then
// one workgroup that selects, buckets and plans), for the small calls route_bucket_fusable()
// accepts (at most 8 tokens).
bool route_bucket_fusable(int T, int k_total, int n_buckets);
hipError_t launch_route_bucket(const void* x, int x_fp16, int T, int H, const float* w_router, const float* bias,
                               int E, int top_k, int n_shared, int32_t* ids, float* weights, float* probs,
                               float* partial, int splits, int n_buckets, int32_t* counts, int32_t* offsets,
                               int32_t* sorted_slot, int32_t* slot_pos, void* table, int rows_per_tile,
                               int64_t n_entries, hipStream_t stream);

// ---- fixed row shapes: zero routing weights and invalid ids on rows past the device row count ----
hipError_t launch_pad_rows(const int32_t* n_rows, int T_shape, int k_total, int32_t* ids, float* weights,
                           hipStream_t stream);

// ---- streaming-read probe (a measurement utility) ----
hipError_t launch_stream_read(const void* buf, uint64_t bytes, uint32_t* sink, hipStream_t stream);

// ---- bucketing ----
constexpr int kBucketChunk = 512;
hipError_t launch_bucket(const int32_t* ids, int n_slots, int n_buckets, int32_t* counts, int32_t* offsets,
                         int32_t* sorted_slot, int32_t* slot_pos, int32_t* ws, hipStream_t stream);
// Whether launch_bucket_plan builds the tile table inside the bucketing launch (one workgroup holds
// all of the slots); otherwise the caller runs the plan launch after it.
bool bucket_plans_inline(int n_slots);
// launch_bucket, and for bucket_plans_inline(n_slots) the expert FFN's tile table (n_entries
// entries of rows_per_tile rows, the entries of ffn_tiles_kernel) from the offsets it just built.
hipError_t launch_bucket_plan(const int32_t* ids, int n_slots, int n_buckets, int32_t* counts, int32_t* offsets,
                              int32_t* sorted_slot, int32_t* slot_pos, int32_t* ws, void* table, int rows_per_tile,
                              int64_t n_entries, hipStream_t stream);

// ---- expert FFN ----
struct ProjDev {
  const uint8_t* w;
  const uint8_t* s;
  int64_t we, wr, se, sr;
  const uint8_t* z;  // INT4 group-32 zero points
  int64_t ze, zr;
  const float* ts;   // NVFP4 tensor scales [n_experts]
};
// Tile plan of one expert-FFN call: 16*mt sorted rows per tile, `tiles` entries in the tile table
// (an upper bound, padded to a multiple of the XCD count).
struct FfnPlan {
  int mt;   // token tiles of 16 per MFMA column block (the kernels' MT)
  int rpt;  // sorted rows (tokens) per tile: 16 * mt, or kTinyT for the tiny down kernel
  int64_t tiles;
  int n_experts;
  bool tile;  // the tile kernels (MXFP4, many rows per expert)
  bool tiny;  // the tiny down kernel (at most kTinyT tokens)
};
constexpr int kTinyT = 4;  // tokens of a call the tiny down kernel takes (at most kTinyT rows per tile)
// Kernel choices that depend on the weights description, as flags for ffn_plan: kPlanBig -- calls
// with many rows per expert may use the 128-token tile kernels (MXFP4 or FP16, whole 128-wide
// chunks, aligned scale rows, 32-bit offsets); kPlanTiny -- calls of at most kTinyT tokens may use
// the tiny down kernel (MXFP4, I a multiple of 512 up to 2048, H a multiple of 64, 16-byte
// aligned scale rows).  The
// FFN entry points and the workspace query must agree, so they all derive the flags from the same
// weights description.
constexpr int kPlanBig = 1, kPlanTiny = 2;
int ffn_plan_opts(int fmt, int T, int k_total, int H, int I, const ProjDev& gate, const ProjDev& up,
                  const ProjDev& down);
FfnPlan ffn_plan(int T, int k_total, int n_experts, int opts);
size_t ffn_table_bytes(int T, int k_total, int n_experts, int opts);
// The tile table of `rows_per_tile`-row tiles for the bucket offsets (entries up to n_entries).
hipError_t launch_ffn_tiles(const int32_t* offsets, int n_experts, int n_rows, int rows_per_tile, int64_t n_entries,
                            void* table, hipStream_t stream);
// The plan builds the tile table in `table`; the gate/up phase reads it and writes h; the down
// phase reads both.
hipError_t launch_ffn_plan(int T, int k_total, int n_experts, int opts, const int32_t* offsets, void* table,
                           hipStream_t stream);
hipError_t launch_ffn_gateup(const void* x, int T, int k_total, int fmt, int n_experts, int opts, int H, int I,
                             ProjDev gate, ProjDev up, const int32_t* sorted_slot, uint16_t* h_hi, uint16_t* h_lo,
                             const void* table, hipStream_t stream);
hipError_t launch_ffn_down(int T, int k_total, int fmt, int n_experts, int opts, int H, int I, ProjDev down,
                           const int32_t* sorted_slot, float* y_slots, const uint16_t* h_hi, const uint16_t* h_lo,
                           const void* table, hipStream_t stream);

// The range-managed FFN (Cascadia Sec. 3.3, Eq. 1): builds its own tile table (non-tile plan) in
// `table`, runs the general kernels with u attenuated by 2^-att_log2 and h rounded to binary16,
// and writes binary16 outputs to y16.
hipError_t launch_ffn_range(const void* x, int T, int k_total, int fmt, int n_experts, int H, int I, ProjDev gate,
                            ProjDev up, ProjDev down, const int32_t* offsets, const int32_t* sorted_slot,
                            uint16_t* h_hi, uint16_t* h_lo, void* table, int att_log2, uint16_t* y16,
                            hipStream_t stream);

// ---- expert FFN, MX mode (MXFP4 weights x MX-quantised activations on scaled MFMAs) ----
int mx_bits(int fmt);                                  // 8, 6 or 4 bits per code; 0 for an unknown format
int64_t mx_tiles(int T, int k_total, int n_experts);   // tile-table entries of an MX call
struct MxFfnArgs {
  int fmt;                                   // moe_mx_format
  const void* x;                             // [T][H] bf16
  int T, k_total, n_experts, H, I;
  ProjDev gate, up, down;
  const int32_t* offsets;
  const int32_t* sorted_slot;
  float* y_slots;
  uint8_t *xq, *xs;                          // x codes [T][H/32 blocks], scales [T][H/32]
  uint8_t *hq, *hs;                          // h codes [T*k_total][I/32 blocks], scales
  void* table;                               // tile table
};
// Quantises a contiguous [n_rows][K] bf16/fp16 matrix into packed codes + E8M0 scales.
hipError_t launch_mx_quantize(const void* x, bool x_fp16, int64_t n_rows, int K, int fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream);
// x quantisation, tile table, gate/up (writes h codes), down (writes y_slots).
hipError_t launch_ffn_mx(const MxFfnArgs& a, hipStream_t stream);

// launch_ffn_mx on x codes and scales that the caller has (a.xq, a.xs are read, a.x is not used).
hipError_t launch_ffn_mx_codes(const MxFfnArgs& a, hipStream_t stream);

// ---- residual addition + RMS norm ----
struct NormArgs {
  const void *x, *residual;  // [T] rows at x_stride / r_stride values; residual may be NULL
  const void* weight;        // [H]
  void *residual_out, *y;    // either may be NULL; y rows are H values apart
  uint8_t *codes, *scales;   // mx != 0
  int64_t x_stride, r_stride, ro_stride, code_row;  // code_row: bytes of a packed row
  int x_dt, r_dt, w_dt, y_dt;                       // moe_dtype
  int T, H, mx;                                     // mx: moe_mx_format, 0 for none
  float eps;
  double inv_h;  // 1 / H
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

// ---- products with 4-bit weights ----
struct LinArgs {
  const uint16_t* x;  // [T] rows of K bf16 values, x_stride values apart
  int64_t x_stride;
  int T, N, K, fmt;
  ProjDev w;          // expert strides unused; ts: one value
  const float* bias;  // [N] or NULL
  void* y;
  int y_dt;
  int64_t y_stride;
  void* ws;
};
size_t linear_workspace_bytes(int fmt, int T, int N, int K);
hipError_t launch_linear(const LinArgs& a, hipStream_t stream);

// ---- attention: rotary positions and cache write, prompts, decoding ----
struct FastDiv {  // n / d for n < 2^31 (attention.hpp)
  uint32_t d, mul, shift;
};
struct HeadsDev {  // moe_heads; p NULL: absent
  void* p;
  int64_t ts, hs;
  int dt;
};
struct RopeArgs {
  const float *cos, *sin;     // [n_positions][R / 2]
  const int32_t* positions;   // [T], or NULL (R = 0)
  int n_positions, R, neighbours;
  int T, Hq, Hkv, D, x_dt;
  HeadsDev in[3], out[3];     // q, k, v
  int fmt, n_slots;           // cache: moe_kv_format, pages * page size
  const int32_t* slots;       // [T], or NULL: no cache
  void *cache_k, *cache_v;
  uint8_t *scale_k, *scale_v;
  int64_t c_page, c_head, c_token, s_page, s_head, s_token;
  FastDiv page_size;
  // set by the launch: runs of eight values of a head, heads of a wave, waves of a token's q, of its k (and v), of all
  int runs, rows_per_wave, q_groups, kv_groups;
  FastDiv groups;
};
hipError_t launch_rope(RopeArgs a, hipStream_t stream);

struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* y;
  float* lse;                 // [Tq][Hq] or NULL
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, y_ts, y_hs;
  const int32_t *cu_q, *cu_k;
  int n_seqs, Tq, Tk, Hq, Hkv, D, f16;
  FastDiv G;                  // Hq / Hkv
  float c;                    // scale * log2(e)
  int causal, window;
  void* ws;
  int parts, part_keys;       // set by the launch: workgroups that share a row's keys, and keys of each
};
size_t prompt_workspace_bytes(int Tq, int Tk, int n_seqs, int Hq, int Hkv, int D);
hipError_t launch_prompt(PromptArgs a, hipStream_t stream);

struct DecodeArgs {
  const uint16_t* q;
  uint16_t* y;
  float* lse;                 // [B][Hq] or NULL
  int64_t q_ts, q_hs, y_ts, y_hs;
  int B, Hq, Hkv, D, G;
  const int32_t* table;       // [B] rows of page numbers
  int64_t table_stride;
  const int32_t* lens;
  int max_len, window, n_pages, fmt;
  const void *cache_k, *cache_v;
  const uint8_t *scale_k, *scale_v;
  int64_t c_page, c_head, c_token, s_page, s_head, s_token;
  FastDiv page_size;
  float c;
  void* ws;
  int parts, part_keys;       // set by the launch
};
size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D, int max_len);
hipError_t launch_decode(DecodeArgs a, hipStream_t stream);

// ---- combine ----
hipError_t launch_combine(const float* y_slots, const float* weights, int T, int k_total, int H, float* y,
                          hipStream_t stream);
hipError_t launch_combine_restore(const uint16_t* y16, const float* weights, int T, int k_total, int H, int att_log2,
                                  float* y, hipStream_t stream);

// ---- decode primitive ----
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* scales, int n_rows, int K, int64_t code_stride,
                          int64_t scale_stride, uint16_t* out, hipStream_t stream);

}  // namespace moe
