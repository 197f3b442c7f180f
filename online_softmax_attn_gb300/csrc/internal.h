// internal.h -- launchers between the C-ABI layer (api.cu) and the kernel
// translation units. Arguments are already validated when these are called.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attn.h"

namespace attn {

// Partial-state workspace carve-up: O~ [rows, S, d], m [rows, S], l [rows, S].
struct PartialLayout {
  size_t o_off, m_off, l_off, total;
};

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline PartialLayout partial_layout(long long rows, int num_splits, int d_h) {
  PartialLayout L;
  L.o_off = 0;
  L.m_off = align256(size_t(rows) * num_splits * d_h * sizeof(float));
  L.l_off = L.m_off + align256(size_t(rows) * num_splits * sizeof(float));
  L.total = L.l_off + align256(size_t(rows) * num_splits * sizeof(float));
  return L;
}

// merge.cu -----------------------------------------------------------------
// n_active == nullptr and seq_lens == nullptr: all splits active.
// seq_lens != nullptr: n_active(row) = split_plan(seq_lens[row / heads_per_seq]),
// with the length clamped into [0, max_len] exactly as the decode kernel does.
// fixed_pps as in split_plan_fixed (0: pages per split from num_splits).
// q_rows != nullptr (a mixed batch's cu_seqlens_q): only rows of sequences
// with one query are merged, each written at token q_rows[row / heads_per_seq].
cudaError_t launch_merge(const float* o_part, const float* m_part, const float* l_part,
                         const int32_t* n_active, const int32_t* seq_lens, int heads_per_seq,
                         int page_size, int max_len, int rows, int num_splits, int d_h, void* o, float* lse,
                         attn_dtype_t out_dtype, cudaStream_t stream, int fixed_pps = 0,
                         const int* pps_dev = nullptr, const int32_t* q_rows = nullptr);
unsigned int merge_read_and_clear_error(cudaStream_t stream, cudaError_t* st);
// Pairwise (O, LSE) merge; arguments validated by the caller.
cudaError_t launch_merge_pair(const void* o_a, const float* lse_a, const void* o_b,
                              const float* lse_b, int rows, int d_h, attn_dtype_t in_dtype,
                              void* o, float* lse, attn_dtype_t out_dtype, cudaStream_t stream);

// decode.cu ----------------------------------------------------------------
struct DecodeArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, h, h_kv, d_h, page_size, num_blocks, max_blocks_per_seq, num_splits;
  float scale;
  float* o_part;
  float* m_part;
  float* l_part;
  int fixed_pps = 0;  // > 0: fixed pages per split (split_plan_fixed)
  const int* pps_dev = nullptr;  // non-null: pages per split read from device memory
  // Non-null (a mixed batch's cu_seqlens_q [B + 1]): only rows with one query
  // are decoded, their query and output at token q_rows[b].
  const int32_t* q_rows = nullptr;
};
// One CTA: the batch's split count by splits_rule, as pages per split of the
// longest row, written to *pps_out (adaptive decode).
cudaError_t launch_decode_plan(const int32_t* seq_lens, const int32_t* q_rows, int B, int h_kv,
                               int max_len, int num_sms, int max_splits, int* pps_out,
                               cudaStream_t stream);
cudaError_t launch_decode_split(const DecodeArgs& a, cudaStream_t stream);
unsigned int decode_read_and_clear_error(cudaStream_t stream, cudaError_t* st);
cudaError_t launch_wait_timeout_selftest(uint64_t limit_ns, cudaStream_t stream);
// One CTA: lets the next kernel start, waits delay_ns, copies n int32.
cudaError_t launch_delayed_copy(int32_t* dst, const int32_t* src, int n, uint64_t delay_ns,
                                cudaStream_t stream);

// cache_e4m3.cu --------------------------------------------------------------
// Tokens packed row after row (cu [B + 1]); row b's are the last of its
// seq_lens[b] positions. Strides in elements.
struct CacheTokens {
  void* k;  // [total, h_kv, d_h], read by the write and written by the read
  void* v;
  long long k_tok, k_head, v_tok, v_head;
  attn_dtype_t dtype;
  const int32_t* block_table;
  const int32_t* cu;
  const int32_t* seq_lens;
  int B, total, h_kv, d_h, num_blocks, max_blocks;
  uint8_t* k_codes;  // [num_blocks, h_kv, 16, d_h]
  uint8_t* v_codes;
  uint8_t* k_exp;    // [num_blocks, h_kv, 16]
  uint8_t* v_exp;
};
cudaError_t launch_cache_write(const CacheTokens& a, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheTokens& a, cudaStream_t stream);
unsigned int cache8_read_and_clear_error(cudaStream_t stream, cudaError_t* st);

// decode_runs.cu -------------------------------------------------------------
constexpr int kRunsMaxCtas = 160;  // bounds the workspace; one CTA per SM
constexpr int kRunsUnit = 1;       // weight of a unit beside its pages (decode_runs.cu)
// Plan (int64: weight per CTA, then the rows' weights' prefix sums [B + 1]), then two
// partial states per CTA: O~ [2 * 160, 8, d_h], m and l [2 * 160, 8].
struct RunsLayout {
  size_t o_off, m_off, l_off, total;
};
inline RunsLayout runs_layout(int B, int d_h) {
  RunsLayout L;
  L.o_off = align256((size_t(B) + 2) * sizeof(long long));
  L.m_off = L.o_off + size_t(2 * kRunsMaxCtas) * 8 * d_h * sizeof(float);
  L.l_off = L.m_off + size_t(2 * kRunsMaxCtas) * 8 * sizeof(float);
  L.total = L.l_off + size_t(2 * kRunsMaxCtas) * 8 * sizeof(float);
  return L;
}
struct DecodeRunsArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const uint8_t* k_exp = nullptr;  // 8-bit cache only
  const uint8_t* v_exp = nullptr;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, h, h_kv, d_h, num_blocks, max_blocks;
  float scale;
  long long* plan;
  float* o_part;
  float* m_part;
  float* l_part;
  float* o_row = nullptr;  // bf16 only: states of units that no run border cuts
  float* m_row = nullptr;
  float* l_row = nullptr;
  void* o = nullptr;       // 8-bit cache only
  float* lse = nullptr;
};
cudaError_t launch_decode8(const DecodeRunsArgs& a, cudaStream_t stream);  // and its merge
unsigned int decode_runs_read_and_clear_error(cudaStream_t stream, cudaError_t* st);

// decode_shared.cu -----------------------------------------------------------
// How the prefix's dense products are cut, from the shape alone: nt row tiles
// of 128 (token, head) rows share a CTA's key tiles, n_rb such row blocks per
// KV head, `groups` equal runs of the (KV head, key tile) pairs, each with one
// CTA per row block; at most s_cap groups touch one head's tiles. The CTAs fill
// the least number of waves over the GPU's 152 SMs whose time per key tile is
// within 5% of the best.
struct SharedPlan {
  int nt, n_rb, groups, s_cap;
};
inline SharedPlan shared_plan(int B, int g, int h_kv) {
  constexpr int kSms = 152;
  SharedPlan p;
  const long long rows = static_cast<long long>(B) * g;
  p.nt = rows > 128 ? 2 : 1;
  p.n_rb = static_cast<int>((rows + p.nt * 128 - 1) / (p.nt * 128));
  auto groups_of = [&](int waves) { return waves * kSms / p.n_rb; };
  auto cost = [&](int waves) { return groups_of(waves) ? double(waves) / groups_of(waves) : 1e30; };
  const int most = p.n_rb / kSms + 4;
  double least = cost(1);
  for (int w = 2; w <= most; ++w) least = cost(w) < least ? cost(w) : least;
  int waves = 1;
  while (cost(waves) > 1.05 * least) ++waves;
  p.groups = groups_of(waves);
  p.s_cap = p.groups / h_kv + 2;
  return p;
}
struct SharedLayout {
  size_t row_o, row_m, row_l, pre_o, pre_m, pre_l, total;  // behind runs_layout
};
inline SharedLayout shared_layout(int B, int h, int h_kv, int d_h) {
  const SharedPlan p = shared_plan(B, h / h_kv, h_kv);
  const size_t rows = size_t(B) * h, pre = size_t(h_kv) * p.s_cap * p.n_rb * 256;
  SharedLayout L;
  L.row_o = align256(runs_layout(B, d_h).total);
  L.row_m = L.row_o + align256(rows * d_h * sizeof(float));
  L.row_l = L.row_m + align256(rows * sizeof(float));
  L.pre_o = L.row_l + align256(rows * sizeof(float));
  L.pre_m = L.pre_o + pre * d_h * sizeof(float);
  L.pre_l = L.pre_m + pre * sizeof(float);
  L.total = L.pre_l + pre * sizeof(float);
  return L;
}
struct SharedArgs {
  DecodeRunsArgs own;  // the rows' own pages, and the workspace of their states
  const int32_t* prefix_table;
  const int32_t* prefix_len;
  int max_prefix_blocks;
  float* pre_o;
  float* pre_m;
  float* pre_l;
};
cudaError_t launch_shared(const SharedArgs& a, cudaStream_t stream);
unsigned int shared_read_and_clear_error(cudaStream_t stream, cudaError_t* st);
// Debug builds: the load (0 K, 1 V, 2 V's second) of the key tile that each CTA does
// not request (-1: none); cudaErrorNotSupported in release builds.
cudaError_t shared_set_stall(int key_tile, int what);

// prefill_simt.cu ----------------------------------------------------------
cudaError_t launch_prefill_f32(const float* q, const float* k, const float* v, float* o,
                               float* lse, int T, int h, int h_kv, int d_h, int causal,
                               float scale, cudaStream_t stream);

// prefill_tc.cu --------------------------------------------------------------
// Workspace carve-up: fp16 copy of V [h_kv, T, d_h], then one int flag per
// (KV head, 128-key tile).
struct PrefillLayout {
  size_t v16_off, flags_off, sched_off, total;
};
PrefillLayout prefill_layout(int T, int h_kv, int d_h);
// workspace == nullptr: every key tile takes the exact bf16 P_hi + P_lo path.
cudaError_t launch_prefill_bf16(const void* q, const void* k, const void* v, void* o, float* lse,
                                int T, int h, int h_kv, int d_h, int causal, float scale,
                                void* workspace, cudaStream_t stream);
// Paged, variable-length prefill (arguments validated by the caller).
struct PagedPrefill {
  const void* q;            // [total_q, h, d_h] bf16
  const void* k_cache;      // [num_blocks, 16, h_kv, d_h] bf16
  const void* v_cache;
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* cu_q;         // [B + 1]
  const int32_t* seq_lens;     // [B]
  int32_t* tile_off;           // [B + 1] workspace
  void* v16;                   // fp16 V copy [B, max_tiles * 128, h_kv, d_h] or nullptr
  int32_t* vwide;              // [B, h_kv, max_tiles] V-format flags (with v16)
  int B, total_q, h, h_kv, d_h, num_blocks, max_blocks, max_q_len, causal;
  float scale;
  void* o;                     // [total_q, h, d_h] bf16
  float* lse;                  // [total_q, h] or nullptr
  int decode_rows_apart = 0;   // nonzero: rows of one query get no query tiles
};
cudaError_t launch_prefill_paged(const PagedPrefill& a, cudaStream_t stream);
unsigned int prefill_read_and_clear_error(cudaStream_t stream, cudaError_t* st);
// Debug builds: the key tile each prefill CTA skips loading K for (-1: none);
// cudaErrorNotSupported in release builds.
cudaError_t prefill_set_stall(int key_tile);
// The fp32 SIMT prefill's error word (debug-build index checks only).
unsigned int simt_read_and_clear_error(cudaStream_t stream, cudaError_t* st);

// tensor maps ---------------------------------------------------------------
// Encodes a tiled tensor map through the driver entry point (no libcuda link).
CUresult encode_tensor_map(CUtensorMap* map, CUtensorMapDataType dtype, int rank, void* base,
                           const uint64_t* dims, const uint64_t* strides_bytes,
                           const uint32_t* box, CUtensorMapSwizzle swizzle);

}  // namespace attn
