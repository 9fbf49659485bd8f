// Host-side interface between the C ABI (gdn_api.cpp) and the kernel
// launchers (*.hip).  Arguments here have already been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

struct ConvParams {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  void* conv_state;
  const int32_t* cu_seqlens;  // nullptr: one sequence
  int64_t total_tokens;
  int32_t n_seqs;
  int32_t channels;
  int32_t width;
  int32_t act;
  int32_t* conv_head;  // [n_seqs] ring heads of conv_state, or null (chronological)
};
hipError_t launch_conv1d(const ConvParams& p, int dtype, hipStream_t stream);

struct DecodeParams {
  const void* x;
  const void* conv_weight;  // nullptr: x already holds q|k|v
  const void* conv_bias;
  void* conv_state;
  const float* g;
  const float* beta;
  void* state;
  void* o;
  int32_t n_seqs;
  int32_t h_qk;
  int32_t h_v;
  int32_t width;
  int32_t act;
  int32_t l2norm;
  float scale;
  int32_t erase;  // 0: erase-off variant, S_t = a_t S_{t-1} + b_t v_t k_t^T
  const int32_t* state_idx;  // [n_seqs] state and conv-state slots, or null (slot n)
  int32_t* conv_head;        // ring heads of the conv-state pool, or null (chronological)
};
hipError_t launch_decode(const DecodeParams& p, int io_dtype, int state_dtype, int d,
                         hipStream_t stream);

struct PrefillParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const float* g;
  const float* beta;
  const void* initial_state;  // fp32 or bf16 (state_bf16)
  void* final_state;
  void* o;
  const int32_t* cu_seqlens;
  int64_t total_tokens;
  int32_t n_seqs;
  int32_t h_qk;
  int32_t h_v;
  int32_t chunk;
  int32_t l2norm;
  float scale;
  void* workspace;
  size_t workspace_bytes;
  int32_t erase;  // 0: erase-off variant (A = 0, U = diag(beta) V)
  int32_t emit_every;        // > 0: the state after every emit_every-th whole chunk
  void* chunk_states;        // [rows, h_v, d_v, d_k] (rows from the plan)
  const int32_t* state_idx;  // [n_seqs] state slots, or null (slot n)
  int32_t state_bf16;        // initial/final/chunk states stored as bf16 (else fp32)
};
// Workspace of gdn_prefill: chunk offsets plus, per (chunk, V head), the
// chunk operands Tb, P and four per-token scalar rows.
size_t prefill_workspace_bytes(int io_dtype, int64_t total_tokens, int n_seqs, int h_v, int d, int chunk,
                               int emit_every);
bool prefill_supported(int io_dtype, int d, int chunk);
hipError_t launch_prefill(const PrefillParams& p, int io_dtype, int d, hipStream_t stream);
// bf16 io at chunk 32 or 64 with n_seqs <= kNoAllocMaxSeqs: the fused kernel
// with its plan arrays in a static per-device array (p.workspace ignored)
constexpr int kNoAllocMaxSeqs = 8192;
hipError_t launch_prefill_noalloc(const PrefillParams& p, int d, hipStream_t stream);

struct PrefillBwdParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const float* g;
  const float* beta;
  const float* initial_state;
  const int32_t* cu_seqlens;
  const void* d_o;
  const float* d_final_state;
  void* dq;
  void* dk;
  void* dv;
  int64_t dq_stride;
  int64_t dk_stride;
  int64_t dv_stride;
  float* dg;
  float* dbeta;
  float* d_initial_state;
  int64_t total_tokens;
  int32_t n_seqs;
  int32_t h_qk;
  int32_t h_v;
  int32_t chunk;
  int32_t l2norm;
  int32_t erase;
  float scale;
  void* workspace;
};
// Workspace of gdn_prefill_backward: every chunk's intermediates, or, for one
// sequence past the budget (2 GiB; GDN_BWD_BUDGET_MB), one window's plus the
// window-start states
size_t prefill_backward_workspace_bytes(int io_dtype, int64_t total_tokens, int n_seqs, int h_qk, int h_v, int d,
                                        int chunk);
hipError_t launch_prefill_backward(const PrefillBwdParams& p, int io_dtype, int d, hipStream_t stream);

struct ConvBwdParams {
  const void* x;
  const void* weight;
  const void* bias;
  const void* conv_state;
  const int32_t* cu_seqlens;
  const void* dy;
  const float* d_new_state;
  void* dx;
  float* dweight;
  float* dbias;
  float* d_conv_state;
  int64_t total_tokens;
  int32_t n_seqs;
  int32_t channels;
  int32_t width;
  int32_t act;
  void* workspace;
};
size_t conv1d_backward_workspace_bytes(int64_t total_tokens, int channels);
hipError_t launch_conv1d_backward(const ConvBwdParams& p, int dtype, hipStream_t stream);

struct NormParams {
  const void* x;
  const void* weight;  // [width] or null
  const void* gate;
  const void* residual;
  void* y;
  void* sum;  // the pre order's residual + scale x
  int64_t x_stride;
  int64_t gate_stride;
  int64_t residual_stride;
  int64_t y_stride;
  int64_t sum_stride;
  int64_t rows;  // tokens * heads, < 2^31
  int32_t heads;
  int32_t width;
  int32_t order;  // 0: norm after the sum, 1: sum after the norm
  int32_t act;    // gate: 1 SiLU, 2 sigmoid
  int32_t weight_bf16;
  float eps;
  float scale;
  float weight_offset;
};
hipError_t launch_norm(const NormParams& p, int dtype, hipStream_t stream);

struct NormBwdParams {
  const void* x;
  const void* weight;
  const void* gate;
  const void* dy;
  const void* d_sum;
  void* dx;
  void* d_residual;
  void* dgate;
  float* dweight;
  int64_t x_stride;
  int64_t gate_stride;
  int64_t dy_stride;
  int64_t d_sum_stride;
  int64_t dx_stride;
  int64_t d_residual_stride;
  int64_t dgate_stride;
  int64_t rows;
  int32_t heads;
  int32_t width;
  int32_t order;
  int32_t act;
  int32_t weight_bf16;
  float eps;
  float scale;
  float weight_offset;
  void* workspace;  // partial dweight rows
};
size_t norm_backward_workspace_bytes(int64_t rows, int width);
hipError_t launch_norm_backward(const NormBwdParams& p, int dtype, hipStream_t stream);

struct RopeParams {
  const void* q;
  const void* k;  // null with h_k = 0
  const void* positions;
  const double* inv_freq;  // [rot / 2]
  void* q_out;
  void* k_out;
  int64_t q_stride;
  int64_t k_stride;
  int64_t q_out_stride;
  int64_t k_out_stride;
  int64_t tokens;
  int32_t pos64;  // positions are int64 (else int32)
  int32_t h_q;
  int32_t h_k;
  int32_t d;
  int32_t rot;
  int32_t half;
  int32_t inverse;
  float mscale;
  int32_t units;  // of a head: set by the launcher
};
hipError_t launch_rope(const RopeParams& p, int dtype, hipStream_t stream);

struct CacheStoreParams {
  const void* k;
  const void* v;
  uint8_t* k_cache;  // [pages, h_kv, page, d]
  uint8_t* v_cache;  // [pages, h_kv, d, page]
  float* k_scale;    // [pages, h_kv]
  float* v_scale;
  const int32_t* page_table;  // [n_seqs, max_pages]
  const int32_t* lens;        // [n_seqs] tokens held before the call
  const int32_t* cu_seqlens;  // or null: tokens / n_seqs new ones for each
  int64_t k_stride;
  int64_t v_stride;
  int64_t tokens;
  int32_t n_seqs;
  int32_t h_kv;
  int32_t d;
  int32_t page;
  int32_t pages;
  int32_t max_pages;
  // set by the launcher: new tokens of a sequence and workgroups for its pages
  int64_t uniform;
  int32_t uniform_slots;
};
hipError_t launch_cache_store(const CacheStoreParams& p, int dtype, hipStream_t stream);

// What decides how a call of gdn_cache_attention is cut up.
struct AttendShape {
  int64_t tokens;
  int32_t n_seqs;
  int32_t h_q;
  int32_t h_kv;
  int32_t d;
  int32_t page;
  int32_t max_pages;
  int32_t ragged;
  int32_t bf16;
  int32_t causal;
  int32_t window;  // 0 (or less): none
};
struct AttendParams {
  const void* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* lens;  // [n_seqs] tokens in the cache, the new ones among them
  const int32_t* cu_seqlens;
  const void* gate;
  void* o;
  float* lse;
  int64_t q_stride;
  int64_t gate_stride;
  int64_t o_stride;
  int64_t tokens;
  int32_t n_seqs;
  int32_t h_q;
  int32_t h_kv;
  int32_t page_shift;
  int32_t pages;
  int32_t max_pages;
  int32_t causal;
  int32_t window;  // 0: none
  float scale_log2;  // scale * log2(e)
  // set by the launcher
  int32_t max_tokens;
  int32_t uniform_tiles;
  int64_t uniform;
  int32_t piece;
  int32_t tile_rows;
  int32_t slots;
  int32_t shares;
  int32_t join_waves;
  float* part_o;    // [pieces, tokens, h_q, d], or [shares + tiles, 16, d]
  float* part_ml;   // a maximum and a sum for each of those rows
  int32_t* places;  // [slots + 1] with shares
};
size_t attend_workspace_bytes(const AttendShape& a);
hipError_t launch_attend(AttendParams p, const AttendShape& a, void* workspace, int dtype, hipStream_t stream);

}  // namespace gdn
