// Host-side launchers of the gfx950 kernels (internal; the public ABI is include/moe_lora.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_lora.h"

namespace moe {

// ---- routing ------------------------------------------------------------
struct RouteArgs {
  const uint16_t *logits;  // (general routing: bf16 or fp32)
  int T, E, K;
  int method;  // moe_lora_routing
  int n_group, topk_group;
  float rsf;
  const float *bias;
  int32_t *ids;
  float *weights;
  int32_t *offsets;
  int32_t *e2p;
  int32_t *p2e;
  int32_t *hist;  // workspace [num_wg][E]
};
size_t route_workspace_bytes(int T, int E, int K);
int route_max_tokens(int E, int K, bool dsv3);
int launch_route(const RouteArgs &a, hipStream_t s);
int launch_zero_offsets(int32_t *offsets, int E, hipStream_t s);

// ---- general routing (scores, bias, groups) ---------------------------------
struct ScoredArgs {
  int score;  // moe_lora_score
  bool f32;   // fp32 logits (else bf16)
  bool renormalize;
  int group_score;
  float scale;
  const float *bias;
};
struct ScoredBackwardArgs {
  const void *logits;
  const int32_t *ids;
  const float *d_weights;
  void *d_logits;
  int T, E, K;
  int score;
  bool f32, renormalize;
  float scale;
};
bool scored_wide(bool bias, int n_group, int group_score);  // whether keys are scores
size_t scored_workspace_bytes(int T, int E, int K, bool groups, bool wide);
int scored_max_tokens();
// RouteArgs: logits (either type), sizes, groups and outputs; method, rsf and bias unused
int launch_route_scored(const RouteArgs &a, const ScoredArgs &s, hipStream_t st);
int launch_route_scored_backward(const ScoredBackwardArgs &a, hipStream_t s);

// ---- permute / finalize ---------------------------------------------------
int launch_permute(const uint16_t *x, const int32_t *p2e, uint16_t *x_perm, int R, int H, int K,
                   hipStream_t s);
int launch_finalize(const uint16_t *y_perm, const float *w, const int32_t *e2p, uint16_t *out,
                    int T, int H, int K, hipStream_t s);

struct FinalizeBackwardArgs {
  const uint16_t *d_out;  // [T, H]
  const uint16_t *y;      // [R, H], or NULL with the checkpoint
  const uint8_t *codes;   // [R, H]
  const uint8_t *exps;    // [R, ceil(H / 32)]
  const float *w;         // [T, K]
  const int32_t *e2p;     // [T * K]
  uint16_t *d_y;          // [R, H]
  float *d_w;             // [T, K]
  int T, H, K, R;
};
int launch_finalize_backward(const FinalizeBackwardArgs &a, hipStream_t s);

// ---- 8-bit checkpoints ------------------------------------------------------------
int launch_checkpoint_pack(long long rows, int cols, const uint16_t *x, uint8_t *codes, uint8_t *exps, hipStream_t s);
int launch_checkpoint_unpack(long long rows, int cols, const uint8_t *codes, const uint8_t *exps, uint16_t *x,
                             hipStream_t s);

// ---- projection with pooled adapters ------------------------------------------------
struct PoolView {
  int S, R;                   // adapters, ranks held for each
  const int32_t *token_slot;  // [T]
  const int32_t *rank;        // [S]
  const float *scaling;       // [S]
};
struct ShrinkArgs {
  const uint16_t *x;  // [T, K], rows ldx apart
  int ldx, T, K;
  const uint16_t *m;  // A [S, R, K], or B [S, K, R]
  PoolView pool;
  uint16_t *out_terms;  // [T, 2, R]: the first bf16 terms of a token, then the second
  float *out_f32;       // [T, R] or NULL
  // where not NULL: the tokens by adapter [T] and the adapters' first places [S + 1], made by
  // a workgroup of the same launch
  int32_t *order, *seg;
};
struct ProjectArgs {
  const uint16_t *x;  // [T, K], rows ldx apart
  int ldx, T, K, N;
  const uint16_t *w;
  PoolView pool;
  const uint16_t *a_or_b;  // the shrink's matrices
  const uint16_t *ext_a;   // the shrink's terms, [T, 2, R]
  const uint16_t *ext_b;   // the expand's matrices
  uint16_t *y;
  int ldy;
};
size_t project_workspace_bytes(int T, int R);
// the shrink over B [S, K, R] and the product with w [K, N], ext_b [S, R, N]
int launch_shrink_transposed(const ShrinkArgs &a, hipStream_t s);
int launch_product_transposed(const ProjectArgs &a, hipStream_t s);

struct AdapterGradArgs {
  const uint16_t *x;  // [T, K], rows ldx apart, or NULL with the checkpoint
  int ldx;
  const uint8_t *codes, *exps;  // [T, K], [T, ceil(K / 32)]
  const uint16_t *dy;           // [T, N], rows ldy apart
  int ldy, K, N;
  const float *u, *v;  // [T, R]
  PoolView pool;
  const int32_t *order, *seg;
  uint16_t *da, *db;  // [S, R, K], [S, N, R]; either may be NULL
  float *part_a, *part_b;
  int parts, tiles_a;
};
struct ProjectBackwardArgs {
  const uint16_t *x;
  int ldx;
  const uint8_t *codes, *exps;
  const uint16_t *dy;
  int ldy, T, K, N;
  const uint16_t *w, *a, *b;
  PoolView pool;
  const float *v;
  uint16_t *dx, *da, *db;
  void *ws;
};
size_t project_backward_workspace_bytes(int T, int K, int N, int S, int R);
int launch_zero16(uint16_t *p, size_t n, hipStream_t s);
int launch_project_backward(const ProjectBackwardArgs &a, hipStream_t s);
int launch_project(const ProjectArgs &a, float *v, hipStream_t s);

// ---- tile-packed expert weights ---------------------------------------------------
int launch_pack_weights_fp8(const moe_lora_dims &d, const uint8_t *w1, const uint8_t *w2, uint8_t *w1p,
                            uint8_t *w2p, hipStream_t s);
int launch_pack_weights(const moe_lora_dims &d, const uint16_t *w1, const uint16_t *w2, uint16_t *w1p,
                        uint16_t *w2p, hipStream_t s);

// ---- expert FFN (grouped GEMMs + LoRA) -----------------------------------------
// fused_only: the workspace (and the call) leave out the decomposed two-stream path
size_t forward_workspace_size(const moe_lora_dims &d, const moe_lora_adapters *lora, bool fused_only = false);
int launch_forward(const moe_lora_dims &d, const uint16_t *x, const uint16_t *x_perm,
                   const int32_t *offsets, const int32_t *p2e, const uint16_t *w1,
                   const uint16_t *w2, const moe_lora_adapters *lora, uint16_t *y_perm, void *ws,
                   size_t ws_bytes, hipStream_t main, hipStream_t side,
                   const moe_lora_options *opts, const float *w1_scale = nullptr,
                   const float *w2_scale = nullptr, bool fused_only = false);

}  // namespace moe
