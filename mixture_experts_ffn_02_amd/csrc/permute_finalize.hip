// Permute (bf16 row gather) and finalize (routing-weighted top-k reduction).
//
// Pages: sglang PR "[LoRA] bf16 MoE-LoRA for trtllm backend ...", Files-changed table
// (permute = bf16 gather of the hidden rows; finalize after the down GEMM); vLLM API
// page "trtllm_lora_moe", _finalize_with_w2_lora (per token, sum over top_k of the
// weighted permuted rows).
//
// Both kernels are HBM-bound row copies: one wavefront moves one 16-byte vector per
// lane per step, so every row is read and written with fully coalesced accesses.
#include "checkpoint.h"
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

// One wavefront per permuted row.
__global__ __launch_bounds__(kRowThreads) void permute_kernel(const uint16_t *__restrict__ x,
                                                              const int32_t *__restrict__ p2e,
                                                              uint16_t *__restrict__ x_perm, int R,
                                                              int H, int K) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int p = (int)block_of_grid() * (kRowThreads / 64) + wave;
  if (p >= R) return;
  const int t = p2e[p] / K;
  const u32x4_t *src = reinterpret_cast<const u32x4_t *>(x + (size_t)t * H);
  u32x4_t *dst = reinterpret_cast<u32x4_t *>(x_perm + (size_t)p * H);
  const int nvec = H / 8;
  for (int v = lane; v < nvec; v += 64) dst[v] = src[v];
}

// One workgroup per token; each thread owns 8 consecutive hidden elements per step.
__global__ __launch_bounds__(kRowThreads) void finalize_kernel(const uint16_t *__restrict__ y,
                                                               const float *__restrict__ w,
                                                               const int32_t *__restrict__ e2p,
                                                               uint16_t *__restrict__ out, int T, int H,
                                                               int K) {
  const int t = (int)block_of_grid();
  if (t >= T) return;
  __shared__ int rows[MOE_LORA_MAX_TOPK];
  __shared__ float wts[MOE_LORA_MAX_TOPK];
  if (threadIdx.x < K) {
    rows[threadIdx.x] = e2p[(size_t)t * K + threadIdx.x];
    wts[threadIdx.x] = w[(size_t)t * K + threadIdx.x];
  }
  __syncthreads();
  const int nvec = H / 8;
  for (int v = threadIdx.x; v < nvec; v += kRowThreads) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < K; ++j) {
      const u32x4_t q = reinterpret_cast<const u32x4_t *>(y + (size_t)rows[j] * H)[v];
      const float wj = wts[j];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[2 * c] += wj * bf16_to_f32(q[c] & 0xffffu);
        acc[2 * c + 1] += wj * bf16_to_f32(q[c] >> 16);
      }
    }
    u32x4_t o;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = pack_bf16x2(acc[2 * c], acc[2 * c + 1]);
    reinterpret_cast<u32x4_t *>(out + (size_t)t * H)[v] = o;
  }
}

// Gradients of finalize: d_y[e2p[t k + j], :] = w[t, j] d_out[t, :] and
// d_w[t, j] = <d_out[t], y[e2p[t k + j]]>.  One workgroup per token; its four wavefronts
// split the k choices, and a wavefront walks the row in 512-wide pieces with the piece of
// d_out in registers for all of its choices (JN of them).  Products and sums in fp32, a
// row's sum in a fixed order.  Bound by HBM: the routed rows are read once (2 bytes a
// value, 1 + 1/32 from a checkpoint) and written once (8192 tokens, top-8, hidden 2048: 121 us
// in bf16, 95 from a checkpoint, 4.7 TB/s; d_y stored past the caches: 121 and 102).
template <int JN, bool CODES>
__global__ __launch_bounds__(kRowThreads) void finalize_backward_kernel(const FinalizeBackwardArgs P) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = (int)block_of_grid(), H = P.H, K = P.K;
  if (t >= P.T) return;
  const int nb = (H + kCkptBlock - 1) / kCkptBlock;
  long long row[JN];
  float w[JN], dot[JN];
  bool on[JN];
#pragma unroll
  for (int i = 0; i < JN; ++i) {
    const int j = wave * JN + i;
    const int p = j < K ? P.e2p[(size_t)t * K + j] : -1;
    on[i] = p >= 0 && p < P.R;  // (a position outside the routed rows takes no part)
    row[i] = on[i] ? p : 0;
    w[i] = on[i] ? P.w[(size_t)t * K + j] : 0.f;
    dot[i] = 0.f;
  }
  for (int h = lane * 8; h < H; h += 512) {
    const u32x4_t d4 = *reinterpret_cast<const u32x4_t *>(P.d_out + (size_t)t * H + h);
    u32x4_t y4[JN];
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      if (!on[i]) continue;
      if constexpr (CODES) {
        const u32x2_t c = *reinterpret_cast<const u32x2_t *>(P.codes + row[i] * H + h);
        y4[i] = ckpt_to_bf16(c, ckpt_scale(P.exps[row[i] * nb + h / kCkptBlock]));
      } else {
        y4[i] = *reinterpret_cast<const u32x4_t *>(P.y + row[i] * H + h);
      }
    }
    float d[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      d[2 * c] = bf16_to_f32(d4[c] & 0xffffu);
      d[2 * c + 1] = bf16_to_f32(d4[c] >> 16);
    }
#pragma unroll
    for (int i = 0; i < JN; ++i) {
      if (!on[i]) continue;
      u32x4_t o;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        dot[i] += d[2 * c] * bf16_to_f32(y4[i][c] & 0xffffu);
        dot[i] += d[2 * c + 1] * bf16_to_f32(y4[i][c] >> 16);
        o[c] = pack_bf16x2(w[i] * d[2 * c], w[i] * d[2 * c + 1]);
      }
      *reinterpret_cast<u32x4_t *>(P.d_y + row[i] * H + h) = o;
    }
  }
#pragma unroll
  for (int i = 0; i < JN; ++i) {
    float v = dot[i];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    const int j = wave * JN + i;
    if (lane == 0 && j < K) P.d_w[(size_t)t * K + j] = v;
  }
}

template <bool CODES>
int launch_fin_bwd(const FinalizeBackwardArgs &a, hipStream_t s) {
  const int per = (a.K + 3) / 4;
  if (per <= 1)
    finalize_backward_kernel<1, CODES><<<grid_of_blocks(a.T), kRowThreads, 0, s>>>(a);
  else if (per <= 2)
    finalize_backward_kernel<2, CODES><<<grid_of_blocks(a.T), kRowThreads, 0, s>>>(a);
  else if (per <= 4)
    finalize_backward_kernel<4, CODES><<<grid_of_blocks(a.T), kRowThreads, 0, s>>>(a);
  else
    finalize_backward_kernel<8, CODES><<<grid_of_blocks(a.T), kRowThreads, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace

int launch_finalize_backward(const FinalizeBackwardArgs &a, hipStream_t s) {
  return a.codes ? launch_fin_bwd<true>(a, s) : launch_fin_bwd<false>(a, s);
}

int launch_permute(const uint16_t *x, const int32_t *p2e, uint16_t *x_perm, int R, int H, int K,
                   hipStream_t s) {
  if (R == 0) return ST_OK;
  const int rows_per_block = kRowThreads / 64;
  permute_kernel<<<grid_of_blocks((R + rows_per_block - 1) / rows_per_block), kRowThreads, 0, s>>>(x, p2e, x_perm, R,
                                                                                                    H, K);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

int launch_finalize(const uint16_t *y_perm, const float *w, const int32_t *e2p, uint16_t *out,
                    int T, int H, int K, hipStream_t s) {
  if (T == 0) return ST_OK;
  finalize_kernel<<<grid_of_blocks(T), kRowThreads, 0, s>>>(y_perm, w, e2p, out, T, H, K);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace moe
