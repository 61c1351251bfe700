// Gradients of the projection with pooled adapters (gfx950), the shared weight frozen:
//
//   u_t = s_a B_a^T dy_t     dx_t = W^T dy_t + A_a^T u_t
//   dA_a = sum_t u_t x_t^T   dB_a = s_a sum_t dy_t v_t^T        (t over the adapter's tokens)
//
// Launches: u (the forward's shrink over B) with the tokens' order by adapter in a workgroup
// of its own beside it, dx (the forward's tiles with transposed weight reads), dA and dB
// together, and their parts' sums where a segment was split.  dA and dB stream x and dy once:
// a wavefront takes 32 tokens x 128 columns as eight rows of 16 bytes per lane, turns the
// 8 x 8 blocks in registers (v_perm), so no LDS is on the way, and multiplies by u or v,
// whose fp32 values enter as three bf16 terms (all of their 24 bits, so the gradients' only
// rounding to 8 bits is their own; the third term: 4096 tokens of four adapters of rank 32 98.8
// -> 99.7 us for the call, of eight of rank 64 116 -> 120).  Sums in fp32; an adapter's tokens are added in a fixed
// order.  Bound by the bytes in flight (4096 tokens, 2048 -> 4096, four adapters of rank 32,
// x in 8 bits: 19-21 us for 42 MB, against 66-70 of dx and 19-21 of u).
#include "checkpoint.h"
#include "project.h"

namespace moe {
namespace {

MOE_DEV uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }

// values of 8 tokens as three bf16 terms, whose sum is the value: the top 8 bits of the 24, the
// next 8, the rest
MOE_DEV void split8(const float (&v)[8], u32x4_t (&t)[3]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float a = v[2 * q], b = v[2 * q + 1];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      t[i][q] = perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
      a -= bf16_to_f32(t[i][q] & 0xffffu);
      b -= bf16_to_f32(t[i][q] >> 16);
    }
  }
}

constexpr int kGradWaves = 8;
constexpr int kGradCols = 128;

// One workgroup: 128 columns of x (dA) or dy (dB), one adapter, RT * 16 ranks, one part of
// the adapter's tokens; its wavefronts take pieces of 32 tokens in turn, each with the next
// piece's rows and the token numbers of the one after it loaded ahead (4096 tokens,
// 2048 -> 4096, rank 32: 1.4 us of the call).
template <int RT, bool FOR_A, bool CODES>
MOE_DEV void adapter_grad_sum(const AdapterGradArgs &P, int c, int r0, int lo, int hi, f32x4_t (&acc)[8][RT]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, grp = lane >> 4;
  const int R = P.pool.R, ld = FOR_A ? P.ldx : P.ldy;
  const float *q = FOR_A ? P.u : P.v;
  const uint16_t *src = FOR_A ? P.x : P.dy;
  const int nb = (P.K + kCkptBlock - 1) / kCkptBlock;
  int p0 = lo + wave * 32, next[8];
  auto tokens = [&](int p) MOE_INLINE {  // (past the end: the first token, its values are cleared)
#pragma unroll
    for (int i = 0; i < 8; ++i) next[i] = P.order[p + grp * 8 + i < hi ? p + grp * 8 + i : lo];
  };
  constexpr bool kCodes = CODES && FOR_A;
  // a piece's rows (codes and exponents where they are a checkpoint) and its u or v
  u32x4_t dn[kCodes ? 1 : 8];
  u32x2_t wn[kCodes ? 8 : 1];
  uint32_t en[kCodes ? 8 : 1];
  float fn[RT][8];
  auto load = [&]() MOE_INLINE {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (kCodes) {
        wn[i] = *reinterpret_cast<const u32x2_t *>(P.codes + (size_t)next[i] * P.K + c);
        en[i] = P.exps[(size_t)next[i] * nb + c / kCkptBlock];
      } else {
        dn[i] = *reinterpret_cast<const u32x4_t *>(src + (size_t)next[i] * ld + c);
      }
    }
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      const int r = min(r0 + k * 16 + row, R - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) fn[k][i] = q[(size_t)next[i] * R + r];
    }
  };
  constexpr int kStep = kGradWaves * 32;
  constexpr bool kAhead = RT <= 2;  // (64 ranks: no registers left)
  if (p0 < hi) {
    tokens(p0);
    if constexpr (kAhead) {
      load();
      tokens(p0 + kStep);
    }
  }
  for (; p0 < hi; p0 += kStep) {
    if constexpr (!kAhead) {
      load();
      tokens(p0 + kStep);
    }
    bool on[8];
    u32x4_t d[8];
    float f[RT][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      on[i] = p0 + grp * 8 + i < hi;
      if constexpr (kCodes)
        d[i] = ckpt_to_bf16(wn[i], ckpt_scale(en[i]));
      else
        d[i] = dn[i];
#pragma unroll
      for (int k = 0; k < RT; ++k) f[k][i] = fn[k][i];
    }
    if constexpr (kAhead) {
      if (p0 + kStep < hi) {
        load();
        tokens(p0 + 2 * kStep);
      }
    }
    // tokens past the segment's end: zeros on both sides
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!on[i]) {
        d[i] = zero_u32x4();
#pragma unroll
        for (int k = 0; k < RT; ++k) f[k][i] = 0.f;
      }
    u32x4_t q3[RT][3];
#pragma unroll
    for (int k = 0; k < RT; ++k) split8(f[k], q3[k]);
    // column j of the lane's 8 x 8 block: its 8 tokens
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x4_t col;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        col[t] = perm(d[2 * t + 1][j >> 1], d[2 * t][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int k = 0; k < RT; ++k)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          acc[j][k] = FOR_A ? mfma_16x16x32(col, q3[k][i], acc[j][k]) : mfma_16x16x32(q3[k][i], col, acc[j][k]);
    }
  }
}

template <int RT, bool CODES>
__global__ __launch_bounds__(kGradWaves * 64) void adapter_grad_kernel(const AdapterGradArgs P) {
  // sums of up to four wavefronts at a time (two, of 64 ranks: LDS)
  constexpr int kJoin = RT <= 2 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) f32x4_t join[kJoin][8 * RT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int R = P.pool.R, chunks = (R + RT * 16 - 1) / (RT * 16);
  const bool for_a = (int)blockIdx.x < P.tiles_a;
  const int c0 = ((int)blockIdx.x - (for_a ? 0 : P.tiles_a)) * kGradCols;
  const int cols = for_a ? P.K : P.N;
  const int slot = blockIdx.y / chunks, r0 = (blockIdx.y % chunks) * (RT * 16);
  const int rank = rank_of(P.pool, slot);
  const int seg0 = P.seg[slot], len = P.seg[slot + 1] - seg0;
  const int each = ((len + P.parts - 1) / P.parts + 31) & ~31;
  const int lo = seg0 + min(len, (int)blockIdx.z * each), hi = seg0 + min(len, ((int)blockIdx.z + 1) * each);
  const int c = min(c0 + row * 8, cols - 8);

  f32x4_t acc[8][RT];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (r0 < rank) {
    if (for_a)
      adapter_grad_sum<RT, true, CODES>(P, c, r0, lo, hi, acc);
    else
      adapter_grad_sum<RT, false, CODES>(P, c, r0, lo, hi, acc);
  }
  // the wavefronts' sums meet in the first one, kJoin of them at a time and then halving
#pragma unroll
  for (int from = kGradWaves - kJoin; from >= kJoin; from -= kJoin) {
    __syncthreads();
    if (wave >= from && wave < from + kJoin)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < RT; ++k) join[wave - from][j * RT + k][lane] = acc[j][k];
    __syncthreads();
    if (wave < kJoin)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < RT; ++k) acc[j][k] += join[wave][j * RT + k][lane];
  }
#pragma unroll
  for (int half = kJoin / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < RT; ++k) join[wave - half][j * RT + k][lane] = acc[j][k];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < RT; ++k) acc[j][k] += join[wave][j * RT + k][lane];
  }
  if (wave != 0) return;
  if (for_a) {
    // lane: rank row; ranks' columns c0 + 8 (4 grp + i) + j are 8 neighbours over j
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      const int r = r0 + k * 16 + row;
      if (r >= R) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int cc = c0 + 8 * (4 * grp + i);
        if (cc >= cols) continue;
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = r < rank ? acc[j][k][i] : 0.f;
        const size_t at = ((size_t)slot * R + r) * P.K + cc;
        if (P.parts > 1) {
          float *w = P.part_a + (size_t)blockIdx.z * P.pool.S * R * P.K + at;
          *reinterpret_cast<f32x4_t *>(w) = f32x4_t{o[0], o[1], o[2], o[3]};
          *reinterpret_cast<f32x4_t *>(w + 4) = f32x4_t{o[4], o[5], o[6], o[7]};
        } else {
          *reinterpret_cast<u32x4_t *>(P.da + at) = u32x4_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                                           pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
        }
      }
    }
  } else {
    // lane: column c0 + 8 row + j; four ranks 4 grp + i
    const float scale = P.pool.scaling[slot];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int nn = c0 + 8 * row + j;
      if (nn >= cols) continue;
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int r = r0 + k * 16 + grp * 4;
        if (r >= R) continue;
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = r + i < rank ? scale * acc[j][k][i] : 0.f;
        const size_t at = ((size_t)slot * P.N + nn) * R + r;
        if (P.parts > 1)
          *reinterpret_cast<f32x4_t *>(P.part_b + (size_t)blockIdx.z * P.pool.S * R * P.N + at) =
              f32x4_t{o[0], o[1], o[2], o[3]};
        else
          *reinterpret_cast<u32x2_t *>(P.db + at) = u32x2_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    }
  }
}

// sums of the parts, in their order, rounded to bf16
__global__ __launch_bounds__(256) void adapter_grad_sum_kernel(const AdapterGradArgs P) {
  const size_t na = P.da ? (size_t)P.pool.S * P.pool.R * P.K : 0, nb = P.db ? (size_t)P.pool.S * P.pool.R * P.N : 0;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < na + nb; i += (size_t)gridDim.x * 1024) {
    const bool a = i < na;
    const size_t at = a ? i : i - na, n = a ? (size_t)P.pool.S * P.pool.R * P.K : (size_t)P.pool.S * P.pool.R * P.N;
    const float *src = (a ? P.part_a : P.part_b) + at;
    f32x4_t v = *reinterpret_cast<const f32x4_t *>(src);
    for (int p = 1; p < P.parts; ++p) v += *reinterpret_cast<const f32x4_t *>(src + p * n);
    *reinterpret_cast<u32x2_t *>((a ? P.da : P.db) + at) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// n (a multiple of 8) 16-bit zeros
__global__ __launch_bounds__(256) void zero16_kernel(u32x4_t *p, size_t n8) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (size_t)gridDim.x * 256) p[i] = zero_u32x4();
}

int ok() { return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP; }

template <bool CODES>
int launch_grad(const AdapterGradArgs &a, int col_tiles, hipStream_t s) {
  const int rt = a.pool.R <= 16 ? 1 : a.pool.R <= 32 ? 2 : 4;
  const dim3 grid(col_tiles, a.pool.S * ((a.pool.R + rt * 16 - 1) / (rt * 16)), a.parts);
  if (rt == 1)
    adapter_grad_kernel<1, CODES><<<grid, kGradWaves * 64, 0, s>>>(a);
  else if (rt == 2)
    adapter_grad_kernel<2, CODES><<<grid, kGradWaves * 64, 0, s>>>(a);
  else
    adapter_grad_kernel<4, CODES><<<grid, kGradWaves * 64, 0, s>>>(a);
  return ok();
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

// Parts an adapter's tokens are cut into, so that few adapters still fill the device: about
// 192 workgroups, at least 256 tokens' worth each (of all tokens), 16 parts at most.
int grad_parts(int T, int K, int N, int S, int R) {
  const int rt = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  const long long wgs = (long long)((K + 127) / 128 + (N + 127) / 128) * S * ((R + rt * 16 - 1) / (rt * 16));
  long long p = (192 + wgs - 1) / wgs;
  const long long most = (T + 255) / 256;
  if (p > most) p = most;
  return (int)(p < 1 ? 1 : p > 16 ? 16 : p);
}

struct Layout {
  size_t ub, u, order, seg, part_a, part_b, total;
  int parts;
};

Layout layout_of(int T, int K, int N, int S, int R) {
  Layout l;
  l.parts = grad_parts(T, K, N, S, R);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += up(n);
    return o;
  };
  l.ub = take((size_t)T * R * 4);
  l.u = take((size_t)T * R * 4);
  l.order = take((size_t)T * 4);
  l.seg = take((size_t)(S + 1) * 4);
  l.part_a = take(l.parts > 1 ? (size_t)l.parts * S * R * K * 4 : 0);
  l.part_b = take(l.parts > 1 ? (size_t)l.parts * S * R * N * 4 : 0);
  l.total = at;
  return l;
}

}  // namespace

int launch_zero16(uint16_t *p, size_t n, hipStream_t s) {
  const size_t blocks = (n / 8 + 255) / 256;
  zero16_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(reinterpret_cast<u32x4_t *>(p), n / 8);
  return ok();
}

size_t project_backward_workspace_bytes(int T, int K, int N, int S, int R) {
  return S > 0 ? layout_of(T, K, N, S, R).total : 0;
}

int launch_project_backward(const ProjectBackwardArgs &a, hipStream_t s) {
  const int S = a.pool.S, R = a.pool.R;
  unsigned char *ws = static_cast<unsigned char *>(a.ws);
  Layout l{};
  if (S > 0) {
    l = layout_of(a.T, a.K, a.N, S, R);
    uint16_t *ub = reinterpret_cast<uint16_t *>(ws + l.ub);
    float *u = reinterpret_cast<float *>(ws + l.u);
    // u over B [S, N, R]: the reduction runs over dy's N columns
    const bool grads = a.da || a.db;
    const ShrinkArgs sh{a.dy, a.ldy, a.T, a.N, a.b, a.pool, ub, u,
                        grads ? reinterpret_cast<int32_t *>(ws + l.order) : nullptr,
                        grads ? reinterpret_cast<int32_t *>(ws + l.seg) : nullptr};
    const int st = launch_shrink_transposed(sh, s);
    if (st != ST_OK) return st;
  }
  if (a.dx) {
    ProjectArgs p{};
    p.x = a.dy;
    p.ldx = a.ldy;
    p.T = a.T;
    p.K = a.N;
    p.N = a.K;
    p.w = a.w;
    p.pool = a.pool;
    p.ext_a = reinterpret_cast<const uint16_t *>(ws + l.ub);
    p.ext_b = a.a;
    p.y = a.dx;
    p.ldy = a.K;
    const int st = launch_product_transposed(p, s);
    if (st != ST_OK) return st;
  }
  if (S == 0 || (!a.da && !a.db)) return ST_OK;
  AdapterGradArgs g{};
  g.x = a.x;
  g.ldx = a.ldx;
  g.codes = a.codes;
  g.exps = a.exps;
  g.dy = a.dy;
  g.ldy = a.ldy;
  g.K = a.K;
  g.N = a.N;
  g.u = reinterpret_cast<const float *>(ws + l.u);
  g.v = a.v;
  g.pool = a.pool;
  g.order = reinterpret_cast<const int32_t *>(ws + l.order);
  g.seg = reinterpret_cast<const int32_t *>(ws + l.seg);
  g.da = a.da;
  g.db = a.db;
  g.part_a = reinterpret_cast<float *>(ws + l.part_a);
  g.part_b = reinterpret_cast<float *>(ws + l.part_b);
  g.parts = l.parts;
  g.tiles_a = a.da ? (a.K + kGradCols - 1) / kGradCols : 0;
  const int col_tiles = g.tiles_a + (a.db ? (a.N + kGradCols - 1) / kGradCols : 0);
  const int st = a.codes ? launch_grad<true>(g, col_tiles, s) : launch_grad<false>(g, col_tiles, s);
  if (st != ST_OK || g.parts == 1) return st;
  const size_t n = (a.da ? (size_t)S * R * a.K : 0) + (a.db ? (size_t)S * R * a.N : 0);
  const size_t blocks = (n / 4 + 255) / 256;
  adapter_grad_sum_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(g);
  return ok();
}

}  // namespace moe
