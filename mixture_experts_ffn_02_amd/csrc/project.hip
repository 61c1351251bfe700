// A dense projection with the low-rank adapter of each token's request beside it (gfx950).
//
//   v_t = A_a x_t,   y_t = W x_t + s_a B_a v_t,   a = token_slot[t]
//
// Two launches.  The shrink writes v (fp32, if the caller keeps it) and bf16(s_a v): 16
// tokens and one adapter per workgroup, K split over its wavefronts and joined in LDS.  The
// rounding of s_a v to bf16 feeds the matrix cores and is the expert layer's own (its
// error is 2^-9 of the delta, below the rounding of y).  The product appends the expand to
// its K loop: one step per adapter among the tile's rows and 64 ranks, with the rows of the
// other adapters masked.  Rows keep token order; requests of a prompt are runs of tokens,
// so a tile meets few adapters.
//
// Up to 256 tokens the weights' stream bounds the call: workgroups of 16 or 32 output
// columns, K split over eight wavefronts, no LDS on the way in.  Above, tiles of up to
// 256 x 256 from double-buffered LDS, filled by DMA loads.
#include <type_traits>

#include "project.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------ shrink
// out[t, r] = sum_k x[t, k] m[slot][...] over a 16-token tile, for its j-th, (j + J)-th ...
// distinct adapter.  TR = 0: m is A [S, R, K] (k contiguous, straight into the MFMA);
// TR = 1: m is B [S, K, R] (r contiguous: a wavefront turns 32 x 16 pieces through LDS).
// Stores s * out in bf16, and fp32 out (scaled if TR) where wanted, zeros past the rank.
constexpr int kShrinkWaves = 8;

template <int RT, bool TR>
__global__ __launch_bounds__(kShrinkWaves * 64) void shrink_kernel(const ShrinkArgs P) {
  constexpr int RP = RT * 16 + 1;
  __shared__ float part[kShrinkWaves / 2][16 * RP];
  __shared__ __attribute__((aligned(16))) uint16_t turn[TR ? kShrinkWaves * 32 * 16 * RT : 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * 16;
  const int row = lane & 15, grp = lane >> 4;
  int rank_row;
  const int t_row = t0 + row;
  int slot_row = t_row < P.T ? adapter_of(P.pool, t_row, rank_row) : -1;
  // rows whose adapter no earlier row of the tile has (bits of lanes 0..15)
  bool first = slot_row >= 0;
#pragma unroll
  for (int i = 0; i < 15; ++i) {
    const int o = __builtin_amdgcn_readlane(slot_row, i);
    if (i < row && o == slot_row) first = false;
  }
  uint32_t todo = (uint32_t)(__ballot(first) & 0xffffull);
  const int R = P.pool.R;
  if (blockIdx.y == 0) {  // rows without an adapter
    for (int i = tid; i < 16 * R; i += kShrinkWaves * 64) {
      const int r = i / R, t = t0 + r;
      int rk;
      if (t < P.T && adapter_of(P.pool, t, rk) < 0) {
        P.out_bf16[(size_t)t * R + i % R] = 0;
        if (P.out_f32) P.out_f32[(size_t)t * R + i % R] = 0.f;
      }
    }
  }
  for (int skip = 0; skip < (int)blockIdx.y && todo; ++skip) todo &= todo - 1;
  const uint16_t *xr = P.x + (size_t)min(t_row, P.T - 1) * P.ldx;
  while (todo) {
    const int slot = __builtin_amdgcn_readlane(slot_row, __ffs(todo) - 1);
    for (int skip = 0; skip < (int)gridDim.y && todo; ++skip) todo &= todo - 1;
    const int rank = rank_of(P.pool, slot);
    for (int r0 = 0; r0 < rank; r0 += RT * 16) {
      f32x4_t acc[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const int steps = (P.K + 31) / 32;
      const uint16_t *mp[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if constexpr (TR) {
          mp[i] = P.m + (size_t)slot * P.K * R + min(r0 + i * 16 + (lane & 1) * 8, R - 8);
        } else {
          mp[i] = P.m + ((size_t)slot * R + min(r0 + i * 16 + row, R - 1)) * P.K;
        }
      }
      // G steps' loads in flight together; the last steps one by one, zeros past K
      auto go = [&](int s, auto count, bool masked) {
        constexpr int G = decltype(count)::value;
        u32x4_t xf[G], mf[G][RT];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int k = (s + g * kShrinkWaves) * 32 + grp * 8;
          const bool in = !masked || k < P.K;
          xf[g] = in ? *reinterpret_cast<const u32x4_t *>(xr + k) : zero_u32x4();
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            if constexpr (TR) {
              const int n = (s + g * kShrinkWaves) * 32 + (lane >> 1);
              mf[g][i] = !masked || n < P.K ? *reinterpret_cast<const u32x4_t *>(mp[i] + (size_t)n * R) : zero_u32x4();
            } else {
              mf[g][i] = in ? *reinterpret_cast<const u32x4_t *>(mp[i] + k) : zero_u32x4();
            }
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if constexpr (TR) {
            // [32][16] pieces of this wavefront, written and read back transposed (LDS
            // operations of one wavefront complete in order)
            uint16_t *tw = turn + wave * (32 * 16 * RT);
#pragma unroll
            for (int i = 0; i < RT; ++i)
              *reinterpret_cast<u32x4_t *>(tw + i * 512 + (lane >> 1) * 16 + (lane & 1) * 8) = mf[g][i];
            wave_lds_fence();
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const uint16_t *p = tw + i * 512 + (grp * 8 + (row >> 2)) * 16 + 4 * (row & 3);
              const u32x2_t lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * 16);
              mf[g][i] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
            }
            wave_lds_fence();
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i] = mfma_16x16x32(xf[g], mf[g][i], acc[i]);
        }
      };
      constexpr int G = RT <= 2 ? 4 : 2;
      int s = wave;
      for (; (s + (G - 1) * kShrinkWaves + 1) * 32 <= P.K; s += G * kShrinkWaves)
        go(s, std::integral_constant<int, G>{}, false);
      for (; s < steps; s += kShrinkWaves) go(s, std::integral_constant<int, 1>{}, true);
      // join the wavefronts' sums, halving their number each time (a fixed order)
#pragma unroll
      for (int half = kShrinkWaves / 2; half >= 1; half >>= 1) {
        __syncthreads();
        if (wave >= half && wave < 2 * half)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) part[wave - half][(grp * 4 + q) * RP + i * 16 + row] = acc[i][q];
        __syncthreads();
        if (wave < half)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] += part[wave][(grp * 4 + q) * RP + i * 16 + row];
      }
      if (wave == 0) {
        const float scale = P.pool.scaling[slot];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int tr = grp * 4 + q, t = t0 + tr;
          if (__shfl(slot_row, tr) != slot || t >= P.T) continue;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const int r = r0 + i * 16 + row;
            if (r >= R) continue;
            const float v = r < rank ? acc[i][q] : 0.f;
            P.out_bf16[(size_t)t * R + r] = (uint16_t)f32_to_bf16(scale * v);
            if (P.out_f32) P.out_f32[(size_t)t * R + r] = TR ? scale * v : v;
          }
        }
      }
    }
    // ranks past the last chunk that the loop above wrote
    if (wave == 0) {
      const int done = (rank + RT * 16 - 1) / (RT * 16) * (RT * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int tr = grp * 4 + q, t = t0 + tr;
        if (__shfl(slot_row, tr) != slot || t >= P.T) continue;
        for (int r = done + row; r < R; r += 16) {
          P.out_bf16[(size_t)t * R + r] = 0;
          if (P.out_f32) P.out_f32[(size_t)t * R + r] = 0.f;
        }
      }
    }
  }
}

// ------------------------------------------------------------------------ few tokens
// y tile of 16 FM tokens x 16 FN columns; eight wavefronts split K (32-wide steps in turn)
// and the tile's adapters, and join in LDS.
constexpr int kFewWaves = 8;

template <int FM, int FN>
__global__ __launch_bounds__(kFewWaves * 64) void project_few_kernel(const ProjectArgs P) {
  constexpr int BM = FM * 16, BN = FN * 16, NT = kFewWaves * 64;
  constexpr int PITCH = BN + 4;
  __shared__ __attribute__((aligned(16))) float red[kFewWaves * BM * PITCH];
  __shared__ int s_slot[BM], s_list[BM];
  __shared__ uint32_t s_bits[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int n0 = blockIdx.x * BN, t0 = blockIdx.y * BM;
  const PoolView &pool = P.pool;
  const int K = P.K, N = P.N;
  const uint16_t *wp[FN], *xp[FM];
#pragma unroll
  for (int j = 0; j < FN; ++j) wp[j] = P.w + (size_t)min(n0 + j * 16 + row, N - 1) * K + grp * 8;
#pragma unroll
  for (int i = 0; i < FM; ++i) xp[i] = P.x + (size_t)min(t0 + i * 16 + row, P.T - 1) * P.ldx + grp * 8;
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // G steps' loads in flight together; the last steps one by one, zeros past K
  auto go = [&](int s, auto count, bool masked) {
    constexpr int G = decltype(count)::value;
    u32x4_t wf[G][FN], xf[G][FM];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int k = (s + g * kFewWaves) * 32;
      const bool in = !masked || k + grp * 8 < K;
#pragma unroll
      for (int j = 0; j < FN; ++j) wf[g][j] = in ? *reinterpret_cast<const u32x4_t *>(wp[j] + k) : zero_u32x4();
#pragma unroll
      for (int i = 0; i < FM; ++i) xf[g][i] = in ? *reinterpret_cast<const u32x4_t *>(xp[i] + k) : zero_u32x4();
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma_16x16x32(wf[g][j], xf[g][i], acc[i][j]);
  };
  constexpr int G = 4;
  int s = wave;
  for (; (s + (G - 1) * kFewWaves + 1) * 32 <= K; s += G * kFewWaves) go(s, std::integral_constant<int, G>{}, false);
  for (; s * 32 < K; s += kFewWaves) go(s, std::integral_constant<int, 1>{}, true);

  const int n_list = tile_adapters<BM, NT>(pool, t0, P.T, s_slot, s_list, s_bits);
  int slot_row[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) slot_row[i] = s_slot[i * 16 + row];
  for (int q = wave; q < n_list; q += kFewWaves) {
    const int slot = __builtin_amdgcn_readfirstlane(s_list[q]);
    const int rank = rank_of(pool, slot);
    for (int r0 = 0; r0 < rank; r0 += 32) {
      const int r = r0 + grp * 8;
      u32x4_t bf[FN], vf[FM];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        bf[j] = zero_u32x4();
        const int n = min(n0 + j * 16 + row, N - 1);
        if (r < rank) bf[j] = *reinterpret_cast<const u32x4_t *>(P.ext_b + ((size_t)slot * N + n) * pool.R + r);
        // ranks past the slot's inside its last 8 (whatever the pool holds there)
        if (r < rank && r + 8 > rank)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (r + 2 * c >= rank) bf[j][c] = 0u;
            else if (r + 2 * c + 1 >= rank) bf[j][c] &= 0xffffu;
          }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        vf[i] = zero_u32x4();
        if (r < rank && slot_row[i] == slot)
          vf[i] = *reinterpret_cast<const u32x4_t *>(P.ext_a + (size_t)(t0 + i * 16 + row) * pool.R + r);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          // (the column of a lane is one token: other requests' tokens take nothing, whatever
          // this adapter holds)
          const f32x4_t d = mfma_16x16x32(bf[j], vf[i], acc[i][j]);
          if (slot_row[i] == slot) acc[i][j] = d;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4_t *>(&red[(wave * BM + i * 16 + row) * PITCH + j * 16 + grp * 4]) = acc[i][j];
  __syncthreads();
  for (int c = tid; c < BM * BN / 4; c += NT) {
    const int t = c / (BN / 4), n = (c % (BN / 4)) * 4;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += *reinterpret_cast<const f32x4_t *>(&red[(w * BM + t) * PITCH + n]);
    if (t0 + t < P.T && n0 + n < N)
      *reinterpret_cast<u32x2_t *>(P.y + (size_t)(t0 + t) * P.ldy + n0 + n) =
          u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// ------------------------------------------------------------------------ many tokens
// One BM x BN tile per workgroup, 64-wide K steps double-buffered in LDS, both operands by
// DMA loads one step ahead (rows of x and W past the matrix repeat its last row, chunks
// past K read zeros).  The expand's steps follow in the same pipeline.
//   NN = 0: w [N, K], ext_b [S, N, R] (reduction contiguous)
//   NN = 1: w [K, N], ext_b [S, R, N] (reduction by rows: operands read transposed from LDS)
// LDS: rows of 64 bf16 in eight 16-byte chunks XOR-swizzled by the row (A, and B when
// NN = 0); for NN = 1 B's rows are BN values whose 32-byte pairs are swizzled by the row
// bits that the lanes of a transposed read differ in.  The DMA writes LDS in lane order, so
// the swizzle picks the source chunk of each lane.
template <int BM, int BN, int WM, int WN, bool NN>
__global__ __launch_bounds__(WM *WN * 64, 2) void project_tile_kernel(const ProjectArgs P) {
  constexpr int NT = WM * WN * 64;
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  constexpr int A_IT = BM * 8 / NT, B_IT = BN * 8 / NT;
  constexpr int BCH = BN / 8;  // chunks per row of B (NN)
  constexpr int SWZ = BN / 16 < 8 ? BN / 16 - 1 : 7;  // its pairs' swizzle stays inside a row
  __shared__ __attribute__((aligned(16))) uint16_t As[2][BM * 64];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[2][BN * 64];
  __shared__ int s_slot[BM], s_list[BM];
  __shared__ uint32_t s_bits[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int row = lane & 15, grp = lane >> 4;

  // tile of this block: blocks are dealt to the XCDs in turn, so each XCD gets a contiguous
  // share, walked in groups of 8 row tiles (their rows and the columns' weights meet in
  // that XCD's L2)
  const int tiles_m = (P.T + BM - 1) / BM, tiles_n = (P.N + BN - 1) / BN;
  const int total = tiles_m * tiles_n, share = (total + 7) >> 3;
  const int L = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= share || L >= total) return;
  const int g8 = L / (8 * tiles_n), in_g = L - g8 * 8 * tiles_n;
  const int gm = min(8, tiles_m - g8 * 8);
  const int t0 = (g8 * 8 + in_g % gm) * BM, n0 = (in_g / gm) * BN;
  const int K = P.K, N = P.N;
  const PoolView &pool = P.pool;

  // byte offsets of this thread's chunks from the step's base addresses
  uint32_t a_off[A_IT], b_off[B_IT];
  int a_k[A_IT], b_k[B_IT];  // reduction index of the chunk inside a step (NN: of its row)
#pragma unroll
  for (int i = 0; i < A_IT; ++i) {
    const int q = i * NT + tid, r = q >> 3, c = (q & 7) ^ (r & 7);
    a_k[i] = c * 8;
    a_off[i] = ((uint32_t)min(r, P.T - 1 - t0) * (uint32_t)P.ldx + c * 8) * 2u;
  }
#pragma unroll
  for (int i = 0; i < B_IT; ++i) {
    const int q = i * NT + tid;
    if constexpr (!NN) {
      const int r = q >> 3, c = (q & 7) ^ (r & 7);
      b_k[i] = c * 8;
      b_off[i] = ((uint32_t)min(r, N - 1 - n0) * (uint32_t)K + c * 8) * 2u;
    } else {
      const int r = q / BCH, c = (q % BCH) ^ ((((r & 3) | ((r >> 1) & 4)) & SWZ) << 1);
      b_k[i] = r;
      b_off[i] = ((uint32_t)r * (uint32_t)N + (uint32_t)min(c * 8, N - 8 - n0)) * 2u;
    }
  }
  const uint16_t *a_base = P.x + (size_t)t0 * P.ldx;
  const uint16_t *b_base = NN ? P.w + n0 : P.w + (size_t)n0 * K;
  const uint32_t a_lds[2] = {lds_byte(&As[0][0]) + wave * 1024, lds_byte(&As[1][0]) + wave * 1024};
  const uint32_t b_lds[2] = {lds_byte(&Bs[0][0]) + wave * 1024, lds_byte(&Bs[1][0]) + wave * 1024};

  auto issue_full = [&](int buf, int k0) {
    const uint16_t *ab = a_base + k0;
    const uint16_t *bb = NN ? b_base + (size_t)k0 * N : b_base + k0;
#pragma unroll
    for (int i = 0; i < A_IT; ++i) dma16(ab, a_off[i], a_lds[buf] + i * NT * 16);
#pragma unroll
    for (int i = 0; i < B_IT; ++i) dma16(bb, b_off[i], b_lds[buf] + i * NT * 16);
  };
  auto issue_tail = [&](int buf, int k0) {  // chunks past K are zeros
    const char *ab = reinterpret_cast<const char *>(a_base + k0);
    const char *bb = reinterpret_cast<const char *>(NN ? b_base + (size_t)k0 * N : b_base + k0);
#pragma unroll
    for (int i = 0; i < A_IT; ++i)
      dma16(k0 + a_k[i] < K ? ab + a_off[i] : reinterpret_cast<const char *>(kZeroChunk), a_lds[buf] + i * NT * 16);
#pragma unroll
    for (int i = 0; i < B_IT; ++i)
      dma16(k0 + b_k[i] < K ? bb + b_off[i] : reinterpret_cast<const char *>(kZeroChunk), b_lds[buf] + i * NT * 16);
  };
  // ranks [r0, r0 + 64) of one adapter
  auto issue_ext = [&](int buf, int slot, int r0, int rank) {
    const char *z = reinterpret_cast<const char *>(kZeroChunk);
#pragma unroll
    for (int i = 0; i < A_IT; ++i) {
      const int r = (i * NT + tid) >> 3;
      const bool on = r0 + a_k[i] < rank && s_slot[r] == slot;
      dma16(on ? reinterpret_cast<const char *>(P.ext_a + (size_t)(t0 + r) * pool.R + r0 + a_k[i]) : z,
            a_lds[buf] + i * NT * 16);
    }
#pragma unroll
    for (int i = 0; i < B_IT; ++i) {
      const char *src = z;
      if constexpr (!NN) {
        const int n = n0 + ((i * NT + tid) >> 3);
        if (r0 + b_k[i] < rank && n < N)
          src = reinterpret_cast<const char *>(P.ext_b + ((size_t)slot * N + n) * pool.R + r0 + b_k[i]);
      } else {
        const int q = i * NT + tid, c = (q % BCH) ^ ((((b_k[i] & 3) | ((b_k[i] >> 1) & 4)) & SWZ) << 1);
        if (r0 + b_k[i] < rank && n0 + c * 8 < N)
          src = reinterpret_cast<const char *>(P.ext_b + ((size_t)slot * pool.R + r0 + b_k[i]) * N + n0 + c * 8);
      }
      dma16(src, b_lds[buf] + i * NT * 16);
    }
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  int a_frag[2], b_frag[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    a_frag[kk] = row * 64 + (((kk * 4 + grp) ^ (row & 7)) << 3);
    b_frag[kk] = a_frag[kk];
  }
  // NN: lane's row of a transposed read is 32 kk + 8 grp + row / 4 (+ 4), whose swizzle is
  // (row / 4) | 4 (grp & 1); columns 4 (row % 4) of a 16-wide piece (one 32-byte pair)
  const int tr_row = grp * 8 + (row >> 2), tr_swz = ((row >> 2) | ((grp & 1) << 2)) & SWZ;

  auto fragments = [&](int buf, int kk, u32x4_t(&af)[FM], u32x4_t(&bf)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      af[i] = *reinterpret_cast<const u32x4_t *>(&As[buf][(wm * WTM + i * 16) * 64 + a_frag[kk]]);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (!NN) {
        bf[j] = *reinterpret_cast<const u32x4_t *>(&Bs[buf][(wn * WTN + j * 16) * 64 + b_frag[kk]]);
      } else {
        const int pair = (wn * WTN) / 16 + j;
        const uint16_t *p = &Bs[buf][(kk * 32 + tr_row) * BN + ((pair ^ tr_swz) << 4) + 4 * (row & 3)];
        const u32x2_t lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * BN);
        bf[j] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  };

  const int steps = (K + 63) / 64;
  if (steps == 1 && K < 64)
    issue_tail(0, 0);
  else
    issue_full(0, 0);
  const int n_list = tile_adapters<BM, NT>(pool, t0, P.T, s_slot, s_list, s_bits);
  const int chunks = (pool.R + 63) / 64;  // 64-rank chunks per adapter
  const int exts = n_list * chunks;
  auto ext_of = [&](int e, int &slot, int &r0, int &rank) {
    slot = __builtin_amdgcn_readfirstlane(s_list[e / chunks]);
    r0 = (e % chunks) * 64;
    rank = rank_of(pool, slot);
  };
  auto main_step = [&](int buf, int s) {
    dma_wait_all();
    __syncthreads();  // step s has landed, and every wavefront has left step s - 1
    if ((s + 2) * 64 <= K) {
      issue_full(buf ^ 1, (s + 1) * 64);
    } else if (s + 1 < steps) {
      issue_tail(buf ^ 1, (s + 1) * 64);
    } else if (exts > 0) {
      int slot, r0, rank;
      ext_of(0, slot, r0, rank);
      issue_ext(buf ^ 1, slot, r0, rank);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4_t af[FM], bf[FN];
      fragments(buf, kk, af, bf);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma_16x16x32(bf[j], af[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int s = 0; s < steps; s += 2) {
    main_step(0, s);
    if (s + 1 < steps) main_step(1, s + 1);
  }
  for (int e = 0; e < exts; ++e) {
    const int buf = (steps + e) & 1;
    int slot, r0, rank;
    ext_of(e, slot, r0, rank);
    const int left = rank - r0;
    dma_wait_all();
    __syncthreads();
    if (e + 1 < exts) {
      int slot2, r02, rank2;
      ext_of(e + 1, slot2, r02, rank2);
      issue_ext(buf ^ 1, slot2, r02, rank2);
    }
    if (!NN && left > 0 && left < 64 && (left & 7) != 0) {
      // ranks past the slot's inside its last 8: zeros, whatever the pool holds there
      for (int n = tid; n < BN; n += NT) {
        uint16_t *p = &Bs[buf][n * 64 + (((left >> 3) ^ (n & 7)) << 3)];
        for (int c = left & 7; c < 8; ++c) p[c] = 0;
      }
      __syncthreads();
    }
    for (int kk = 0; kk < 2 && kk * 32 < left; ++kk) {
      u32x4_t af[FM], bf[FN];
      fragments(buf, kk, af, bf);
      // a lane's column is one token: those of other requests take nothing from this
      // adapter, whatever it holds
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const bool mine = s_slot[wm * WTM + i * 16 + row] == slot;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const f32x4_t d = mfma_16x16x32(bf[j], af[i], acc[i][j]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = mine ? d[q] : acc[i][j][q];
        }
        __builtin_amdgcn_sched_barrier(0);  // (a row of tiles at a time: few temporaries)
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int t = t0 + wm * WTM + i * 16 + row;
    if (t >= P.T) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + wn * WTN + j * 16 + grp * 4;
      if (n < N)
        *reinterpret_cast<u32x2_t *>(P.y + (size_t)t * P.ldy + n) =
            u32x2_t{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
    }
  }
}

int ok() { return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP; }

constexpr int kFewTokens = 256;

template <bool TR>
int launch_shrink(const ShrinkArgs &a, hipStream_t s) {
  // a decode-sized batch takes a workgroup per (tile, adapter): up to 16 adapters meet in a
  // tile of 16 requests; in longer batches a tile's few adapters follow each other
  const dim3 grid((a.T + 15) / 16, a.T <= 1024 ? 16 : 1);
  if (a.pool.R <= 16)
    shrink_kernel<1, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  else if (a.pool.R <= 32)
    shrink_kernel<2, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  else
    shrink_kernel<4, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  return ok();
}

template <int FN>
int launch_few(const ProjectArgs &a, hipStream_t s) {
  const int fm = a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4;
  const dim3 grid((a.N + FN * 16 - 1) / (FN * 16), (a.T + fm * 16 - 1) / (fm * 16));
  if (fm == 1)
    project_few_kernel<1, FN><<<grid, kFewWaves * 64, 0, s>>>(a);
  else if (fm == 2)
    project_few_kernel<2, FN><<<grid, kFewWaves * 64, 0, s>>>(a);
  else
    project_few_kernel<4, FN><<<grid, kFewWaves * 64, 0, s>>>(a);
  return ok();
}

template <int BM, int BN, int WM, int WN, bool NN>
int launch_tiles(const ProjectArgs &a, hipStream_t s) {
  const int total = ((a.T + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  project_tile_kernel<BM, BN, WM, WN, NN><<<((total + 7) >> 3) * 8, WM * WN * 64, 0, s>>>(a);
  return ok();
}

template <bool NN>
int launch_product(const ProjectArgs &a, hipStream_t s) {
  auto tiles = [&](int b) { return (long long)((a.T + b - 1) / b) * ((a.N + b - 1) / b); };
  if (tiles(256) >= 192) return launch_tiles<256, 256, 2, 4, NN>(a, s);
  if (tiles(128) >= 160) return launch_tiles<128, 128, 2, 2, NN>(a, s);
  return launch_tiles<64, 64, 2, 2, NN>(a, s);
}

}  // namespace

int launch_shrink_transposed(const ShrinkArgs &a, hipStream_t s) { return launch_shrink<true>(a, s); }
int launch_product_transposed(const ProjectArgs &a, hipStream_t s) { return launch_product<true>(a, s); }

size_t project_workspace_bytes(int T, int R) { return ((size_t)T * R * 2 + 255) & ~(size_t)255; }

int launch_project(const ProjectArgs &a, float *v, hipStream_t s) {
  if (a.pool.S > 0) {
    const ShrinkArgs sh{a.x, a.ldx, a.T, a.K, a.a_or_b, a.pool, const_cast<uint16_t *>(a.ext_a), v};
    const int st = launch_shrink<false>(sh, s);
    if (st != ST_OK) return st;
  }
  if (a.T <= kFewTokens)
    return (a.N + 31) / 32 >= 96 ? launch_few<2>(a, s) : launch_few<1>(a, s);
  return launch_product<false>(a, s);
}

}  // namespace moe
