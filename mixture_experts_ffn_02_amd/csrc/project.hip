// A dense projection with the low-rank adapter of each token's request beside it (gfx950).
//
//   v_t = A_a x_t,   y_t = W x_t + s_a B_a v_t,   a = token_slot[t]
//
// Two launches.  The shrink writes v (fp32, if the caller keeps it) and s_a v for the matrix
// cores, as two bf16 terms: 16 tokens and one adapter per workgroup, K split over its
// wavefronts and joined in LDS.  The terms hold s_a v to 2^-16 of it, the size of the fp32
// sums' own error; one rounding to bf16 would move y where the delta is not small beside W x.
// The product appends the expand to its K loop: two steps, one for each term, per 64 ranks of
// the adapters among the tile's rows (one step where they come to 32), with the rows of the
// other adapters masked.  Rows keep token order; requests of a prompt are runs of tokens, so a
// tile meets few adapters.
//
// Small calls (a few tokens, or few output tiles) are bound by the weights' stream and
// latency: workgroups of 16 to 64 output columns, K split over eight wavefronts.  Larger ones
// take tiles of up to 256 x 256 from double-buffered LDS, filled by DMA loads.
#include "project.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------ shrink
// out[t, r] = sum_k x[t, k] m[slot][...] over a 16-token tile, for its j-th, (j + J)-th ...
// distinct adapter.  TR = 0: m is A [S, R, K] (k contiguous); TR = 1: m is B [S, K, R] (r
// contiguous: read back transposed from LDS).  Stores the terms of s * out, and fp32 out
// (scaled if TR) where wanted, zeros past the rank.  Each wavefront takes a run of 64-wide K
// steps, G of them in flight, loaded with neighbouring lanes on neighbouring bytes and turned
// into MFMA operands through LDS of its own.
constexpr int kShrinkWaves = 8;

template <int RT, int MT, bool TR>
__global__ __launch_bounds__(kShrinkWaves * 64, 2) void shrink_kernel(const ShrinkArgs P) {
  constexpr int RP = RT * 16 + 1;
  constexpr int G = (RT <= 2 ? 4 : 2) / MT;
  constexpr int ROWS = 16 * MT, XI = 2 * MT;
  constexpr int kStage = kShrinkWaves * (ROWS + RT * 16) * 64 * 2, kPart = kShrinkWaves * ROWS * RP * 4;
  __shared__ __attribute__((aligned(16))) unsigned char smem[kStage > kPart ? kStage : kPart];
  __shared__ int s_slot[ROWS];
  float *part = reinterpret_cast<float *>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (TR && P.order) {  // the first workgroup orders the tokens
    static_assert((kShrinkWaves + 1) * (MOE_LORA_MAX_POOL_SLOTS + 1) * 4 <= sizeof(smem), "order in the stages' LDS");
    if (blockIdx.x == 0) {
      if (blockIdx.y == 0)
        order_tokens<kShrinkWaves * 64>(P.pool, P.T, P.order, P.seg, reinterpret_cast<int *>(smem));
      return;
    }
  }
  const int t0 = ((int)blockIdx.x - (TR && P.order ? 1 : 0)) * ROWS;
  const int row = lane & 15, grp = lane >> 4;
  const int lr = lane >> 3, lc = lane & 7;  // this lane's row of eight, and 16-byte chunk
  const int st_off = lr * 64 + ((lc ^ lr) << 3);
  const int steps = (P.K + 63) / 64, per = (steps + kShrinkWaves - 1) / kShrinkWaves;
  const int s_begin = min(steps, wave * per), s_end = min(steps, s_begin + per);
  const uint16_t *xr[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) xr[i] = P.x + (size_t)min(t0 + i * 8 + lr, P.T - 1) * P.ldx + lc * 8;
  u32x4_t xg[G][XI];
  auto load_x = [&](int g, int s) MOE_INLINE {  // zeros past the run or K
    const bool in = s < s_end && s * 64 + lc * 8 < P.K;
#pragma unroll
    for (int i = 0; i < XI; ++i) xg[g][i] = in ? *reinterpret_cast<const u32x4_t *>(xr[i] + s * 64) : zero_u32x4();
  };
  // the first rows are on their way while the adapters are looked up (64 tokens, 2048 -> 4096:
  // 0.3 us of the call)
#pragma unroll
  for (int g = 0; g < G; ++g) load_x(g, s_begin + g);
  bool fresh = true;  // those loads serve the first adapter
  // lane r < ROWS: row r's adapter; rows whose adapter no earlier row has (bits of those lanes)
  int rank_row = 0;
  const int t_row = t0 + lane;
  const int slot_row = lane < ROWS && t_row < P.T ? adapter_of(P.pool, t_row, rank_row) : -1;
  bool first = slot_row >= 0;
#pragma unroll
  for (int i = 0; i < ROWS - 1; ++i) {
    const int o = __builtin_amdgcn_readlane(slot_row, i);
    if (i < lane && o == slot_row) first = false;
  }
  uint32_t todo = (uint32_t)__ballot(first);
  if (tid < ROWS) s_slot[tid] = slot_row;
  const int R = P.pool.R;
  __syncthreads();
  if (blockIdx.y == 0) {  // rows without an adapter
    for (int i = tid; i < ROWS * R; i += kShrinkWaves * 64) {
      const int r = i / R, t = t0 + r;
      if (t < P.T && s_slot[r] < 0) {
        store_terms(P.out_terms + (size_t)t * 2 * R, R, i % R, 0.f);
        if (P.out_f32) P.out_f32[(size_t)t * R + i % R] = 0.f;
      }
    }
  }
  for (int skip = 0; skip < (int)blockIdx.y && todo; ++skip) todo &= todo - 1;
  uint16_t *stage = reinterpret_cast<uint16_t *>(smem) + wave * (ROWS + RT * 16) * 64;
  uint16_t *stage_m = stage + ROWS * 64;
  while (todo) {
    const int lead = __ffs(todo) - 1, slot = __builtin_amdgcn_readlane(slot_row, lead);
    for (int skip = 0; skip < (int)gridDim.y && todo; ++skip) todo &= todo - 1;
    const int rank = __builtin_amdgcn_readlane(rank_row, lead);
    const float scale = P.pool.scaling[slot];
    for (int r0 = 0; r0 < rank; r0 += RT * 16) {
      f32x4_t acc[MT][RT];
#pragma unroll
      for (int h = 0; h < MT; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[h][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      // TR: a step's rows n, each 2 RT chunks of 8 ranks; else 16 RT rank rows of 8 chunks
      const uint16_t *mp[2 * RT];
      int m_n[2 * RT];
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        const int q = i * 64 + lane;
        m_n[i] = q / (2 * RT);
        if constexpr (TR)
          mp[i] = P.m + ((size_t)slot * P.K + m_n[i]) * R + min(r0 + (q % (2 * RT)) * 8, R - 8);
        else
          mp[i] = P.m + ((size_t)slot * R + min(r0 + i * 8 + lr, R - 1)) * P.K + lc * 8;
      }
      u32x4_t mg[G][2 * RT];
      auto load_m = [&](int g, int s) MOE_INLINE {
        const bool in = s < s_end && s * 64 + lc * 8 < P.K;
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) {
          if constexpr (TR)
            mg[g][i] = s < s_end && s * 64 + m_n[i] < P.K
                           ? *reinterpret_cast<const u32x4_t *>(mp[i] + (size_t)s * 64 * R)
                           : zero_u32x4();
          else
            mg[g][i] = in ? *reinterpret_cast<const u32x4_t *>(mp[i] + s * 64) : zero_u32x4();
        }
      };
      if (!fresh) {
#pragma unroll
        for (int g = 0; g < G; ++g) load_x(g, s_begin + g);
      }
      fresh = false;
#pragma unroll
      for (int g = 0; g < G; ++g) load_m(g, s_begin + g);
      __syncthreads();  // the last round's sums have been read
      for (int s0 = s_begin; s0 < s_end; s0 += G) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (s0 + g >= s_end) break;
#pragma unroll
          for (int i = 0; i < XI; ++i) *reinterpret_cast<u32x4_t *>(stage + i * 512 + st_off) = xg[g][i];
#pragma unroll
          for (int i = 0; i < 2 * RT; ++i)
            *reinterpret_cast<u32x4_t *>(stage_m + i * 512 + (TR ? lane * 8 : st_off)) = mg[g][i];
          if (s0 + g + G < s_end) {
            load_x(g, s0 + g + G);
            load_m(g, s0 + g + G);
          }
          wave_lds_fence();
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int off = row * 64 + (((kk * 4 + grp) ^ (row & 7)) << 3);
            u32x4_t xf[MT];
#pragma unroll
            for (int h = 0; h < MT; ++h) xf[h] = *reinterpret_cast<const u32x4_t *>(stage + h * 16 * 64 + off);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              u32x4_t mf;
              if constexpr (TR) {
                const uint16_t *p = stage_m + (kk * 32 + grp * 8 + (row >> 2)) * (16 * RT) + i * 16 + 4 * (row & 3);
                const u32x2_t lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * 16 * RT);
                mf = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
              } else {
                mf = *reinterpret_cast<const u32x4_t *>(stage_m + i * 16 * 64 + off);
              }
#pragma unroll
              for (int h = 0; h < MT; ++h) acc[h][i] = mfma_16x16x32(xf[h], mf, acc[h][i]);
            }
          }
          wave_lds_fence();
        }
      }
      // join the wavefronts' sums (in their order)
      __syncthreads();
#pragma unroll
      for (int h = 0; h < MT; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) part[(wave * ROWS + h * 16 + grp * 4 + q) * RP + i * 16 + row] = acc[h][i][q];
      __syncthreads();
      for (int c = tid; c < ROWS * RT * 16; c += kShrinkWaves * 64) {
        const int tr = c / (RT * 16), rc = c % (RT * 16), t = t0 + tr, r = r0 + rc;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kShrinkWaves; ++w) v += part[(w * ROWS + tr) * RP + rc];
        if (s_slot[tr] != slot || r >= R) continue;
        if (r >= rank) v = 0.f;
        store_terms(P.out_terms + (size_t)t * 2 * R, R, r, scale * v);
        if (P.out_f32) P.out_f32[(size_t)t * R + r] = TR ? scale * v : v;
      }
    }
    // ranks past the last chunk that the loop above wrote
    const int done = (rank + RT * 16 - 1) / (RT * 16) * (RT * 16);
    if (done < R) {
      for (int c = tid; c < ROWS * (R - done); c += kShrinkWaves * 64) {
        const int tr = c / (R - done), t = t0 + tr, r = done + c % (R - done);
        if (s_slot[tr] != slot) continue;
        store_terms(P.out_terms + (size_t)t * 2 * R, R, r, 0.f);
        if (P.out_f32) P.out_f32[(size_t)t * R + r] = 0.f;
      }
    }
  }
}

// ------------------------------------------------------------------------ few tokens
// y tile of 16 FM tokens x 16 FN columns; W wavefronts split K (a run of 64-wide steps each,
// G of them in flight) and the tile's adapters, and join in LDS.  The first steps' loads are
// out before the tile's adapters are listed, and the first adapters' before the steps'
// products.  Eight neighbouring lanes load 128 contiguous bytes of a row, and each wavefront
// turns its steps into MFMA operands through LDS of its own: loads in the operands' order
// (neighbouring lanes in different rows) take one lane per cycle in the address path and
// bounded the call (64 tokens, 2048 -> 4096, in 64 x 32 tiles without adapters: 13.6 us, 9.8 so).
template <int FM, int FN, int W, int G>
__global__ __launch_bounds__(W * 64) void project_few_kernel(const ProjectArgs P) {
  constexpr int BM = FM * 16, BN = FN * 16, NT = W * 64;
  constexpr int PITCH = BN + 4;
  constexpr int ROWS = BM + BN, IT = ROWS / 8;  // x rows, then w rows
  constexpr int kStage = W * ROWS * 64 * 2, kRed = W * BM * PITCH * 4;
  __shared__ __attribute__((aligned(16))) unsigned char smem[kStage > kRed ? kStage : kRed];
  __shared__ int s_slot[BM], s_list[BM];
  __shared__ uint32_t s_bits[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int n0 = blockIdx.x * BN, t0 = blockIdx.y * BM;
  const PoolView &pool = P.pool;
  const int K = P.K, N = P.N;
  uint16_t *stage = reinterpret_cast<uint16_t *>(smem) + wave * ROWS * 64;
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int steps = (K + 63) / 64, per = (steps + W - 1) / W;
  const int s_begin = min(steps, wave * per), s_end = min(steps, s_begin + per);
  const int lr = lane >> 3, lc = lane & 7;  // this lane's row of eight, and 16-byte chunk
  const uint16_t *src[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = i * 8 + lr;
    src[i] = r < BM ? P.x + (size_t)min(t0 + r, P.T - 1) * P.ldx : P.w + (size_t)min(n0 + r - BM, N - 1) * K;
    src[i] += lc * 8;
  }
  const int st_off = lr * 64 + ((lc ^ lr) << 3);
  u32x4_t rg[G][IT];
  auto load = [&](int g, int s) {  // zeros past the run or K
    const bool in = s < s_end && s * 64 + lc * 8 < K;
#pragma unroll
    for (int i = 0; i < IT; ++i) rg[g][i] = in ? *reinterpret_cast<const u32x4_t *>(src[i] + s * 64) : zero_u32x4();
  };
#pragma unroll
  for (int g = 0; g < G; ++g) load(g, s_begin + g);
  const int n_list = tile_adapters<BM, NT>(pool, t0, P.T, s_slot, s_list, s_bits);

  // the expand: 32 ranks of Q adapters' rows at a time
  constexpr int Q = 2;
  u32x4_t vf[FM][2], bf[Q][FN];
  int slot[Q], rank[Q];
  auto load_v = [&](int r0) {
    const int r = r0 + grp * 8;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        vf[i][h] = r < pool.R ? *reinterpret_cast<const u32x4_t *>(
                                    P.ext_a + ((size_t)min(t0 + i * 16 + row, P.T - 1) * 2 + h) * pool.R + r)
                              : zero_u32x4();
  };
  auto load_b = [&](int r0, int q0) {
    const int r = r0 + grp * 8;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int at = q0 + q * W;
      const int entry = at < n_list ? __builtin_amdgcn_readfirstlane(s_list[at]) : 0;
      slot[q] = list_slot(entry);
      rank[q] = list_rank(entry);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = min(n0 + j * 16 + row, N - 1);
        bf[q][j] = r < rank[q] ? *reinterpret_cast<const u32x4_t *>(P.ext_b + ((size_t)slot[q] * N + n) * pool.R + r)
                               : zero_u32x4();
      }
    }
  };
  if (wave < n_list) {
    load_v(0);
    load_b(0, wave);
  }
  for (int s0 = s_begin; s0 < s_end; s0 += G) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (s0 + g >= s_end) break;
#pragma unroll
      for (int i = 0; i < IT; ++i) *reinterpret_cast<u32x4_t *>(stage + i * 512 + st_off) = rg[g][i];
      if (s0 + g + G < s_end) load(g, s0 + g + G);
      wave_lds_fence();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int off = row * 64 + (((kk * 4 + grp) ^ (row & 7)) << 3);
        u32x4_t wf[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) wf[j] = *reinterpret_cast<const u32x4_t *>(stage + (BM + j * 16) * 64 + off);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const u32x4_t xf = *reinterpret_cast<const u32x4_t *>(stage + i * 16 * 64 + off);
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mfma_16x16x32(wf[j], xf, acc[i][j]);
        }
      }
      wave_lds_fence();
    }
  }
  if (wave < n_list) {
    int slot_row[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) slot_row[i] = s_slot[i * 16 + row];
    for (int r0 = 0; r0 < pool.R; r0 += 32) {
      const int r = r0 + grp * 8;
      if (r0 > 0) load_v(r0);
      for (int q0 = wave; q0 < n_list; q0 += Q * W) {
        if (r0 > 0 || q0 > wave) load_b(r0, q0);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if (r0 >= rank[q]) continue;
          // ranks past the adapter's inside its last 8: zeros, whatever the pool holds there
          if ((rank[q] & 7) != 0 && r < rank[q] && r + 8 > rank[q])
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (r + 2 * c >= rank[q]) bf[q][j][c] = 0u;
                else if (r + 2 * c + 1 >= rank[q]) bf[q][j][c] &= 0xffffu;
              }
          // a lane's column is one token: those of other requests take nothing from this
          // adapter, whatever it holds
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              f32x4_t d = mfma_16x16x32(bf[q][j], vf[i][0], acc[i][j]);
              d = mfma_16x16x32(bf[q][j], vf[i][1], d);
              if (slot_row[i] == slot[q]) acc[i][j] = d;
            }
        }
      }
    }
  }
  float *red = reinterpret_cast<float *>(smem);
  __syncthreads();  // the stages are free
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
    for (int w = 0; w < W; ++w) v += *reinterpret_cast<const f32x4_t *>(&red[(w * BM + t) * PITCH + n]);
    if (t0 + t < P.T && n0 + n < N)
      *reinterpret_cast<u32x2_t *>(P.y + (size_t)(t0 + t) * P.ldy + n0 + n) =
          u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// ------------------------------------------------------------------------ many tokens
// 8 outputs of a token whose adapter may hold what is not finite: NaN where a row (column,
// NN) of the adapter's expand does.  Rare: the tile found such a value.
template <bool NN>
MOE_DEV void restore_odd(const ProjectArgs &P, int slot, int n, u32x4_t &v) {
  if (slot < 0) return;
  const int rank = rank_of(P.pool, slot), R = P.pool.R;
  for (int i = 0; i < 8; ++i) {
    bool odd = false;
    for (int r = 0; r < rank; ++r) {
      const uint16_t b = NN ? P.ext_b[((size_t)slot * R + r) * P.N + n + i] : P.ext_b[((size_t)slot * P.N + n + i) * R + r];
      odd |= (b & 0x7f80u) == 0x7f80u;
    }
    if (odd) v[i >> 1] = (v[i >> 1] & (i & 1 ? 0x0000ffffu : 0xffff0000u)) | (0x7fc0u << (16 * (i & 1)));
  }
}

// One BM x BN tile per workgroup, 64-wide K steps buffered in LDS, both operands by DMA
// loads one step ahead (rows of x and W past the matrix repeat its last row, chunks
// past K read zeros; small tiles three steps ahead).  The expand's steps follow in the same
// pipeline.
//   NN = 0: w [N, K], ext_b [S, N, R] (reduction contiguous)
//   NN = 1: w [K, N], ext_b [S, R, N] (reduction by rows: operands read transposed from LDS)
// LDS: rows of 64 bf16 in eight 16-byte chunks XOR-swizzled by the row (A, and B when
// NN = 0); for NN = 1 B's rows are BN values whose 32-byte pairs are swizzled by the row
// bits that the lanes of a transposed read differ in.  The DMA writes LDS in lane order, so
// the swizzle picks the source chunk of each lane.
template <int BM, int BN, int WM, int WN, bool NN>
__global__ __launch_bounds__(WM *WN * 64, BM * BN / (WM * WN) > 8192 ? 1 : 2) void project_tile_kernel(const ProjectArgs P) {
  constexpr int NT = WM * WN * 64;
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  constexpr int A_IT = BM * 8 / NT, B_IT = BN * 8 / NT;
  constexpr int BCH = BN / 8;  // chunks per row of B (NN)
  constexpr int SWZ = BN / 16 < 8 ? BN / 16 - 1 : 7;  // its pairs' swizzle stays inside a row
  constexpr bool kRing = BM * BN <= 4096;
  constexpr int NB = kRing ? 4 : 2;  // steps held in LDS
  __shared__ __attribute__((aligned(16))) uint16_t smem[NB * (BM + BN) * 64];
  uint16_t(*As)[BM * 64] = reinterpret_cast<uint16_t(*)[BM * 64]>(smem);
  uint16_t(*Bs)[BN * 64] = reinterpret_cast<uint16_t(*)[BN * 64]>(smem + NB * BM * 64);
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
  const int t0 = __builtin_amdgcn_readfirstlane((g8 * 8 + in_g % gm) * BM);
  const int n0 = __builtin_amdgcn_readfirstlane((in_g / gm) * BN);
  const int K = P.K, N = P.N;
  const PoolView &pool = P.pool;

  // byte offsets of this thread's chunks from the step's base addresses
  uint32_t a_off[A_IT], b_off[B_IT];
  // reduction index of chunk i of this thread inside a step (NN: of its row of B)
  auto a_k = [&](int i) MOE_INLINE {
    const int q = i * NT + tid;
    return ((q & 7) ^ ((q >> 3) & 7)) * 8;
  };
  auto b_k = [&](int i) MOE_INLINE { return NN ? (i * NT + tid) / BCH : a_k(i); };
#pragma unroll
  for (int i = 0; i < A_IT; ++i) {
    const int q = i * NT + tid, r = q >> 3, c = (q & 7) ^ (r & 7);
    a_off[i] = ((uint32_t)min(r, P.T - 1 - t0) * (uint32_t)P.ldx + c * 8) * 2u;
  }
#pragma unroll
  for (int i = 0; i < B_IT; ++i) {
    const int q = i * NT + tid;
    if constexpr (!NN) {
      const int r = q >> 3, c = (q & 7) ^ (r & 7);
      b_off[i] = ((uint32_t)min(r, N - 1 - n0) * (uint32_t)K + c * 8) * 2u;
    } else {
      const int r = q / BCH, c = (q % BCH) ^ ((((r & 3) | ((r >> 1) & 4)) & SWZ) << 1);
      b_off[i] = ((uint32_t)r * (uint32_t)N + (uint32_t)min(c * 8, N - 8 - n0)) * 2u;
    }
  }
  const uint16_t *a_base = P.x + (size_t)t0 * P.ldx;
  const uint16_t *b_base = NN ? P.w + n0 : P.w + (size_t)n0 * K;
  auto a_lds = [&](int buf) MOE_INLINE { return lds_byte(&As[0][0]) + wave * 1024 + buf * (BM * 128); };
  auto b_lds = [&](int buf) MOE_INLINE { return lds_byte(&Bs[0][0]) + wave * 1024 + buf * (BN * 128); };

  auto issue_full = [&](int buf, int k0) MOE_INLINE {
    const uint16_t *ab = a_base + k0;
    const uint16_t *bb = NN ? b_base + (size_t)k0 * N : b_base + k0;
#pragma unroll
    for (int i = 0; i < A_IT; ++i) dma16(ab, a_off[i], a_lds(buf) + i * NT * 16);
#pragma unroll
    for (int i = 0; i < B_IT; ++i) dma16(bb, b_off[i], b_lds(buf) + i * NT * 16);
  };
  auto issue_tail = [&](int buf, int k0) MOE_INLINE {  // chunks past K are zeros
    const char *ab = reinterpret_cast<const char *>(a_base + k0);
    const char *bb = reinterpret_cast<const char *>(NN ? b_base + (size_t)k0 * N : b_base + k0);
#pragma unroll
    for (int i = 0; i < A_IT; ++i)
      dma16(k0 + a_k(i) < K ? ab + a_off[i] : reinterpret_cast<const char *>(kZeroChunk), a_lds(buf) + i * NT * 16);
#pragma unroll
    for (int i = 0; i < B_IT; ++i)
      dma16(k0 + b_k(i) < K ? bb + b_off[i] : reinterpret_cast<const char *>(kZeroChunk), b_lds(buf) + i * NT * 16);
  };
  // A group of the expand holds `per` adapters of up to 32 ranks side by side, or 64 ranks of
  // one: ranks [r0, r0 + 64) of the adapters at [first, first + count) of the list.  (A group
  // for each adapter: 8192 tokens of 8 mixed adapters of rank 16, 2048 -> 4096: 230 us, 170
  // so; dx of 64 tokens of 32 adapters 61 us, 28 so.)  It takes two steps over the same rows
  // of B: the first terms of s v, then the second.  Where all of the tile's adapters come to
  // 32 ranks (packed) one step does: A holds the first terms in its lower half and the second
  // in its upper, and both meet B's lower half.
  const int R = pool.R, per = R <= 32 ? 64 / R : 1;
  bool packed = false;  // known once the adapters are listed
  const uint32_t inv = (65536u + R - 1) / R;  // k / R = k inv >> 16 for k < 64 (R >= 8: off by less than 1 / R)
  // reduction index k of a group: its adapter (slot | rank << 16) and rank there; false: none
  auto ext_at = [&](int first, int count, int r0, int k, int &entry, int &r) MOE_INLINE {
    const int j = per > 1 ? (int)((uint32_t)k * inv >> 16) : 0;
    r = r0 + k - j * R;
    entry = s_list[first + min(j, count - 1)];
    return j < count && r < list_rank(entry);
  };
  // a term of a group's s v into buf, and where buf2 >= 0 the next one into buf2
  auto issue_ext_a = [&](int buf, int buf2, int first, int count, int r0, int term) MOE_INLINE {
    static_assert(NT % 64 == 0, "a thread's chunks of rows of 64 are at one reduction index");
    int entry, r;
    const int k = packed ? a_k(0) & 31 : a_k(0);
    if (packed) term = a_k(0) >> 5;
    const bool live = ext_at(first, count, r0, k, entry, r);
    const uint16_t *src = P.ext_a + (size_t)t0 * 2 * R + term * R + r;
    int own[A_IT];  // (read before the loads, which nothing is moved across)
#pragma unroll
    for (int i = 0; i < A_IT; ++i) own[i] = s_slot[(i * NT + tid) >> 3];
#pragma unroll
    for (int i = 0; i < A_IT; ++i) {
      const int t = (i * NT + tid) >> 3;
      const bool on = live && own[i] == list_slot(entry);
      const void *z = kZeroChunk, *p = src + (size_t)t * 2 * R;
      dma16(on ? p : z, a_lds(buf) + i * NT * 16);
      if (buf2 >= 0) dma16(on ? static_cast<const uint16_t *>(p) + R : z, a_lds(buf2) + i * NT * 16);
    }
  };
  auto issue_ext_b = [&](int buf, int first, int count, int r0) MOE_INLINE {
    const char *z = reinterpret_cast<const char *>(kZeroChunk);
    int entry, r;
    const bool live = ext_at(first, count, r0, a_k(0), entry, r);
    const char *src[B_IT];
#pragma unroll
    for (int i = 0; i < B_IT; ++i) {
      if constexpr (!NN) {
        const int n = n0 + ((i * NT + tid) >> 3);
        const uint16_t *p = P.ext_b + ((size_t)list_slot(entry) * N + n) * R + r;
        src[i] = live && n < N ? reinterpret_cast<const char *>(p) : z;
      } else {
        const int q = i * NT + tid, c = (q % BCH) ^ ((((b_k(i) & 3) | ((b_k(i) >> 1) & 4)) & SWZ) << 1);
        const bool on = ext_at(first, count, r0, b_k(i), entry, r) && n0 + c * 8 < N;
        const uint16_t *p = P.ext_b + ((size_t)list_slot(entry) * R + r) * N + n0 + c * 8;
        src[i] = on ? reinterpret_cast<const char *>(p) : z;
      }
    }
#pragma unroll
    for (int i = 0; i < B_IT; ++i) dma16(src[i], b_lds(buf) + i * NT * 16);
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // a lane's chunk of a half kk in rows of 64: chunk (4 kk + grp) ^ (row % 8) of row `row`
  const int frag0 = row * 64 + ((grp ^ (row & 7)) << 3);
  auto frag = [&](int kk) MOE_INLINE { return frag0 ^ (kk << 5); };
  // NN: lane's row of a transposed read is 32 kk + 8 grp + row / 4 (+ 4), whose swizzle is
  // (row / 4) | 4 (grp & 1); columns 4 (row % 4) of a 16-wide piece (one 32-byte pair)
  const int tr_row = grp * 8 + (row >> 2), tr_swz = ((row >> 2) | ((grp & 1) << 2)) & SWZ;

  // the c-th of the reads that bring one 32-wide half's operands into registers
  constexpr int kReads = FM + (NN ? 2 * FN : FN);
  auto read2 = [&](int a_buf, int a_kk, int b_buf, int b_kk, int c, u32x4_t(&af)[FM], u32x4_t(&bf)[FN]) MOE_INLINE {
    if (c < FM) {
      af[c] = *reinterpret_cast<const u32x4_t *>(&As[a_buf][(wm * WTM + c * 16) * 64 + frag(a_kk)]);
    } else if constexpr (!NN) {
      bf[c - FM] = *reinterpret_cast<const u32x4_t *>(&Bs[b_buf][(wn * WTN + (c - FM) * 16) * 64 + frag(b_kk)]);
    } else {
      const int j = (c - FM) >> 1, h = (c - FM) & 1;
      const int pair = (wn * WTN) / 16 + j;
      const u32x2_t v = lds_read_tr(
          &Bs[b_buf][(b_kk * 32 + tr_row + 4 * h) * BN + ((pair ^ tr_swz) << 4) + 4 * (row & 3)]);
      bf[j][2 * h] = v[0];
      bf[j][2 * h + 1] = v[1];
    }
  };
  auto read = [&](int buf, int kk, int c, u32x4_t(&af)[FM], u32x4_t(&bf)[FN]) MOE_INLINE {
    read2(buf, kk, buf, kk, c, af, bf);
  };

  // Pipeline of a step: its first half's operands are in registers when it begins; the
  // second half's are read among the first half's products, then the next step's data must
  // have landed (one barrier: also every wavefront has left this buffer), and the DMA of the
  // step after it goes out into this buffer among the second half's products, with the reads
  // of the next step's first operands.  (DMA loads in one burst instead held the products
  // up: 8192 x 2048 -> 4096 in 137 us against 129, dx of 4096 x 4096 -> 2048 in 69 against 61.)
  const int steps = (K + 63) / 64, full = K / 64;
  // groups of an adapter of more than 32 ranks: 1 << two
  static_assert(MOE_LORA_MAX_POOL_RANK <= 128, "two groups at most");
  const int two = R > 64 ? 1 : 0;
  int adapters = 0, exts = 0;        // (exts: steps of the expand) known once the adapters are listed
  // the e-th group of the expand; left: its reduction's length (may be 0 or less)
  auto ext_of = [&](int e, int &first, int &count, int &r0, int &left) MOE_INLINE {
    first = per > 1 ? e * per : e >> two;
    count = min(per, adapters - first);
    r0 = per > 1 ? 0 : (e & two) * 64;
    left = per > 1 ? count * R : list_rank(__builtin_amdgcn_readfirstlane(s_list[first])) - r0;
  };
  // step h of the expand: its group and term.  Its A goes where any step's does; a group's B,
  // which two steps read, into the buffer of its own count (free: the step that had it before
  // is at least a buffer's turn behind).
  auto group_of = [&](int h) MOE_INLINE { return packed ? h : h >> 1; };
  auto term_of = [&](int h) MOE_INLINE { return packed ? 0 : h & 1; };
  auto ext_b_buf = [&](int h) MOE_INLINE { return (steps + group_of(h)) & (NB - 1); };
  auto issue = [&](int buf, int s) MOE_INLINE {
    if (s < full) {
      issue_full(buf, s * 64);
    } else if (s < steps) {
      issue_tail(buf, s * 64);
    } else if (s < steps + exts) {
      const int h = s - steps;
      int first, count, r0, left;
      ext_of(group_of(h), first, count, r0, left);
      issue_ext_a(buf, -1, first, count, r0, term_of(h));
      if (term_of(h) == 0) issue_ext_b(ext_b_buf(h), first, count, r0);
    }
  };
  issue(0, 0);
  adapters = tile_adapters<BM, NT>(pool, t0, P.T, s_slot, s_list, s_bits);
  packed = adapters * R <= 32;
  exts = (per > 1 ? (adapters + per - 1) / per : adapters << two) * (packed ? 1 : 2);
  if (tid == 0) s_bits[0] = 0u;  // from here on: whether an adapter holds what is not finite
  // The expand.  Other requests' rows of the A operand are zeros; so that nothing that an
  // adapter holds reaches them as 0 * inf or 0 * NaN, what is not finite in its rows is taken
  // out here and marks the adapter, whose outputs get it back at the end.  (Selecting
  // accumulators by row instead kept them out of the accumulation registers.)
  auto clean = [&](int buf, int first, int count, int r0) MOE_INLINE {
    bool odd = false;
    int ranks = 64;  // of the chunk's adapter, from the chunk's first on
    if constexpr (!NN) {
      int entry, r;
      ranks = ext_at(first, count, r0, b_k(0), entry, r) ? list_rank(entry) - r : 0;
    }
    uint32_t ones = 0;  // (an exponent of ones carries into the sign's place)
#pragma unroll
    for (int i = 0; i < B_IT; ++i) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(&Bs[buf][(i * NT + tid) * 8]);
#pragma unroll
      for (int c = 0; c < 4; ++c) ones |= (v[c] & 0x7f807f80u) + 0x00800080u;
    }
    if ((ones & 0x80008000u) == 0u && ranks >= 8) return;
#pragma unroll 1
    for (int i = 0; i < B_IT; ++i) {
      u32x4_t *p = reinterpret_cast<u32x4_t *>(&Bs[buf][(i * NT + tid) * 8]);
      u32x4_t v = *p;
      bool change = false;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t half_mask = c & 1 ? 0xffff0000u : 0x0000ffffu;
        // (NN = 0: ranks past the adapter's, whatever the pool holds there)
        const bool past = !NN && c >= ranks;
        const bool bad = (v[c >> 1] & half_mask & 0x7f807f80u) == (half_mask & 0x7f807f80u);
        odd |= bad && !past;
        change |= bad || past;
        v[c >> 1] &= bad || past ? ~half_mask : 0xffffffffu;
      }
      if (change) *p = v;
    }
    if (odd) atomicOr(&s_bits[0], 1u);
  };
  u32x4_t af1[FM], bf1[FN];
  // the products of a step of the expand, whose A is in a_buf; left: its group's
  auto expand = [&](int h, int a_buf, int left) MOE_INLINE {
    const int b_buf = ext_b_buf(h);
#pragma unroll 1
    for (int kk = 0; kk < 2 && (packed || kk * 32 < left); ++kk) {
#pragma unroll
      for (int c = 0; c < kReads; ++c) read2(a_buf, kk, b_buf, packed ? 0 : kk, c, af1, bf1);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma_16x16x32(bf1[j], af1[i], acc[i][j]);
    }
  };
  // clears a group's B of what is not finite before its first step
  auto prepare_ext = [&](int h, int &left) MOE_INLINE {
    int first, count, r0;
    ext_of(group_of(h), first, count, r0, left);
    if (left > 0 && term_of(h) == 0) {
      clean(ext_b_buf(h), first, count, r0);
      __syncthreads();
    }
  };
  // A small tile's steps are short beside the loads' latency: four of them in LDS, three on
  // their way (dx without adapters, 64 tokens, 4096 -> 2048: 32.1 -> 24.4 us; 512: 33 -> 25).
  if constexpr (kRing) {
    // loads of a wavefront for one step: A_IT + B_IT, A_IT for the expand's second one
    constexpr int kLoads = A_IT + B_IT;
    static_assert(NB == 4, "two steps on their way behind the one that is waited for");
    const int groups = packed ? exts : exts >> 1;
    exts = min(exts, 2);  // the first group's go out in the main loop, the others' whole one group ahead
    const int total = steps + exts;
#pragma unroll 1
    for (int s = 1; s < NB - 1; ++s) issue(s, s);
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      if (s + NB - 2 >= total)
        dma_wait_all();
      else if (s + NB - 2 > steps)
        dma_wait<kLoads + A_IT>();
      else
        dma_wait<2 * kLoads>();
      __syncthreads();
      issue((s + NB - 1) & (NB - 1), s + NB - 1);
      const int buf = s & (NB - 1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int c = 0; c < kReads; ++c) read(buf, kk, c, af1, bf1);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mfma_16x16x32(bf1[j], af1[i], acc[i][j]);
      }
    }
    // (a group's two steps together: its addresses are found once, and one barrier serves both)
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      const int at = steps + 2 * g;
      dma_wait_all();
      __syncthreads();
      if (g + 1 < groups) {
        int first, count, r0, left;
        ext_of(g + 1, first, count, r0, left);
        issue_ext_a((at + 2) & (NB - 1), (at + 3) & (NB - 1), first, count, r0, 0);
        issue_ext_b(ext_b_buf(2 * (g + 1)), first, count, r0);
      }
      int left;
      prepare_ext(packed ? g : 2 * g, left);
      expand(packed ? g : 2 * g, at & (NB - 1), left);
      if (!packed) expand(2 * g + 1, (at + 1) & (NB - 1), left);
    }
  } else {
    dma_wait_all();
    __syncthreads();
    issue(1, 1);
    u32x4_t af0[FM], bf0[FN];
#pragma unroll
    for (int c = 0; c < kReads; ++c) read(0, 0, c, af0, bf0);

    // the g-th of SEG shares of a full step's DMA loads
    auto dma_one = [&](auto dc, int dbuf, const uint16_t *ab, const uint16_t *bb, int live) MOE_INLINE {
      constexpr int d = decltype(dc)::value;
      if constexpr (d < A_IT)
        dma16_if<d * NT * 16>(live, ab, a_off[d], a_lds(dbuf));
      else
        dma16_if<(d - A_IT) * NT * 16>(live, bb, b_off[d - A_IT], b_lds(dbuf));
    };
    // products of one half among the reads of (buf, kk); with dma, also among the DMA loads at
    // k0 into dbuf
    auto half = [&](u32x4_t(&af)[FM], u32x4_t(&bf)[FN], int buf, int kk, u32x4_t(&an)[FM], u32x4_t(&bn)[FN], auto dma,
                    int dbuf, int k0, int live) MOE_INLINE {
      constexpr bool kDma = decltype(dma)::value;
      constexpr int SEG = kDma ? 8 : 1;  // pieces that the scheduler keeps in order
      const uint16_t *ab = a_base + k0;
      const uint16_t *bb = NN ? b_base + (size_t)k0 * N : b_base + k0;
      __builtin_amdgcn_sched_barrier(0);
      static_for<0, SEG>([&](auto gc) MOE_INLINE {
        constexpr int g = decltype(gc)::value;
        if constexpr (kDma)
          static_for<g * (A_IT + B_IT) / SEG, (g + 1) * (A_IT + B_IT) / SEG>(
              [&](auto dc) MOE_INLINE { dma_one(dc, dbuf, ab, bb, live); });
#pragma unroll
        for (int c = g * kReads / SEG; c < (g + 1) * kReads / SEG; ++c) read(buf, kk, c, an, bn);
#pragma unroll
        for (int m = g * FM * FN / SEG; m < (g + 1) * FM * FN / SEG; ++m)
          acc[m / FN][m % FN] = mfma_16x16x32(bf[m % FN], af[m / FN], acc[m / FN][m % FN]);
#pragma unroll
        for (int c = 0; c < kReads / SEG; ++c) {  // an LDS read, then a share of the products
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, FM * FN / kReads, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    // (two steps to an iteration and the branches of issue() between the halves: with both
    // halves in one basic block, or one step to an iteration, the register allocator moved
    // accumulators about on every step)
    auto main_step = [&](int buf, int s) MOE_INLINE {
      half(af0, bf0, buf, 1, af1, bf1, std::false_type{}, 0, 0, 0);
      dma_wait_all();
      __syncthreads();
      int left = s + 2 - full;
      asm volatile("" : "+v"(left));
      const int more = (int)((uint32_t)__builtin_amdgcn_readfirstlane(left) >> 31);
      if (!more) issue(buf, s + 2);
      // (past the last step the reads bring what nothing uses)
      half(af1, bf1, buf ^ 1, 0, af0, bf0, std::true_type{}, buf, more * (s + 2) * 64, more);
    };
#pragma unroll 1
    for (int s = 0; s < steps; s += 2) {
      main_step(0, s);
      if (s + 1 < steps) main_step(1, s + 1);
    }

#pragma unroll 1
    for (int h = 0; h < exts; ++h) {
      const int buf = (steps + h) & 1;
      int left;
      prepare_ext(h, left);
      expand(h, buf, left);
      if (h + 1 < exts) {
        dma_wait_all();
        __syncthreads();
        if (h + 2 < exts) issue(buf, steps + h + 2);
      }
    }
  }
  // The tile leaves through LDS (rows of BN bf16, 16-byte chunks XOR-swizzled by the row), so
  // that neighbouring lanes store neighbouring bytes.
  constexpr int OCH = BN / 8, OSW = OCH < 16 ? OCH - 1 : 15;
  __syncthreads();
  const bool odd_adapter = s_bits[0] != 0u;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r = wm * WTM + i * 16 + row;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int c = (wn * WTN + j * 16) / 8 + (grp >> 1);
      *reinterpret_cast<u32x2_t *>(&smem[r * BN + ((c ^ (r & OSW)) << 3) + (grp & 1) * 4]) =
          u32x2_t{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int q = tid; q < BM * OCH; q += NT) {
    const int r = q / OCH, c = q % OCH, t = t0 + r, n = n0 + c * 8;
    if (t < P.T && n < N) {
      u32x4_t v = *reinterpret_cast<const u32x4_t *>(&smem[r * BN + ((c ^ (r & OSW)) << 3)]);
      if (odd_adapter) restore_odd<NN>(P, s_slot[r], n, v);
      *reinterpret_cast<u32x4_t *>(P.y + (size_t)t * P.ldy + n) = v;
    }
  }
}

int ok() { return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP; }

template <int MT, bool TR>
int launch_shrink_ranks(const ShrinkArgs &a, hipStream_t s) {
  const dim3 grid((a.T + 16 * MT - 1) / (16 * MT) + (TR && a.order ? 1 : 0), MT == 1 ? 16 : 1);
  if (a.pool.R <= 16)
    shrink_kernel<1, MT, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  else if (a.pool.R <= 32)
    shrink_kernel<2, MT, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  else
    shrink_kernel<4, MT, TR><<<grid, kShrinkWaves * 64, 0, s>>>(a);
  return ok();
}

// A decode-sized batch takes a workgroup per (tile of 16, adapter): up to 16 adapters meet
// in 16 requests.  In longer batches a tile's few adapters follow each other, and tiles of 32
// tokens halve the reads of the adapters (4096 x 4096, rank 32, over B: 17.5 us in tiles of
// 16, 12.6 of 32; the same 19 us either way where x comes from HBM).  Two steps in flight
// there: four spill (18 us).
template <bool TR>
int launch_shrink(const ShrinkArgs &a, hipStream_t s) {
  return a.T <= 1024 ? launch_shrink_ranks<1, TR>(a, s) : launch_shrink_ranks<2, TR>(a, s);
}

template <int FM, int FN, int W, int G>
int launch_few_tile(const ProjectArgs &a, hipStream_t s) {
  const dim3 grid((a.N + FN * 16 - 1) / (FN * 16), (a.T + FM * 16 - 1) / (FM * 16));
  project_few_kernel<FM, FN, W, G><<<grid, W * 64, 0, s>>>(a);
  return ok();
}

// The smallest tiles that all run at once (one workgroup to a compute unit): more of the
// device loads, and each workgroup less; wider tiles beyond, since a workgroup reads its
// tokens' rows of x whole.  (Inputs in no cache, without adapters: 64 tokens, 2048 -> 4096 in
// tiles of 64 x 32, 32 x 32 and 32 x 16: 10.4, 8.4 and 9.2 us; 64 tokens, 2048 -> 1024 in 64
// x 32, 32 x 16 and 16 x 16: 8.0, 5.2 and 4.4; 128 tokens, 2048 -> 4096 in 64 x 32 and 32 x
// 32: 10.5 and 11.1; 256 tokens, 2048 -> 4096 in 64 x 32 and 64 x 64: 16.4 and 12.6.)
int launch_few(const ProjectArgs &a, hipStream_t s) {
  auto fits = [&](int tokens, int cols) {
    return (long long)((a.T + tokens - 1) / tokens) * ((a.N + cols - 1) / cols) <= 256;
  };
  if (fits(16, 16)) return launch_few_tile<1, 1, 8, 2>(a, s);
  if (a.T <= 16) return launch_few_tile<1, 2, 8, 2>(a, s);
  if (fits(32, 16)) return launch_few_tile<2, 1, 8, 2>(a, s);
  if (a.T <= 32 || fits(32, 32)) return launch_few_tile<2, 2, 8, 1>(a, s);
  return fits(64, 32) ? launch_few_tile<4, 2, 8, 1>(a, s) : launch_few_tile<4, 4, 8, 1>(a, s);
}

// Whether the few-token kernel takes the call: while its widest tiles all run at once (512
// tokens, 4096 -> 2048, 8 mixed adapters: 31.7 us against 36.3 in LDS tiles; 2048 -> 4096, two
// rounds of workgroups: 33.9 against 32.0).
bool takes_few(const ProjectArgs &a) {
  return a.T <= 32 || (long long)((a.T + 63) / 64) * ((a.N + 63) / 64) <= 256;
}

template <int BM, int BN, int WM, int WN, bool NN>
int launch_tiles(const ProjectArgs &a, hipStream_t s) {
  const int total = ((a.T + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  project_tile_kernel<BM, BN, WM, WN, NN><<<((total + 7) >> 3) * 8, WM * WN * 64, 0, s>>>(a);
  return ok();
}

// The largest tiles that still come to most of a round of workgroups; 32 x 32 while all of
// those run at once, two to a compute unit (dx with adapters, 64 tokens, 4096 -> 2048: 40.4 us
// in tiles of 64, 28.5 of 32; 512 tokens, 2048 -> 1024, 512 tiles of 32: 21.4 and 19.5; 512,
// 4096 -> 2048, 1024 tiles: 33.5 and 45).  The 256 x 256 tiles of dx spill registers outside
// their main loop and are the faster ones all the same (8192 tokens, 2048 -> 4096: 132 us, 161 in
// tiles of 128; 4096 -> 4096: 245 and 299; 8 mixed adapters: 208 and 239), but for some counts
// just above a round of workgroups (5000 tokens, 4096 -> 4096, 320 tiles: 212 and 189).
template <bool NN>
int launch_product(const ProjectArgs &a, hipStream_t s) {
  auto tiles = [&](int b) { return (long long)((a.T + b - 1) / b) * ((a.N + b - 1) / b); };
  if (tiles(256) >= 192) return launch_tiles<256, 256, 2, 2, NN>(a, s);
  if (tiles(128) >= 160) return launch_tiles<128, 128, 2, 2, NN>(a, s);
  // (calls of the forward form with fewer tiles go to the few-token kernel)
  if constexpr (NN) {
    if (tiles(32) <= 512) return launch_tiles<32, 32, 2, 2, NN>(a, s);
  }
  return launch_tiles<64, 64, 2, 2, NN>(a, s);
}

}  // namespace

int launch_shrink_transposed(const ShrinkArgs &a, hipStream_t s) { return launch_shrink<true>(a, s); }
int launch_product_transposed(const ProjectArgs &a, hipStream_t s) { return launch_product<true>(a, s); }

size_t project_workspace_bytes(int T, int R) { return ((size_t)T * R * 4 + 255) & ~(size_t)255; }

int launch_project(const ProjectArgs &a, float *v, hipStream_t s) {
  if (a.pool.S > 0) {
    const ShrinkArgs sh{a.x, a.ldx, a.T, a.K, a.a_or_b, a.pool, const_cast<uint16_t *>(a.ext_a), v, nullptr, nullptr};
    const int st = launch_shrink<false>(sh, s);
    if (st != ST_OK) return st;
  }
  if (takes_few(a)) return launch_few(a, s);
  return launch_product<false>(a, s);
}

}  // namespace moe
