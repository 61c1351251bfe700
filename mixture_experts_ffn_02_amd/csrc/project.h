// Shared pieces of the pooled-adapter projection kernels (gfx950).
#pragma once

#include <type_traits>

#include "common.h"
#include "kernels.h"

// (a lambda of a kernel left out of line would take its captures through memory)
#define MOE_INLINE __attribute__((always_inline))

namespace moe {

// 16 zero bytes for lanes whose chunk lies outside its matrix (a masked lane still reads)
__device__ __attribute__((aligned(16))) static const uint32_t kZeroChunk[4] = {0u, 0u, 0u, 0u};

// One 16-byte chunk per lane from global memory straight into LDS: lane l writes LDS bytes
// [lds + 16 l, lds + 16 l + 16).  Counts in vmcnt like any load; nothing waits here.
MOE_DEV void dma16(const void *src, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(src), "s"(lds)
      : "memory");
}
// the same with a wave-uniform base and a 32-bit byte offset per lane
MOE_DEV void dma16(const void *base, uint32_t off, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(base), "s"(lds)
      : "memory");
}
// The same, to lds + LDS, where on is not 0 and nothing where it is (wave-uniform), without a
// branch.  For code that all 64 lanes run: the mask is set back to all of them.
template <int LDS>
MOE_DEV void dma16_if(int on, const void *base, uint32_t off, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_add_u32 m0, %3, %5\n\t"
      "s_cmp_lg_u32 %4, 0\n\t"
      "s_cselect_b64 exec, -1, 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b64 exec, -1\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(base), "s"(lds), "s"(on), "n"(LDS)
      : "memory", "scc");
}
// until at most N of the wavefront's loads are on their way (they land in order)
template <int N>
MOE_DEV void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
MOE_DEV void dma_wait_all() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// f(integral_constant<D>) for D = BEGIN .. END - 1
template <int BEGIN, int END, class F>
MOE_DEV void static_for(F f) {
  if constexpr (BEGIN < END) {
    f(std::integral_constant<int, BEGIN>{});
    static_for<BEGIN + 1, END>(f);
  }
}

MOE_DEV uint32_t lds_byte(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// Transposed LDS read: each group of 16 lanes reads a 4 x 16 block of 16-bit values, lane i
// giving the address of row i / 4, columns 4 (i % 4) .. + 3; it receives column i's 4 rows.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
MOE_DEV u32x2_t lds_read_tr(const uint16_t *p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4_t *)p));
}

// orders one wavefront's own LDS writes and reads
MOE_DEV void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A value as two bf16 terms: of finite values the pair is off by at most 2^-16 of the value;
// one that bf16 holds as an infinity, and a NaN, has a second term of 0 (so that inf * b keeps
// its sign).  Stored at rank r of a token's terms: R first ones, then R second.
MOE_DEV void store_terms(uint16_t *terms, int R, int r, float v) {
  const uint32_t hi = f32_to_bf16(v);
  const float rest = (hi & 0x7f80u) == 0x7f80u ? 0.f : v - bf16_to_f32(hi);
  terms[r] = (uint16_t)hi;
  terms[R + r] = (uint16_t)f32_to_bf16(rest);
}

// slot of a token with an adapter of positive rank, else -1; its rank
MOE_DEV int adapter_of(const PoolView &P, int t, int &rank) {
  const int s = P.token_slot[t];
  rank = 0;
  if (s < 0 || s >= P.S) return -1;
  const int r = P.rank[s];
  rank = r < P.R ? r : P.R;
  return rank > 0 ? s : -1;
}
MOE_DEV int rank_of(const PoolView &P, int s) {
  const int r = P.rank[s];
  return r < P.R ? r : P.R;
}

// The tokens with an adapter, by adapter and ascending inside one, into order; where each
// adapter's tokens begin into seg [S + 1].  Called by one workgroup of NT threads; hist:
// (NT / 64 + 1) * (S + 1) ints of LDS.
template <int NT>
MOE_DEV void order_tokens(const PoolView &P, int T, int32_t *order, int32_t *seg, int *hist) {
  constexpr int W = NT / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = P.S + 1;
  int *start = hist + W * n;
  for (int i = tid; i < W * n; i += NT) hist[i] = 0;
  __syncthreads();
  const int per = (T + W - 1) / W;
  const int t0 = min(T, wave * per), t1 = min(T, t0 + per);
  int rank;
  for (int t = t0 + lane; t < t1; t += 64) {
    const int s = adapter_of(P, t, rank);
    if (s >= 0) atomicAdd(&hist[wave * n + s], 1);
  }
  __syncthreads();
  for (int s = tid; s < n; s += NT) {
    int run = 0;
    for (int w = 0; w < W; ++w) {
      const int c = hist[w * n + s];
      hist[w * n + s] = run;
      run += c;
    }
    start[s] = run;
  }
  __syncthreads();
  if (wave == 0) {  // exclusive scan over the adapters
    const int each = (n + 63) / 64;
    int local = 0;
    for (int q = 0; q < each; ++q) local += lane * each + q < n ? start[lane * each + q] : 0;
    int incl = local;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    int run = incl - local;
    for (int q = 0; q < each; ++q) {
      const int s = lane * each + q;
      if (s < n) {
        const int c = start[s];
        start[s] = run;
        seg[s] = run;
        run += c;
      }
    }
  }
  __syncthreads();
  int *mine = hist + wave * n;
  int bits = 0;
  while ((1 << bits) < P.S) ++bits;
  const uint64_t lt = (1ull << lane) - 1;
  for (int b = t0; b < t1; b += 64) {
    const int t = b + lane;
    const int s = t < t1 ? adapter_of(P, t, rank) : -1;
    const bool on = s >= 0;
    uint64_t peers = __ballot(on);
    for (int q = 0; q < bits; ++q) {
      const bool bit = on && ((s >> q) & 1);
      const uint64_t m = __ballot(bit);
      peers &= bit ? m : ~m;
    }
    int at = 0;
    if (on) at = mine[s];
    wave_lds_fence();
    if (on) {
      order[start[s] + at + __popcll(peers & lt)] = t;
      if ((peers & lt) == 0ull) mine[s] = at + __popcll(peers);
    }
    wave_lds_fence();
  }
}

// Distinct adapters of a tile's rows, thread r giving row r's (slot -1: none): row slots into
// s_slot, the list of slot | rank << 16 in ascending order into s_list, its length returned
// (uniform).  Called by the whole workgroup; s_bits: 16 words.
template <int ROWS, int NT>
MOE_DEV int list_adapters(int s, int rank, int *s_slot, int *s_list, uint32_t *s_bits) {
  static_assert(ROWS <= NT, "one row per thread");
  const int tid = threadIdx.x;
  if (tid < 16) s_bits[tid] = 0u;
  __syncthreads();
  uint32_t before = 0;
  if (tid < ROWS) {
    s_slot[tid] = s;
    if (s >= 0) before = atomicOr(&s_bits[s >> 5], 1u << (s & 31));
  }
  __syncthreads();
  int n = 0, at = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const int c = __popc(s_bits[w]);
    at += w < (s >> 5) ? c : 0;
    n += c;
  }
  // the row that set its adapter's bit lists it
  if (s >= 0 && !((before >> (s & 31)) & 1u))
    s_list[at + __popc(s_bits[s >> 5] & ((1u << (s & 31)) - 1u))] = s | (rank << 16);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(n);
}
template <int ROWS, int NT>
MOE_DEV int tile_adapters(const PoolView &P, int t0, int T, int *s_slot, int *s_list, uint32_t *s_bits) {
  const int tid = threadIdx.x;
  int s = -1, rank = 0;
  if (tid < ROWS && P.S > 0 && t0 + tid < T) s = adapter_of(P, t0 + tid, rank);
  return list_adapters<ROWS, NT>(s, rank, s_slot, s_list, s_bits);
}
MOE_DEV int list_slot(int entry) { return entry & 0xffff; }
MOE_DEV int list_rank(int entry) { return entry >> 16; }

}  // namespace moe
