// Expert-sorted pack of the routing kernels (gfx950): per-wave expert counts in LDS, their
// prefixes, and the stable scatter of each wave's expanded rows.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kRouteThreads = 1024;
constexpr int kMaxRouteWg = 256;  // workgroups of one routing launch

struct RouteParams {
  RouteArgs a;
  int tok_per_wg;
  int num_wg;
};

// inclusive sum over the lanes of a wavefront: shifts inside the 16-lane rows, then row ends
// into the rows above (no LDS round trip per step)
MOE_DEV int wave_scan_add(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Second launch of a multi-workgroup batch (route_finish_kernel): block-relative positions
// become final ones.
int launch_route_finish(const RouteParams &P, hipStream_t s);

// Called by a whole workgroup after its waves filled hist_w [waves][E] (counts of the
// wave's tokens [w_begin, w_end)) and ids_l [tokens][K], and after a barrier.  tot and
// wgbase: E ints each.
template <bool MULTI>
MOE_DEV void pack_block(const RouteArgs &a, int32_t *hist_w, const int32_t *ids_l, int32_t *tot,
                        int32_t *wgbase, int waves, int threads, int t_begin, int w_begin, int w_end) {
  const int E = a.E, K = a.K;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // ---- per-wave starting positions inside this workgroup, workgroup totals
  for (int e = tid; e < E; e += threads) {
    int run = 0;
    for (int w = 0; w < waves; ++w) {
      const int c = hist_w[w * E + e];
      hist_w[w * E + e] = run;
      run += c;
    }
    tot[e] = run;
    if (MULTI) a.hist[(size_t)blockIdx.x * E + e] = run;
  }
  __syncthreads();
  if (!MULTI && wave == 0) {
    // one workgroup: offsets are the exclusive scan of its totals
    const int per_lane = (E + 63) / 64;
    int local = 0;
    for (int q = 0; q < per_lane; ++q) {
      const int e = lane * per_lane + q;
      local += (e < E) ? tot[e] : 0;
    }
    const int incl = wave_scan_add(local);
    int run = incl - local;
    for (int q = 0; q < per_lane; ++q) {
      const int e = lane * per_lane + q;
      if (e < E) {
        a.offsets[e] = run;
        wgbase[e] = run;
        run += tot[e];
      }
    }
    if (lane == 63) a.offsets[E] = incl;
  }
  if (MULTI)
    for (int e = tid; e < E; e += threads) wgbase[e] = 0;
  __syncthreads();

  // ---- stable scatter of this wave's expanded rows.  One workgroup writes final
  // positions; with several, each writes its positions relative to its own block
  // (into e2p) and the second launch adds the global bases.
  int32_t *start = hist_w + wave * E;
  const int j0 = w_begin * K, j1 = w_end * K;
  const int jl0 = t_begin * K;
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
  for (int base = j0; base < j1; base += 64) {
    const int j = base + lane;
    const bool valid = j < j1;
    const int e = valid ? ids_l[j - jl0] : 0;
    uint64_t peers = __ballot(valid);
    for (int bb = 0; bb < nbits; ++bb) {
      const bool bit = (e >> bb) & 1;
      const uint64_t m = __ballot(valid && bit);
      peers &= bit ? m : ~m;
    }
    const int rank = __popcll(peers & lt);
    int sp = 0;
    if (valid) sp = start[e];
    __builtin_amdgcn_wave_barrier();
    if (valid) {
      const int pos = wgbase[e] + sp + rank;
      a.e2p[j] = pos;
      if (!MULTI) a.p2e[pos] = j;
      if ((peers & lt) == 0ull) start[e] = sp + __popcll(peers);
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace moe
