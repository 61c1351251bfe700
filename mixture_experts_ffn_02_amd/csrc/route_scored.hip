// General expert routing (gfx950): softmax or sigmoid scores, a balance bias, groups by
// their best or two best experts, top-k, optional renormalisation; and the gradient of the
// chosen weights to the logits.
//
// Forward.  key = score + bias, or the logit itself without a bias (both scores grow with
// the logit).  A token is owned by LPT lanes: a whole wavefront, or one 16-lane DPP row so
// that one instruction stream selects for four tokens.  Each lane holds EPL consecutive
// experts as order-preserving unsigned keys (0 = not selectable), so a selection step is
// a local max, a max over the lanes and a ballot; equal keys go to the lowest lane, which
// holds the lowest index.  Keys with a bias, and groups scored by two, are defined in fp64:
// a first choice is made on their fp32 values, whose error is known, and stands if every
// difference that decided something is larger than two such errors; else (about one token
// in some hundreds, and exact ties) the token is chosen again on fp64 keys, as two 32-bit
// words.  The weights are fp32, from the log scores relative to the largest chosen one when
// renormalised (nothing underflows in the sum).  The expert-sorted pack is the one of
// moe_lora_route.
//
// Bound: at 1 to 64 tokens one workgroup's latency (one launch; 1 token, 256 experts, sigmoid,
// bias, 4 of 8 groups: 8.5 us); above, the selection's vector instructions (two launches;
// 16384 tokens, 128 experts, softmax: 11 + 5 us).
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "route_pack.h"

namespace moe {
namespace {

constexpr int kScoredOneWg = 64;     // batches up to this run in one workgroup and one launch
constexpr int kScoredOneWgWide = 16; // the same with keys of fp64
constexpr int kScoredMaxTok = 256;   // tokens of one workgroup (its ids live in LDS)

template <int CTRL>
MOE_DEV uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
  return o > v ? o : v;
}
// max over the LPT lanes of a token, in all of them: quad swaps, rotations by 4 and 8 inside
// the 16-lane rows, then (64 lanes) rows 0 and 2 into their neighbours, row 1 into the upper
// half, and the last lane's value to all.  (The runtime's wave reduction walks the lanes one
// by one: a selection step took 0.47 us with it.)
template <int LPT>
MOE_DEV uint32_t lanes_max_u32(uint32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x124>(v);
  v = dpp_max<0x128>(v);
  if constexpr (LPT == 64) {
    v = dpp_max<0x142>(v);  // row_bcast:15
    v = dpp_max<0x143>(v);  // row_bcast:31
    v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
  return v;
}

template <int CTRL>
MOE_DEV float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int LPT>
MOE_DEV float lanes_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x124>(v);
  v = dpp_add<0x128>(v);
  if constexpr (LPT == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
template <int LPT>
MOE_DEV double lanes_sum_f64(double v) {
#pragma unroll
  for (int m = 1; m < LPT; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// order-preserving map of a float (NaN greatest, -0 equal to +0); never 0
MOE_DEV uint32_t f32_key(float v) {
  if (v != v) return 0xffffffffu;
  if (v == 0.f) v = 0.f;
  const uint32_t u = __float_as_uint(v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
MOE_DEV float key_f32(uint32_t k) {
  return k == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}
MOE_DEV uint64_t f64_key(double v) {
  if (v != v) return ~0ull;
  if (v == 0.0) v = 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
// max of two floats over the lanes; a NaN anywhere is ignored (the sums carry it)
template <int LPT>
MOE_DEV float lanes_max(float v) {
  return key_f32(lanes_max_u32<LPT>(v != v ? 1u : f32_key(v)));
}

// One selection step: the largest key m among this token's lanes (ties to the lowest index).
// Returns true in the one lane that owns it, with its local index; that key is cleared.
// lanes, lower: the ballot bits of the token's lanes, and of those below this one.
template <int LPT, int N, bool WIDE>
MOE_DEV bool take_best(uint32_t (&hi)[N], uint32_t (&lo)[N], uint64_t lanes, uint64_t lower, uint32_t &m, int &at) {
  uint32_t best = hi[0];
#pragma unroll
  for (int i = 1; i < N; ++i) best = hi[i] > best ? hi[i] : best;
  m = lanes_max_u32<LPT>(best);
  bool mine = best == m;
  uint64_t who = __ballot(mine) & lanes;
  uint32_t ml = 0;
  bool by_low = false;
  if constexpr (WIDE) {
    int same = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) same += hi[i] == m;
    if (__ballot(same > 1 || (who & (who - 1)) != 0) != 0) {  // some token's high words tie
      uint32_t bl = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) bl = (hi[i] == m && lo[i] > bl) ? lo[i] : bl;
      ml = lanes_max_u32<LPT>(mine ? bl : 0u);
      mine = mine && bl == ml;
      who = __ballot(mine) & lanes;
      by_low = true;
    }
  }
  if constexpr (LPT == 64) {
    // no branch: the owner is one lane of the wavefront
    const bool own = lane_id() == __builtin_ctzll(who | (1ull << 63));
#pragma unroll
    for (int i = N - 1; i >= 0; --i) at = hi[i] == m && (!WIDE || !by_low || lo[i] == ml) ? i : at;
#pragma unroll
    for (int i = 0; i < N; ++i) hi[i] = own && at == i ? 0u : hi[i];
    return own;
  }
  if (!mine || (who & lower) != 0) return false;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) at = hi[i] == m && (!WIDE || !by_low || lo[i] == ml) ? i : at;
#pragma unroll
  for (int i = 0; i < N; ++i) hi[i] = at == i ? 0u : hi[i];
  return true;
}

// Whether fp32 keys a >= b (order keys of values) decide as the fp64 ones do.  In half steps of
// 2^-24, around values of at most 1: exp and the division take some six (a sigmoid is off by
// less than 2^-21.4, a sum of two by 2^-20.4), a softmax sum 36 at most (32 terms in a lane and
// four joins, 512 experts on 16 lanes), so a softmax score is off by less than 2^-18.5; with
// groups (64 lanes: 8 terms and six joins) by less than 2^-19.5, and a sum of two keys by
// 2^-18.5.  Adding the bias takes a half step of the key.  A difference above slack (2^-19 of
// sigmoids, 2^-17 else; of sums, and 2^-20 of the largest key in one) + 2^-20 of the keys is
// larger than two such errors.  Ties and what is not finite are not decided.
MOE_DEV bool decided(uint32_t a, uint32_t b, float slack) {
  const float x = key_f32(a), y = key_f32(b);
  return x - y > slack + 0x1p-20f * fmaxf(fabsf(x), fabsf(y)) && fabsf(x) < 1e30f;
}

// orders one wavefront's own LDS writes and reads
MOE_DEV void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

MOE_DEV float load_logit(const void *p, size_t i, bool f32) {
  return f32 ? static_cast<const float *>(p)[i] : bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}

// N consecutive logits of a row from expert e0 (-inf past the last): whole vectors where every
// lane's run starts aligned and ends inside the row, else one by one (which takes the
// address path one lane a cycle)
template <int N>
MOE_DEV void load_logits(const void *p, size_t row, int e0, int E, bool f32, float (&x)[N]) {
  if (N > 1 && E % N == 0) {
    if (e0 >= E) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = -INFINITY;
    } else if (f32) {
      constexpr int V = N < 4 ? N : 4;
      typedef float vec __attribute__((ext_vector_type(V)));
      const vec *v = reinterpret_cast<const vec *>(static_cast<const float *>(p) + row + e0);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = v[i / V][i % V];
    } else {
      constexpr int V = N < 8 ? N : 8;
      typedef uint16_t vec __attribute__((ext_vector_type(V)));
      const vec *v = reinterpret_cast<const vec *>(static_cast<const uint16_t *>(p) + row + e0);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = bf16_to_f32(v[i / V][i % V]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? load_logit(p, row + e0 + i, f32) : -INFINITY;
  }
}

MOE_DEV float log_sigmoid(float x) { return fminf(x, 0.f) - log1pf(expf(-fabsf(x))); }

struct ScoredParams {
  RouteParams r;
  ScoredArgs s;
};

// LDS (dynamic): hist [waves][E] int | tot [E] | wgbase [E] | ids [tokens][K] int
//                | group keys [waves][E] double (groups)
template <int LPT, int EPL, bool WIDE, bool MULTI>
__global__ __launch_bounds__(kRouteThreads) void scored_kernel(const ScoredParams P) {
  const RouteArgs &a = P.r.a;
  const ScoredArgs &s = P.s;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int E = a.E, K = a.K;
  const int threads = blockDim.x, waves = threads >> 6;
  constexpr int TPW = 64 / LPT;  // tokens of a wave at a time
  int32_t *hist_w = reinterpret_cast<int32_t *>(smem);
  int32_t *tot = hist_w + waves * E;
  int32_t *wgbase = tot + E;
  int32_t *ids_l = wgbase + E;
  double *grp = reinterpret_cast<double *>(
      smem + (((size_t)(waves * E + 2 * E + P.r.tok_per_wg * K) * 4 + 15) & ~(size_t)15));

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane / LPT, ll = lane % LPT;
  for (int i = tid; i < waves * E; i += threads) hist_w[i] = 0;
  __syncthreads();
  const int t_begin = blockIdx.x * P.r.tok_per_wg;
  const int t_end = min(a.T, t_begin + P.r.tok_per_wg);
  const int tpw = (P.r.tok_per_wg + waves - 1) / waves;
  const int w_begin = min(t_end, t_begin + wave * tpw);
  const int w_end = min(t_end, w_begin + tpw);
  const uint64_t lanes = LPT == 64 ? ~0ull : (0xffffull << (lane & 48));
  const uint64_t lower = lanes & ((1ull << lane) - 1);
  const bool sigmoid = s.score == MOE_LORA_SCORE_SIGMOID;
  const float slack = sigmoid ? 0x1p-19f : 0x1p-17f;
  const bool grouped = LPT == 64 && a.n_group > 1;  // (groups run on whole wavefronts)

  for (int t0 = w_begin; t0 < w_end; t0 += TPW) {
    const bool tv = t0 + sub < w_end;
    const int t = tv ? t0 + sub : w_begin;
    int32_t *id_row = ids_l + (t - t_begin) * K;
    float x[EPL];
    const size_t row = (size_t)t * E;
    load_logits<EPL>(a.logits, row, ll * EPL, E, s.f32, x);
    float bias[WIDE ? EPL : 1];
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) bias[i] = s.bias && ll * EPL + i < E ? s.bias[ll * EPL + i] : 0.f;
    }
    // softmax over all experts: largest logit and sum
    float mx = 0.f, total = 1.f;
    float px[EPL];
    if (!sigmoid && (!s.renormalize || WIDE)) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
      mx = lanes_max<LPT>(m);
      if (mx == -INFINITY) mx = 0.f;  // every expert masked
      total = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        px[i] = expf(x[i] - mx);
        total += ll * EPL + i < E ? px[i] : 0.f;
      }
      total = lanes_sum<LPT>(total);
      total = total == 0.f ? 1.f : total;
    }

    int chosen = 0;  // LPT = 64: lane j's j-th expert
    // The choice on keys of 32 bits, or (exact) of 64 where WIDE.  Returns whether it stands.
    auto choose = [&](auto exact) __attribute__((always_inline)) {
      constexpr bool F64 = decltype(exact)::value;
      bool sure = true;
      uint32_t hi[EPL], lo[EPL];
      float gk32[EPL];
      if constexpr (F64) {
        double p[EPL], sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const bool in = ll * EPL + i < E;
          p[i] = in ? (sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : exp((double)x[i] - (double)mx)) : 0.0;
          sum += p[i];
        }
        if (!sigmoid) {
          sum = lanes_sum_f64<LPT>(sum);
          sum = sum == 0.0 ? 1.0 : sum;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = ll * EPL + i;
          const double key = (sigmoid ? p[i] : p[i] / sum) + (double)bias[i];
          if (grouped && e < E) grp[wave * E + e] = key;
          // without a bias only the groups need the scores: experts compare by logit
          const uint64_t k = s.bias ? f64_key(key) : (uint64_t)f32_key(x[i]) << 32;
          hi[i] = e < E ? (uint32_t)(k >> 32) : 0u;
          lo[i] = e < E ? (uint32_t)k : 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = ll * EPL + i;
          gk32[i] = x[i];
          if constexpr (WIDE) gk32[i] = (sigmoid ? 1.f / (1.f + expf(-x[i])) : px[i] / total) + bias[i];
          hi[i] = e < E ? f32_key(WIDE && s.bias ? gk32[i] : x[i]) : 0u;
          lo[i] = 0u;
          if (grouped && e < E) grp[wave * E + e] = (double)gk32[i];
        }
      }
      if (grouped) {
        wave_lds_order();
        // lanes split over the groups, then joined: lpg lanes (a power of two) scan a group
        const int per = E / a.n_group;
        int lpg = 1;
        while (lpg * 2 * a.n_group <= 64 && lpg < per) lpg *= 2;
        const int g = lane / lpg;
        double b0 = -INFINITY, b1 = -INFINITY;
        if (g < a.n_group) {
          for (int q = lane % lpg; q < per; q += lpg) {
            const double v = grp[wave * E + g * per + q];
            if (v > b0 || v != v) {
              b1 = b0;
              b0 = v;
            } else if (v > b1) {
              b1 = v;
            }
          }
        }
        for (int m = 1; m < lpg; m <<= 1) {
          const double o0 = __shfl_xor(b0, m), o1 = __shfl_xor(b1, m);
          const bool up = o0 > b0 || o0 != o0;
          b1 = up ? (b0 > o1 ? b0 : o1) : (b1 > o0 ? b1 : o0);
          b0 = up ? o0 : b0;
        }
        const double gv = (s.group_score == 2 && per > 1) ? b0 + b1 : b0;
        const bool head = g < a.n_group && lane % lpg == 0;
        uint64_t kept = 0;
        uint32_t m = 0;
        int at = 0;
        uint32_t gh[1], gl[1] = {0u};
        if constexpr (F64) {
          const uint64_t gk = f64_key(gv);
          gh[0] = head ? (uint32_t)(gk >> 32) : 0u;
          gl[0] = (uint32_t)gk;
        } else {
          gh[0] = head ? f32_key((float)gv) : 0u;  // (a sum of two fp32 keys: one more half step)
        }
        for (int r = 0; r < a.topk_group; ++r)
          kept |= __ballot(take_best<64, 1, F64>(gh, gl, ~0ull, (1ull << lane) - 1, m, at));  // the groups' first lanes
        if constexpr (WIDE && !F64) {
          // (keys of opposite sign may leave a small sum: their own roundings count)
          const float size = head && s.group_score == 2 ? fmaxf(fabsf((float)b0), per > 1 ? fabsf((float)b1) : 0.f) : 0.f;
          if (a.topk_group < a.n_group)
            sure = decided(m, lanes_max_u32<64>(gh[0]), slack + 0x1p-20f * lanes_max<64>(size));
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = ll * EPL + i;
          const int ge = e < E ? e / per : 0;
          if (!((kept >> (ge * lpg)) & 1ull)) hi[i] = 0u;
        }
        __builtin_amdgcn_wave_barrier();
      }
      uint32_t taken = 0;  // lane j of the token: its j-th key
      for (int j = 0; j < K; ++j) {
        int at = 0;
        uint32_t m;
        const bool own = take_best<LPT, EPL, F64>(hi, lo, lanes, lower, m, at);
        if constexpr (LPT == 64) {
          const int e = __builtin_amdgcn_readlane(ll * EPL + at, __builtin_ctzll(__ballot(own)));
          chosen = lane == j ? e : chosen;
        } else if (own && tv) {
          id_row[j] = ll * EPL + at;
        }
        if constexpr (WIDE && !F64) taken = ll == j ? m : taken;
      }
      if constexpr (WIDE && !F64) {
        if (s.bias) {
          uint32_t best = hi[0];
#pragma unroll
          for (int i = 1; i < EPL; ++i) best = hi[i] > best ? hi[i] : best;
          best = lanes_max_u32<LPT>(best);
          // each key taken against the next, the last against the best that is left
          uint32_t next = (uint32_t)__shfl((int)taken, lane + 1);
          next = ll == K - 1 ? best : next;
          sure = sure && (ll >= K || (ll == K - 1 && best == 0u) || decided(taken, next, slack));
        }
      }
      return sure;
    };
    const bool sure = choose(std::false_type{});
    if constexpr (WIDE) {
      if (__ballot(!sure) != 0) choose(std::true_type{});
    }
    // lane j < K of the token: its j-th expert and weight
    const bool mine = ll < K;
    int id = 0;
    if constexpr (LPT == 64) {
      id = mine ? chosen : 0;
      if (mine) id_row[ll] = id;
    } else {
      wave_lds_order();
      id = mine ? id_row[ll] : 0;
    }
    const float xc = mine ? load_logit(a.logits, row + id, s.f32) : 0.f;
    float w;
    if (s.renormalize) {
      const float z = !mine ? -INFINITY : sigmoid ? log_sigmoid(xc) : xc;
      float zm = lanes_max<LPT>(z);
      if (zm == -INFINITY) zm = 0.f;
      const float q = mine ? expf(z - zm) : 0.f;
      const float qs = lanes_sum<LPT>(q);
      w = q / (qs == 0.f ? 1.f : qs);
    } else if (sigmoid) {
      w = 1.f / (1.f + expf(-xc));
    } else {
      w = expf(xc - mx) / total;
    }
    if (mine && tv) {
      a.ids[(size_t)t * K + ll] = id;
      a.weights[(size_t)t * K + ll] = s.scale * w;
      atomicAdd(&hist_w[wave * E + id], 1);
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  pack_block<MULTI>(a, hist_w, ids_l, tot, wgbase, waves, threads, t_begin, w_begin, w_end);
}

// Gradient of the weights to the logits, g_j = dL/dw_j of the j-th chosen expert:
//   softmax             dl_e = c p_e (sum_{j: id_j = e} g_j - sum_j g_j p_{id_j})
//   softmax, renorm     dl_{id_j} += c q_j (g_j - sum_i q_i g_i),  q = softmax over the chosen
//   sigmoid             dl_{id_j} += c s_j (1 - s_j) g_j
//   sigmoid, renorm     dl_{id_j} += c q_j (1 - s_j) (g_j - sum_i q_i g_i),  q = s / sum s
// The k terms of a token meet in an LDS row of E floats: of equal ids the first lane writes
// their sum (taken in j order, so results do not depend on timing), and the row leaves as
// whole vectors.  Bound by latency (8192 x 128 fp32, 8.9 MB: 5 us).
template <int LPT, int VEC, int CH>
__global__ __launch_bounds__(256) void scored_backward_kernel(const ScoredBackwardArgs P) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int TPW = 64 / LPT;
  const int E = P.E, K = P.K;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane / LPT, ll = lane % LPT;
  const int pitch = (E + 3) & ~3;
  float *at = reinterpret_cast<float *>(smem) + (wave * TPW + sub) * pitch;
  const long long t = (block_of_grid() * 4 + wave) * TPW + sub;
  const bool tv = t < P.T;
  const size_t row = (size_t)(tv ? t : 0) * E;
  const bool sigmoid = P.score == MOE_LORA_SCORE_SIGMOID;
  const bool dense = !sigmoid && !P.renormalize;

  for (int e = ll * VEC; e < E; e += LPT * VEC)
#pragma unroll
    for (int q = 0; q < VEC; ++q) at[e + q] = 0.f;
  // lane j: the j-th chosen expert (an index outside the experts takes no part)
  int id = -1;
  float g = 0.f;
  if (tv && ll < K) {
    id = P.ids[(size_t)t * K + ll];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) g = P.d_weights[(size_t)t * K + ll];
  }
  float x[CH][VEC];
  float mx = 0.f, inv = 0.f;
  if (dense) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * LPT + ll) * VEC;
      if (VEC == 4 && e < E) {
        if (P.f32) {
          const f32x4_t v = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(P.logits) + row + e);
#pragma unroll
          for (int q = 0; q < VEC; ++q) x[c][q] = v[q];
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(P.logits) + row + e);
#pragma unroll
          for (int q = 0; q < VEC; ++q) x[c][q] = bf16_to_f32((v[q >> 1] >> (16 * (q & 1))) & 0xffffu);
        }
      } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) x[c][q] = e + q < E ? load_logit(P.logits, row + e + q, P.f32) : -INFINITY;
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) m = fmaxf(m, x[c][q]);
    }
    mx = lanes_max<LPT>(m);
    if (mx == -INFINITY) mx = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        x[c][q] = expf(x[c][q] - mx);  // 0 past the last expert
        sum += x[c][q];
      }
    sum = lanes_sum<LPT>(sum);
    inv = 1.f / (sum == 0.f ? 1.f : sum);
  } else {
    const float xc = id >= 0 ? load_logit(P.logits, row + id, P.f32) : -INFINITY;
    const float rest = sigmoid ? 1.f / (1.f + expf(xc)) : 1.f;  // 1 - s
    if (P.renormalize) {
      const float z = sigmoid ? log_sigmoid(xc) : xc;
      float zm = lanes_max<LPT>(z);
      if (zm == -INFINITY) zm = 0.f;
      float q = id >= 0 ? expf(z - zm) : 0.f;
      const float qs = lanes_sum<LPT>(q);
      q = q / (qs == 0.f ? 1.f : qs);
      g = q * (g - lanes_sum<LPT>(q * g)) * rest;
    } else {
      g = g * rest / (1.f + expf(-xc));
    }
    if (id < 0) g = 0.f;
  }
  // equal ids: the first lane carries the sum
  bool first = id >= 0;
  float sum_g = 0.f;
  for (int j = 0; j < K; ++j) {
    const int src = sub * LPT + j;
    const int oid = __shfl(id, src);
    const float og = __shfl(g, src);
    if (oid == id) {
      sum_g += og;
      if (j < ll) first = false;
    }
  }
  wave_lds_order();
  if (first) at[id] = sum_g;
  wave_lds_order();
  float d[CH][VEC];
  float dot = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      const int e = (c * LPT + ll) * VEC + q;
      d[c][q] = e < E ? at[e] : 0.f;
      if (dense) {
        x[c][q] *= inv;
        dot += x[c][q] * d[c][q];
      }
    }
  if (dense) dot = lanes_sum<LPT>(dot);
  if (!tv) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * LPT + ll) * VEC;
    float o[VEC];
#pragma unroll
    for (int q = 0; q < VEC; ++q) o[q] = P.scale * (dense ? x[c][q] * (d[c][q] - dot) : d[c][q]);
    if (VEC == 4) {
      if (e < E) {
        if (P.f32)
          *reinterpret_cast<f32x4_t *>(static_cast<float *>(P.d_logits) + row + e) = f32x4_t{o[0], o[1], o[2], o[3]};
        else
          *reinterpret_cast<u32x2_t *>(static_cast<uint16_t *>(P.d_logits) + row + e) =
              u32x2_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    } else if (e < E) {
      if (P.f32)
        static_cast<float *>(P.d_logits)[row + e] = o[0];
      else
        static_cast<uint16_t *>(P.d_logits)[row + e] = (uint16_t)f32_to_bf16(o[0]);
    }
  }
}

struct Plan {
  int waves, tok_per_wg, num_wg, lpt;
  size_t lds;
};

// Lanes per token: groups take a whole wavefront (their keys' LDS rows, one per wave, would
// not fit for four tokens at 512 experts), and so do k > 16 (one lane per chosen expert)
// and batches too small to fill the device with four tokens a wave.  One workgroup and one
// launch up to 64 tokens; up to 16 where the keys are scores, whose choice takes a wavefront
// longer (64 tokens, 256 experts in 8 groups: 38 us in one workgroup, 19 in four and a second
// launch).
Plan plan_scored(int T, int E, int K, bool groups, bool wide) {
  Plan p;
  p.lpt = (groups || K > 16 || T <= 4096) ? 64 : 16;
  const int per = 64 / p.lpt;
  if (T <= (wide ? kScoredOneWgWide : kScoredOneWg)) {
    p.waves = T < 16 ? T : 16;
    p.tok_per_wg = T;
    p.num_wg = 1;
  } else {
    p.waves = 16;
    p.tok_per_wg = 16 * per;
    int n = (T + p.tok_per_wg - 1) / p.tok_per_wg;
    if (n > kMaxRouteWg) {
      p.tok_per_wg = (T + kMaxRouteWg - 1) / kMaxRouteWg;
      n = (T + p.tok_per_wg - 1) / p.tok_per_wg;
    }
    p.num_wg = n;
  }
  p.lds = ((size_t)(p.waves * E + 2 * E + p.tok_per_wg * K) * 4 + 15) & ~(size_t)15;
  if (groups) p.lds += (size_t)p.waves * E * sizeof(double);
  return p;
}

template <int LPT, int EPL, bool WIDE, bool MULTI>
int launch_one(const ScoredParams &P, const Plan &p, hipStream_t s) {
  // (the attribute is per device and kernel, and cheap: set when the default does not do)
  if (p.lds > 64 * 1024 &&
      hipFuncSetAttribute((const void *)scored_kernel<LPT, EPL, WIDE, MULTI>,
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds) != hipSuccess)
    return ST_HIP;
  scored_kernel<LPT, EPL, WIDE, MULTI><<<p.num_wg, p.waves * 64, p.lds, s>>>(P);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

template <int LPT, int EPL>
int launch_keys(const ScoredParams &P, const Plan &p, bool wide, hipStream_t s) {
  if (p.num_wg > 1)
    return wide ? launch_one<LPT, EPL, true, true>(P, p, s) : launch_one<LPT, EPL, false, true>(P, p, s);
  return wide ? launch_one<LPT, EPL, true, false>(P, p, s) : launch_one<LPT, EPL, false, false>(P, p, s);
}

template <int LPT>
int launch_experts(const ScoredParams &P, const Plan &p, bool wide, hipStream_t s) {
  const int need = (P.r.a.E + LPT - 1) / LPT;
  if (need <= 1) return launch_keys<LPT, 1>(P, p, wide, s);
  if (need <= 2) return launch_keys<LPT, 2>(P, p, wide, s);
  if (need <= 4) return launch_keys<LPT, 4>(P, p, wide, s);
  if (need <= 8) return launch_keys<LPT, 8>(P, p, wide, s);
  if constexpr (LPT == 16) {
    if (need <= 16) return launch_keys<LPT, 16>(P, p, wide, s);
    return launch_keys<LPT, 32>(P, p, wide, s);
  }
  return ST_UNSUPPORTED;
}

template <int LPT, int VEC>
int launch_backward(const ScoredBackwardArgs &a, hipStream_t s) {
  const int per_wg = 4 * (64 / LPT);
  const int chunks = (a.E + LPT * VEC - 1) / (LPT * VEC);
  const size_t lds = (size_t)per_wg * ((a.E + 3) & ~3) * sizeof(float);
  const dim3 grid = grid_of_blocks(((long long)a.T + per_wg - 1) / per_wg);
#define MOE_BWD(CH) scored_backward_kernel<LPT, VEC, CH><<<grid, 256, lds, s>>>(a)
  if (chunks <= 1)
    MOE_BWD(1);
  else if (chunks <= 2)
    MOE_BWD(2);
  else if (chunks <= 4)
    MOE_BWD(4);
  else
    MOE_BWD(8);
#undef MOE_BWD
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace

size_t scored_workspace_bytes(int T, int E, int K, bool groups, bool wide) {
  const Plan p = plan_scored(T, E, K, groups, wide);
  return p.num_wg > 1 ? (size_t)p.num_wg * E * sizeof(int32_t) : 0;
}

bool scored_wide(bool bias, int n_group, int group_score) { return bias || (n_group > 1 && group_score == 2); }

int scored_max_tokens() { return kMaxRouteWg * kScoredMaxTok; }

int launch_route_scored(const RouteArgs &a, const ScoredArgs &s, hipStream_t st) {
  const bool groups = a.n_group > 1;
  // fp64 keys: where a bias or a group's sum of two compares scores
  const bool wide = scored_wide(s.bias != nullptr, a.n_group, s.group_score);
  const Plan p = plan_scored(a.T, a.E, a.K, groups, wide);
  ScoredParams P;
  P.r.a = a;
  P.r.tok_per_wg = p.tok_per_wg;
  P.r.num_wg = p.num_wg;
  P.s = s;
  const int r = p.lpt == 64 ? launch_experts<64>(P, p, wide, st) : launch_experts<16>(P, p, wide, st);
  if (r != ST_OK || p.num_wg == 1) return r;
  return launch_route_finish(P.r, st);
}

int launch_route_scored_backward(const ScoredBackwardArgs &a, hipStream_t s) {
  // four tokens per wave where a token's chosen experts and logits fit 16 lanes
  const bool vec = a.E % 4 == 0;
  if (a.K <= 16 && a.E <= (vec ? 512 : 128))
    return vec ? launch_backward<16, 4>(a, s) : launch_backward<16, 1>(a, s);
  return vec ? launch_backward<64, 4>(a, s) : launch_backward<64, 1>(a, s);
}

}  // namespace moe
