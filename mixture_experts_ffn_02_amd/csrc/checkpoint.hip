// 8-bit checkpoints of bf16 rows (gfx950).
//
// Of each 32 neighbours of a row: e = the smallest exponent (at least -117) with
// max|x| <= 448 * 2^e, code = E4M3(x * 2^-e) rounded to nearest even.  The scale is a power
// of two, so x * 2^-e is exact, a value is rounded once (at most 2^-4 of it), and decoding
// into bf16 is exact.  The exponent comes from the largest magnitude's bits alone.
//
// One thread holds 8 values (a 16-byte load), four neighbouring lanes a block; the maximum
// joins over them with two DPP moves.  Bound by HBM: 2 bytes read and 1 + 1/32 written per
// value (packing), the reverse for unpacking.  The codes, read a whole pass later, are stored
// past the caches, and so are large unpacked rows (65536 x 2048 with the inputs in no cache:
// packing 71.5 -> 70.1 us, unpacking 73.5 -> 70.9, 5.8 TB/s; with the same inputs again, which
// then stay in the memory-side cache, 72.8 -> 60.9 and 74.8 -> 58.0).
#include "checkpoint.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;  // loads in flight per thread

MOE_DEV uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);  // xor 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);  // xor 2
  return o > v ? o : v;
}

MOE_DEV uint32_t max16(uint32_t a) {
  const uint32_t lo = a & 0x7fffu, hi = (a >> 16) & 0x7fffu;
  return lo > hi ? lo : hi;
}

// the codes of 8 values and, through biased, their block's exponent.  All four lanes of a
// block call it.
MOE_DEV u32x2_t encode8(const u32x4_t &x, uint32_t &biased) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = max16(x[i]);
    m = v > m ? v : m;
  }
  m = quad_max(m);
  // rare: not-finite values, or magnitudes that would round up to 2^128
  const bool odd = m >= 0x7f78u;
  u32x4_t f = x;
  uint32_t bad = 0;  // bit i: value i is not finite
  if (__ballot(odd) != 0) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t b = (x[i >> 1] >> (16 * (i & 1))) & 0xffffu;
      if ((b & 0x7fffu) >= 0x7f80u) {
        bad |= 1u << i;
        b = 0;
      } else if ((b & 0x7fffu) > 0x7f70u) {
        m = 0x7f78u;                   // the block's exponent is that of the value itself
        b = (b & 0x8000u) | 0x7f70u;   // 240 * 2^120, the largest code whose value is finite
      }
      const uint32_t a = b & 0x7fffu;
      m = a > m ? a : m;
      f[i >> 1] = (f[i >> 1] & (i & 1 ? 0x0000ffffu : 0xffff0000u)) | (b << (16 * (i & 1)));
    }
    m = quad_max(m);
  }
  const uint32_t e8 = (m >> 7) + ((m & 127u) > 96u ? 1u : 0u);  // mantissa above 1.75
  biased = e8 > (uint32_t)kCkptMinExp + 8u ? e8 - 8u : (uint32_t)kCkptMinExp;
  const float inv = __uint_as_float((254u - biased) << 23);
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(f[2 * h] << 16) * inv,
                                        __uint_as_float(f[2 * h] & 0xffff0000u) * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(f[2 * h + 1] << 16) * inv,
                                        __uint_as_float(f[2 * h + 1] & 0xffff0000u) * inv, w, true);
    c[h] = (uint32_t)w;
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((bad >> i) & 1u) c[i >> 2] = (c[i >> 2] & ~(0xffu << (8 * (i & 3)))) | (0x7fu << (8 * (i & 3)));
  }
  return c;
}

// Threads of a workgroup: `across` of them (a multiple of 4) over a row's 8-value chunks,
// `down` rows side by side; each thread takes kRowsPerThread row groups.
struct CkptShape {
  long long rows;
  int cols, blocks;   // blocks of 32 per row
  int across, down;   // across * down <= kThreads
};

template <bool PACK, bool NT>
__global__ __launch_bounds__(kThreads) void checkpoint_kernel(const CkptShape S, const uint16_t *__restrict__ src,
                                                              uint16_t *__restrict__ dst,
                                                              uint8_t *__restrict__ codes_out,
                                                              uint8_t *__restrict__ exps_out,
                                                              const uint8_t *__restrict__ codes_in,
                                                              const uint8_t *__restrict__ exps_in) {
  const int r = threadIdx.x / S.across, c0 = threadIdx.x % S.across;
  if (r >= S.down) return;  // (whole blocks of four lanes: across is a multiple of 4)
  const long long row0 = (long long)blockIdx.x * (S.down * kRowsPerThread) + r;
  for (int c = c0; c < S.blocks * 4; c += S.across) {
    const bool in = c * 8 < S.cols;
    if constexpr (PACK) {
      u32x4_t x[kRowsPerThread];
#pragma unroll
      for (int u = 0; u < kRowsPerThread; ++u) {
        const long long row = row0 + u * S.down;
        x[u] = zero_u32x4();
        if (in && row < S.rows) x[u] = *reinterpret_cast<const u32x4_t *>(src + row * S.cols + c * 8);
      }
#pragma unroll
      for (int u = 0; u < kRowsPerThread; ++u) {
        const long long row = row0 + u * S.down;
        uint32_t biased;
        const u32x2_t w = encode8(x[u], biased);
        if (row < S.rows) {
          if (in) store_stream<NT>(reinterpret_cast<u32x2_t *>(codes_out + row * S.cols + c * 8), w);
          if ((c & 3) == 0) exps_out[row * S.blocks + (c >> 2)] = (uint8_t)biased;
        }
      }
    } else {
      u32x2_t w[kRowsPerThread];
      uint32_t e[kRowsPerThread];
#pragma unroll
      for (int u = 0; u < kRowsPerThread; ++u) {
        const long long row = row0 + u * S.down;
        w[u] = u32x2_t{0u, 0u};
        e[u] = 127u;
        if (in && row < S.rows) {
          w[u] = *reinterpret_cast<const u32x2_t *>(codes_in + row * S.cols + c * 8);
          e[u] = exps_in[row * S.blocks + (c >> 2)];
        }
      }
#pragma unroll
      for (int u = 0; u < kRowsPerThread; ++u) {
        const long long row = row0 + u * S.down;
        if (in && row < S.rows)
          store_stream<NT>(reinterpret_cast<u32x4_t *>(dst + row * S.cols + c * 8), ckpt_to_bf16(w[u], ckpt_scale(e[u])));
      }
    }
  }
}

CkptShape shape_of(long long rows, int cols) {
  CkptShape s;
  s.rows = rows;
  s.cols = cols;
  s.blocks = (cols + kCkptBlock - 1) / kCkptBlock;
  s.across = s.blocks * 4 < kThreads ? s.blocks * 4 : kThreads;
  s.down = kThreads / s.across;
  return s;
}

unsigned grid_of(const CkptShape &s) {
  const long long per = (long long)s.down * kRowsPerThread;
  return (unsigned)((s.rows + per - 1) / per);
}

}  // namespace

int launch_checkpoint_pack(long long rows, int cols, const uint16_t *x, uint8_t *codes, uint8_t *exps, hipStream_t s) {
  const CkptShape S = shape_of(rows, cols);
  checkpoint_kernel<true, true><<<grid_of(S), kThreads, 0, s>>>(S, x, nullptr, codes, exps, nullptr, nullptr);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

int launch_checkpoint_unpack(long long rows, int cols, const uint8_t *codes, const uint8_t *exps, uint16_t *x,
                             hipStream_t s) {
  const CkptShape S = shape_of(rows, cols);
  if ((size_t)rows * cols * 2 > kStreamBytes)
    checkpoint_kernel<false, true><<<grid_of(S), kThreads, 0, s>>>(S, nullptr, x, nullptr, nullptr, codes, exps);
  else
    checkpoint_kernel<false, false><<<grid_of(S), kThreads, 0, s>>>(S, nullptr, x, nullptr, nullptr, codes, exps);
  return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace moe
