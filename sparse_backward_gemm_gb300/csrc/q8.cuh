// 8-bit activation checkpoints: the number format, as device helpers.
//
// 32 consecutive values of a row share one power of two.  Its exponent e is
// the smallest integer >= -120 with max|v| <= L * 2^e, where L is the largest
// 8-bit value (448 for e4m3, 127 for int8); a code is v * 2^-e rounded to the
// nearest 8-bit value, ties to even, and the exponent is kept as the byte
// e + 127.  A group that holds a NaN or an infinity gets the byte 255 and
// decodes to NaN everywhere.  At the top of the range no code stands for 2^128,
// which is no bf16 or f32 number: int8 exponents end at 121, and the codes under
// the largest exponent at 240 (e4m3) and 127.
//
// Why a power of two and not max|v| / L: scaling by it is exact, so a code is
// one rounding of v with no case that depends on how a division rounds, and
// decoding is exact in bf16 (an e4m3 value has 4 significant bits, an int8
// value 7, and the smallest product, 2^-129, is a bf16 denormal).  It costs
// int8 at most one bit (half a bit on average); e4m3 keeps its relative
// precision.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace collider {

constexpr int kQ8Group = 32;
constexpr int kQ8E4m3 = 0, kQ8Int8 = 1;

// the largest exponent byte (but 255), and the largest code value under it
template <int FMT>
constexpr int kQ8TopByte = FMT == kQ8E4m3 ? 247 : 248;
template <int FMT>
constexpr float kQ8TopCode = FMT == kQ8E4m3 ? 240.f : 127.f;
// exponent byte of a group whose largest magnitude is amax >= 0 (NaN or
// infinite: 255).  amax = 1.f * 2^(E-127): L = 1.75 * 2^8 or 1.984375 * 2^6.
template <int FMT>
__device__ __forceinline__ int q8_exp_byte(float amax) {
  const unsigned u = __float_as_uint(amax) & 0x7fffffffu;
  if (u >= 0x7f800000u) return 255;
  const int E = (int)(u >> 23), over = (u & 0x7fffffu) > (FMT == kQ8E4m3 ? 0x600000u : 0x7e0000u);
  return min(max(E + over - (FMT == kQ8E4m3 ? 8 : 6), 7), kQ8TopByte<FMT>);
}
// 2^-(byte - 127) for a byte q8_exp_byte gave (7..248)
__device__ __forceinline__ float q8_inv_scale(int byte) { return __uint_as_float((unsigned)(254 - byte) << 23); }
// 2^(byte - 127) for any byte; 255 is NaN
__device__ __forceinline__ float q8_scale(unsigned byte) {
  const unsigned u = byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23;
  return __uint_as_float(u);
}

// 8 codes of 8 values already scaled by 2^-e
template <int FMT>
__device__ __forceinline__ uint2 q8_encode8(const float* v) {
  uint2 c;
  unsigned* w = reinterpret_cast<unsigned*>(&c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (FMT == kQ8E4m3) {
      const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
      const unsigned hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
      w[k] = lo | (hi << 16);
    } else {
      // v + 1.5 * 2^23 rounds v to a whole number (ties to even) in the low bits
      unsigned b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(v[4 * k + i], 12582912.f));
      w[k] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
  }
  return c;
}

// the 8 values of 8 codes, times scale
template <int FMT>
__device__ __forceinline__ void q8_decode8(uint2 c, float scale, float* v) {
  const unsigned* w = reinterpret_cast<const unsigned*>(&c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (FMT == kQ8E4m3) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k] >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[4 * k + 2 * i] = __fmul_rn(f.x, scale);
        v[4 * k + 2 * i + 1] = __fmul_rn(f.y, scale);
      }
    } else {
      // byte b ^ 0x80 under the exponent of 2^23 is 2^23 + 128 + b
      const unsigned u = w[k] ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[4 * k + i] =
            __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)), 8388736.f), scale);
    }
  }
}

// The j-th (from 0) token that is not in the ascending list idx[0..nk), found
// by the whole warp: the number r of kept tokens before it is the first r with
// idx[r] - r > j.  32 probes a round.  In range for any list: j + r < j + nk + 1.
__device__ __forceinline__ int filtered_token(const int32_t* idx, int nk, int j) {
  int lo = 0, hi = nk;   // the answer r lies in [lo, hi]
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;   // probes lo, lo + step, ...
    const int past = at >= hi || idx[at] - at > j;
    const unsigned m = __ballot_sync(0xffffffffu, past);
    const int first = m ? __ffs(m) - 1 : 32;   // the first probe past j
    if (first == 0) { hi = lo; break; }
    const int nlo = lo + (first - 1) * step + 1;
    const int nhi = min(hi, lo + first * step);
    lo = nlo;
    hi = nhi;
  }
  return j + lo;
}

}  // namespace collider
