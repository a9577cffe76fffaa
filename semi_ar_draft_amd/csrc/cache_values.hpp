// Values of a key-value cache: to e4m3 and to MXFP4 (e2m1 values with a power of
// two for each 32 of them), and what the kernels that write them share.
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace dspark {

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  bf16x2_t r;
  r[0] = (__bf16)lo;                                     // to nearest even
  r[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

// The bf16 values of a word.
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = low_bf16(w[i]);
    f[2 * i + 1] = high_bf16(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
}

// x / s as the e4m3 value nearest the exact quotient (ties to even, larger
// magnitudes kept at 448, NaN as NaN).  A float quotient q may have been
// rounded onto a border between two e4m3 values that the exact quotient
// misses, so its last bit is made sticky: with r = x - q s (its sign is
// exact) nonzero, an even q moves one step towards the exact quotient; an
// odd q lies on no border (those end in zeros).
__device__ __forceinline__ float quotient_sticky(float x, float s, float rs) {
  const float q0 = x * rs;
  // infinities, and what stays beyond 448 whatever the last bits are
  if (!(__builtin_fabsf(q0) < 512.0f)) return q0 != q0 ? q0 : __builtin_copysignf(448.0f, q0);
  const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, x), rs, q0);
  const float r = __builtin_fmaf(-q, s, x);
  const uint32_t u = __float_as_uint(q);
  // r with the sign of x: |q| falls short of |x / s|
  const bool up = (__float_as_uint(r) ^ __float_as_uint(x)) >> 31 == 0;
  const bool move = r != 0.0f && (u & 1u) == 0 && (u << 1) != 0;
  const float t = __uint_as_float(move ? (up ? u + 1 : u - 1) : u);
  return __builtin_fminf(__builtin_fmaxf(t, -448.0f), 448.0f);
}

// A double as a float whose last bit is set where it is not exact: rounded to
// a type of fewer bits (whose borders end in zeros) it goes where the double
// itself would.
__device__ __forceinline__ float to_odd(double y) {
  const float f = (float)y;
  const double r = y - (double)f;                        // NaN for an infinite y: stays as it is
  const uint32_t u = __float_as_uint(f);
  const bool even = (u & 1u) == 0;
  // (0 with a remainder, from below the least float, moves away from 0 as well)
  const bool up = (r > 0) == (y > 0);
  return __uint_as_float(even && (r > 0 || r < 0) ? (up || (u << 1) == 0 ? u + 1 : u - 1) : u);
}

__device__ __forceinline__ uint32_t pack4_e4m3(const float (&q)[4]) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  return (uint32_t)w;
}

// Eight values over s as e4m3.
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], float s, float rs) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient_sticky(x[4 * j + i], s, rs);
    w[j] = pack4_e4m3(q);
  }
  return make_uint2(w[0], w[1]);
}

// The largest x of the four lanes of a quad, all of which have to be active.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t y = __builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false);   // quad_perm [1, 0, 3, 2]
  const uint32_t m = x > y ? x : y;
  const uint32_t z = __builtin_amdgcn_update_dpp(m, m, 0x4E, 0xF, 0xF, false);   // quad_perm [2, 3, 0, 1]
  return m > z ? m : z;
}

// Eight values of a block whose 32 a quad of lanes holds, as e2m1 codes: the
// word of this lane's and the byte of the block's power.  The power is the
// least 2^e whose 7 is no less than the largest magnitude A = m 2^x: e = x - 2,
// or x - 1 where m > 1.75, so every value, the largest too, is off by half
// the distance of its neighbours at most; e stays within -120 .. 125 (results
// normal floats, 6 2^e finite; what passes 6 2^125, infinities too, becomes
// that).  A block of zeros has the power 1, one with a NaN the byte 255 and
// codes 0.
__device__ __forceinline__ uint32_t to_mxfp4(const float (&x)[8], unsigned char& power) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;   // larger for larger magnitudes, above all for NaN
    top = u > top ? u : top;
  }
  top = quad_max(top);
  int b = (int)((top + 0x1FFFFFu) >> 23) - 2;            // a mantissa above 0.75 carries
  b = top == 0 ? 127 : b < 7 ? 7 : b > 252 ? 252 : b;
  const float p = __uint_as_float((uint32_t)b << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], p, 0);   // ties to even, magnitudes above 6 kept at 6
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], p, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], p, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], p, 3);
  const bool nan = top > 0x7F800000u;
  power = nan ? 255 : (unsigned char)b;
  return nan ? 0 : w;
}

// Eight e2m1 codes times 2^(power - 127) as bf16 (255: NaN): exact.
__device__ __forceinline__ uint4 from_mxfp4(uint32_t w, unsigned char power) {
  const float p = __uint_as_float((uint32_t)power << 23);
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 3)));
}

}  // namespace dspark
