// Keys and values of a step's packed rows into their slots of the paged
// cache, as bf16 or rounded to e4m3 with a scale per head.
//
// A copy with a scattered destination: bound by memory (at a step's few
// rows by the launch).  A thread owns 16 bytes of the key cache and of the
// value cache, so both tensors' loads are in flight together, and consecutive
// threads write consecutive bytes of a token's head.  Measured: 16381 rows of 8
// heads of 128 into e4m3, 101 MB, 24.4 us (4.1 TB/s, a copy reaches 4.8); a
// step's rows of 128 requests 3.3 us.
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

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

__device__ __forceinline__ uint32_t pack4(const float (&q)[4]) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
  return (uint32_t)w;
}

template <int E4M3>
__device__ __forceinline__ uint4 to_cache(const uint16_t* p, float s, float rs) {
  if constexpr (!E4M3) return *reinterpret_cast<const uint4*>(p);
  const uint4 x[2] = {reinterpret_cast<const uint4*>(p)[0], reinterpret_cast<const uint4*>(p)[1]};
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w0 = j & 1 ? x[j >> 1].z : x[j >> 1].x, w1 = j & 1 ? x[j >> 1].w : x[j >> 1].y;
    const float v[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u), __uint_as_float(w1 << 16),
                        __uint_as_float(w1 & 0xFFFF0000u)};
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient_sticky(v[i], s, rs);
    out[j] = pack4(q);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int E4M3>
__global__ __launch_bounds__(kCacheThreads) void cache_write_impl(const CacheWriteArgs a) {
  const unsigned i = blockIdx.x * kCacheThreads + threadIdx.x;
  const unsigned row = i / (unsigned)a.chunks;
  if (row >= (unsigned)a.n_rows) return;
  const unsigned c = i - row * (unsigned)a.chunks;
  const int slot = a.slot[row];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1 && c == 0) atomicOr(a.err, kErrSlot);
    return;
  }
  constexpr int kElems = E4M3 ? 16 : 8;
  const int h = c >> a.chunk_shift;
  const int d0 = (c & ((1 << a.chunk_shift) - 1)) * kElems;
  const int64_t to = (int64_t)(slot >> a.page_shift) * a.c_page + (int64_t)(slot & ((1 << a.page_shift) - 1)) * a.c_tok +
                     (int64_t)h * a.c_head + (E4M3 ? d0 : 2 * d0);
  float ks = 1.0f, vs = 1.0f;
  if constexpr (E4M3) {
    if (a.k_scale) ks = a.k_scale[h];
    if (a.v_scale) vs = a.v_scale[h];
  }
  const uint4 k = to_cache<E4M3>(a.k + row * a.k_row + h * a.k_head + d0, ks, 1.0f / ks);
  const uint4 v = to_cache<E4M3>(a.v + row * a.v_row + h * a.v_head + d0, vs, 1.0f / vs);
  *reinterpret_cast<uint4*>(a.kc + to) = k;
  *reinterpret_cast<uint4*>(a.vc + to) = v;
}

}  // namespace

const void* cache_write_kernel(int e4m3) {
  return e4m3 ? (const void*)&cache_write_impl<1> : (const void*)&cache_write_impl<0>;
}

}  // namespace dspark
