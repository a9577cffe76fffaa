// Keys and values of a step's packed rows into their slots of the paged
// cache, as bf16, rounded to e4m3 with a scale per head, or to e2m1 with a
// power of two for each 32 of them (MXFP4); and rows of a cache back as bf16.
//
// Copies with a scattered side: bound by memory (at a step's few
// rows by the launch).  A thread owns 16 bytes of the key cache and of the
// value cache (MXFP4: 4, of eight values, whose block's largest the lanes of
// a quad find together), so both tensors' loads are in flight together, and
// consecutive threads write consecutive bytes of a token's head.  Measured:
// 16381 rows of 8 heads of 128 into e4m3, 101 MB, 24.4 us (4.1 TB/s, a copy
// reaches 4.8); a step's rows of 128 requests 3.3 us; 32749 rows of 8 heads of
// 128 back from MXFP4, 170 MB of which 134 are written, 34.9 us (4.9 TB/s);
// 63 rows into MXFP4 3.0, back 2.8.
#include "cache_values.hpp"

namespace dspark {
namespace {

// 16 bytes of a bf16 or e4m3 cache.
template <int F>
__device__ __forceinline__ uint4 to_cache(const uint16_t* p, float s, float rs) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  if constexpr (F == kCacheBf16) return x;
  const uint4 y = reinterpret_cast<const uint4*>(p)[1];
  float f[2][8];
  unpack8(x, f[0]);
  unpack8(y, f[1]);
  const uint2 lo = to_e4m3(f[0], s, rs), hi = to_e4m3(f[1], s, rs);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Where a thread's values stand: row, chunk, head, first value; place in the cache.  Whether there is one.
struct Spot {
  unsigned row;
  int h, d0, page, place;
  int64_t to;
};

__device__ __forceinline__ bool find(const CacheWriteArgs& a, int elems, Spot& s) {
  const unsigned i = blockIdx.x * kCacheThreads + threadIdx.x;
  s.row = i / (unsigned)a.chunks;
  if (s.row >= (unsigned)a.n_rows) return false;
  const unsigned c = i - s.row * (unsigned)a.chunks;
  const int slot = a.slot[s.row];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1 && c == 0) atomicOr(a.err, kErrSlot);
    return false;
  }
  s.h = c >> a.chunk_shift;
  s.d0 = (c & ((1 << a.chunk_shift) - 1)) * elems;
  s.page = slot >> a.page_shift;
  s.place = slot & ((1 << a.page_shift) - 1);
  s.to = (int64_t)s.page * a.c_page + (int64_t)s.place * a.c_tok + (int64_t)s.h * a.c_head;
  return true;
}

template <int F>
__global__ __launch_bounds__(kCacheThreads) void cache_write_impl(const CacheWriteArgs a) {
  Spot s;
  if (!find(a, F == kCacheE4m3 ? 16 : 8, s)) return;
  float ks = 1.0f, vs = 1.0f;
  if constexpr (F == kCacheE4m3) {
    if (a.k_scale) ks = a.k_scale[s.h];
    if (a.v_scale) vs = a.v_scale[s.h];
  }
  const uint4 k = to_cache<F>(a.k + s.row * a.k_row + s.h * a.k_head + s.d0, ks, 1.0f / ks);
  const uint4 v = to_cache<F>(a.v + s.row * a.v_row + s.h * a.v_head + s.d0, vs, 1.0f / vs);
  const int64_t at = s.to + (F == kCacheE4m3 ? s.d0 : 2 * s.d0);
  *reinterpret_cast<uint4*>(a.kc + at) = k;
  *reinterpret_cast<uint4*>(a.vc + at) = v;
}

__global__ __launch_bounds__(kCacheThreads) void cache_write_mxfp4_impl(const CacheWritePowers p) {
  const CacheWriteArgs& a = p.w;
  Spot s;
  if (!find(a, 8, s)) return;
  const uint4 xk = *reinterpret_cast<const uint4*>(a.k + s.row * a.k_row + s.h * a.k_head + s.d0);
  const uint4 xv = *reinterpret_cast<const uint4*>(a.v + s.row * a.v_row + s.h * a.v_head + s.d0);
  float k[8], v[8];
  unpack8(xk, k);
  unpack8(xv, v);
  unsigned char pk, pv;
  const uint32_t wk = to_mxfp4(k, pk), wv = to_mxfp4(v, pv);
  *reinterpret_cast<uint32_t*>(a.kc + s.to + s.d0 / 2) = wk;
  *reinterpret_cast<uint32_t*>(a.vc + s.to + s.d0 / 2) = wv;
  if ((threadIdx.x & 3) == 0) {
    const int64_t at = s.page * p.s_page + s.h * p.s_head + (int64_t)s.place * p.blocks + s.d0 / 32;
    p.k_power[at] = pk;
    p.v_power[at] = pv;
  }
}

// Eight values of a cache as bf16: the product with an e4m3 cache's scale is
// rounded to float32 and that to bf16, MXFP4 values are exact.
template <int F>
__device__ __forceinline__ uint4 from_cache(const unsigned char* p, float s, unsigned char power) {
  if constexpr (F == kCacheBf16) {
    return *reinterpret_cast<const uint4*>(p);
  } else if constexpr (F == kCacheMxfp4) {
    return from_mxfp4(*reinterpret_cast<const uint32_t*>(p), power);
  } else {
    typedef __attribute__((ext_vector_type(2))) float f32x2_t;
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    const f32x2_t f[4] = {__builtin_amdgcn_cvt_pk_f32_fp8(x.x, false), __builtin_amdgcn_cvt_pk_f32_fp8(x.x, true),
                          __builtin_amdgcn_cvt_pk_f32_fp8(x.y, false), __builtin_amdgcn_cvt_pk_f32_fp8(x.y, true)};
    return make_uint4(pack2_bf16(f[0][0] * s, f[0][1] * s), pack2_bf16(f[1][0] * s, f[1][1] * s),
                      pack2_bf16(f[2][0] * s, f[2][1] * s), pack2_bf16(f[3][0] * s, f[3][1] * s));
  }
}

template <int F>
__global__ __launch_bounds__(kCacheThreads) void cache_read_impl(const CacheReadArgs a) {
  const unsigned i = blockIdx.x * kCacheThreads + threadIdx.x;
  const unsigned row = i / (unsigned)a.chunks;
  if (row >= (unsigned)a.n_rows) return;
  const unsigned c = i - row * (unsigned)a.chunks;
  const int slot = a.slot[row];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1 && c == 0) atomicOr(a.err, kErrSlot);
    return;
  }
  const int h = c >> a.chunk_shift;
  const int d0 = (c & ((1 << a.chunk_shift) - 1)) * 8;
  const int page = slot >> a.page_shift, place = slot & ((1 << a.page_shift) - 1);
  const int64_t from = (int64_t)page * a.c_page + (int64_t)place * a.c_tok + (int64_t)h * a.c_head +
                       (F == kCacheBf16 ? 2 * d0 : F == kCacheE4m3 ? d0 : d0 / 2);
  float ks = 1.0f, vs = 1.0f;
  unsigned char kp = 0, vp = 0;
  if constexpr (F == kCacheE4m3) {
    if (a.k_scale) ks = a.k_scale[h];
    if (a.v_scale) vs = a.v_scale[h];
  }
  if constexpr (F == kCacheMxfp4) {
    const int64_t at = page * a.s_page + h * a.s_head + (int64_t)place * a.blocks + d0 / 32;
    kp = a.k_power[at];
    vp = a.v_power[at];
  }
  const uint4 k = from_cache<F>(a.kc + from, ks, kp), v = from_cache<F>(a.vc + from, vs, vp);
  *reinterpret_cast<uint4*>(a.k + row * a.k_row + h * a.k_head + d0) = k;
  *reinterpret_cast<uint4*>(a.v + row * a.v_row + h * a.v_head + d0) = v;
}

}  // namespace

const void* cache_write_kernel(int type) {
  return type == kCacheMxfp4  ? (const void*)&cache_write_mxfp4_impl
         : type == kCacheE4m3 ? (const void*)&cache_write_impl<kCacheE4m3>
                              : (const void*)&cache_write_impl<kCacheBf16>;
}

const void* cache_read_kernel(int type) {
  return type == kCacheMxfp4  ? (const void*)&cache_read_impl<kCacheMxfp4>
         : type == kCacheE4m3 ? (const void*)&cache_read_impl<kCacheE4m3>
                              : (const void*)&cache_read_impl<kCacheBf16>;
}

}  // namespace dspark
