// Rotary positions of a step's packed rows: queries and keys to new rows (or in
// place), or queries so and keys and values into their cache slots.
//
// Pair j of a row at position t is turned by a = t f_j: (x0, x1) -> factor
// (x0 cos a - x1 sin a, x1 cos a + x0 sin a).  A far position's angle needs more
// than 24 bits, so turns = t f_j / 2 pi, their fraction, the sine and cosine and
// their products with the factor are float64; a workgroup works them out once for its rows and keeps them in
// LDS, where every head reads them (a row's 64 pairs, 40 heads: a sine and
// cosine for 40 pairs).  What becomes bf16 is turned in float32; keys that a
// cache rounds to 8 or 4 bits in float64, so that a value near a border between
// two of those goes to the side of the exact one.
//
// Bound by memory: 16381 rows of 40 heads of 128 62.4 us (335 MB, 5.4 TB/s, a
// copy of 2 GiB reaches 4.9); 8190 rows, 32 heads to rows and 8 into a bf16 cache
// 40.4 (5.0 TB/s), into e4m3 45.2, into MXFP4 44.4 (4.0), where the keys' float64
// part does not hide whole; a step's 821 rows 6.2.  A row a workgroup: its sines,
// a quarter of its threads' work, pass under the loads of its values, and several
// workgroups of a CU are at different stages (four rows 69.0 us against 62.4).
#include "cache_values.hpp"

namespace dspark {
namespace {

// floor(n / d) for n, d < 2^16, m = 2^32 / d rounded up (d = 1: 0).
__device__ __forceinline__ unsigned divide(unsigned n, unsigned m) { return m ? __umulhi(n, m) : n; }

template <typename T>
__device__ __forceinline__ T turned0(T x0, T x1, T c, T s) { return __builtin_fma(-x1, s, x0 * c); }
template <>
__device__ __forceinline__ float turned0(float x0, float x1, float c, float s) { return __builtin_fmaf(-x1, s, x0 * c); }
template <typename T>
__device__ __forceinline__ T turned1(T x0, T x1, T c, T s) { return __builtin_fma(x0, s, x1 * c); }
template <>
__device__ __forceinline__ float turned1(float x0, float x1, float c, float s) { return __builtin_fmaf(x0, s, x1 * c); }

struct Angle32 {
  float c, s;
};
struct Angle64 {
  double c, s;
};

// factor (cos, sin) of the pairs of this workgroup's rows, [rows][rot / 2].
template <bool WIDE>
__device__ __forceinline__ void angles(const RopeArgs& a, int row0, Angle32* t32, Angle64* t64) {
  const unsigned pairs = a.rot / 2;
  for (unsigned i = threadIdx.x; i < a.rows * pairs; i += kRopeThreads) {
    const unsigned r = divide(i, a.pairs_inv), j = i - r * pairs;
    const int row = row0 + (int)r;
    const int pos = row < a.n_rows ? a.pos[row] : -1;
    if (pos < -1 && j == 0) atomicOr(a.err, kErrPos);
    const double turns = (double)pos * (a.freq[j] * 0.15915494309189533577);   // 1 / 2 pi
    const double part = turns - __builtin_rint(turns);
    double s, c;
    sincospi(part + part, &s, &c);
    c *= a.factor;
    s *= a.factor;
    t32[i] = {(float)c, (float)s};
    if constexpr (WIDE) t64[i] = {c, s};
  }
}

// Heads of this workgroup's rows turned: unit u < rot / 16 of a head is its
// pairs 8 u .. 8 u + 7, the others are eight values that stay as they are.  A
// thread has one unit of every `slots`-th head; a head's values are loaded
// while the one before it is turned, the first one's while the angles are
// worked out, whatever the row's position is, which only the store waits for.
template <bool PAIRED>
struct Heads {
  const RopeArgs& a;
  const Angle32* t32;
  int row0;
  unsigned heads, slots, u, it, row_in;
  bool turned;
  int at0, at1;
  uint16_t* out;                 // of the loaded head; null: none
  uint4 x0, x1;

  __device__ __forceinline__ Heads(const RopeArgs& a_, const Angle32* t, int row0_) : a(a_), t32(t), row0(row0_) {
    heads = a.heads_q + a.heads_k;
    slots = kRopeThreads / a.units;
    it = divide(threadIdx.x, a.units_inv);
    u = threadIdx.x - it * a.units;
    if (it >= slots) it = 1u << 16;                      // a thread too many
    turned = (int)u < a.rot / 16;
    at0 = !turned ? a.rot + 8 * ((int)u - a.rot / 16) : PAIRED ? 16 * u : 8 * u;
    at1 = !turned ? at0 : PAIRED ? at0 + 8 : at0 + a.rot / 2;
    load();
  }

  __device__ __forceinline__ void load() {
    out = nullptr;
    if (it >= a.rows * heads) return;
    row_in = divide(it, a.heads_inv);
    const unsigned head = it - row_in * heads;
    const int row = row0 + (int)row_in;
    if (row >= a.n_rows) return;
    const bool is_k = head >= (unsigned)a.heads_q;
    const int64_t h = is_k ? head - a.heads_q : head;
    const uint16_t* in = is_k ? a.k + row * a.k_row + h * a.k_head : a.q + row * a.q_row + h * a.q_head;
    out = is_k ? a.ko + row * a.ko_row + h * a.ko_head : a.qo + row * a.qo_row + h * a.qo_head;
    x0 = *reinterpret_cast<const uint4*>(in + at0);
    x1 = *reinterpret_cast<const uint4*>(in + at1);
  }

  // (the angles are there)
  __device__ __forceinline__ void turn() {
    while (it < a.rows * heads) {
      const uint4 w0 = x0, w1 = x1;
      uint16_t* to = out;
      const unsigned r = row_in;
      it += slots;
      load();
      if (!to) continue;
      const Angle32* t = t32 + r * (a.rot / 2) + 8 * u;
      if (a.pos[row0 + (int)r] < 0) continue;
      if (!turned) {
        *reinterpret_cast<uint4*>(to + at0) = w0;
        continue;
      }
      float x[2][8], y[2][8];
      unpack8(w0, x[0]);
      unpack8(w1, x[1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Angle32 w = t[i];
        if constexpr (PAIRED) {
          const float x0 = x[i >> 2][2 * (i & 3)], x1 = x[i >> 2][2 * (i & 3) + 1];
          y[i >> 2][2 * (i & 3)] = turned0(x0, x1, w.c, w.s);
          y[i >> 2][2 * (i & 3) + 1] = turned1(x0, x1, w.c, w.s);
        } else {
          y[0][i] = turned0(x[0][i], x[1][i], w.c, w.s);
          y[1][i] = turned1(x[0][i], x[1][i], w.c, w.s);
        }
      }
      *reinterpret_cast<uint4*>(to + at0) = pack8(y[0]);
      *reinterpret_cast<uint4*>(to + at1) = pack8(y[1]);
    }
  }
};

// Eight turned values of a key, from those eight (x) and (halves) their
// partners (xp): values 8 c .. of a head.
template <bool PAIRED, typename T, typename A>
__device__ __forceinline__ void turn_chunk(const RopeArgs& a, int c, const float (&x)[8], const float (&xp)[8], const A* t,
                                           T (&y)[8]) {
  const int half = a.rot / 16;
  if (c >= 2 * half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (T)x[i];
  } else if constexpr (PAIRED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const A w = t[4 * c + i];
      y[2 * i] = turned0<T>((T)x[2 * i], (T)x[2 * i + 1], w.c, w.s);
      y[2 * i + 1] = turned1<T>((T)x[2 * i], (T)x[2 * i + 1], w.c, w.s);
    }
  } else {
    const bool second = c >= half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const A w = t[8 * (second ? c - half : c) + i];
      y[i] = second ? turned1<T>((T)xp[i], (T)x[i], w.c, w.s) : turned0<T>((T)x[i], (T)xp[i], w.c, w.s);
    }
  }
}

// y / s as e4m3: the quotient of the doubles (one more step than the product
// with the reciprocal, which may miss a border that the quotient is), odd.
__device__ __forceinline__ uint2 to_e4m3_wide(const double (&y)[8], double s) {
  const double rs = 1.0 / s;
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = y[4 * j + i], q0 = x * rs;
      const double q1 = __builtin_fma(__builtin_fma(-q0, s, x), rs, q0);
      const float t = to_odd(__builtin_isfinite(q0) ? q1 : q0);
      q[i] = t != t ? t : __builtin_fminf(__builtin_fmaxf(t, -448.0f), 448.0f);
    }
    w[j] = pack4_e4m3(q);
  }
  return make_uint2(w[0], w[1]);
}

// Keys turned and values as they are into the cache, eight of each a thread;
// loaded as the heads above are.
template <bool PAIRED, int F>
struct CacheHeads {
  const RopeWriteArgs& w;
  const RopeArgs& a;
  int row0, c;
  unsigned slots, it, row_in, h;
  bool there;
  uint4 xk, xo, xv;

  __device__ __forceinline__ CacheHeads(const RopeWriteArgs& w_, int row0_) : w(w_), a(w_.r), row0(row0_) {
    const unsigned chunks = w.d / 8;                     // 8, 16 or 32: a quad's threads have one token and head
    slots = kRopeThreads / chunks;
    c = threadIdx.x & (chunks - 1);
    it = threadIdx.x / chunks;
    load();
  }

  __device__ __forceinline__ void load() {
    there = false;
    if (it >= a.rows * (unsigned)w.heads_kv) return;
    row_in = divide(it, w.heads_kv_inv);
    h = it - row_in * w.heads_kv;
    const int row = row0 + (int)row_in;
    if (row >= a.n_rows) return;
    there = true;
    const int half = a.rot / 16;
    const uint16_t* kp = a.k + row * a.k_row + h * a.k_head;
    xk = *reinterpret_cast<const uint4*>(kp + 8 * c);
    xv = *reinterpret_cast<const uint4*>(w.v + row * w.v_row + h * w.v_head + 8 * c);
    // (halves: the partners of the pairs)
    const int co = PAIRED || c >= 2 * half ? c : c < half ? c + half : c - half;
    xo = *reinterpret_cast<const uint4*>(kp + 8 * co);
  }

  __device__ __forceinline__ void write(const Angle32* t32, const Angle64* t64) {
    const int half = a.rot / 16;
    while (it < a.rows * (unsigned)w.heads_kv) {
      const uint4 gk = xk, go = xo, gv = xv;
      const unsigned r = row_in, head = h;
      const bool now = there;
      it += slots;
      load();
      if (!now) continue;
      const int row = row0 + (int)r;
      const int slot = w.slot[row];
      if (a.pos[row] < 0) continue;
      if (slot < 0 || slot >= w.n_slots) {
        if (slot != -1 && c == 0 && head == 0) atomicOr(a.err, kErrSlot);
        continue;
      }
      const int page = slot >> w.page_shift, place = slot & ((1 << w.page_shift) - 1);
      const int64_t to = (int64_t)page * w.c_page + (int64_t)place * w.c_tok + (int64_t)head * w.c_head;
      float x[8], xp[8], v[8];
      unpack8(gk, x);
      unpack8(go, xp);
      const unsigned row_t = r * (a.rot / 2);
      if constexpr (F == kCacheBf16) {
        float y[8];
        turn_chunk<PAIRED>(a, c, x, xp, t32 + row_t, y);
        *reinterpret_cast<uint4*>(w.kc + to + 16 * c) = c < 2 * half ? pack8(y) : gk;
        *reinterpret_cast<uint4*>(w.vc + to + 16 * c) = gv;
      } else {
        double y[8];
        turn_chunk<PAIRED>(a, c, x, xp, t64 + row_t, y);
        unpack8(gv, v);
        if constexpr (F == kCacheE4m3) {
          const float ks = w.k_scale ? w.k_scale[head] : 1.0f, vs = w.v_scale ? w.v_scale[head] : 1.0f;
          *reinterpret_cast<uint2*>(w.kc + to + 8 * c) = to_e4m3_wide(y, (double)ks);
          *reinterpret_cast<uint2*>(w.vc + to + 8 * c) = to_e4m3(v, vs, 1.0f / vs);
        } else {
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = to_odd(y[i]);
          unsigned char pk, pv;
          const uint32_t codes_k = to_mxfp4(z, pk), codes_v = to_mxfp4(v, pv);
          *reinterpret_cast<uint32_t*>(w.kc + to + 4 * c) = codes_k;
          *reinterpret_cast<uint32_t*>(w.vc + to + 4 * c) = codes_v;
          if ((c & 3) == 0) {
            const int64_t at = page * w.s_page + head * w.s_head + (int64_t)place * (w.d / 32) + c / 4;
            w.k_power[at] = pk;
            w.v_power[at] = pv;
          }
        }
      }
    }
  }
};

template <bool PAIRED>
__global__ __launch_bounds__(kRopeThreads) void rope_impl(const RopeArgs a) {
  __shared__ Angle32 t32[kRopeTable];
  const int row0 = blockIdx.x * a.rows;
  Heads<PAIRED> heads(a, t32, row0);
  angles<false>(a, row0, t32, nullptr);
  __syncthreads();
  heads.turn();
}

template <bool PAIRED, int F>
__global__ __launch_bounds__(kRopeThreads) void rope_write_impl(const RopeWriteArgs w) {
  const RopeArgs& a = w.r;
  constexpr bool kWide = F != kCacheBf16;
  __shared__ Angle32 t32[kRopeTable];
  __shared__ Angle64 t64[kWide ? kRopeTable : 1];
  const int row0 = blockIdx.x * a.rows;
  CacheHeads<PAIRED, F> cache(w, row0);
  Heads<PAIRED> heads(a, t32, row0);
  angles<kWide>(a, row0, t32, t64);
  __syncthreads();
  cache.write(t32, t64);
  heads.turn();
}

template <bool PAIRED>
const void* rope_write_fn(int type) {
  return type == kCacheMxfp4  ? (const void*)&rope_write_impl<PAIRED, kCacheMxfp4>
         : type == kCacheE4m3 ? (const void*)&rope_write_impl<PAIRED, kCacheE4m3>
                              : (const void*)&rope_write_impl<PAIRED, kCacheBf16>;
}

}  // namespace

const void* rope_kernel(int paired) { return paired ? (const void*)&rope_impl<true> : (const void*)&rope_impl<false>; }
const void* rope_write_kernel(int paired, int type) { return paired ? rope_write_fn<true>(type) : rope_write_fn<false>(type); }

}  // namespace dspark
