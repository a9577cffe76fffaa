// Attention of packed rows over a paged key-value cache.
//
// [summary] section 5 (the flattened verify batch).  Row i of request b (K[b]
// + 1 rows: one token, a verify batch, or a draft block that sees itself)
// takes, for each of its query heads,
//     o = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),
//     s_t = (scale log2 e k_scale) q . k_t,
// over the tokens t it sees, in one pass with a running m (a row's sums are
// rescaled only when some score passes m by more than 8, so p_t stays within
// 2^8 of the largest and the products keep their bits).
//
// Work: a tile is the rows of one request that share a cache head (rows times
// heads per group, 16 MT of them at a time, so that a key is read once for
// all of a tile) over the request's tokens in steps of 32.  All tiles of the
// batch stand in one line, request by request, each as long as its steps and
// what it costs besides them, and every wave takes an equal stretch of the
// line, so that ragged lengths load the chip evenly without the host knowing
// them.  The four waves of a workgroup have neighbouring stretches and join
// what they share of a tile in LDS when they are done; what a workgroup shares
// with its neighbours it leaves in memory, and a second launch adds the pieces
// up in the order of their tokens.
//
// One workgroup a CU, one wave a SIMD (MXFP4: two, where the registers hold
// them, one step ahead each): its registers hold the next two steps' keys and
// values in flight (64 to 128 KB a CU), which is what the memory's
// latency asks for; with more waves the older ones of a SIMD are served first
// and the younger ones finish alone (measured: two workgroups a CU 139 us
// against 131 on 128 requests of 64 to 8192 tokens, 137 against 96 on equal
// lengths of 1024).
//
// Scores are formed transposed, S^T = K Q^T, and so is the product, O^T =
// V^T P^T: then the accumulators of the first product (a lane: one query,
// tokens 4 g + i of the two 16-token halves, g = lane / 16) are in place as
// the second's operand, whose eight products per lane may be taken in any
// order of tokens as long as the values come in the same order.  A lane loads
// its eight tokens' values at D / 16 neighbouring places, whole cache lines
// per token, and exchanges rows for columns within its own registers.  No
// key, value or score passes through LDS.
//
// Measured: 128 requests of 64 to 8192 tokens, up to 8 rows, 32 query and 8
// cache heads of 128, 107 us and 6 for the second launch (537 MB, each key and
// value read once; 6.1 TB/s on 64 requests of 8192), bound by memory, with heads
// of 256 both launches 214 (5.0 TB/s), in e4m3 138 (4.0); 6 requests of 60000 to
// 131000 tokens in e4m3, 64 rows a tile, 105 and 11 us, bound by the issue of
// vector instructions (about 255, and 64 matrix ones, a step); 48 draft blocks
// of 7 positions, heads of 64, 19.5 and 4 us, bound by the latency of finding a
// stretch and its first keys.  Over MXFP4 (a quarter of bf16's bytes), both
// launches, the first 62 us (pages that keep a head's tokens together 55), the
// long ones 116, the blocks 16.5.  The long ones: a wave's vector instructions
// (48% of a SIMD's time) and its products (30%), a value being 4 bits to widen
// and a weight two products, run one after the other with one wave a SIMD.  The
// first: neither (37 and 18%), nor memory (56 us all in the caches); of the two waves of
// a SIMD the older ends after 35 us, the younger after 42, the last one after 50, and
// 9 us are the join.  The blocks: the latencies of the books (2 us), the first loads (2),
// of two or three steps (5) and of the launches.
#include "common.hpp"
#include "internal.hpp"
#include "power_place.hpp"

namespace dspark {
namespace {

constexpr int kStep = 32;        // tokens of a step
constexpr int kWaves = kAttendThreads / 64;
// What a tile costs besides its steps, in steps, and the steps of a wave's
// stretch at least.  128 requests of 64 to 8192 tokens: 117 us with a cost of
// 1, 119 with 2, 123 with 4; one row of one request of up to 1200 tokens: 14.2 us
// with at least 1 step, 16.1 with 2 (a wave's first step waits for its loads,
// the second is nearly free, but so is the wave that would take it).
// Over MXFP4, whose steps are shorter beside it, costs of 1 / 2 / 3 / 4 on those requests, tokens before heads and heads
// before tokens: 62.7 / 63.6 / 61.2 / 60.9 and 57.4 / 54.5 / 55.2 / 54.9 us; one row each 53.3 / 53.8 / 54.7 / 53.2 and
// 40.2 / 39.2 / 40.3 / 40.2; of up to 600 tokens 25.5 / 23.9 / 24.7 / 26.1 and 25.0 / 23.8 / 24.9 / 25.8; one row of one
// request 13.4 / 12.5 / 13.4 / 13.6; 256 of 2 rows, heads of 64, 33.6 / 32.9 / 30.9 / 32.5 and 31.0 / 27.0 / 26.9 / 27.6; 64
// with heads of 256 32.8 / 34.3 / 34.4 / 34.0.
template <int F>
constexpr int kCost = F == kCacheMxfp4 ? 2 : 1;
constexpr int kMinSteps = 1;

__device__ __forceinline__ f32x4_t mfma(const uint4 a, const uint4 b, const f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ f32x4_t mfma_f16(const uint4 a, const uint4 b, const f32x4_t c) {
  typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0,
                                                0);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
  f16x2_t r;
  r[0] = (_Float16)lo;                                   // to nearest even
  r[1] = (_Float16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  bf16x2_t r;
  r[0] = (__bf16)lo;                                     // to nearest even
  r[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

// A load past the caches, or (KEEP) into them.
template <bool KEEP, typename T>
__device__ __forceinline__ T load_as(const unsigned char* p) {
  if constexpr (KEEP) return *reinterpret_cast<const T*>(p);
  return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}

template <bool KEEP>
__device__ __forceinline__ uint2 load8(const unsigned char* p) {
  typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
  const u32x2_t v = load_as<KEEP, u32x2_t>(p);
  return make_uint2(v[0], v[1]);
}

template <bool KEEP>
__device__ __forceinline__ uint4 load16(const unsigned char* p) {
  typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
  const u32x4_t v = load_as<KEEP, u32x4_t>(p);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The bits of the infinite and NaN ones among the two bf16 or four e4m3
// values of a word.
__device__ __forceinline__ uint32_t odd_bf16(uint32_t x) {
  return ((x & 0x7F80u) == 0x7F80u ? 0x0000FFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ uint32_t odd_e4m3(uint32_t x) {
  return ((((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
}

// The bit pattern of 2^(b - 127) as the conversions below read it (the exponent's eight bits alone), b the byte of x that
// a rotation by `turn` = (8 place + 9) % 32 bits brings there.
__device__ __forceinline__ float power_at(uint32_t x, unsigned turn) {
  return __uint_as_float(__builtin_amdgcn_alignbit(x, x, turn));
}
// The bits of the codes (of a word of eight) that are infinite or NaN in bf16 times the power of a byte: all of 255's, of
// 2^127 those from 2 on, of 2^126 those from 4 on, none of a lower one.
__device__ __forceinline__ uint32_t odd_codes(uint32_t w, unsigned byte) {
  if (byte == 255) return 0xFFFFFFFFu;
  const uint32_t m = byte == 254 ? w >> 2 : byte == 253 ? w >> 2 & w >> 1 : 0u;
  return (m & 0x11111111u) * 15u;
}

// Two e2m1 values (byte c of w) times a power of two as bf16: exact from 2^-126 on, NaN for a byte of 255.
__device__ __forceinline__ uint32_t widen4(uint32_t w, float s, int c) {
  switch (c) {                                           // (the place is an immediate)
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  }
}

// Two e4m3 values (the low or high half of w) as bf16 or f16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}
template <bool HI>
__device__ __forceinline__ uint32_t widen_f16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

typedef const __attribute__((address_space(4))) int32_t* uniform_ptr;   // scalar loads

// The rows of request b: none where a length, row or count is out of range.
struct Rows {
  int n, len, row0, bad;
};

template <typename P>
__device__ __forceinline__ Rows request_rows(const AttendArgs& a, P K, P len, P offs, int b) {
  Rows r;
  int k = a.K ? K[b] : a.gamma;
  r.len = len[b];
  r.row0 = a.offs ? offs[b] : b * (a.gamma + 1);
  r.bad = 0;
  if (k < -1 || k > a.gamma) {
    r.bad = kErrK;
    k = k < -1 ? -1 : a.gamma;
  }
  r.n = k + 1;
  if (r.n > 0 && (r.len < 0 || (int64_t)r.len + r.n > (int64_t)a.cols << a.page_shift)) {
    r.bad |= kErrCache;
    r.n = 0;
  }
  if (r.n > 0 && (r.row0 < 0 || (int64_t)r.row0 + r.n > a.n_rows)) {
    r.bad |= kErrRow;
    r.n = 0;
  }
  return r;
}

// The places of a step: where its groups of G tokens that a page holds whole (8,
// or 16 where the pages have them) begin, in bytes from the beginning of a
// cache and (MXFP4) of its powers.
template <int F, int G>
struct At {
  int64_t v[32 / G];
};
template <int G>
struct At<kCacheMxfp4, G> {
  int64_t v[32 / G], s[32 / G];
};
// The lane's group of half s: uniform where a half is one group, else by `second`.
template <int G>
__device__ __forceinline__ int64_t in_half(const int64_t (&at)[32 / G], int s, bool second) {
  if constexpr (G == 16) return at[s];
  const int64_t lo = at[2 * s], hi = at[2 * s + 1];
  return second ? hi : lo;
}

// Keys and values of a step as a lane has them loaded.
template <int D, int F, int G>
struct Loaded {
  static constexpr bool kBf16 = F == kCacheBf16, kFp4 = F == kCacheMxfp4;
  static constexpr int kBits = kBf16 ? 16 : kFp4 ? 4 : 8;
  static constexpr int KB = D * kBits / 32 < 16 ? D * kBits / 32 : 16;   // bytes of a lane's load of a key
  static constexpr int KW = D * kBits / 32 / KB;         // such loads of a key per lane
  static constexpr int VB = D * kBits / 128;             // bytes of a value per lane
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int NB = D / 32;                      // blocks that share a power of two (MXFP4)
  // A head of a token that is less than a line of the caches: with tokens
  // before heads another wave has the line's rest (128 requests of 64 to
  // 8192 tokens 66.6 us against 69.6, 48 draft blocks with heads of 64 18.9 against 21.1;
  // of 128 bytes 78.7 against 76.9).
  static constexpr bool kKeep = kFp4 && D * kBits / 8 < 128;
  uint4 k[2][KW];
  uint32_t v[8][VW];
  uint32_t ks[kFp4 ? 2 : 1][KW];                         // MXFP4: powers of the keys' blocks,
  uint32_t vs[kFp4 ? 8 : 1];                             // of the values' (see take_v)

  // A lane's keys: token lane % 16 of either half, `kl` its place in a group.
  __device__ __forceinline__ void load_k(const unsigned char* kc, const unsigned char* sc, const At<F, G>& at, unsigned kl,
                                         int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const unsigned char* p = kc + in_half<G>(at.v, s, lane & 8) + kl;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        if constexpr (KB == 8) {
          const uint2 x = load8<kKeep>(p);
          k[s][w] = make_uint4(x.x, x.y, 0, 0);
        } else {
          k[s][w] = load16<kKeep>(p + 64 * w);
        }
      }
      if constexpr (kFp4) {
        const unsigned at_s = (unsigned)(lane & (G - 1)) * NB + (D == 64 ? lane >> 5 : lane >> 4);
        const unsigned char* ps = sc + in_half<G>(at.s, s, lane & 8) + at_s;
#pragma unroll
        for (int w = 0; w < KW; ++w) ks[s][w] = ps[4 * w];
      }
    }
  }

  // A lane's values: tokens 4 g + i of either half, `vl` the first one's place in its group.
  __device__ __forceinline__ void load_v(const unsigned char* vc, const unsigned char* sc, const At<F, G>& at,
                                         unsigned vl, int64_t c_tok, int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const unsigned char* p = vc + in_half<G>(at.v, s, lane & 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (groups of 16: a uniform address and 32 bits of a lane's own)
        const unsigned char* pt = G == 16 ? p + (vl + i * (unsigned)c_tok) : p + vl + i * c_tok;
        uint32_t(&w)[VW] = v[4 * s + i];
        if constexpr (VB == 2) {
          w[0] = load_as<kKeep, uint16_t>(pt);
        } else if constexpr (VW == 1) {
          w[0] = load_as<kKeep, uint32_t>(pt);
        } else if constexpr (VW == 2) {
          const uint2 x = load8<kKeep>(pt);
          w[0] = x.x;
          w[1] = x.y;
        } else {
#pragma unroll
          for (int c = 0; c < VW / 4; ++c) {
            const uint4 x = load16<kKeep>(pt + 16 * c);
            w[4 * c] = x.x;
            w[4 * c + 1] = x.y;
            w[4 * c + 2] = x.z;
            w[4 * c + 3] = x.w;
          }
        }
      }
      if constexpr (kFp4) {
        // the powers of one of the four tokens: take_v exchanges them within the quad
        const unsigned token = 4 * (lane >> 4 & (G / 4 - 1)) + (lane & 3);
        const unsigned char* ps = sc + in_half<G>(at.s, s, lane & 32) + token * NB;
        if constexpr (D == 64) vs[4 * s] = *reinterpret_cast<const uint16_t*>(ps);
        else vs[4 * s] = *reinterpret_cast<const uint32_t*>(ps + (D == 256 ? lane >> 1 & 4 : 0));
      }
    }
  }

  // MXFP4: the bits of the powers of the lane's tokens, out of what its quad has loaded.
  __device__ __forceinline__ void take_v(int lane) {
    if constexpr (!kFp4) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      // the byte of the lane's block, which is the quad's where a quad has 32 values at most
      const unsigned turn = (8 * (D == 64 ? lane >> 3 & 1 : D == 128 ? lane >> 2 & 3 : lane >> 1 & 3) + 9) & 31;
      const uint32_t w = D == 256 ? vs[4 * s] : __float_as_uint(power_at(vs[4 * s], turn));
      const uint32_t of[4] = {from_quad<0x00>(w), from_quad<0x55>(w), from_quad<0xAA>(w), from_quad<0xFF>(w)};
#pragma unroll
      for (int i = 0; i < 4; ++i) vs[4 * s + i] = D == 256 ? __float_as_uint(power_at(of[i], turn)) : of[i];
    }
  }
  // x of another lane of the quad (a quad_perm pattern).
  template <int P>
  __device__ __forceinline__ static uint32_t from_quad(uint32_t x) {
    return __builtin_amdgcn_update_dpp(x, x, P, 0xF, 0xF, false);
  }

  // Where product ks's values of lane's group begin in a key and a query.
  __device__ __forceinline__ static int first(int ks, int lane) {
    const int g = lane >> 4;
    if constexpr (kBf16) return 32 * ks + 8 * g;
    if constexpr (kFp4) return D == 64 ? 16 * g + 8 * ks : 128 * (ks >> 2) + 32 * g + 8 * (ks & 3);
    return 64 * (ks >> 1) + 16 * g + 8 * (ks & 1);
  }

  // The key operand of product ks: 16 tokens (a lane: its token's values from first(ks) on).
  __device__ __forceinline__ uint4 key(int s, int ks) const {
    if constexpr (kBf16) return k[s][ks];
    if constexpr (kFp4) {
      const uint4 w = k[s][ks >> 2];
      const uint32_t x = (ks & 3) == 0 ? w.x : (ks & 3) == 1 ? w.y : (ks & 3) == 2 ? w.z : w.w;
      const float p = __uint_as_float(this->ks[s][ks >> 2] << 23);
      return make_uint4(widen4(x, p, 0), widen4(x, p, 1), widen4(x, p, 2), widen4(x, p, 3));
    }
    const uint4 w = k[s][ks >> 1];
    const uint32_t lo = ks & 1 ? w.z : w.x, hi = ks & 1 ? w.w : w.y;
    return make_uint4(widen<false>(lo), widen<true>(lo), widen<false>(hi), widen<true>(hi));
  }

  // The value operands of blocks dt and dt + 1, bf16 or (e4m3) f16: rows d =
  // D / 16 r + dt of V^T (r = lane % 16), the lane's eight tokens in pairs.
  __device__ __forceinline__ void values(int dt, uint4 (&f)[2]) const {
    uint32_t x[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F == kCacheE4m3) {
        const uint32_t e = v[2 * j][dt / 4], o = v[2 * j + 1][dt / 4];
        const uint32_t w = __builtin_amdgcn_perm(o, e, dt & 2 ? 0x07030602u : 0x05010400u);
        x[0][j] = widen_f16<false>(w);
        x[1][j] = widen_f16<true>(w);
      } else {
        uint32_t e, o;
        if constexpr (kFp4) {
          e = widen4(v[2 * j][dt / 8], __uint_as_float(vs[2 * j]), dt / 2 & 3);
          o = widen4(v[2 * j + 1][dt / 8], __uint_as_float(vs[2 * j + 1]), dt / 2 & 3);
        } else {
          e = v[2 * j][dt / 2];
          o = v[2 * j + 1][dt / 2];
        }
        x[0][j] = __builtin_amdgcn_perm(o, e, 0x05040100u);
        x[1][j] = __builtin_amdgcn_perm(o, e, 0x07060302u);
      }
    }
    f[0] = make_uint4(x[0][0], x[0][1], x[0][2], x[0][3]);
    f[1] = make_uint4(x[1][0], x[1][1], x[1][2], x[1][3]);
  }

  // Takes infinite and NaN values out; whether there were any.
  __device__ __forceinline__ uint32_t take_odd() {
    uint32_t odd = 0;
    if constexpr (kFp4) {
      // (vs: the powers' bytes from bit 23 on, anything around them)
      uint32_t top = 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) top = max(top, vs[t] & 0x7F800000u);
      if (__builtin_expect(!__any(top >= 253u << 23), 1)) return 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const unsigned byte = vs[t] >> 23 & 255;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t x = odd_codes(v[t][w], byte);
          odd |= x;
          v[t][w] &= ~x;
        }
        if (byte == 255) vs[t] = 0x3F800000u;
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t x = kBf16 ? odd_bf16(v[t][w]) : odd_e4m3(v[t][w]);
          odd |= x;
          v[t][w] &= ~x;
        }
    }
    return odd;
  }
};

// Where the groups of a step begin in a cache.  A page holds whole groups; one
// behind the last token is taken as the last group,
// and places of a group behind the last token are read and masked.  Page ids
// are uniform: scalar loads, whose wait is none of the key and value loads'.
template <int G>
struct Groups {
  int id[32 / G];
  __device__ __forceinline__ static int first(int base, int j, int last) { return min(base + G * j, last & ~(G - 1)); }
  __device__ __forceinline__ void load(const AttendArgs& a, const int32_t* table, int base, int last) {
    const uniform_ptr t = (uniform_ptr)(uintptr_t)table;
#pragma unroll
    for (int j = 0; j < 32 / G; ++j) id[j] = t[first(base, j, last) >> a.page_shift];
  }
  // The places of the step at `base` whose ids are loaded.
  template <int D, int F>
  __device__ __forceinline__ void place(const AttendArgs& a, int base, int last, At<F, G>& at) const {
#pragma unroll
    for (int j = 0; j < 32 / G; ++j) {
      int p = id[j];
      if ((unsigned)p >= (unsigned)a.n_pages) {
        atomicOr(a.err, kErrPage);
        p = 0;
      }
      at.v[j] = (int64_t)p * a.c_page + (int64_t)(first(base, j, last) & ((1 << a.page_shift) - 1)) * a.c_tok;
      if constexpr (F == kCacheMxfp4)
        at.s[j] = power_place(p, a.Hkv, 0, a.page_shift, first(base, j, last) & ((1 << a.page_shift) - 1), D / 32);
    }
  }
};

template <int D, int MT, int F, int G>
struct Tile {
  using In = Loaded<D, F, G>;
  static constexpr bool E4M3 = F == kCacheE4m3;
  static constexpr int kRows = 16 * MT;
  static constexpr int KS = D / 32;                      // products of 32 values per score
  static constexpr int DT = D / 16;                      // 16-wide blocks of a value row
  // m stands this far below the row's maximum (in the exponent) when it is set.  The weights over an e4m3 cache
  // are f16 in the second product: a row's largest lies between 2^7 and 2^15, below 65504, and what f16 cannot
  // hold of the small ones is 2^-32 of it.  (From maxima of 2^25 on, where a float's step is 4, the largest may lie
  // as low as 2^-8; from 2^28 on, where it is 32, it may pass 65504.)
  static constexpr float kHead = E4M3 ? 7.0f : 0.0f;

  uint4 q[MT][KS];
  f32x4_t o[MT][DT];
  float m[MT], l[MT];
  int lim[MT];                                           // last token a query sees
  uint32_t odd;                                          // infinite or NaN values were taken out

  __device__ __forceinline__ void load_q(const AttendArgs& a, const Rows& r, int h, int rt, int lane) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = rt * kRows + mt * 16 + (lane & 15);
      const bool ok = row < a.group * r.n;
      const int i = ok ? row / a.group : 0, hh = ok ? row - i * a.group : 0;
      const uint16_t* p = a.q + (int64_t)(r.row0 + i) * a.q_row + (int64_t)(h * a.group + hh) * a.q_head;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        q[mt][ks] = ok ? *reinterpret_cast<const uint4*>(p + In::first(ks, lane)) : make_uint4(0, 0, 0, 0);
      }
      lim[mt] = a.causal ? r.len + i : r.len + r.n - 1;
    }
  }

  __device__ __forceinline__ void reset() {
    odd = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = -INFINITY;
      l[mt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[mt][dt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }

  // Scores, p and sums of the 32 tokens at `base`, in `in`; `tail`: some query
  // may not see some of them.  next_k and next_v load a later step's keys and
  // values into it once these are used.
  template <typename NextK, typename NextV>
  __device__ __forceinline__ void step(In& in, int base, bool tail, float sc, int lane, NextK next_k, NextV next_v) {
    const int g = lane >> 4;
    f32x4_t s[MT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 kf = in.key(h, ks);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          s[mt][h] = mfma(kf, q[mt][ks], ks == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : s[mt][h]);
      }
    next_k();
    // exponents against the maximum so far (0 where nothing was seen yet: then
    // every p of a masked token is 2^-inf = 0 too)
    float ref[MT], top[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      ref[mt] = m[mt] == -INFINITY ? 0.0f : m[mt];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[mt][h][i] = __builtin_fmaf(s[mt][h][i], sc, -ref[mt]);
    }
    if (tail) {
      asm volatile("");                                  // a branch: few steps take it
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 16 * h + 4 * g + i > lim[mt]) s[mt][h][i] = -INFINITY;
    }
    bool grows = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float x = fmaxf(fmaxf(s[mt][0][0], s[mt][0][1]), fmaxf(s[mt][0][2], s[mt][0][3]));
      x = fmaxf(x, fmaxf(fmaxf(s[mt][1][0], s[mt][1][1]), fmaxf(s[mt][1][2], s[mt][1][3])));
      top[mt] = x + ref[mt];
      // (the difference, not top > m + 15, which rounds past the limit of f16 where m is large; before
      // the first score it is infinite, or NaN where nothing is seen)
      grows |= top[mt] - m[mt] > 8.0f + kHead;
    }
    if (__any(grows)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x = fmaxf(top[mt], shfl_xor(top[mt], 16));
        x = fmaxf(x, shfl_xor(x, 32));
        const float mn = fmaxf(m[mt], x - kHead);
        const float f = mn == m[mt] ? 1.0f : fast_exp2(m[mt] - mn);
        const float up = (m[mt] == -INFINITY ? 0.0f : m[mt]) - (mn == -INFINITY ? 0.0f : mn);
        m[mt] = mn;
        l[mt] *= f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][h][i] += up;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[mt][dt] *= f;
      }
    }
    // The weights of the second product.  bf16 and MXFP4 values: a weight is the sum of
    // two bf16 numbers, its leading 8 bits and the rest to nearest, off by
    // 2^-15 of it at most (rounded to one, 2^-8 of it, they cost as much as the
    // rounding of the result does).  Over a bf16 cache the rest is that of 1 + 2^-16 times the
    // weight (a.unrest takes the factor out of the result): positive wherever
    // the weight is, since 0 times an infinite value is NaN.  e4m3 values are
    // exact in f16, whose 11 bits leave 2^-11 of a weight, far below the
    // rounding of the values that such a cache holds.  (MXFP4 values are not, for their powers: where those
    // of a step span no more than f16 does, one product would do, 109 us against 119 on 6 requests of 60000
    // to 131000 tokens, 69.5 against 69.3 on 128 of 64 to 8192; but a way around for the others costs
    // the common case more than that.)
    uint4 p[MT], rest[E4M3 ? 1 : MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float e[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[4 * h + i] = fast_exp2(s[mt][h][i]);
      l[mt] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      uint32_t w[4], x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (E4M3) {
          w[j] = pack_f16(e[2 * j], e[2 * j + 1]);
        } else {
          constexpr float kFactor = F == kCacheBf16 ? kRestFactor : 1.0f;
          const uint32_t a = __float_as_uint(e[2 * j]), b = __float_as_uint(e[2 * j + 1]);
          w[j] = __builtin_amdgcn_perm(b, a, 0x07060302u);
          x[j] = pack_bf16(__builtin_fmaf(e[2 * j], kFactor, -__uint_as_float(a & 0xFFFF0000u)),
                           __builtin_fmaf(e[2 * j + 1], kFactor, -__uint_as_float(b & 0xFFFF0000u)));
        }
      }
      p[mt] = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (!E4M3) rest[mt] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    // a token that a query does not see must not reach it, but 0 times
    // infinity or NaN is NaN: such values are left out here and added to the
    // results that see them at the end
    in.take_v(lane);
    if (tail) odd |= in.take_odd();
#pragma unroll
    for (int dt = 0; dt < DT; dt += 2) {
      uint4 f[2];
      in.values(dt, f);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (E4M3) {
            o[mt][dt + c] = mfma_f16(f[c], p[mt], o[mt][dt + c]);
          } else {
            o[mt][dt + c] = mfma(f[c], p[mt], o[mt][dt + c]);
            o[mt][dt + c] = mfma(f[c], rest[mt], o[mt][dt + c]);
          }
        }
    }
    next_v();
  }
};

// Steps loaded ahead: two, or one where two and the sums pass the registers.
// (More of the small steps cost more at a piece's beginning than they hide: three
// 24.0, four 26.5 us against 23.4 on 48 draft blocks with heads of 64.)
// Over MXFP4 with two waves a SIMD one: 69.3 us against 69.6 on 128 requests of
// 64 to 8192 tokens, 71.5 against 77.3 in pages of 8, where two pass the registers.
template <int D, int MT, int F>
constexpr int kAhead = (D * MT >= 512 && F == kCacheBf16) || F == kCacheMxfp4 ? 1 : 2;

// A wave's steps s0 .. s1 - 1 of a tile: the rows of request r at cache head h, row tile rt.
struct Piece {
  Rows r;
  int h, rt, n_s, s0, s1;        // n_s: steps of the whole tile
  int64_t real0;                 // where they begin in the line
  const int32_t* table;          // the request's pages
  __device__ __forceinline__ int last() const { return min(s1 * kStep, r.len + r.n) - 1; }
};

template <int D, int MT, int F, int G>
__global__ __launch_bounds__(kAttendThreads, attend_waves(D, MT, F)) void attend_impl(const AttendArgs a) {
  using T = Tile<D, MT, F, G>;
  using In = Loaded<D, F, G>;
  constexpr bool E4M3 = F == kCacheE4m3, kFp4 = F == kCacheMxfp4;
  constexpr int kRows = T::kRows, DT = T::DT, kTileCost = kCost<F>;
  __shared__ int64_t sums[kWaves];
  __shared__ Rows start_rows[kWaves];
  __shared__ int start_b[kWaves], start_off[kWaves];
  __shared__ f32x4_t share_o[kWaves - 1][MT * DT][64];    // what waves 1 .. 3 begin with of a tile
  __shared__ float2 share_ml[kWaves - 1][kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups of one XCD (every eighth) have neighbouring stretches: a line of the cache that two heads share
  // is in its L2 when the second asks (128 requests of 64 to 8192 tokens 62.7 us against 66.7).
  const unsigned block = kFp4 && gridDim.x % 8 == 0 ? xcd_block() : blockIdx.x;
  // a lane's place in a group: its key's and its first value's
  const unsigned kl = (unsigned)(lane & (G - 1)) * (unsigned)a.c_tok + In::KB * (lane >> 4);
  const unsigned vl = 4 * (lane >> 4 & (G / 4 - 1)) * (unsigned)a.c_tok + In::VB * (lane & 15);

  // the line: what every request adds to it, and where the four stretches of
  // this workgroup's waves begin
  const int per = (a.B + kAttendThreads - 1) / kAttendThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto row_tiles = [&](const Rows& r) { return (a.group * r.n + kRows - 1) / kRows; };
  auto steps = [&](const Rows& r) { return (r.len + r.n + kStep - 1) / kStep; };
  auto length = [&](const Rows& r) -> int64_t {
    return r.n <= 0 ? 0 : (int64_t)a.Hkv * row_tiles(r) * (steps(r) + kTileCost);
  };
  int64_t mine = 0;
  Rows r{0, 0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    r = request_rows(a, a.K, a.len, a.offs, b);
    if (r.bad && block == 0) atomicOr(a.err, r.bad);
    mine += length(r);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(incl, o, 64);
    if (lane >= o) incl += u;
  }
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  const int64_t workers = (int64_t)gridDim.x * kWaves;
  const int64_t chunk = max((int64_t)kTileCost + kMinSteps, (total + workers - 1) / workers);
  const int64_t group_chunk = kWaves * chunk, group_u0 = block * group_chunk;
  if (group_u0 >= total) {
    if (tid == 0) a.joins[block].n = 0;
    return;
  }
  for (int w = 0; w < kWaves; ++w) {
    const int64_t u0 = group_u0 + w * chunk;
    if (u0 < before || u0 >= before + mine) continue;
    int64_t base = before;
    int b = b0;
    if (per > 1)                                         // else r is the request still
      for (;; ++b) {
        r = request_rows(a, a.K, a.len, a.offs, b);
        const int64_t n = length(r);
        if (u0 < base + n) break;
        base += n;
      }
    start_b[w] = b;
    start_off[w] = (int)(u0 - base);
    start_rows[w] = r;
  }
  __syncthreads();
  // MXFP4: powers, [n_pages][Hkv][page][D / 32]
  const unsigned char* k_power = reinterpret_cast<const unsigned char*>(a.k_scale);
  const unsigned char* v_power = reinterpret_cast<const unsigned char*>(a.v_scale);
  const int64_t power_head = (int64_t)(D / 32) << a.page_shift;
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const int64_t u0 = group_u0 + wave * chunk, u1 = min(total, u0 + chunk);
  const uniform_ptr uK = (uniform_ptr)(uintptr_t)a.K, ulen = (uniform_ptr)(uintptr_t)a.len,
                    uoffs = (uniform_ptr)(uintptr_t)a.offs;
  T t;
  Piece now;                                             // the piece at hand

  // A lane: query lane % 16 of each block, values DT (4 g + i) + dt.
  auto write = [&]() {
    const float vs = E4M3 && a.v_scale ? a.v_scale[now.h] : 1.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int grow = now.rt * kRows + mt * 16 + (lane & 15);
      if (grow >= a.group * now.r.n) continue;
      const int i = grow / a.group, hh = grow - i * a.group;
      const float inv = vs * a.unrest / t.l[mt];
      uint16_t* op = a.out + (int64_t)(now.r.row0 + i) * a.o_row + (int64_t)(now.h * a.group + hh) * a.o_head +
                     4 * DT * (lane >> 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[DT / 2];
#pragma unroll
        for (int c = 0; c < DT / 2; ++c) w[c] = pack_bf16(t.o[mt][2 * c][j] * inv, t.o[mt][2 * c + 1][j] * inv);
        if constexpr (DT == 4) {
          reinterpret_cast<uint2*>(op)[j] = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int c = 0; c < DT / 8; ++c)
            reinterpret_cast<uint4*>(op + j * DT)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
      }
      if (a.lse && lane < 16)
        a.lse[(int64_t)(now.r.row0 + i) * a.Hq + now.h * a.group + hh] = (t.m[mt] + fast_log2(t.l[mt])) * kLn2;
    }
  };
  // A workgroup leaves at most two pieces in memory: what it begins with and what it ends with.
  auto leave = [&]() {
    float* part = a.part + (int64_t)(2 * block + (group_u0 < now.real0 - kTileCost ? 1 : 0)) * (kRows * (D + 2));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (lane < 16) *reinterpret_cast<float2*>(part + 2 * (mt * 16 + lane)) = make_float2(t.m[mt], t.l[mt]);
      f32x4_t* pp = reinterpret_cast<f32x4_t*>(part + 2 * kRows) + mt * DT * 64 + lane;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) pp[dt * 64] = t.o[mt][dt];
    }
  };

  bool owner = false;                                    // the tile at hand goes on in the next wave
  if (u0 < total) {
    int b = uniform(start_b[wave]);
    r = Rows{uniform(start_rows[wave].n), uniform(start_rows[wave].len), uniform(start_rows[wave].row0), 0};
    int off = uniform(start_off[wave]);                  // place in request b's part of the line (below 2^31)
    int64_t u = u0;
    // the stretch's next piece, if it has one
    auto take = [&](Piece& p) {
      while (u < u1) {
        while (r.n <= 0) r = request_rows(a, uK, ulen, uoffs, ++b);   // u < u1 <= total: one follows
        const int n_rt = row_tiles(r), size = steps(r) + kTileCost;
        const int seg = off / size, x0 = off - seg * size;
        const int x1 = (int)min((int64_t)size, x0 + (u1 - u));
        p.r = r;
        p.n_s = size - kTileCost;
        p.h = seg / n_rt;
        p.rt = seg - p.h * n_rt;
        p.s0 = max(0, x0 - kTileCost);
        p.s1 = x1 - kTileCost;
        p.real0 = u - x0 + kTileCost;
        p.table = a.table + b * a.tstride;
        if (u == group_u0 && lane == 0) {
          // of the workgroups whose stretches begin within a tile's steps the
          // first has it joined: its predecessor's piece, its own ..
          AttendJoin j{0, 0, 0, 0, 0, 0};
          if (p.s0 > 0 && group_u0 - group_chunk <= p.real0) {
            j.row0 = r.row0;
            j.rows = a.group * r.n - p.rt * kRows;
            j.h = p.h;
            j.rt = p.rt;
            j.n = (int)((p.real0 + p.n_s - 1) / group_chunk) - (int)block + 2;
            j.slot = 2 * ((int)block - 1) + (group_u0 - group_chunk < p.real0 - kTileCost ? 1 : 0);
          }
          a.joins[block] = j;
        }
        u += x1 - x0;
        off += x1 - x0;
        if (off == a.Hkv * n_rt * size) {
          off = 0;
          ++b;
          if (u < u1) r = request_rows(a, uK, ulen, uoffs, b);
        }
        if (p.s1 > 0) return true;                       // else none of the tile's steps falls to this stretch
      }
      return false;
    };
    constexpr int N = kAhead<D, MT, F>;
    In in[N];
    Groups<G> ids[N + 1];
    At<F, G> at;
    // a piece's first steps: page ids, then queries, keys and values
    auto ask = [&](const Piece& p) {
#pragma unroll
      for (int i = 0; i <= N; ++i) ids[i].load(a, p.table, (p.s0 + i) * kStep, p.last());
    };
    auto begin = [&](const Piece& p) {
      const unsigned char *kc = a.kc + (int64_t)p.h * a.c_head, *vc = a.vc + (int64_t)p.h * a.c_head;
      const unsigned char *ksc = k_power + p.h * power_head, *vsc = v_power + p.h * power_head;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ids[i].template place<D>(a, (p.s0 + i) * kStep, p.last(), at);
        in[i].load_k(kc, ksc, at, kl, lane);
        if (i == 0) t.load_q(a, p.r, p.h, p.rt, lane);
        in[i].load_v(vc, vsc, at, vl, a.c_tok, lane);
      }
    };
    bool have = take(now);
    if (have) {
      ask(now);
      begin(now);
    }
    while (have) {
      Piece next = now;
      have = take(next);
      t.reset();
      const int L = now.r.len + now.r.n, h = now.h;
      const float sc = a.scale2 * (E4M3 && a.k_scale ? a.k_scale[h] : 1.0f);
      const unsigned char *kc = a.kc + (int64_t)h * a.c_head, *vc = a.vc + (int64_t)h * a.c_head;
      const unsigned char *ksc = k_power + h * power_head, *vsc = v_power + h * power_head;
      const int full = a.causal ? now.r.len : L - 1;     // tokens up to `full` are seen by every row
      const int last = now.last();
      Groups<G> id = ids[N];
      if (have) ask(next);
      int base = now.s0 * kStep;
      for (;;) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          t.step(
              in[i], base, base + kStep - 1 > full, sc, lane,
              [&]() {
                // (with 64 rows the branch costs more register copies than the loads: those are
                // the last tokens once more)
                if (MT < 4 && base + N * kStep > last) return;
                id.template place<D>(a, base + N * kStep, last, at);
                id.load(a, now.table, base + (N + 1) * kStep, last);
                in[i].load_k(kc, ksc, at, kl, lane);
              },
              [&]() {
                if (MT == 4 || base + N * kStep <= last) in[i].load_v(vc, vsc, at, vl, a.c_tok, lane);
              });
          base += kStep;
          if (base > last) goto done;
        }
      }
    done:
      if (__any(t.odd != 0)) {
        // the values left out above, to the rows that see them: only steps that
        // reach past `full` leave any out
        for (int tk = max(now.s0 * kStep, (full + 1) & ~(kStep - 1)); tk <= last; ++tk) {
          const int page = now.table[tk >> a.page_shift];
          const unsigned char* p = vc + (int64_t)((unsigned)page < (unsigned)a.n_pages ? page : 0) * a.c_page +
                                   (int64_t)(tk & ((1 << a.page_shift) - 1)) * a.c_tok;
          if constexpr (kFp4) {
            // 0 times them all: NaN for those that were left out.  (The lane's D / 4 values of a token have one
            // power, or one for each half of them.)
            const unsigned char* ps = vsc + power_place((unsigned)page < (unsigned)a.n_pages ? page : 0, a.Hkv, 0, a.page_shift,
                                                        tk & ((1 << a.page_shift) - 1), D / 32) + (D / 4) * (lane >> 4) / 32;
            const uint16_t* pw = reinterpret_cast<const uint16_t*>(p) + DT * (lane >> 4);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if (tk > t.lim[mt]) continue;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float s = __uint_as_float((uint32_t)ps[D == 256 ? i / 2 : 0] << 23);
#pragma unroll
                for (int dt = 0; dt < DT; dt += 2) {
                  const uint32_t x = widen4(pw[(DT * i + dt) / 4], s, dt / 2 & 1);
                  t.o[mt][dt][i] = __builtin_fmaf(__uint_as_float(x << 16), 0.0f, t.o[mt][dt][i]);
                  t.o[mt][dt + 1][i] = __builtin_fmaf(__uint_as_float(x & 0xFFFF0000u), 0.0f, t.o[mt][dt + 1][i]);
                }
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int dt = 0; dt < DT; ++dt) {
                const int d = DT * (4 * (lane >> 4) + i) + dt;
                const uint32_t x = E4M3 ? widen<false>(p[d]) & 0xFFFFu : reinterpret_cast<const uint16_t*>(p)[d];
                const float y = (x & 0x7F80u) == 0x7F80u ? __uint_as_float(x << 16) : 0.0f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  if (tk <= t.lim[mt]) t.o[mt][dt][i] += y;
              }
          }
        }
      }
      if (have) begin(next);                             // under way while this piece is finished
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        t.l[mt] += shfl_xor(t.l[mt], 16);
        t.l[mt] += shfl_xor(t.l[mt], 32);
      }
      owner = now.s1 < now.n_s;                          // the stretch ends within the tile
      if (now.s0 > 0 && wave > 0) {
        // begun by an earlier wave of this workgroup, which joins it
        owner = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (lane < 16) share_ml[wave - 1][mt * 16 + lane] = make_float2(t.m[mt], t.l[mt]);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) share_o[wave - 1][mt * DT + dt][lane] = t.o[mt][dt];
        }
      } else if (!owner) {
        if (now.s0 == 0) write();
        else leave();
      }
      if (have) now = next;
    }
  }
  __syncthreads();
  if (!owner) return;
  // the pieces of the waves after this one that the tile reaches
  const int64_t last_u = now.real0 + now.n_s - 1;
  const int to = (int)min((int64_t)kWaves - 1, (last_u - group_u0) / chunk);
  for (int w = wave + 1; w <= to; ++w) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float2 ml = share_ml[w - 1][mt * 16 + (lane & 15)];
      const float mn = fmaxf(t.m[mt], ml.x);
      const float f = t.m[mt] == -INFINITY ? 0.0f : fast_exp2(t.m[mt] - mn);
      const float g = ml.x == -INFINITY ? 0.0f : fast_exp2(ml.x - mn);
      t.m[mt] = mn;
      t.l[mt] = t.l[mt] * f + ml.y * g;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) t.o[mt][dt] = t.o[mt][dt] * f + share_o[w - 1][mt * DT + dt][lane] * g;
    }
  }
  if (now.real0 >= group_u0 && last_u < group_u0 + group_chunk) write();
  else leave();
}

// Adds up the pieces of the tiles that several workgroups share: a workgroup for
// 16 rows, a wave of it for a quarter of their values, eight pieces in flight,
// or three where no more are left (12 and six: 1 us less where a tile has
// eleven, 0.3 more where it has two or three).  Bound by latency: a tile's
// place, then its pieces, 3.5 to 10 us.
template <int D>
__global__ __launch_bounds__(kAttendThreads) void attend_join_impl(const AttendArgs a) {
  constexpr int DT = D / 16, kV = DT / 4;
  const AttendJoin d = a.joins[blockIdx.x];
  const int lane = threadIdx.x & 63, mt = blockIdx.y, rows = a.rows;
  if (d.n == 0 || mt * 16 >= d.rows) return;
  const int row = mt * 16 + (lane & 15), dt0 = (threadIdx.x >> 6) * kV, size = rows * (D + 2);
  float M = -INFINITY, L = 0.0f;
  f32x4_t acc[kV];
#pragma unroll
  for (int c = 0; c < kV; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kPieces = 8, kFew = 3;
  for (int j0 = 0; j0 < d.n; j0 += kPieces) {
    float2 ml[kPieces];
    f32x4_t y[kPieces][kV];
    auto load = [&](int j) {
      // the first piece stands alone, the others at the beginnings of the stretches after it
      const int i = min(j0 + j, d.n - 1);
      const float* p = a.part + (int64_t)(i == 0 ? d.slot : (d.slot & ~1) + 2 * i) * size;
      ml[j] = *reinterpret_cast<const float2*>(p + 2 * row);
#pragma unroll
      for (int c = 0; c < kV; ++c)
        y[j][c] = reinterpret_cast<const f32x4_t*>(p + 2 * rows)[(mt * DT + dt0 + c) * 64 + lane];
    };
#pragma unroll
    for (int j = 0; j < kFew; ++j) load(j);
    if (d.n - j0 > kFew) {
#pragma unroll
      for (int j = kFew; j < kPieces; ++j) load(j);
    } else {
#pragma unroll
      for (int j = kFew; j < kPieces; ++j) {
        ml[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int c = 0; c < kV; ++c) y[j][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
    float mn = M;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) mn = fmaxf(mn, ml[j].x);
    if (j0 > 0) {
      const float f = M == -INFINITY ? 0.0f : fast_exp2(M - mn);
      L *= f;
#pragma unroll
      for (int c = 0; c < kV; ++c) acc[c] *= f;
    }
    M = mn;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const bool there = j0 + j < d.n;
      const float f = ml[j].x == -INFINITY ? 0.0f : fast_exp2(ml[j].x - M);
      L += there ? f * ml[j].y : 0.0f;
#pragma unroll
      for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[c][i] += there ? y[j][c][i] * f : 0.0f;
    }
  }
  if (row >= d.rows) return;
  const int grow = d.rt * rows + row, q = grow / a.group, hh = grow - q * a.group;
  const float inv = (a.v_scale ? a.v_scale[d.h] : 1.0f) * a.unrest / L;
  uint16_t* op = a.out + (int64_t)(d.row0 + q) * a.o_row + (int64_t)(d.h * a.group + hh) * a.o_head +
                 4 * DT * (lane >> 4) + dt0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kV == 1) {
      op[i * DT] = (uint16_t)pack_bf16(acc[0][i] * inv, 0.0f);
    } else {
#pragma unroll
      for (int c = 0; c < kV; c += 2)
        *reinterpret_cast<uint32_t*>(op + i * DT + c) = pack_bf16(acc[c][i] * inv, acc[c + 1][i] * inv);
    }
  }
  if (a.lse && threadIdx.x < 16)
    a.lse[(int64_t)(d.row0 + q) * a.Hq + d.h * a.group + hh] = (M + fast_log2(L)) * kLn2;
}

template <int D, int MT>
const void* attend_fn(int type, int g) {
  return type == kCacheE4m3   ? (const void*)&attend_impl<D, MT, kCacheE4m3, 8>
         : type == kCacheBf16 ? (const void*)&attend_impl<D, MT, kCacheBf16, 8>
         : g == 8             ? (const void*)&attend_impl<D, MT, kCacheMxfp4, 8>
                              : (const void*)&attend_impl<D, MT, kCacheMxfp4, 16>;
}

}  // namespace

const void* attend_kernel(int d, int mt, int type, int page) {
  const int g = page < 16 ? 8 : 16;
  if (d == 64) return mt == 1 ? attend_fn<64, 1>(type, g) : mt == 2 ? attend_fn<64, 2>(type, g) : attend_fn<64, 4>(type, g);
  if (d == 128) return mt == 1 ? attend_fn<128, 1>(type, g) : mt == 2 ? attend_fn<128, 2>(type, g) : attend_fn<128, 4>(type, g);
  return mt == 1 ? attend_fn<256, 1>(type, g) : attend_fn<256, 2>(type, g);
}

const void* attend_join_kernel(int d) {
  return d == 64 ? (const void*)&attend_join_impl<64> : d == 128 ? (const void*)&attend_join_impl<128>
                                                                : (const void*)&attend_join_impl<256>;
}

}  // namespace dspark
