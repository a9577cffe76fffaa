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
// One workgroup a CU, one wave a SIMD: its registers hold the next two steps'
// keys and values in flight (64 to 128 KB a CU), which is what the memory's
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
// stretch and its first keys.
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

constexpr int kStep = 32;        // tokens of a step
constexpr int kWaves = kAttendThreads / 64;
// What a tile costs besides its steps, in steps, and the steps of a wave's
// stretch at least.  128 requests of 64 to 8192 tokens: 117 us with a cost of
// 1, 119 with 2, 123 with 4; one row of one request of up to 1200 tokens: 14.2 us
// with at least 1 step, 16.1 with 2 (a wave's first step waits for its loads,
// the second is nearly free, but so is the wave that would take it).
constexpr int kTileCost = 1, kMinSteps = 1;

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

__device__ __forceinline__ uint4 load16(const unsigned char* p) {
  typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
  const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
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

// Keys and values of a step as a lane has them loaded.
template <int D, int E4M3>
struct Loaded {
  static constexpr int KW = E4M3 ? D / 64 : D / 32;      // 16-byte loads of a key per lane
  static constexpr int VW = D / 16 * (E4M3 ? 1 : 2) / 4; // words of a value per lane
  uint4 k[2][KW];
  uint32_t v[8][VW];

  // A lane's keys: token lane % 16 of either half, `kl` its place in a group.
  __device__ __forceinline__ void load_k(const unsigned char* kc, const int64_t (&at)[4], unsigned kl, int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t lo = at[2 * s], hi = at[2 * s + 1];
      const unsigned char* p = kc + (lane & 8 ? hi : lo) + kl;
#pragma unroll
      for (int w = 0; w < KW; ++w) k[s][w] = load16(p + 64 * w);
    }
  }

  // A lane's values: tokens 4 g + i of either half, `vl` the first one's place in its group.
  __device__ __forceinline__ void load_v(const unsigned char* vc, const int64_t (&at)[4], unsigned vl, int64_t c_tok,
                                         int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t lo = at[2 * s], hi = at[2 * s + 1];
      const unsigned char* p = vc + (lane & 32 ? hi : lo) + vl;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* pt = p + i * c_tok;
        uint32_t(&w)[VW] = v[4 * s + i];
        if constexpr (VW == 1) {
          w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(pt));
        } else if constexpr (VW == 2) {
          typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
          const u32x2_t x = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(pt));
          w[0] = x[0];
          w[1] = x[1];
        } else {
#pragma unroll
          for (int c = 0; c < VW / 4; ++c) {
            const uint4 x = load16(pt + 16 * c);
            w[4 * c] = x.x;
            w[4 * c + 1] = x.y;
            w[4 * c + 2] = x.z;
            w[4 * c + 3] = x.w;
          }
        }
      }
    }
  }

  // The key operand of product ks: 16 tokens (a lane: its token's values 32 ks
  // + 8 g ..; e4m3: 64 (ks / 2) + 16 g + 8 (ks % 2) .., the order of the queries too).
  __device__ __forceinline__ uint4 key(int s, int ks) const {
    if constexpr (!E4M3) return k[s][ks];
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
      if constexpr (!E4M3) {
        const uint32_t e = v[2 * j][dt / 2], o = v[2 * j + 1][dt / 2];
        x[0][j] = __builtin_amdgcn_perm(o, e, 0x05040100u);
        x[1][j] = __builtin_amdgcn_perm(o, e, 0x07060302u);
      } else {
        const uint32_t e = v[2 * j][dt / 4], o = v[2 * j + 1][dt / 4];
        const uint32_t w = __builtin_amdgcn_perm(o, e, dt & 2 ? 0x07030602u : 0x05010400u);
        x[0][j] = widen_f16<false>(w);
        x[1][j] = widen_f16<true>(w);
      }
    }
    f[0] = make_uint4(x[0][0], x[0][1], x[0][2], x[0][3]);
    f[1] = make_uint4(x[1][0], x[1][1], x[1][2], x[1][3]);
  }

  // Takes infinite and NaN values out; whether there were any.
  __device__ __forceinline__ uint32_t take_odd() {
    uint32_t odd = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t x = E4M3 ? odd_e4m3(v[t][w]) : odd_bf16(v[t][w]);
        odd |= x;
        v[t][w] &= ~x;
      }
    return odd;
  }
};

// Where the four groups of eight tokens of a step begin in a cache.  A page
// holds whole groups; one behind the last token is taken as the last group,
// and places of a group behind the last token are read and masked.  Page ids
// are uniform: scalar loads, whose wait is none of the key and value loads'.
struct Groups {
  int id[4];
  __device__ __forceinline__ static int first(int base, int j, int last) { return min(base + 8 * j, last & ~7); }
  __device__ __forceinline__ void load(const AttendArgs& a, const int32_t* table, int base, int last) {
    const uniform_ptr t = (uniform_ptr)(uintptr_t)table;
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = t[first(base, j, last) >> a.page_shift];
  }
  // Bytes from the cache's beginning, for the step at `base` whose ids are loaded.
  __device__ __forceinline__ void place(const AttendArgs& a, int base, int last, int64_t (&at)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int p = id[j];
      if ((unsigned)p >= (unsigned)a.n_pages) {
        atomicOr(a.err, kErrPage);
        p = 0;
      }
      at[j] = (int64_t)p * a.c_page + (int64_t)(first(base, j, last) & ((1 << a.page_shift) - 1)) * a.c_tok;
    }
  }
};

template <int D, int MT, int E4M3>
struct Tile {
  using In = Loaded<D, E4M3>;
  static constexpr int kRows = 16 * MT;
  static constexpr int KS = D / 32;                      // products of 32 values per score
  static constexpr int DT = D / 16;                      // 16-wide blocks of a value row
  // m stands this far below the row's maximum (in the exponent) when it is set.  The weights of an e4m3 cache
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
        const int d = E4M3 ? 64 * (ks >> 1) + 16 * (lane >> 4) + 8 * (ks & 1) : 32 * ks + 8 * (lane >> 4);
        q[mt][ks] = ok ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
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
    // The weights of the second product.  bf16 values: a weight is the sum of
    // two bf16 numbers, its leading 8 bits and the rest to nearest, off by
    // 2^-15 of it at most (rounded to one, 2^-8 of it, they cost as much as the
    // rounding of the result does).  The rest is that of 1 + 2^-16 times the
    // weight (a.unrest takes the factor out of the result): positive wherever
    // the weight is, since 0 times an infinite value is NaN.  e4m3 values are
    // exact in f16, whose 11 bits leave 2^-11 of a weight, far below the
    // rounding of the values that such a cache holds.
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
          const uint32_t a = __float_as_uint(e[2 * j]), b = __float_as_uint(e[2 * j + 1]);
          w[j] = __builtin_amdgcn_perm(b, a, 0x07060302u);
          x[j] = pack_bf16(__builtin_fmaf(e[2 * j], kRestFactor, -__uint_as_float(a & 0xFFFF0000u)),
                           __builtin_fmaf(e[2 * j + 1], kRestFactor, -__uint_as_float(b & 0xFFFF0000u)));
        }
      }
      p[mt] = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (!E4M3) rest[mt] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    // a token that a query does not see must not reach it, but 0 times
    // infinity or NaN is NaN: such values are left out here and added to the
    // results that see them at the end
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
template <int D, int MT, int E4M3>
constexpr int kAhead = D * MT >= 512 && !E4M3 ? 1 : 2;

// A wave's steps s0 .. s1 - 1 of a tile: the rows of request r at cache head h, row tile rt.
struct Piece {
  Rows r;
  int h, rt, n_s, s0, s1;        // n_s: steps of the whole tile
  int64_t real0;                 // where they begin in the line
  const int32_t* table;          // the request's pages
  __device__ __forceinline__ int last() const { return min(s1 * kStep, r.len + r.n) - 1; }
};

template <int D, int MT, int E4M3>
__global__ __launch_bounds__(kAttendThreads, 1) void attend_impl(const AttendArgs a) {
  using T = Tile<D, MT, E4M3>;
  using In = Loaded<D, E4M3>;
  constexpr int kRows = T::kRows, DT = T::DT;
  __shared__ int64_t sums[kWaves];
  __shared__ Rows start_rows[kWaves];
  __shared__ int start_b[kWaves], start_off[kWaves];
  __shared__ f32x4_t share_o[kWaves - 1][MT * DT][64];    // what waves 1 .. 3 begin with of a tile
  __shared__ float2 share_ml[kWaves - 1][kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a lane's place in a group of eight tokens: its key's and its first value's
  const unsigned kl = (unsigned)(lane & 7) * (unsigned)a.c_tok + 16 * (lane >> 4);
  const unsigned vl = 4 * (lane >> 4 & 1) * (unsigned)a.c_tok + 4 * In::VW * (lane & 15);

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
    if (r.bad && blockIdx.x == 0) atomicOr(a.err, r.bad);
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
  const int64_t group_chunk = kWaves * chunk, group_u0 = blockIdx.x * group_chunk;
  if (group_u0 >= total) {
    if (tid == 0) a.joins[blockIdx.x].n = 0;
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
    float* part = a.part + (int64_t)(2 * blockIdx.x + (group_u0 < now.real0 - kTileCost ? 1 : 0)) * (kRows * (D + 2));
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
            j.n = (int)((p.real0 + p.n_s - 1) / group_chunk) - (int)blockIdx.x + 2;
            j.slot = 2 * ((int)blockIdx.x - 1) + (group_u0 - group_chunk < p.real0 - kTileCost ? 1 : 0);
          }
          a.joins[blockIdx.x] = j;
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
    constexpr int N = kAhead<D, MT, E4M3>;
    In in[N];
    Groups ids[N + 1];
    int64_t at[4];
    // a piece's first steps: page ids, then queries, keys and values
    auto ask = [&](const Piece& p) {
#pragma unroll
      for (int i = 0; i <= N; ++i) ids[i].load(a, p.table, (p.s0 + i) * kStep, p.last());
    };
    auto begin = [&](const Piece& p) {
      const unsigned char *kc = a.kc + (int64_t)p.h * a.c_head, *vc = a.vc + (int64_t)p.h * a.c_head;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ids[i].place(a, (p.s0 + i) * kStep, p.last(), at);
        in[i].load_k(kc, at, kl, lane);
        if (i == 0) t.load_q(a, p.r, p.h, p.rt, lane);
        in[i].load_v(vc, at, vl, a.c_tok, lane);
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
      const int full = a.causal ? now.r.len : L - 1;     // tokens up to `full` are seen by every row
      const int last = now.last();
      Groups id = ids[N];
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
                id.place(a, base + N * kStep, last, at);
                id.load(a, now.table, base + (N + 1) * kStep, last);
                in[i].load_k(kc, at, kl, lane);
              },
              [&]() {
                if (MT == 4 || base + N * kStep <= last) in[i].load_v(vc, at, vl, a.c_tok, lane);
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
// 16 rows, a wave of it for a quarter of their values, eight pieces in flight
// (16: 1 us more where a tile has two or three pieces, no less where it has
// eleven).  Bound by latency: a tile's place, then its pieces, 4 to 11 us.
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
  constexpr int kPieces = 8;
  for (int j0 = 0; j0 < d.n; j0 += kPieces) {
    float2 ml[kPieces];
    f32x4_t y[kPieces][kV];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      // the first piece stands alone, the others at the beginnings of the stretches after it
      const int i = min(j0 + j, d.n - 1);
      const float* p = a.part + (int64_t)(i == 0 ? d.slot : (d.slot & ~1) + 2 * i) * size;
      ml[j] = *reinterpret_cast<const float2*>(p + 2 * row);
#pragma unroll
      for (int c = 0; c < kV; ++c)
        y[j][c] = reinterpret_cast<const f32x4_t*>(p + 2 * rows)[(mt * DT + dt0 + c) * 64 + lane];
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
const void* attend_fn(int e4m3) {
  return e4m3 ? (const void*)&attend_impl<D, MT, 1> : (const void*)&attend_impl<D, MT, 0>;
}

}  // namespace

const void* attend_kernel(int d, int mt, int e4m3) {
  if (d == 64) return mt == 1 ? attend_fn<64, 1>(e4m3) : mt == 2 ? attend_fn<64, 2>(e4m3) : attend_fn<64, 4>(e4m3);
  if (d == 128) return mt == 1 ? attend_fn<128, 1>(e4m3) : mt == 2 ? attend_fn<128, 2>(e4m3) : attend_fn<128, 4>(e4m3);
  return mt == 1 ? attend_fn<256, 1>(e4m3) : attend_fn<256, 2>(e4m3);
}

const void* attend_join_kernel(int d) {
  return d == 64 ? (const void*)&attend_join_impl<64> : d == 128 ? (const void*)&attend_join_impl<128>
                                                                : (const void*)&attend_join_impl<256>;
}

}  // namespace dspark
