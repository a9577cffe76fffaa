// Attention of packed rows over a paged key-value cache.
//
// [summary] section 5 (the flattened verify batch).  Row i of request b (K[b]
// + 1 rows: one token, a verify batch, or a draft block that sees itself)
// takes, for each of its query heads,
//     o = sum_t p_t v_t / sum_t p_t,   p_t = 2^(s_t - m),
//     s_t = (scale log2 e k_scale) q . k_t,
// over the tokens t it sees, in one pass with a running m (a row's sums are
// rescaled only when some score passes m by more than 8, so p_t stays below
// 2^8 and the products keep their bits).
//
// Work: a tile is the rows of one request that share a cache head (rows times
// heads per group, 16 MT of them at a time, so that a key is read once for
// all of them) over the request's tokens in units of 128.  All units of the
// batch stand in one line, request by request, and every workgroup takes an
// equal stretch of it, so that ragged lengths load the chip evenly without the
// host knowing them; a tile that falls to several workgroups is joined from
// its pieces by a second launch.
//
// In a workgroup each of the four waves takes 32 tokens of a unit.  Scores
// are formed transposed, S^T = K Q^T, and so is the product, O^T = V^T P^T:
// then the accumulators of the first product (a lane: one query, tokens 4 g + i
// of the two 16-token halves, g = lane / 16) are in place as the second's
// operand, whose eight products per lane may be taken in any order of tokens as
// long as the values come in the same order.  A lane loads its eight tokens'
// values at D / 16 neighbouring places, whole cache lines per token, and
// exchanges rows for columns within its own registers.  No key, value or score
// passes through LDS.
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

constexpr int kUnit = 128;       // tokens of a unit: 4 waves of 32

__device__ __forceinline__ f32x4_t mfma(const uint4 a, const uint4 b, const f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  bf16x2_t r;
  r[0] = (__bf16)lo;                                     // to nearest even
  r[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

// Two e4m3 values (the low or high half of w) as bf16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// The rows of request b: none where a length, row or count is out of range.
struct Rows {
  int n, len, row0;
};

__device__ __forceinline__ Rows request_rows(const AttendArgs& a, int b, bool report) {
  Rows r;
  int k = a.K ? a.K[b] : a.gamma;
  r.len = a.len[b];
  r.row0 = a.offs ? a.offs[b] : b * (a.gamma + 1);
  int bad = 0;
  if (k < -1 || k > a.gamma) {
    bad = kErrK;
    k = k < -1 ? -1 : a.gamma;
  }
  r.n = k + 1;
  if (r.n > 0 && (r.len < 0 || (int64_t)r.len + r.n > (int64_t)a.cols << a.page_shift)) {
    bad |= kErrCache;
    r.n = 0;
  }
  if (r.n > 0 && (r.row0 < 0 || (int64_t)r.row0 + r.n > a.n_rows)) {
    bad |= kErrRow;
    r.n = 0;
  }
  if (bad && report) atomicOr(a.err, bad);
  return r;
}

template <int D, int MT, int E4M3>
struct Tile {
  static constexpr int kRows = 16 * MT;
  static constexpr int KS = D / 32;                      // products of 32 values per score
  static constexpr int DT = D / 16;                      // 16-wide blocks of a value row
  static constexpr int KW = E4M3 ? KS / 2 : KS;          // 16-byte loads of a key per lane
  static constexpr int VW = DT * (E4M3 ? 1 : 2) / 4;     // words of a value per lane
  static constexpr int kSize = E4M3 ? 1 : 2;

  uint4 k[2][KW];
  uint32_t v[8][VW];
  uint4 q[MT][KS];
  f32x4_t o[MT][DT];
  float m[MT], l[MT];
  int lim[MT];                                           // last token a query sees
  int kid[2], vid[2];                                    // page ids of the next tile's tokens

  // Page ids of the tile of 32 tokens at `base`, tokens past `last` taken as
  // `last` (they are masked): the lane's two key tokens and two runs of four
  // value tokens, which a page of 8 or more holds whole.
  __device__ __forceinline__ void load_ids(const AttendArgs& a, const int32_t* table, int base, int last, int lane) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      kid[s] = table[min(base + 16 * s + (lane & 15), last) >> a.page_shift];
      vid[s] = table[min(base + 16 * s + 4 * (lane >> 4), last) >> a.page_shift];
    }
  }

  __device__ __forceinline__ int64_t page_base(const AttendArgs& a, int id) {
    if ((unsigned)id >= (unsigned)a.n_pages) {
      atomicOr(a.err, kErrPage);
      id = 0;
    }
    return (int64_t)id * a.c_page;
  }

  __device__ __forceinline__ void load_k(const AttendArgs& a, const unsigned char* kc, int base, int last, int lane) {
    const int in_page = (1 << a.page_shift) - 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int t = min(base + 16 * s + (lane & 15), last);
      const unsigned char* p = kc + page_base(a, kid[s]) + (int64_t)(t & in_page) * a.c_tok + 16 * (lane >> 4);
#pragma unroll
      for (int w = 0; w < KW; ++w) k[s][w] = *reinterpret_cast<const uint4*>(p + 64 * w);
    }
  }

  __device__ __forceinline__ void load_v(const AttendArgs& a, const unsigned char* vc, int base, int last, int lane) {
    const int in_page = (1 << a.page_shift) - 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const unsigned char* p = vc + page_base(a, vid[s]) + 4 * VW * (lane & 15);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = min(base + 16 * s + 4 * (lane >> 4) + i, last);
        const unsigned char* pt = p + (int64_t)(t & in_page) * a.c_tok;
        uint32_t(&w)[VW] = v[4 * s + i];
        if constexpr (VW == 1) {
          w[0] = *reinterpret_cast<const uint32_t*>(pt);
        } else if constexpr (VW == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(pt);
          w[0] = x.x;
          w[1] = x.y;
        } else {
#pragma unroll
          for (int c = 0; c < VW / 4; ++c) {
            const uint4 x = reinterpret_cast<const uint4*>(pt)[c];
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
  // + 8 g ..; e4m3: 64 (ks / 2) + 16 g + 8 (ks % 2) .., the order of q below).
  __device__ __forceinline__ uint4 key(int s, int ks) const {
    if constexpr (!E4M3) return k[s][ks];
    const uint4 w = k[s][ks >> 1];
    const uint32_t lo = ks & 1 ? w.z : w.x, hi = ks & 1 ? w.w : w.y;
    return make_uint4(widen<false>(lo), widen<true>(lo), widen<false>(hi), widen<true>(hi));
  }

  // The value operands of blocks dt and dt + 1: rows d = DT r + dt of V^T (r =
  // lane % 16), the lane's eight tokens in pairs.
  __device__ __forceinline__ void values(int dt, uint4 (&f)[2]) const {
    uint32_t x[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!E4M3) {
        const uint32_t e = v[2 * j][dt / 2], o2 = v[2 * j + 1][dt / 2];
        x[0][j] = __builtin_amdgcn_perm(o2, e, 0x05040100u);
        x[1][j] = __builtin_amdgcn_perm(o2, e, 0x07060302u);
      } else {
        const uint32_t e = v[2 * j][dt / 4], o2 = v[2 * j + 1][dt / 4];
        const uint32_t w = __builtin_amdgcn_perm(o2, e, dt & 2 ? 0x07030602u : 0x05010400u);
        x[0][j] = widen<false>(w);
        x[1][j] = widen<true>(w);
      }
    }
    f[0] = make_uint4(x[0][0], x[0][1], x[0][2], x[0][3]);
    f[1] = make_uint4(x[1][0], x[1][1], x[1][2], x[1][3]);
  }

  // The bits of the infinite and NaN ones among the two bf16 or four e4m3
  // values of a word.
  static __device__ __forceinline__ uint32_t odd_bf16(uint32_t x) {
    return ((x & 0x7F80u) == 0x7F80u ? 0x0000FFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
  }
  static __device__ __forceinline__ uint32_t odd_e4m3(uint32_t x) {
    return ((((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
  }

  __device__ __forceinline__ bool odd_values() const {
    uint32_t any = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int w = 0; w < VW; ++w) any |= E4M3 ? odd_e4m3(v[t][w]) : odd_bf16(v[t][w]);
    return any != 0;
  }

  __device__ __forceinline__ void add_odd_values(int base, int lane, const uint4 (&p)[MT]) {
    const int g = lane >> 4;
#pragma unroll
    for (int dt = 0; dt < DT; dt += 2) {
      uint4 f[2];
      values(dt, f);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        f[c] = make_uint4(f[c].x & odd_bf16(f[c].x), f[c].y & odd_bf16(f[c].y), f[c].z & odd_bf16(f[c].z),
                          f[c].w & odd_bf16(f[c].w));
#pragma unroll 1
      for (int t = 0; t < 32; ++t) {
        const int e = (t & 3) + (t >> 4) * 4, gt = (t >> 2) & 3;
        uint32_t keep[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) keep[j] = g == gt && e >> 1 == j ? (e & 1 ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 vf = make_uint4(f[c].x & keep[0], f[c].y & keep[1], f[c].z & keep[2], f[c].w & keep[3]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 pf = make_uint4(p[mt].x & keep[0], p[mt].y & keep[1], p[mt].z & keep[2], p[mt].w & keep[3]);
            const f32x4_t x = mfma(vf, pf, f32x4_t{0.f, 0.f, 0.f, 0.f});
            const bool seen = base + t <= lim[mt];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][dt + c][i] += seen ? x[i] : 0.0f;
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int w = 0; w < VW; ++w) v[t][w] &= ~(E4M3 ? odd_e4m3(v[t][w]) : odd_bf16(v[t][w]));
  }

  __device__ __forceinline__ void start(const AttendArgs& a, const Rows& r, int h, int rt, int lane) {
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
      m[mt] = -INFINITY;
      l[mt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[mt][dt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }

  // Scores, p and sums of the tile at `base`; `tail`: some query may not see
  // some token of it.  `next` loads the following tile's keys once this one's
  // are used, and then its values.
  template <typename NextK, typename NextV>
  __device__ __forceinline__ void step(int base, bool tail, float sc, int lane, NextK next_k, NextV next_v) {
    const int g = lane >> 4;
    f32x4_t s[MT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 kf = key(h, ks);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          s[mt][h] = mfma(kf, q[mt][ks], ks == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : s[mt][h]);
      }
    next_k();
    if (tail) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 16 * h + 4 * g + i > lim[mt]) s[mt][h][i] = -INFINITY;
    }
    float top[MT];
    bool grows = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float x = fmaxf(fmaxf(s[mt][0][0], s[mt][0][1]), fmaxf(s[mt][0][2], s[mt][0][3]));
      x = fmaxf(x, fmaxf(fmaxf(s[mt][1][0], s[mt][1][1]), fmaxf(s[mt][1][2], s[mt][1][3])));
      top[mt] = x * sc;
      grows |= top[mt] > m[mt] + 8.0f;
    }
    if (__any(grows)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x = fmaxf(top[mt], shfl_xor(top[mt], 16));
        x = fmaxf(x, shfl_xor(x, 32));
        const float mn = fmaxf(m[mt], x);
        const float f = mn == m[mt] ? 1.0f : fast_exp2(m[mt] - mn);
        m[mt] = mn;
        l[mt] *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[mt][dt] *= f;
      }
    }
    uint4 p[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float ref = m[mt] == -INFINITY ? 0.0f : m[mt];   // nothing seen yet: every p is 2^-inf = 0
      float e[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[4 * h + i] = fast_exp2(__builtin_fmaf(s[mt][h][i], sc, -ref));
      l[mt] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      // p as bf16 for the second product: half a unit of 2^-8 of each term, of
      // either sign, below the rounding of the bf16 result
      p[mt] = make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
    }
    // a token that a query does not see must not reach it, but 0 times
    // infinity or NaN is NaN: such values are taken out of the tile and added
    // one token at a time where they are seen
    if (tail && __any(odd_values())) add_odd_values(base, lane, p);
#pragma unroll
    for (int dt = 0; dt < DT; dt += 2) {
      uint4 f[2];
      values(dt, f);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][dt + c] = mfma(f[c], p[mt], o[mt][dt + c]);
    }
    next_v();
  }
};

// Workgroups of a variant that a CU is to hold (its registers are allotted
// for them).
template <int D, int MT>
constexpr int kPerCu = D * MT <= 128 ? 3 : D * MT <= 256 && D < 256 ? 2 : 1;

template <int D, int MT, int E4M3>
__global__ __launch_bounds__(kAttendThreads, (kPerCu<D, MT>)) void attend_impl(const AttendArgs a) {
  using T = Tile<D, MT, E4M3>;
  constexpr int kRows = T::kRows, DT = T::DT;
  __shared__ float4 red[4][DT][64];
  __shared__ float wm[4][kRows], wl[4][kRows];
  __shared__ int64_t sums[kAttendThreads / 64];
  __shared__ int start_b;
  __shared__ int64_t start_off;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  // units of every request, and where this workgroup's stretch begins
  const int per = (a.B + kAttendThreads - 1) / kAttendThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto units = [&](const Rows& r) -> int {
    if (r.n <= 0) return 0;
    return a.Hkv * ((a.group * r.n + kRows - 1) / kRows) * ((r.len + r.n + kUnit - 1) / kUnit);
  };
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += units(request_rows(a, b, blockIdx.x == 0));
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
  for (int w = 0; w < kAttendThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  int64_t chunk = (total + gridDim.x - 1) / gridDim.x;
  if (chunk < a.min_units) chunk = a.min_units;
  const int64_t u0 = blockIdx.x * chunk;
  const int64_t u1 = u0 + chunk < total ? u0 + chunk : total;
  if (u0 >= total) {
    if (tid == 0) {
      AttendPiece d;
      d.t0 = 0;
      a.pieces[blockIdx.x] = d;
    }
    return;
  }
  if (u0 >= before && u0 < before + mine) {
    int64_t base = before;
    for (int b = b0; b < b1; ++b) {
      const int n = units(request_rows(a, b, false));
      if (u0 < base + n) {
        start_b = b;
        start_off = u0 - base;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  int b = start_b, off = (int)start_off;
  int slot = 0;
  bool first = true;
  for (int64_t u = u0; u < u1;) {
    Rows r = request_rows(a, b, false);
    while (r.n <= 0) r = request_rows(a, ++b, false);    // u < u1 <= total: one follows
    const int L = r.len + r.n;
    const int n_rt = (a.group * r.n + kRows - 1) / kRows, n_t = (L + kUnit - 1) / kUnit;
    const int seg = off / n_t, t0 = off - seg * n_t;
    const int t1 = (int)(u1 - u < n_t - t0 ? t0 + (u1 - u) : n_t);
    const int h = seg / n_rt, rt = seg - h * n_rt;
    const bool whole = t0 == 0 && t1 == n_t;
    if (first && tid == 0) {
      AttendPiece d;
      d.b = b;
      d.h = h;
      d.rt = rt;
      d.n_t = n_t;
      d.t0 = t0;
      d.unit0 = u - t0;
      d.chunk = chunk;
      a.pieces[blockIdx.x] = d;
    }

    // this wave's tiles of 32 tokens: every fourth
    T t;
    t.start(a, r, h, rt, lane);
    const float sc = a.scale2 * (E4M3 && a.k_scale ? a.k_scale[h] : 1.0f);
    const int32_t* table = a.table + b * a.tstride;
    const unsigned char* kc = a.kc + (int64_t)h * a.c_head;
    const unsigned char* vc = a.vc + (int64_t)h * a.c_head;
    const int full = a.causal ? r.len : L - 1;           // tokens up to `full` are seen by every row
    int base = (t0 * 4 + wave) * 32;
    const int end = min(t1 * kUnit, L), last = end - 1;
    if (base < end) {
      t.load_ids(a, table, base, last, lane);
      t.load_k(a, kc, base, last, lane);
      t.load_v(a, vc, base, last, lane);
      t.load_ids(a, table, base + kUnit, last, lane);
      // the tile after the last one is token `last` over and over: loads
      // without a branch, of one cache line a lane group
      for (; base < end; base += kUnit)
        t.step(
            base, base + 31 > full, sc, lane, [&]() { t.load_k(a, kc, base + kUnit, last, lane); },
            [&]() {
              t.load_v(a, vc, base + kUnit, last, lane);
              t.load_ids(a, table, base + 2 * kUnit, last, lane);
            });
    }

    // the four waves' sums, 16 queries at a time
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float l = t.l[mt];
      l += shfl_xor(l, 16);
      l += shfl_xor(l, 32);
      if (lane < 16) {
        wm[wave][mt * 16 + lane] = t.m[mt];
        wl[wave][mt * 16 + lane] = l;
      }
    }
    const float vs = E4M3 && a.v_scale ? a.v_scale[h] : 1.0f;
    float* part = a.part + ((int64_t)blockIdx.x * 2 + slot) * (kRows * (D + 2));
    // thread: query tid / 16, values DT (tid % 16) ..
    const int qi = tid >> 4, rr = tid & 15;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        red[wave][dt][lane] = make_float4(t.o[mt][dt][0], t.o[mt][dt][1], t.o[mt][dt][2], t.o[mt][dt][3]);
      __syncthreads();
      const int row = mt * 16 + qi;
      float M = wm[0][row];
#pragma unroll
      for (int w = 1; w < 4; ++w) M = fmaxf(M, wm[w][row]);
      float f[4], lsum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = wm[w][row] == -INFINITY ? 0.0f : fast_exp2(wm[w][row] - M);
        lsum += f[w] * wl[w][row];
      }
      float acc[DT];
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float* y = reinterpret_cast<const float*>(&red[w][dt][(rr >> 2) * 16 + qi]);
          x += f[w] * y[rr & 3];
        }
        acc[dt] = x;
      }
      const int grow = rt * kRows + row;
      if (grow < a.group * r.n) {
        if (whole) {
          const int i = grow / a.group, hh = grow - i * a.group;
          const float inv = vs / lsum;
          uint16_t* op = a.out + (int64_t)(r.row0 + i) * a.o_row + (int64_t)(h * a.group + hh) * a.o_head + DT * rr;
          uint32_t w[DT / 2];
#pragma unroll
          for (int c = 0; c < DT / 2; ++c) w[c] = pack_bf16(acc[2 * c] * inv, acc[2 * c + 1] * inv);
          if constexpr (DT == 4) {
            *reinterpret_cast<uint2*>(op) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int c = 0; c < DT / 8; ++c)
              reinterpret_cast<uint4*>(op)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          }
          if (a.lse && rr == 0)
            a.lse[(int64_t)(r.row0 + i) * a.Hq + h * a.group + hh] = (M + fast_log2(lsum)) * kLn2;
        } else {
          if (rr == 0) {
            part[row] = M;
            part[kRows + row] = lsum;
          }
          float4* pp = reinterpret_cast<float4*>(part + 2 * kRows + row * D + DT * rr);
#pragma unroll
          for (int c = 0; c < DT / 4; ++c)
            pp[c] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
        }
      }
    }
    __syncthreads();
    u += t1 - t0;
    off += t1 - t0;
    slot = 1;
    first = false;
    if (off == a.Hkv * n_rt * n_t) {
      ++b;
      off = 0;
    }
  }
}

// Joins the pieces of one tile: those of workgroups w - 1, w, .. where w is
// the first whose stretch begins inside the tile.  A wave per row; pieces are
// added in the order of their tokens.
template <int D>
__global__ __launch_bounds__(kAttendThreads) void attend_join_impl(const AttendArgs a) {
  const int rows = a.rows;
  const int w = blockIdx.x + 1;
  const AttendPiece d = a.pieces[w];
  if (d.t0 == 0 || d.unit0 < (w - 1) * d.chunk) return;
  const Rows r = request_rows(a, d.b, false);
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.y * (kAttendThreads / 64) + (threadIdx.x >> 6);
  const int grow = d.rt * rows + row;
  if (grow >= a.group * r.n) return;
  const int n = (int)((d.unit0 + d.n_t - 1) / d.chunk) - (w - 1) + 1;
  const int size = rows * (D + 2);
  // piece j: workgroup w - 1 + j; the first may be the second of its workgroup
  const int skip = d.unit0 == (w - 1) * d.chunk ? 0 : 1;
  auto piece = [&](int j) { return a.part + ((int64_t)(w - 1 + j) * 2 + (j == 0 ? skip : 0)) * size; };
  float M = -INFINITY;
  for (int j = lane; j < n; j += 64) M = fmaxf(M, piece(j)[row]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) M = fmaxf(M, shfl_xor(M, o));
  float L = 0.0f, acc[D / 64];
#pragma unroll
  for (int c = 0; c < D / 64; ++c) acc[c] = 0.0f;
  for (int j0 = 0; j0 < n; j0 += 64) {
    float f = 0.0f;
    if (j0 + lane < n) {
      const float* p = piece(j0 + lane);
      f = p[row] == -INFINITY ? 0.0f : fast_exp2(p[row] - M);
      L += f * p[rows + row];
    }
    const int m = min(64, n - j0);
#pragma unroll 4
    for (int j = 0; j < m; ++j) {
      const float fj = __shfl(f, j, 64);
      const float* p = piece(j0 + j) + 2 * rows + row * D;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float y = p[(D / 64) * lane + c];
        acc[c] += fj * y;
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) L += shfl_xor(L, o);
  const int i = grow / a.group, hh = grow - i * a.group;
  const float inv = (a.v_scale ? a.v_scale[d.h] : 1.0f) / L;
  uint16_t* op = a.out + (int64_t)(r.row0 + i) * a.o_row + (int64_t)(d.h * a.group + hh) * a.o_head;
  if constexpr (D == 64) {
    op[lane] = (uint16_t)pack_bf16(acc[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int c = 0; c < D / 128; ++c)
      reinterpret_cast<uint32_t*>(op)[(D / 128) * lane + c] = pack_bf16(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[(int64_t)(r.row0 + i) * a.Hq + d.h * a.group + hh] = (M + fast_log2(L)) * kLn2;
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
