// Penalties for repeated tokens, biases and grammar masks on logit rows.
//
// [blog] "形式化定义" (the target scores every drafted position of a request in
// one pass): row i of a request follows its history and the drafts x_1 .. x_i,
// so its penalties count those drafts too.  With c the number of times entry
// v was written (history behind the prompt, and x_1 .. x_i) and `seen` whether
// it occurs there or in the prompt:
//     l1 = seen ? (l > 0 ? l / rep : l rep) : l
//     out = allowed ? max(l1 - freq c - pres [c > 0] + bias, kMasked) : kMasked
//
// Bound by memory: every logit is read and its float32 written once.  A
// workgroup takes a slice of the vocabulary of one request for all of its
// rows.  It counts the history's tokens of its slice in LDS (integers: any
// order of the additions gives the same counts), one word an entry, read once
// for the request's rows together; a word of zero is an entry that no rule but
// the mask touches.  Entries whose count differs between the rows (drafted
// tokens) or that carry a bias are marked in their word, and the thread that
// marks one works it out for every row; the pass over the slice leaves them
// out (worked out inside that pass, one entry held up its whole wave: 301 us
// against 166 on 1024 rows of 151936 bf16 logits with 32 biases and a mask).
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

constexpr uint32_t kPrompt = 0x80000000u, kSpecial = 0x40000000u, kCount = 0x3FFFFFFFu;

// Four logits of a row (a uniform pointer) at entry v; rows are read once.
template <int BF16>
__device__ __forceinline__ f32x4_t load4(const char* row, unsigned v) {
  if constexpr (BF16) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
    const u32x2_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(row + 2 * v));
    return f32x4_t{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                   __uint_as_float(w[1] & 0xFFFF0000u)};
  }
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(row + 4 * v));
}

template <int BF16>
__device__ __forceinline__ float load1(const char* row, unsigned v) {
  if constexpr (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[v]);
  return reinterpret_cast<const float*>(row)[v];
}

struct Penalty {
  float rep, inv, freq, pres;    // inv: 1 / rep
};

__device__ __forceinline__ float penalised(float x, uint32_t word, const Penalty& p) {
  const float c = (float)(word & kCount);
  // x / rep: the reciprocal's product and its remainder, within a unit of the
  // last place (1.5 where x is subnormal); rep is normal
  const float q = x * p.inv;
  const float d = __builtin_fmaf(__builtin_fmaf(-q, p.rep, x), p.inv, q);
  const float y = x > 0.0f ? (d == d ? d : q) : x * p.rep;
  return y - p.freq * c - (c > 0.0f ? p.pres : 0.0f);
}

// y where bit e of `bits` is set, else kMasked.
__device__ __forceinline__ float allowed(float y, uint32_t bits, int e) {
  const uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)bits, e, 1);
  return __uint_as_float((__float_as_uint(y) & m) | (__float_as_uint(kMasked) & ~m));
}

// NaN stays; the lowest values and -infinity become kMasked.
__device__ __forceinline__ float at_least_masked(float x) { return x < kMasked ? kMasked : x; }

// Sum of the biases of entry v (ids ascending, equal ids in order).
__device__ __forceinline__ float bias_of(const int32_t* ids, const float* values, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ids[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  float s = 0.0f;
  for (; lo < n && ids[lo] == v; ++lo) s += values[lo];
  return s;
}

template <int BF16>
__global__ __launch_bounds__(kConstrainThreads) void constrain_impl(const ConstrainArgs a) {
  __shared__ __align__(16) uint32_t count[kConstrainMaxSlice];
  __shared__ int32_t drafted[kMaxGamma];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int v0 = blockIdx.x * a.slice, v1 = min(a.V, v0 + a.slice);
  const bool report = blockIdx.x == 0;

  // rows of the request
  int n = a.n_pos;
  if (a.K) {
    int k = a.K[b];
    if (k < -1 || k >= a.n_pos) {
      if (report && tid == 0) atomicOr(a.err, kErrK);
      k = k < -1 ? -1 : a.n_pos - 1;
    }
    n = k + 1;
  }
  int64_t row0 = (int64_t)b * a.n_pos;                   // mask rows and packed rows
  if (a.offs) {
    row0 = a.offs[b];
    if (n > 0 && (row0 < 0 || row0 + n > a.n_rows)) {
      if (report && tid == 0) atomicOr(a.err, kErrRow);
      return;
    }
  }
  if (n <= 0) return;

  // the counts of this slice
  for (int i = tid * 4; i < a.slice; i += kConstrainThreads * 4) *reinterpret_cast<uint4*>(count + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (a.hist) {
    int len = a.n_hist[b];
    if (len < 0 || len > a.hist_max) {
      if (report && tid == 0) atomicOr(a.err, kErrHist);
      len = len < 0 ? 0 : a.hist_max;
    }
    const int prompt = a.n_prompt ? a.n_prompt[b] : 0;
    const int32_t* h = a.hist + b * a.hist_stride;
    constexpr int kUnroll = 8;
    for (int i0 = tid; i0 < len; i0 += kUnroll * kConstrainThreads) {
      int t[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) t[u] = h[min(i0 + u * kConstrainThreads, len - 1)];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kConstrainThreads;
        if (report && (unsigned)t[u] >= (unsigned)a.V) atomicOr(a.err, kErrToken);
        if (i < len && t[u] >= v0 && t[u] < v1) {
          if (i < prompt) atomicOr(&count[t[u] - v0], kPrompt);
          else atomicAdd(&count[t[u] - v0], 1u);
        }
      }
    }
  }
  const int n_draft = a.tokens ? n - 1 : 0;
  if (tid < n_draft) {
    drafted[tid] = a.tokens[b * a.tok_stride + tid];
    if (report && (unsigned)drafted[tid] >= (unsigned)a.V) atomicOr(a.err, kErrToken);
  }
  const float rep = a.rep ? a.rep[b] : 1.0f;
  const bool rep_ok = rep >= 0x1p-126f && rep < INFINITY;   // (a subnormal one's reciprocal is infinite)
  if (!rep_ok && report && tid == 0) atomicOr(a.err, kErrPenalty);
  Penalty pen;
  pen.rep = rep_ok ? rep : 1.0f;
  pen.inv = 1.0f / pen.rep;
  pen.freq = a.freq ? a.freq[b] : 0.0f;
  pen.pres = a.pres ? a.pres[b] : 0.0f;
  int n_bias = 0;
  const int64_t bias_row = (int64_t)b * a.bias_stride;
  if (a.bias_id) {
    n_bias = a.n_bias ? a.n_bias[b] : a.bias_max;
    if (n_bias < 0 || n_bias > a.bias_max) {
      if (report && tid == 0) atomicOr(a.err, kErrHist);
      n_bias = n_bias < 0 ? 0 : a.bias_max;
    }
  }
  __syncthreads();

  auto in_row = [&](int i) {
    return static_cast<const char*>(a.in) + (a.offs ? (row0 + i) * a.in_k : b * a.in_b + i * a.in_k) * (BF16 ? 2 : 4);
  };
  auto out_row = [&](int i) {
    return reinterpret_cast<char*>(a.out) + (a.offs ? (row0 + i) * a.out_k : b * a.out_b + i * a.out_k) * 4;
  };
  auto mask_row = [&](int i) {
    return reinterpret_cast<const uint8_t*>(a.mask + (a.offs ? (row0 + i) * a.mask_k : b * a.mask_b + i * a.mask_k));
  };

  // the marked entries: drafted tokens, then biases
  for (int j = tid; j < n_draft + n_bias; j += kConstrainThreads) {
    const int v = j < n_draft ? drafted[j] : a.bias_id[bias_row + j - n_draft];
    if (report && j >= n_draft) {
      if ((unsigned)v >= (unsigned)a.V) atomicOr(a.err, kErrToken);
      if (j > n_draft && a.bias_id[bias_row + j - n_draft - 1] > v) atomicOr(a.err, kErrBias);
    }
    if (v < v0 || v >= v1) continue;
    const uint32_t w = atomicOr(&count[v - v0], kSpecial);
    if (w & kSpecial) continue;                          // another thread's
    const float bias = n_bias > 0 ? bias_of(a.bias_id + bias_row, a.bias_val + bias_row, n_bias, v) : 0.0f;
    uint32_t c = w;
    for (int i = 0; i < n; ++i) {
      if (i > 0 && i <= n_draft) c += drafted[i - 1] == v ? 1u : 0u;
      float x = load1<BF16>(in_row(i), v);
      if (c) x = penalised(x, c, pen);
      x = at_least_masked(x + bias);
      if (a.mask) x = allowed(x, mask_row(i)[v >> 3], v & 7);
      reinterpret_cast<float*>(out_row(i))[v] = x;
    }
  }
  __syncthreads();

  // the others: four entries a thread, rows in groups so that several rows'
  // loads are in flight
  constexpr int kGroup = 8;
  for (int v = v0 + 4 * tid; v < v1; v += 4 * kConstrainThreads) {
    const uint4 w4 = *reinterpret_cast<const uint4*>(count + (v - v0));
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    const uint32_t any = w[0] | w[1] | w[2] | w[3];
    if (v + 4 > a.V) {
      for (int i = 0; i < n; ++i)
        for (int e = 0; v + e < a.V; ++e) {
          if (w[e] & kSpecial) continue;
          float y = load1<BF16>(in_row(i), v + e);
          if (w[e]) y = penalised(y, w[e], pen);
          y = at_least_masked(y);
          if (a.mask) y = allowed(y, mask_row(i)[(v + e) >> 3], (v + e) & 7);
          reinterpret_cast<float*>(out_row(i))[v + e] = y;
        }
      continue;
    }
    const bool touched = __any(any != 0);
    for (int i0 = 0; i0 < n; i0 += kGroup) {
      f32x4_t x[kGroup];
      uint32_t bits[kGroup];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const int i = min(i0 + u, n - 1);
        x[u] = load4<BF16>(in_row(i), v);
        bits[u] = a.mask ? mask_row(i)[(unsigned)v >> 3] : 0xFFu;
      }
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const f32x4_t was = x[u];
        if (touched) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = penalised(x[u][e], w[e], pen);
            x[u][e] = w[e] ? y : x[u][e];
          }
        }
        const uint32_t nibble = bits[u] >> (v & 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[u][e] = allowed(at_least_masked(x[u][e]), nibble, e);
        // in place, what stays as it is need not be written again
        bool write = i0 + u < n;
        if (!BF16 && a.in_place) {
          bool same = true;
#pragma unroll
          for (int e = 0; e < 4; ++e) same = same && __float_as_uint(was[e]) == __float_as_uint(x[u][e]);
          write = write && !same;
        }
        if (write) {
          char* p = out_row(i0 + u) + 4 * (unsigned)v;
          if (!(any & kSpecial)) {
            __builtin_nontemporal_store(x[u], reinterpret_cast<f32x4_t*>(p));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(w[e] & kSpecial)) reinterpret_cast<float*>(p)[e] = x[u][e];
          }
        }
      }
    }
  }
}

}  // namespace

const void* constrain_kernel(int bf16) {
  return bf16 ? (const void*)&constrain_impl<1> : (const void*)&constrain_impl<0>;
}

}  // namespace dspark
