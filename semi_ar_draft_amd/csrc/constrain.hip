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
// tokens) or that carry a bias are marked in their word and worked out one by
// one.
#include "common.hpp"
#include "internal.hpp"

namespace dspark {
namespace {

constexpr uint32_t kPrompt = 0x80000000u, kSpecial = 0x40000000u, kCount = 0x3FFFFFFFu;

template <int BF16>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  if constexpr (BF16) {
    typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
    const u32x2_t w =
        __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + i));
    return make_float4(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                       __uint_as_float(w[1] & 0xFFFF0000u));
  }
  const f32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i));
  return make_float4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store4(float* p, const float (&y)[4]) {
  __builtin_nontemporal_store(f32x4_t{y[0], y[1], y[2], y[3]}, reinterpret_cast<f32x4_t*>(p));
}

template <int BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float penalised(float x, uint32_t word, const Penalty& p) {
  const float c = (float)(word & kCount);
  const float y = x > 0.0f ? x / p.rep : x * p.rep;
  return y - p.freq * c - (c > 0.0f ? p.pres : 0.0f);
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
    const int t = a.tokens[b * a.tok_stride + tid];
    drafted[tid] = t;
    if (report && (unsigned)t >= (unsigned)a.V) atomicOr(a.err, kErrToken);
    if (t >= v0 && t < v1) atomicOr(&count[t - v0], kSpecial);
  }
  int n_bias = 0;
  const int32_t* bias_id = a.bias_id + (int64_t)b * a.bias_stride;
  const float* bias_val = a.bias_val + (int64_t)b * a.bias_stride;
  if (a.bias_id) {
    n_bias = a.n_bias ? a.n_bias[b] : a.bias_max;
    if (n_bias < 0 || n_bias > a.bias_max) {
      if (report && tid == 0) atomicOr(a.err, kErrHist);
      n_bias = n_bias < 0 ? 0 : a.bias_max;
    }
    for (int i = tid; i < n_bias; i += kConstrainThreads) {
      const int t = bias_id[i];
      if (report && (unsigned)t >= (unsigned)a.V) atomicOr(a.err, kErrToken);
      if (report && i > 0 && bias_id[i - 1] > t) atomicOr(a.err, kErrBias);
      if (t >= v0 && t < v1) atomicOr(&count[t - v0], kSpecial);
    }
  }
  Penalty pen{a.rep ? a.rep[b] : 1.0f, a.freq ? a.freq[b] : 0.0f, a.pres ? a.pres[b] : 0.0f};
  if (!(pen.rep > 0.0f) || !(pen.rep < INFINITY)) {
    if (report && tid == 0) atomicOr(a.err, kErrPenalty);
    pen.rep = 1.0f;
  }
  __syncthreads();

  // out of an entry of row i whose word is w
  auto value = [&](float x, uint32_t w, int i, int v) -> float {
    if (w & kSpecial) {
      uint32_t c = w & (kPrompt | kCount);
      for (int j = 0; j < min(i, n_draft); ++j) c += drafted[j] == v ? 1u : 0u;
      if (c) x = penalised(x, c, pen);
      if (n_bias > 0) x += bias_of(bias_id, bias_val, n_bias, v);
    } else if (w) {
      x = penalised(x, w, pen);
    }
    return at_least_masked(x);
  };

  // rows in groups, so that several rows' loads are in flight
  constexpr int kGroup = 4;
  auto in_row = [&](int i) { return a.offs ? (row0 + i) * a.in_k : b * a.in_b + i * a.in_k; };
  auto out_row = [&](int i) { return a.offs ? (row0 + i) * a.out_k : b * a.out_b + i * a.out_k; };
  auto mask_row = [&](int i) {
    return reinterpret_cast<const uint8_t*>(a.mask + (a.offs ? (row0 + i) * a.mask_k : b * a.mask_b + i * a.mask_k));
  };
  for (int v = v0 + 4 * tid; v < v1; v += 4 * kConstrainThreads) {
    const uint4 w4 = *reinterpret_cast<const uint4*>(count + (v - v0));
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    const uint32_t any = w[0] | w[1] | w[2] | w[3];
    if (v + 4 <= a.V) {
      for (int i0 = 0; i0 < n; i0 += kGroup) {
        float4 x[kGroup];
        uint32_t bits[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          const int i = min(i0 + u, n - 1);
          x[u] = load4<BF16>(a.in, in_row(i) + v);
          bits[u] = a.mask ? mask_row(i)[v >> 3] >> (v & 4) : 0xFu;
        }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          const int i = i0 + u;
          float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = any ? value(y[e], w[e], i, v + e) : at_least_masked(y[e]);
            y[e] = bits[u] >> e & 1u ? y[e] : kMasked;
          }
          if (i < n) store4(a.out + out_row(i) + v, y);
        }
      }
    } else {
      for (int i = 0; i < n; ++i)
        for (int e = 0; v + e < a.V; ++e) {
          const float y = value(load1<BF16>(a.in, in_row(i) + v + e), w[e], i, v + e);
          const bool allowed = !a.mask || mask_row(i)[(v + e) >> 3] >> ((v + e) & 7) & 1u;
          a.out[out_row(i) + v + e] = allowed ? y : kMasked;
        }
    }
  }
}

}  // namespace

const void* constrain_kernel(int bf16) {
  return bf16 ? (const void*)&constrain_impl<1> : (const void*)&constrain_impl<0>;
}

}  // namespace dspark
