// Log probabilities of given tokens, entropy and the best alternatives of rows of
// logits on gfx950 (draft_branch_logprobs).
//
// One pass over a row: a lane keeps the running maximum m of its elements, l =
// sum e^(z - m) and s = sum e^(z - m) (z - m), from which lse = f m + ln l and the
// entropy ln l - s / l (both terms at least 0, so a peaked row's small entropy
// does not drown in lse).  The best alternatives cost the pass nothing: the k-th
// largest of the lanes' maxima is a bound that at least k elements reach, and only
// lanes whose maximum reaches it can hold one of the best k, so after the pass the
// elements of those few lanes are read once more.
#include <algorithm>
#include <cmath>

#include "../../include/draftbranch.h"
#include "layer.h"

namespace {

using namespace dl;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTop = DB_MAX_TOP;
constexpr int kRoom = 1024;                 // candidates that LDS holds, and entries of a row's parts
constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kLowest = -3.4028234663852886e38f;   // m before the first element: finite, so no inf - inf arises
constexpr float kLeast = -200.0f;           // exponents below give a weight of 0 anyway; keeps 0 * inf out of s

struct LogprobArgs {
  const void* x;
  int64_t ld;
  int M, N;
  float scale;
  const float* scales;
  const int32_t* tokens;
  int n_tok, top;
  float *logprob, *lse, *entropy;
  int32_t* top_id;
  float* top_logprob;
  int parts;            // of a row
  float* part;          // [M][parts][4]: m, l, s of a part
  uint64_t* part_top;   // [M][parts][top] keys, best first
};

// m, l and s; exponents are those of 2, c = f log2(e).
struct Sum {
  float m, l, s;
};
__device__ __forceinline__ Sum joined(const Sum& a, const Sum& b, float c) {
  const float m = fmaxf(a.m, b.m), ta = fmaxf((a.m - m) * c, kLeast), tb = fmaxf((b.m - m) * c, kLeast);
  const float wa = __builtin_amdgcn_exp2f(ta), wb = __builtin_amdgcn_exp2f(tb);
  return {m, a.l * wa + b.l * wb, (a.s + a.l * ta) * wa + (b.s + b.l * tb) * wb};
}

// A key orders elements by value, then by the lower index; 0 is below every element's
// (-inf, which no key is made of, would be the lowest).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o); }
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  x = x == 0.0f ? 0.0f : x;   // -0 is 0
  return (uint64_t)ordered(x) << 32 | (uint32_t)~index;
}

// A row's elements in vectors of 16 bytes as memory is aligned: vector v holds
// elements v * kPer - shift .. + kPer - 1, the first and last perhaps in part.
template <class T>
struct RowOf {
  static constexpr int kPer = 16 / sizeof(T);
  const T* x;
  int n, shift, vectors;
  __device__ __forceinline__ RowOf(const LogprobArgs& A, int m) {
    x = static_cast<const T*>(A.x) + (int64_t)m * A.ld;
    n = A.N;
    shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    vectors = (n + shift + kPer - 1) / kPer;
  }
  static __device__ __forceinline__ float number(T t);
  __device__ __forceinline__ float at(int i) const { return number(x[i]); }
  // the elements of vector v; -inf in the places of those that are not the row's
  __device__ __forceinline__ void load(int v, float (&e)[kPer]) const {
    const int i0 = v * kPer - shift;
    if (i0 >= 0 && i0 + kPer <= n) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(x + i0);
      expand(w, e);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) e[k] = i0 + k >= 0 && i0 + k < n ? at(i0 + k) : -INFINITY;
    }
  }
  static __device__ __forceinline__ void expand(u32x4 w, float (&e)[kPer]);
};
template <>
__device__ __forceinline__ float RowOf<float>::number(float t) { return t; }
template <>
__device__ __forceinline__ float RowOf<uint16_t>::number(uint16_t t) { return __uint_as_float((uint32_t)t << 16); }
template <>
__device__ __forceinline__ void RowOf<float>::expand(u32x4 w, float (&e)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ void RowOf<uint16_t>::expand(u32x4 w, float (&e)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) e[2 * i] = bf16_lo(w[i]), e[2 * i + 1] = bf16_hi(w[i]);
}

// The `top` largest of n keys in LDS, best first, to out[0 .. top - 1] (0 past the
// last): a key's place is the number of larger ones.
__device__ __forceinline__ void sort_keys(const uint64_t* keys, int n, int top, uint64_t* out) {
  for (int i = threadIdx.x; i < top; i += kThreads) out[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t mine = keys[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += keys[j] > mine;
    if (place < top) out[place] = mine;
  }
  __syncthreads();
}

struct Shared {
  Sum sums[kWaves];
  uint64_t bests[kThreads];      // a lane's largest element's key
  uint64_t keys[kRoom];
  uint64_t out[kTop];
  uint16_t lanes[kThreads];      // those that may hold one of the best
  int n_lanes, n_keys;
  uint64_t most;
};

__device__ __forceinline__ float factor_of(const LogprobArgs& A, int m) { return A.scales ? A.scale * A.scales[m] : A.scale; }

// The row's results, from its sum and its best keys (in LDS).
template <class T>
__device__ __forceinline__ void finish(const LogprobArgs& A, int m, const RowOf<T>& row, Sum t, float f, const uint64_t* best) {
  const int tid = threadIdx.x;
  const bool bad = !(f > 0.0f && f < INFINITY) || t.l != t.l, none = t.l == 0.0f;
  const float nan = __builtin_nanf(""), log_l = logf(t.l);
  auto logprob = [&](float x) { return bad ? nan : none ? -INFINITY : (x - t.m) * f - log_l; };
  if (tid == 0) {
    A.lse[m] = bad ? nan : none ? -INFINITY : f * t.m + log_l;
    A.entropy[m] = bad ? nan : none ? 0.0f : log_l - kLn2 * t.s / t.l;
  }
  for (int i = tid; i < A.n_tok; i += kThreads) {
    const int token = A.tokens[(size_t)m * A.n_tok + i];
    const bool here = (unsigned)token < (unsigned)A.N;
    A.logprob[(size_t)m * A.n_tok + i] = bad ? nan : here ? logprob(row.at(here ? token : 0)) : -INFINITY;
  }
  for (int i = tid; i < A.top; i += kThreads) {
    const uint64_t k = best[i];
    A.top_id[(size_t)m * A.top + i] = bad || k == 0 ? -1 : (int)~(uint32_t)k;
    A.top_logprob[(size_t)m * A.top + i] = bad ? nan : k == 0 ? -INFINITY : logprob(value_of((uint32_t)(k >> 32)));
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs A) {
  __shared__ Shared lds;
  constexpr int kPer = RowOf<T>::kPer;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m = blockIdx.x / A.parts, part = blockIdx.x % A.parts;
  const RowOf<T> row(A, m);
  const float f = factor_of(A, m), c = f * kLog2e;
  const int v0 = (int)((int64_t)row.vectors * part / A.parts), v1 = (int)((int64_t)row.vectors * (part + 1) / A.parts);
  Sum t{kLowest, 0.0f, 0.0f};
  int best_at = -1;        // vector of the lane's largest element
  for (int v = v0 + tid; v < v1; v += kThreads) {
    float e[kPer];
    row.load(v, e);
    float most = e[0];
#pragma unroll
    for (int k = 1; k < kPer; ++k) most = fmaxf(most, e[k]);
    if (most > t.m || (best_at < 0 && most > -INFINITY)) {
      const float d = fmaxf((t.m - most) * c, kLeast), w = __builtin_amdgcn_exp2f(d);
      t.s = (t.s + t.l * d) * w;
      t.l *= w;
      t.m = most;
      best_at = v;
    }
    float l = 0.0f, s = 0.0f;   // the vector's own first: eight times fewer roundings at the size of the whole sum
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float d = (e[k] - t.m) * c, w = __builtin_amdgcn_exp2f(d);
      l += w;
      s = fmaf(w, fmaxf(d, kLeast), s);
    }
    t.l += l;
    t.s += s;
  }
  // the workgroup's sum, in the lanes' and waves' order
  Sum all = t;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const Sum other{__shfl_xor(all.m, by), __shfl_xor(all.l, by), __shfl_xor(all.s, by)};
    all = joined(all, other, c);
  }
  if (lane == 0) lds.sums[wave] = all;
  if (tid == 0) lds.n_lanes = lds.n_keys = 0;
  if (A.top > 0) {
    uint64_t key = 0;
    if (best_at >= 0) {
      float e[kPer];
      row.load(best_at, e);
#pragma unroll
      for (int k = kPer - 1; k >= 0; --k)
        if (e[k] == t.m) key = key_of(e[k], best_at * kPer - row.shift + k);
    }
    lds.bests[tid] = key;
  }
  __syncthreads();
  all = lds.sums[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) all = joined(all, lds.sums[w], c);
  if (A.top > 0) {
    // lanes whose largest is among the `top` largest of the lanes'; the last of them is the bound
    const uint64_t mine = lds.bests[tid];
    int place = 0;
    for (int i = 0; i < kThreads; ++i) place += lds.bests[i] > mine;
    if (mine != 0 && place < A.top) lds.lanes[atomicAdd(&lds.n_lanes, 1)] = (uint16_t)tid;
    if (tid == 0) lds.most = 1;      // fewer lanes than `top` hold an element: every one's elements above -inf
    __syncthreads();
    if (mine != 0 && place == A.top - 1) lds.most = mine;
    __syncthreads();
    const uint64_t bound = lds.most;
    const int lanes = lds.n_lanes, per_lane = (v1 - v0 + kThreads - 1) / kThreads;
    auto each = [&](auto&& take) {      // the keys of those lanes' elements that reach the bound
      for (int i = tid; i < lanes * per_lane; i += kThreads) {
        const int v = v0 + lds.lanes[i % lanes] + i / lanes * kThreads;
        if (v >= v1) continue;
        float e[kPer];
        row.load(v, e);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const uint64_t key = key_of(e[k], v * kPer - row.shift + k);
          if (e[k] > -INFINITY && key >= bound) take(key);
        }
      }
    };
    each([&](uint64_t key) {
      const int at = atomicAdd(&lds.n_keys, 1);
      if (at < kRoom) lds.keys[at] = key;
    });
    __syncthreads();
    if (lds.n_keys <= kRoom) {
      sort_keys(lds.keys, lds.n_keys, A.top, lds.out);
    } else {
      // more than there is room for: the largest below the one before, again and again
      uint64_t last = ~(uint64_t)0;
      for (int i = 0; i < A.top; ++i) {
        uint64_t most = 0;
        each([&](uint64_t key) { most = key < last && key > most ? key : most; });
#pragma unroll
        for (int by = 1; by < 64; by *= 2) {
          const uint64_t other = __shfl_xor((unsigned long long)most, by);
          most = other > most ? other : most;
        }
        if (lane == 0) lds.bests[wave] = most;
        __syncthreads();
        most = lds.bests[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) most = lds.bests[w] > most ? lds.bests[w] : most;
        if (tid == 0) lds.out[i] = most;
        last = most;
        __syncthreads();
      }
    }
  }
  if (A.parts == 1) {
    finish(A, m, row, all, f, lds.out);
    return;
  }
  const size_t at = (size_t)m * A.parts + part;
  if (tid == 0) {
    A.part[at * 4] = all.m;
    A.part[at * 4 + 1] = all.l;
    A.part[at * 4 + 2] = all.s;
  }
  for (int i = tid; i < A.top; i += kThreads) A.part_top[at * A.top + i] = lds.out[i];
}

// A row from its parts.
template <class T>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(LogprobArgs A) {
  __shared__ uint64_t keys[kRoom], out[kTop];
  __shared__ Sum sums[kThreads];
  const int tid = threadIdx.x, m = blockIdx.x;
  const RowOf<T> row(A, m);
  const float f = factor_of(A, m), c = f * kLog2e;
  const int entries = A.parts * A.top;
  for (int i = tid; i < entries; i += kThreads) keys[i] = A.part_top[(size_t)m * entries + i];
  if (tid < A.parts) {
    const float* p = A.part + ((size_t)m * A.parts + tid) * 4;
    sums[tid] = Sum{p[0], p[1], p[2]};
  }
  __syncthreads();
  Sum all = sums[0];
  for (int i = 1; i < A.parts; ++i) all = joined(all, sums[i], c);
  if (A.top > 0) sort_keys(keys, entries, A.top, out);
  finish(A, m, row, all, f, out);
}

// Parts of a row: enough for `kFill` workgroups in all, of 2,048 elements at
// least, and no more than the join has room for.
constexpr int kFill = 1024, kLeastPart = 2048;
int parts_of(int M, int N, int top) {
  const int most = std::min(kThreads, top > 0 ? kRoom / top : kThreads);
  return std::max(1, std::min({most, (kFill + M - 1) / std::max(M, 1), N / kLeastPart}));
}
size_t part_bytes(int M, int parts, int top) {
  return parts == 1 ? 0 : (size_t)M * parts * (16 + 8 * (size_t)top);
}

int check_logits(const char* who, int M, int N, int top) {
  if (M < 0 || M > DL_MAX_ROWS) return dh::fail(DH_ESHAPE, "%s: M must be in 0..%d (got %d)", who, DL_MAX_ROWS, M);
  if (N < 1 || N > DB_MAX_VOCAB) return dh::fail(DH_ESHAPE, "%s: N must be in 1..%d (got %d)", who, DB_MAX_VOCAB, N);
  if (top < 0 || top > DB_MAX_TOP) return dh::fail(DH_EUNSUP, "%s: top must be in 0..%d (got %d)", who, DB_MAX_TOP, top);
  return DH_OK;
}

template <class T>
void launch(const LogprobArgs& A, hipStream_t s) {
  hipLaunchKernelGGL(logprobs_kernel<T>, dim3((unsigned)A.M * A.parts), dim3(kThreads), 0, s, A);
  if (A.parts > 1) hipLaunchKernelGGL(logprobs_join_kernel<T>, dim3(A.M), dim3(kThreads), 0, s, A);
}

}  // namespace

extern "C" {

int draft_branch_logprobs_workspace_bytes(int M, int N, int top, size_t* bytes) {
  if (!bytes) return dh::fail(DH_EINVAL, "logprobs_workspace_bytes: null pointer");
  const int rc = check_logits("logprobs_workspace_bytes", M, N, top);
  if (rc) return rc;
  // fewer rows, logits or alternatives may make more parts, but rows * parts stays below 2 kFill
  // and an alternative more takes 8 bytes of each
  *bytes = M == 0 ? 0 : (size_t)2 * kFill * (16 + 8 * (size_t)top);
  return dh::ok();
}

int draft_branch_logprobs(const void* logits, int type, int64_t ld, int M, int N, float scale, const float* scales,
                          const int32_t* tokens, int n_tok, int top, float* logprob, float* lse, float* entropy,
                          int32_t* top_id, float* top_logprob, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "logprobs";
  const int rc = check_logits(who, M, N, top);
  if (rc) return rc;
  if (type != DB_BF16 && type != DB_FP32) return dh::fail(DH_EUNSUP, "logprobs: type must be DB_BF16 or DB_FP32 (got %d)", type);
  if (n_tok < 0 || n_tok > DB_MAX_TOKENS) return dh::fail(DH_EUNSUP, "logprobs: n_tok must be in 0..%d (got %d)", DB_MAX_TOKENS, n_tok);
  if (ld < N) return dh::fail(DH_EINVAL, "logprobs: the row stride is %lld, below its %d logits", (long long)ld, N);
  if (!(scale > 0.0f) || !std::isfinite(scale)) return dh::fail(DH_EINVAL, "logprobs: scale must be finite and > 0");
  if (M == 0) return dh::ok();
  if (!logits || !lse || !entropy || (n_tok > 0 && (!tokens || !logprob)) || (top > 0 && (!top_id || !top_logprob)))
    return dh::fail(DH_EINVAL, "logprobs: null pointer");
  if (!aligned(logits, type == DB_BF16 ? 2 : 4) || !aligned(scales, 4) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(top_id, 4) || !aligned(top_logprob, 4))
    return dh::fail(DH_EINVAL, "logprobs: tensors must be aligned to their elements");
  LogprobArgs A{logits, ld, M, N, scale, scales, tokens, n_tok, top, logprob, lse, entropy, top_id, top_logprob, parts_of(M, N, top), nullptr, nullptr};
  const size_t need = part_bytes(M, A.parts, top);
  if (need > 0) {
    if (!workspace || !aligned(workspace, 16)) return dh::fail(DH_EINVAL, "logprobs: workspace must be a 16-byte aligned pointer");
    if (workspace_bytes < need)
      return dh::fail(DH_EINVAL, "logprobs: workspace of %zu bytes is below the %zu needed", workspace_bytes, need);
    A.part = static_cast<float*>(workspace);
    A.part_top = reinterpret_cast<uint64_t*>(static_cast<unsigned char*>(workspace) + (size_t)M * A.parts * 16);
  }
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (type == DB_BF16)
    launch<uint16_t>(A, st);
  else
    launch<float>(A, st);
  return launched("logprobs_kernel");
}

}  // extern "C"
