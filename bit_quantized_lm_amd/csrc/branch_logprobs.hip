// Log probabilities of given tokens, entropy and the best alternatives of rows of
// logits on gfx950 (draft_branch_logprobs).
//
// One pass over a row: a lane keeps the running maximum m of its elements, l =
// sum e^(z - m) and s = sum e^(z - m) (z - m), from which lse = f m + ln l and the
// entropy ln l - s / l (both terms at least 0, so a peaked row's small entropy
// does not drown in lse).  The best alternatives cost the pass little: the k-th
// largest of the lanes' maxima is a bound that at least k elements reach, so after
// the first steps only elements that reach theirs are put down, and the few that
// reach the bound of all steps are put in order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/draftbranch.h"
#include "layer.h"

namespace {

using namespace dl;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTop = DB_MAX_TOP;
constexpr int kRoom = 1024;                 // keys that LDS holds, and entries of a row's parts
constexpr int kList = 512;                  // vectors put down
constexpr int kAtOnce = 2;                  // vectors of a lane a step; the next step's are on their way
constexpr int kFirstSteps = 4, kMoreSteps = 16;   // before the first bound, and before a closer one
constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;
constexpr float kLowest = -3.4028234663852886e38f;   // m of nothing: finite, so no inf - inf arises
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

// A row: `head` elements up to the first 16-byte boundary, `vectors` of 16 bytes, and
// `tail` elements behind them.
template <class T>
struct RowOf {
  static constexpr int kPer = 16 / sizeof(T);
  const T* x;
  int n, head, vectors, tail;
  __device__ __forceinline__ RowOf(const LogprobArgs& A, int m) {
    x = static_cast<const T*>(A.x) + (int64_t)m * A.ld;
    n = A.N;
    head = min((int)((0 - reinterpret_cast<uintptr_t>(x)) & 15) / (int)sizeof(T), n);
    vectors = (n - head) / kPer;
    tail = n - head - vectors * kPer;
  }
  static __device__ __forceinline__ float number(T t);
  static __device__ __forceinline__ u32x4 nothing();   // -inf throughout
  static __device__ __forceinline__ void expand(u32x4 w, float (&e)[kPer]);
  static __device__ __forceinline__ u32x4 packed(const float (&e)[kPer]);   // expand's input again
  __device__ __forceinline__ float at(int i) const { return number(x[i]); }
  __device__ __forceinline__ const u32x4* at_vector(int v) const { return reinterpret_cast<const u32x4*>(x + head) + v; }
  __device__ __forceinline__ u32x4 raw(int v) const { return *at_vector(v); }
  __device__ __forceinline__ int index(int v, int k) const { return head + v * kPer + k; }
  // the elements beside the vectors: edge i of head + tail
  __device__ __forceinline__ int edge(int i) const { return i < head ? i : n - tail + i - head; }
};
template <>
__device__ __forceinline__ float RowOf<float>::number(float t) { return t; }
template <>
__device__ __forceinline__ float RowOf<uint16_t>::number(uint16_t t) { return __uint_as_float((uint32_t)t << 16); }
template <>
__device__ __forceinline__ u32x4 RowOf<float>::nothing() { return u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}; }
template <>
__device__ __forceinline__ u32x4 RowOf<uint16_t>::nothing() { return u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
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

template <>
__device__ __forceinline__ u32x4 RowOf<float>::packed(const float (&e)[4]) {
  return u32x4{__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3])};
}
template <>
__device__ __forceinline__ u32x4 RowOf<uint16_t>::packed(const float (&e)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(e[2 * i]) >> 16 | (__float_as_uint(e[2 * i + 1]) & 0xFFFF0000u);
  return w;
}

// One instruction each; fmaxf and fminf first make their arguments canonical.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// A bound that at least k of n numbers reach and hardly more, by one wave: the k-th
// largest, found bit by bit, or the prefix of it that exactly k reach; 0 where only
// k of all would do.  at(i): number i, n at most 64 K.
template <int K, class At>
__device__ __forceinline__ uint32_t bound_of(int n, int k, const At at) {
  const int lane = threadIdx.x & 63;
  uint32_t x[K], bound = 0;
#pragma unroll
  for (int j = 0; j < K; ++j) x[j] = j * 64 + lane < n ? at(j * 64 + lane) : 0u;
  int some = 0;
#pragma unroll
  for (int j = 0; j < K; ++j) some += (int)__popcll(__ballot(x[j] > 0u));
  if (some <= k) return 0u;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = bound | 1u << bit;
    int count = 0;
#pragma unroll
    for (int j = 0; j < K; ++j) count += (int)__popcll(__ballot(x[j] >= trial));
    if (count >= k) bound = trial;
    if (count == k) break;
  }
  return bound;
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
  u32x4 raw[kList];              // vectors with an element that reached the bound of their step
  int at[kList];                 // and which they are; ~i: element i, in the first place
  uint64_t kept[kRoom];          // keys of their elements that reach the last one
  uint64_t out[kTop];
  uint32_t most[kThreads];       // a lane's largest element, 0: none
  uint32_t bound;
  int n_list, n_kept;
};

// A lane's sums while it passes over the row, under the largest element so far: its
// weight is 1 exactly, which a peaked row's small results need.
struct Running {
  float most = -INFINITY, at = kLowest, l = 0.0f, s = 0.0f;   // at: most, finite
  __device__ __forceinline__ void see(float x, float c) {   // the largest element of a step
    if (!(x > most)) return;
    const float d = fmaxf((at - x) * c, kLeast), w = __builtin_amdgcn_exp2f(d);
    s = (s + l * d) * w;
    l *= w;
    most = at = x;
  }
  __device__ __forceinline__ void add(float x, float c) {
    const float d = (x - at) * c, w = __builtin_amdgcn_exp2f(d);
    l += w;
    s = fmaf(w, fmaxf(d, kLeast), s);
  }
  __device__ __forceinline__ Sum sum() const { return {at, l, s}; }
};

__device__ __forceinline__ float factor_of(const LogprobArgs& A, int m) { return A.scales ? A.scale * A.scales[m] : A.scale; }

// The row's results, from its sum and its best keys (in LDS).
template <class T>
__device__ __forceinline__ void finish(const LogprobArgs& A, int m, const RowOf<T>& row, Sum t, float f, const uint64_t* best) {
  const int tid = threadIdx.x;
  // the exponents' factor has to be a number too, of rows without an element as of others
  const bool bad = !(f > 0.0f && f * kLog2e < INFINITY) || t.l != t.l, none = t.l == 0.0f;
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

// The row's best where more elements reach the bound than LDS holds (many equal
// ones): the largest below the one before, again and again.
template <class T>
__device__ __forceinline__ void pick_one_by_one(const RowOf<T>& row, int v0, int v1, int edges, int top, Shared& lds) {
  constexpr int kPer = RowOf<T>::kPer;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint64_t last = ~(uint64_t)0;
  for (int i = 0; i < top; ++i) {
    uint64_t most = 0;
    auto look = [&](float x, int index) {
      const uint64_t key = key_of(x, index);
      if (x > -INFINITY && key < last && key > most) most = key;
    };
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float e[kPer];
      RowOf<T>::expand(row.raw(v), e);
#pragma unroll
      for (int k = 0; k < kPer; ++k) look(e[k], row.index(v, k));
    }
    if (tid < edges) look(row.at(row.edge(tid)), row.edge(tid));
#pragma unroll
    for (int by = 1; by < 64; by *= 2) {
      const uint64_t other = __shfl_xor((unsigned long long)most, by);
      most = other > most ? other : most;
    }
    if (lane == 0) lds.kept[wave] = most;
    __syncthreads();
    most = lds.kept[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) most = lds.kept[w] > most ? lds.kept[w] : most;
    if (tid == 0) lds.out[i] = most;
    last = most;
    __syncthreads();
  }
}

// The workgroup's sum, in the lanes' and waves' order, in every thread.
__device__ __forceinline__ Sum sum_of_all(Sum t, float c, Sum (&of_wave)[kWaves]) {
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const Sum other{__shfl_xor(t.m, by), __shfl_xor(t.l, by), __shfl_xor(t.s, by)};
    t = joined(t, other, c);
  }
  if ((threadIdx.x & 63) == 0) of_wave[threadIdx.x >> 6] = t;
  __syncthreads();
  t = of_wave[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) t = joined(t, of_wave[w], c);
  return t;
}

// kOnce: rows of many steps, whose loads go past the caches (2,048 rows of 124,160: 102 us
// so, 107 through them); a row's parts are looked at again.
template <class T, bool kOnce>
__global__ __launch_bounds__(kThreads, 8) void logprobs_kernel(LogprobArgs A) {
  __shared__ Shared lds;
  constexpr int kPer = RowOf<T>::kPer, kStep = kAtOnce * kThreads;
  const int tid = threadIdx.x, wave = tid >> 6;
  const int m = blockIdx.x / A.parts, part = blockIdx.x % A.parts;
  const RowOf<T> row(A, m);
  const float f = factor_of(A, m), c = f * kLog2e;
  const int v0 = (int)((int64_t)row.vectors * part / A.parts), v1 = (int)((int64_t)row.vectors * (part + 1) / A.parts);
  const int edges = part == 0 ? row.head + row.tail : 0;   // a lane's each
  if (tid == 0) lds.n_list = lds.n_kept = 0;
  u32x4 next[kAtOnce];
  auto load = [&](int v) { return kOnce ? __builtin_nontemporal_load(row.at_vector(v)) : *row.at_vector(v); };
  auto fetch = [&](int base) {
    if (base + kStep <= v1) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) next[u] = load(base + tid + u * kThreads);
    } else {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        next[u] = RowOf<T>::nothing();
        if (base + tid + u * kThreads < v1) next[u] = load(base + tid + u * kThreads);
      }
    }
  };
  fetch(v0);
  const float edge = tid < edges ? row.at(row.edge(tid)) : -INFINITY;
  Running t;
  // reached by nothing, +inf neither: before the first bound nothing is put down, and the
  // counters' zeros are only there from the first barrier on, which that bound comes behind
  float bound = __builtin_nanf("");
  auto put_down = [&](int v, const float (&e)[kPer]) {
    const int at = atomicAdd(&lds.n_list, 1);
    if (at < kList) lds.raw[at] = RowOf<T>::packed(e), lds.at[at] = v;
  };
  auto most_of = [](const float (&e)[kPer]) {
    float most = max3(e[0], e[1], e[2]);
#pragma unroll
    for (int k = 3; k + 1 < kPer; k += 2) most = max3(most, e[k], e[k + 1]);
    return max3(most, most, e[kPer - 1]);
  };
  // the bound of the lanes' maxima so far, and (again) what reaches it of the vectors before v
  auto raise = [&](bool again, int v) {
    lds.most[tid] = t.most > -INFINITY ? ordered(t.most == 0.0f ? 0.0f : t.most) : 0u;   // -0 is 0
    __syncthreads();
    if (wave == 0) {
      const uint32_t b = bound_of<kThreads / 64>(kThreads, A.top, [&](int i) { return lds.most[i]; });
      if (tid == 0) lds.bound = b;
    }
    __syncthreads();
    bound = value_of(lds.bound);
    if (!(bound >= kLowest)) bound = kLowest;   // none, or a prefix that is no number: every element above -inf
    if (!again || !(t.most >= bound)) return;
    auto look = [&](int u, u32x4 raw) {
      float e[kPer];
      RowOf<T>::expand(raw, e);
      if (most_of(e) >= bound) put_down(u, e);
    };
    if (edge >= bound) {
      float e[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) e[k] = k == 0 ? edge : -INFINITY;
      put_down(~row.edge(tid), e);
    }
    for (int u0 = v0 + tid; u0 < v; u0 += 4 * kThreads) {
      u32x4 raw[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) raw[u] = row.raw(min(u0 + u * kThreads, v - 1));
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (u0 + u * kThreads < v) look(u0 + u * kThreads, raw[u]);
    }
  };
  t.see(edge, c);
  if (tid < edges) t.add(edge, c);
  int step = 0;
  for (int base = v0; base < v1; base += kStep, ++step) {
    if ((step == kFirstSteps || step == kMoreSteps) && A.top > 0) raise(step == kFirstSteps, base);
    float e[kAtOnce][kPer], most[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) RowOf<T>::expand(next[u], e[u]);
    fetch(base + kStep);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) most[u] = most_of(e[u]);
    float top = most[0], low = e[0][0];
#pragma unroll
    for (int u = 1; u < kAtOnce; ++u) top = fmaxf(top, most[u]);
#pragma unroll
    for (int i = 1; i + 1 < kAtOnce * kPer; i += 2) low = min3(low, e[i / kPer][i % kPer], e[(i + 1) / kPer][(i + 1) % kPer]);
    low = min3(low, low, e[kAtOnce - 1][kPer - 1]);
    t.see(top, c);
    if (top >= bound) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (most[u] >= bound) put_down(base + tid + u * kThreads, e[u]);
    }
    auto add = [&](auto clean) {   // clean: every exponent is finite, and 0 times it 0
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        float l = 0.0f, s = 0.0f;   // the vector's own first: eight times fewer roundings at the size of the whole sum
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const float d = (e[u][k] - t.at) * c, w = __builtin_amdgcn_exp2f(d);
          l += w;
          s = fmaf(w, decltype(clean)::value ? d : fmaxf(d, kLeast), s);
        }
        t.l += l;
        t.s += s;
      }
    };
    if (__all((low - t.at) * c > kLowest))
      add(std::true_type{});
    else
      add(std::false_type{});
  }
  if (A.top > 0) {
    raise(step <= kFirstSteps, v1);   // after more steps, what reaches this bound has reached the first and is put down
    __syncthreads();
    if (lds.n_list > kList && step > kFirstSteps) {   // far more reached the first
      __syncthreads();
      if (tid == 0) lds.n_list = 0;
      raise(true, v1);
      __syncthreads();
    }
    const int listed = lds.n_list;
    for (int i = tid; i < min(listed, kList) * kPer; i += kThreads) {
      float e[kPer];
      RowOf<T>::expand(lds.raw[i / kPer], e);
      float x = e[0];
#pragma unroll
      for (int k = 1; k < kPer; ++k) x = i % kPer == k ? e[k] : x;
      if (x >= bound) {
        const int at = atomicAdd(&lds.n_kept, 1);
        const int v = lds.at[i / kPer];
        if (at < kRoom) lds.kept[at] = key_of(x, v < 0 ? ~v : row.index(v, i % kPer));
      }
    }
    __syncthreads();
    if (listed <= kList && lds.n_kept <= kRoom)
      sort_keys(lds.kept, lds.n_kept, A.top, lds.out);
    else
      pick_one_by_one(row, v0, v1, edges, A.top, lds);
  }
  const Sum all = sum_of_all(t.sum(), c, lds.sums);
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
  __shared__ uint64_t keys[kRoom], kept[kRoom], out[kTop];
  __shared__ Sum sums[kWaves];
  __shared__ uint32_t bound;
  __shared__ int n_kept;
  const int tid = threadIdx.x, m = blockIdx.x;
  const RowOf<T> row(A, m);
  const float f = factor_of(A, m), c = f * kLog2e;
  const int entries = A.parts * A.top;
  Sum t{kLowest, 0.0f, 0.0f};
  if (tid < A.parts) {
    const float* p = A.part + ((size_t)m * A.parts + tid) * 4;
    t = Sum{p[0], p[1], p[2]};
  }
  for (int i = tid; i < entries; i += kThreads) keys[i] = A.part_top[(size_t)m * entries + i];
  if (tid == 0) n_kept = 0;
  const Sum all = sum_of_all(t, c, sums);   // its barrier is the keys' too
  if (A.top > 0) {
    if (tid < 64) {
      // of the parts' first ones, if they are as many as are asked for: what reaches it is in few parts
      const uint32_t b = A.parts >= A.top ? bound_of<kThreads / 64>(A.parts, A.top, [&](int i) { return (uint32_t)(keys[i * A.top] >> 32); })
                                          : bound_of<kRoom / 64>(entries, A.top, [&](int i) { return (uint32_t)(keys[i] >> 32); });
      if (tid == 0) bound = b;
    }
    __syncthreads();
    for (int i = tid; i < entries; i += kThreads)
      if (keys[i] != 0 && (uint32_t)(keys[i] >> 32) >= bound) kept[atomicAdd(&n_kept, 1)] = keys[i];
    __syncthreads();
    sort_keys(kept, n_kept, A.top, out);
  }
  finish(A, m, row, all, f, out);
}

// Parts of a row: a step each where that makes up to half of what the card runs at
// once, else four steps each and no more than the card runs, in either case no more
// than the join has room for.  Steps of 4,096 bf16 logits, alternatives 8: 8 rows of
// 32,000 12.1 us so and 19.5 in parts of four steps, 72 of 32,000 13.4 and 20.8; 72 of
// 124,160 22.3 in steps and 18.7 in fours, 128 of them 23.3 and 21.1, 600 of 32,000
// 30.6 and 29.0.
constexpr int kFill = 2048;
int parts_of(int M, int N, int top, int type) {
  const int most = std::min(kThreads, top > 0 ? kRoom / top : kThreads), per = type == DB_BF16 ? 8 : 4;
  const int steps = (N + kAtOnce * kThreads * per - 1) / (kAtOnce * kThreads * per);
  const bool few = (int64_t)M * steps <= kFill / 2;
  return std::max(1, std::min({most, kFill / std::max(M, 1), few ? steps : (steps + 3) / 4}));
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
  if (A.parts == 1) {
    hipLaunchKernelGGL((logprobs_kernel<T, true>), dim3((unsigned)A.M), dim3(kThreads), 0, s, A);
  } else {
    hipLaunchKernelGGL((logprobs_kernel<T, false>), dim3((unsigned)A.M * A.parts), dim3(kThreads), 0, s, A);
    hipLaunchKernelGGL(logprobs_join_kernel<T>, dim3(A.M), dim3(kThreads), 0, s, A);
  }
}

}  // namespace

extern "C" {

int draft_branch_logprobs_workspace_bytes(int M, int N, int top, size_t* bytes) {
  if (!bytes) return dh::fail(DH_EINVAL, "logprobs_workspace_bytes: null pointer");
  const int rc = check_logits("logprobs_workspace_bytes", M, N, top);
  if (rc) return rc;
  // fewer rows or alternatives may make more parts, but rows * parts stays up to kFill
  // and an alternative more takes 8 bytes of each
  *bytes = M == 0 ? 0 : (size_t)kFill * (16 + 8 * (size_t)top);
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
  LogprobArgs A{logits, ld, M, N, scale, scales, tokens, n_tok, top, logprob, lse, entropy, top_id, top_logprob, parts_of(M, N, top, type), nullptr, nullptr};
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
