// A tile of attention over the 8-bit cache: rows of queries against a range of a
// sequence's tokens, with the running reference and sum of the softmax.  Used by
// every kernel that attends (not part of the public ABI).
#pragma once

#include "layer.h"

namespace dl {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------- tokens
struct Range {   // groups of 32 tokens a tile sees: `ns` groups from s0 on, then g0 .. g0 + n - ns - 1
  int s0, ns, g0, n;
};

// The tokens of one sequence that a tile's rows see, and where they are: the row
// at position p those at j <= p, of these only j > p - window and j < sinks where
// window > 0.  kSplit: of two sequences' table rows, the positions below `split` (the
// groups `shared` counts, which come first) from row `lead`, the others from row
// `seq`; a group that holds positions of both comes twice.
template <bool kSplit>
struct Tokens {
  const Batch& b;
  const Cache& c;
  int seq, head;
  Range see;
  int window, sinks;
  Range shared = {};
  int lead = 0, split = 0;

  static __device__ __forceinline__ int at(const Range& r, int n) { return n < r.ns ? n + r.s0 : n - r.ns + r.g0; }
  __device__ __forceinline__ bool before(int n) const { return kSplit && n < shared.n; }   // among the shared groups
  __device__ __forceinline__ int group_at(int n) const { return before(n) ? at(shared, n) : at(see, kSplit ? n - shared.n : n); }
  __device__ __forceinline__ int row_at(int n) const { return before(n) ? lead : seq; }
  __device__ __forceinline__ int lo_at(int n) const { return kSplit && !before(n) ? split : 0; }
  __device__ __forceinline__ int hi_at(int n) const { return before(n) ? split : INT32_MAX; }
  // whether some row at p_first .. p_last does not see some of the tokens of group n, first .. first + 31
  __device__ __forceinline__ bool hides(int n, int first, int p_first, int p_last) const {
    return first + 31 > p_first || (window > 0 && first <= p_last - window && first + 31 >= sinks) ||
           (kSplit && (first < lo_at(n) || first + 31 >= hi_at(n)));
  }
};

// --------------------------------------------------------------- conversions
// Code bytes (value + 128) as fp16: 0x6400 | u is 1024 + u, and subtracting
// 1152 leaves the signed code exactly.
__device__ __forceinline__ u32x2 codes_to_half4(uint32_t a) {
  const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) - off),
               __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) - off)};
}
__device__ __forceinline__ half8 codes_to_half(uint32_t a, uint32_t b) {
  const u32x2 x = codes_to_half4(a), y = codes_to_half4(b);
  return __builtin_bit_cast(half8, u32x4{x[0], x[1], y[0], y[1]});
}

__device__ __forceinline__ f32x4 mfma(half8 a, half8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A lane's 16 bytes of KiB `f` of the codes at `at` (one address for the wave).
constexpr int kOnce = 2;   // nt: read by this workgroup alone, not worth keeping
template <int kPolicy>
__device__ __forceinline__ u32x4 load_codes(const uint8_t* at, int f) {
  const __amdgpu_buffer_rsrc_t b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(at), 0, 0x7FFFFFFF, 0x00027000);
  return __builtin_amdgcn_raw_buffer_load_b128(b, (threadIdx.x & 63) * 16, f * 1024, kPolicy);
}

// A row's query fragments, lane (hi, lo) holding elements 64 f + 16 hi ..
// + 15 of the tile's row lo, as fp16 scaled by 2^-e so that the row's largest
// element is in [2^14, 2^15).  Returns scale_log2 * 2^e.  A zero row keeps 1;
// an infinite or NaN element makes its own row NaN and no other, through what is
// returned: infinite scores of one sign alone would be a row that sees nothing.
template <int D>
__device__ __forceinline__ float load_query(const uint16_t* __restrict__ row, bool valid, float scale_log2, half8 (&frag)[D / 32]) {
  const int hi = (threadIdx.x & 63) >> 4;
  u32x4 raw[D / 32];
  uint32_t top = 0;
#pragma unroll
  for (int f = 0; f < D / 32; ++f) {
    raw[f] = valid ? *reinterpret_cast<const u32x4*>(row + f / 2 * 64 + hi * 16 + (f & 1) * 8) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(raw[f][i] & 0x7FFFu, (raw[f][i] >> 16) & 0x7FFFu));
  }
  top = max(top, __shfl_xor(top, 16));
  top = max(top, __shfl_xor(top, 32));
  const int e = max((int)(top >> 7) - 127, -100) - 14;   // a row below 2^-100 stays below 2^14
  const float up = __builtin_ldexpf(1.0f, -e);
#pragma unroll
  for (int f = 0; f < D / 32; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      frag[f][2 * i] = (_Float16)(bf16_lo(raw[f][i]) * up);
      frag[f][2 * i + 1] = (_Float16)(bf16_hi(raw[f][i]) * up);
    }
  return top >= 0x7F80u ? __builtin_nanf("") : __builtin_ldexpf(scale_log2, e);
}

// Online softmax of one row: weights are 2^(x - m) with x = z log2(e) +
// log2(value scale), so that a weight times a value code is the value's whole
// share, whatever its page's scale, and m near the running maximum of x; l sums
// the weights over the value scales again.  m is set kHead below the maximum
// and stays until a weight passes 2^kFit, which a lane's sum of them tells: most
// steps then need neither a maximum nor a rescaling, weights fit fp16 (its
// largest is just under 2^16), and one keeps its 11 bits down to 2^-21 of the
// largest.
constexpr float kHead = 7.0f, kFit = 15.0f, kMost = 0x1p15f;
constexpr float kLowest = -0x1p127f;   // m before the first visible token; finite, so no inf - inf arises

// What the scores take of a page's two scales.  One that is not finite makes the
// key scale NaN, and with it the scores of the rows that see the page; a hidden
// token's weight is formed from the value scale's logarithm, which stays finite.
struct PageScales {
  float ks, lv, rv;   // key scale, log2(value scale), 1 / (value scale)
};
__device__ __forceinline__ PageScales page_scales(float ks, float vs) {
  const float nan_if_not_finite = (ks - ks) + (vs - vs), v = fminf(fmaxf(vs, kMinScale), 0x1p126f);
  return {ks + nan_if_not_finite, __builtin_amdgcn_logf(v), __builtin_amdgcn_rcpf(v)};
}

// What is common to a group's scores: where its tokens are and its scales.
struct Group {
  int id, first;       // page (-1: nothing there), position of token 0
  float ks, lv, rv;    // key scale, log2(value scale), 1 / (value scale)
  bool edge;           // some row does not see some of its tokens
  int lo, hi;          // only positions lo .. hi - 1 of it count (kSplit)
};

// A group's weights of all row tiles, from its scores x in code units.  In
// three steps, so that a caller can put other work between them: hidden scores
// to -inf; weights under the present references; and, where some weight may have
// passed 2^kFit, which the lanes' sums tell, the references and what was summed
// under them moved and the weights formed again.  One test for all tiles: tile by
// tile, each waits for the one before.
template <int N>
struct Weights {
  float c[N], p[N][8], sum[N];   // scale of x, weights, this lane's sum of them

  template <bool kSplit>
  __device__ __forceinline__ void hide(const Tokens<kSplit>& A, const Group& g, f32x4 (&x)[N][2], const float (&qs)[N], const int (&pos)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) c[t] = g.ks * qs[t];
    if (!g.edge) return;
    const int hi = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < N; ++t) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = g.first + hi * 4 + (j >> 2) * 16 + (j & 3);
        // & and |, not && and ||: selects, no branch a score
        const bool seen = (g.id >= 0) & (at <= pos[t]) & ((A.window == 0) | (at > pos[t] - A.window) | (at < A.sinks)) &
                          (!kSplit | ((at >= g.lo) & (at < g.hi)));
        x[t][j >> 2][j & 3] = seen ? x[t][j >> 2][j & 3] * c[t] : -INFINITY;
      }
      c[t] = 1.0f;
    }
  }

  // A score's exponent, rounded as a reference is. form() does not round the product:
  // a reference of 2^28 may be 16 off it, and a weight from such a difference is
  // anything from 0 to infinity.
  static __device__ __forceinline__ float rounded(float x, float c, float lv) {
#pragma clang fp contract(off)
    const float z = x * c;
    return z + lv;
  }

  // weights `from` .. `to` - 1 of the 8 N
  __device__ __forceinline__ void form(const Group& g, const f32x4 (&x)[N][2], const float (&m)[N], int from = 0, int to = 8 * N) {
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) {
      if (i < from || i >= to) continue;
      const int t = i / 8, j = i % 8;
      p[t][j] = __builtin_amdgcn_exp2f(fmaf(x[t][j >> 2][j & 3], c[t], g.lv - m[t]));
      sum[t] = j == 0 ? p[t][j] : sum[t] + p[t][j];
    }
  }

  template <int C>
  __device__ __forceinline__ void settle(const Group& g, const f32x4 (&x)[N][2], float (&m)[N], float (&l)[N], f32x4 (&o)[N][C], half8 (&w)[N]) {
    float most = sum[0];
#pragma unroll
    for (int t = 1; t < N; ++t) most = fmaxf(most, sum[t]);
    if (__any(most > kMost)) {
#pragma unroll
      for (int t = 0; t < N; ++t) {
        float top = x[t][0][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, x[t][j >> 2][j & 3]);
        top = rounded(top, c[t], g.lv);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // by each row's own maximum, whichever row asked: rows do not touch each other's bits
        const float next = top > m[t] + kFit ? top - kHead : m[t], down = __builtin_amdgcn_exp2f(m[t] - next);
        m[t] = next;
        l[t] *= down;
#pragma unroll
        for (int i = 0; i < C; ++i) o[t][i] *= down;
      }
#pragma unroll
      for (int t = 0; t < N; ++t) {
        sum[t] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[t] += p[t][j] = __builtin_amdgcn_exp2f(rounded(x[t][j >> 2][j & 3], c[t], g.lv - m[t]));
      }
    }
#pragma unroll
    for (int t = 0; t < N; ++t) {
      l[t] = fmaf(sum[t], g.rv, l[t]);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[t][j] = (_Float16)p[t][j];
    }
  }
};

// ------------------------------------------------------- few rows: streaming
// 16 rows against a stream of groups of 32 tokens.  Each wave takes every W-th
// group of its workgroup's part or run, straight from global memory into the
// fragments (each load instruction 1 KiB without gaps), a step ahead, so
// nothing is shared until the waves' results are joined.  S^T = K Q^T puts a
// row's weights into the lanes and order that the next product takes its columns
// in (O^T = V^T P^T), so they never leave their registers.
//
// Bound by memory: 64 slots over 0.95 GB of cache 157 us, 6.1 TB/s against 6.9 for
// a plain read of 1 GiB.  Loads marked as not worth keeping: 58 us instead of 66
// for one row over 131,072 tokens (268 MB), whose time is now 48 us, 37 of them
// reading (7.2 TB/s), the rest beginning, handing over and joining 31 parts.
template <int F>
struct Bytes {   // a lane's codes of one group
  u32x4 k[F], v[F];
};

// Rows 0 .. rows - 1 of a tile against the groups from .. to - 1 of what they see
// (positions p_first .. p_last), each of the W waves its own of them (W = 1: the wave
// is alone with the tile).  place(r, pos) gives row
// r's queries and position (-1 past the last row); finish(o, m, l) takes this wave's
// share, within the function, so that o never leaves its registers (handed back as
// an argument it spilled 19 of 256).
template <int D, int W, int kPolicy, bool kSplit, class Place, class Finish>
__device__ __forceinline__ void stream_tile(const Tokens<kSplit> A, int from, int to, int rows, int p_first, int p_last, float scale_log2,
                                            const Place place, const Finish finish) {
  constexpr int F = D / 32, C = D / 16;
  const int wave = W == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, lo = lane & 15;
  const size_t page_bytes = (size_t)D << A.c.page_shift;

  // lane i: page and scales of the wave's i-th group from `base`, 64 at a time
  int base = from + wave, id_mine;
  PageScales mine_scales;
  auto look = [&] {
    const int n = base + lane * W;
    id_mine = n < to ? page_id(A.b, A.c.n_pages, A.row_at(n), A.group_at(n) >> (A.c.page_shift - 5)) : -1;
    const size_t at = (size_t)max(id_mine, 0) * A.c.hkv + A.head;
    mine_scales = page_scales(A.c.ks[at], A.c.vs[at]);   // of one that is not there page 0's, which step() hides
  };
  auto load = [&](int i, Bytes<F>& b) {   // of a group that is not there page 0's bytes, which step() hides
    const size_t off = ((size_t)max(__builtin_amdgcn_readlane(id_mine, i), 0) * A.c.hkv + A.head) * page_bytes +
                       (size_t)(A.group_at(base + i * W) & ((1 << (A.c.page_shift - 5)) - 1)) * 32 * D;
#pragma unroll
    for (int f = 0; f < F; ++f) b.k[f] = load_codes<kPolicy>(A.c.k + off, f);
#pragma unroll
    for (int f = 0; f < F; ++f) b.v[f] = load_codes<kPolicy>(A.c.v + off, f);
  };
  // the first codes are on their way before the queries are looked at
  Bytes<F> even, odd;
  if (base < to) {
    look();
    load(0, even);
  }
  half8 qf[F], pf[1];
  float qs[1], m[1] = {kLowest}, l[1] = {0.0f};
  int pos[1];
  f32x4 o[1][C];
  {
    const uint16_t* row = place(lo, pos[0]);
    qs[0] = load_query<D>(row, lo < rows, scale_log2, qf);
#pragma unroll
    for (int c = 0; c < C; ++c) o[0][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  auto step = [&](int i, const Bytes<F>& b) {
    const int n = base + i * W, first = A.group_at(n) * 32, id = __builtin_amdgcn_readlane(id_mine, i);
    const Group group{id, first, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.ks), i)),
                      __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.lv), i)),
                      __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.rv), i)),
                      id < 0 || A.hides(n, first, p_first, p_last), A.lo_at(n), A.hi_at(n)};
    f32x4 s[1][2] = {{{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}}};
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int half = f / (D / 64), c = f % (D / 64);
      s[0][half] = mfma(codes_to_half(b.k[f][0], b.k[f][1]), qf[2 * c], s[0][half]);
      s[0][half] = mfma(codes_to_half(b.k[f][2], b.k[f][3]), qf[2 * c + 1], s[0][half]);
    }
    Weights<1> weights;
    weights.hide(A, group, s, qs, pos);
    weights.form(group, s, m);
    weights.settle(group, s, m, l, o, pf);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      o[0][2 * f] = mfma(codes_to_half(b.v[f][0], b.v[f][1]), pf[0], o[0][2 * f]);
      o[0][2 * f + 1] = mfma(codes_to_half(b.v[f][2], b.v[f][3]), pf[0], o[0][2 * f + 1]);
    }
  };
  while (base < to) {
    const int count = min(64, (to - base + W - 1) / W);
    for (int i = 0; i < count; i += 2) {
      if (i + 1 < count) load(i + 1, odd);
      step(i, even);
      if (i + 1 >= count) break;
      if (i + 2 < count) load(i + 2, even);
      step(i + 1, odd);
    }
    base += 64 * W;
    if (base < to) {
      look();
      load(0, even);
    }
  }
  finish(o, m, l);
}

// -------------------------------------------------------- many rows: shared
// R = 16 NQ W rows: each wave holds NQ tiles of 16 rows, and the workgroup's
// waves share the key and value fragments, converted to fp16 once, through LDS.
//
// A step works on one group of 32 tokens.  The matrix cores and the vector
// units run side by side only where one wave's instructions alternate between
// them (two waves a SIMD, each with its products and its exponentials in blocks,
// overlapped in a fifth of the matrix cycles), so a step forms the next group's
// scores between the exponentials of its own, and sums its own values between the
// conversions of the codes to come.  Bundle n is what step n needs from LDS: the
// keys of group n + 1 and the values of group n.  Bundles alternate between two
// places: while one is read, the next one's codes are converted into the other and
// the one after that is on its way from memory in registers; one barrier a step.
//
// A prompt of 4096 rows, 40 on 8 heads of 128, takes 190 to 200 us (860 to 900
// TFLOP/s against 1,240 for a large bf16 matrix product).  Neither kind of unit is
// full: of a SIMD's busy cycles 40% have a matrix instruction and about half a
// vector one (per group and wave 32 matrix instructions, 512 cycles, and about 115
// vector ones, 650 cycles: four each, an exponential sixteen), 38% of the matrix
// cycles with a vector instruction beside them; with products and exponentials in
// blocks that was 19%, and 212 us.  What is left is overlap.
template <int D, int NQ, int W>
struct Shared {
  static constexpr int R = 16 * NQ * W, F = D / 32, kThreads = 64 * W;
  static constexpr int kPer = 2 * F / W;            // KiB of codes a wave carries of a bundle: keys are the first F, then values
  static constexpr int kBundle = 2 * F * 128;       // 16-byte fragments of a bundle
  static constexpr int kTable = kThreads;           // groups whose page and scales are at hand
  static constexpr size_t kLds = (2 * (size_t)kBundle + kTable) * 16;
  static_assert(2 * F % W == 0, "every wave carries as many codes");
};

// Rows 0 .. rows - 1 of a tile against the groups from .. to - 1 of what they see:
// finish(o, m, l) takes those of this wave's rows (positions w_first .. w_last).  Every
// thread of the workgroup calls it; `stage` is the workgroup's LDS, free before.
template <int D, int NQ, int W, bool kSplit, class Place, class Finish>
__device__ __forceinline__ void shared_tile(const Tokens<kSplit> A, int from, int to, int rows, int w_first, int w_last, float scale_log2,
                                            const Place place, u32x4* stage, const Finish finish) {
  using S = Shared<D, NQ, W>;
  constexpr int F = S::F, C = D / 16;
  u32x4* table = stage + 2 * S::kBundle;   // number in the code arrays, key scale, log2 and reciprocal of the value scale
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, lo = lane & 15;
  const int mine0 = wave * 16 * NQ;    // this wave's own rows; none of them: it only carries codes
  const bool working = mine0 < rows;
  const int in_page = (1 << (A.c.page_shift - 5)) - 1;
  int table_at = 0;   // group of the table's first entry
  auto fill = [&](int n) {
    const int i = max(n + tid, from), g = A.group_at(i);
    const int id = i < to ? page_id(A.b, A.c.n_pages, A.row_at(i), g >> (A.c.page_shift - 5)) : -1;
    const size_t at = (size_t)max(id, 0) * A.c.hkv + A.head;
    const PageScales scales = page_scales(A.c.ks[at], A.c.vs[at]);   // of one that is not there page 0's, hidden later
    const int where = id < 0 ? -1 : (int)((at << (A.c.page_shift - 5)) + (g & in_page));
    __syncthreads();
    table[tid] = u32x4{(uint32_t)where, __float_as_uint(scales.ks), __float_as_uint(scales.lv), __float_as_uint(scales.rv)};
    table_at = n;
    __syncthreads();
  };
  auto entry = [&](int n) { return table[n - table_at]; };
  using Raw = u32x4[S::kPer];
  // a bundle: the keys at `k`, the values at `v` (numbers of groups in the code
  // arrays; one that is not there: the arrays' first, hidden later)
  auto load = [&](int k, int v, Raw& raw) {
#pragma unroll
    for (int u = 0; u < S::kPer; ++u) {
      const int unit = u * W + wave;
      const bool key = unit < F;
      raw[u] = load_codes<0>((key ? A.c.k : A.c.v) + (size_t)max(key ? k : v, 0) * (32 * D), unit % F);
    }
  };
  auto uniform = [](uint32_t x) { return (int)__builtin_amdgcn_readfirstlane((int)x); };
  // the first codes are on their way before the queries are looked at
  Raw one, two;
  int at[4];
  if (from < to) {
    fill(from);
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = uniform(entry(from + i)[0]);
    load(at[0], at[0], one);   // of bundle from - 1 only the keys are used
    load(at[1], at[0], two);
  }

  half8 qf[NQ][F];
  float qs[NQ], m[NQ], l[NQ];
  int pos[NQ];
  f32x4 o[NQ][C];
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int r = mine0 + t * 16 + lo;
    const uint16_t* row = place(r, pos[t]);
    qs[t] = load_query<D>(row, r < rows, scale_log2, qf[t]);
    m[t] = kLowest;
    l[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // pieces `from` .. `to` - 1 of the 4 kPer that the wave's codes are converted in
  u32x4 made[2];
  auto store = [&](int n, const Raw& raw, int from, int to) {
#pragma unroll
    for (int i = 0; i < 4 * S::kPer; ++i) {
      if (i < from || i >= to) continue;
      const u32x2 h = codes_to_half4(raw[i / 4][i % 4]);
      made[i / 2 % 2][i % 2 * 2] = h[0];
      made[i / 2 % 2][i % 2 * 2 + 1] = h[1];
      if (i % 2) stage[(n & 1) * S::kBundle + (i / 4 * W + wave) * 128 + i / 2 % 2 * 64 + lane] = made[i / 2 % 2];
    }
  };
  // Products of a bundle's C key or value fragments, other() work between them;
  // `ring` holds the first kRing fragments when it begins and those of `then`
  // when it ends.  The compiler keeps the order: arithmetic on its own may pass,
  // matrix instructions and LDS reads may not.
  constexpr int kRing = 4;
  half8 ring[kRing];
  auto fetch = [&](const u32x4* at, int i) { ring[i % kRing] = __builtin_bit_cast(half8, at[i * 64]); };
  auto products = [&](const u32x4* at, const u32x4* then, auto product, auto other) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      product(i, ring[i % kRing]);
      if (i + kRing < C)
        fetch(at, i + kRing);
      else if (then)
        fetch(then, i + kRing - C);
      other(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // scores of the keys in bundle n
  auto score = [&](f32x4 (&s)[NQ][2]) {
    return [&](int i, half8 k) {
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        f32x4& to = s[t][i / (D / 32)];
        to = mfma(k, qf[t][i % (D / 32)], i % (D / 32) ? to : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      }
    };
  };
  auto bundle = [&](int n) { return stage + (n & 1) * S::kBundle + lane; };
  // What a step needs of the table is read a step before: `here` is the entry of
  // its group, `far` that of the keys it loads; the values it loads are those of
  // the keys loaded by the step before.
  u32x4 here;
  uint32_t far;
  int v_at;
  // `ready` holds bundle n + 1's codes, `coming` takes bundle n + 2's
  auto step = [&](int n, f32x4 (&now)[NQ][2], f32x4 (&next)[NQ][2], const Raw& ready, Raw& coming) {
    const int k_at = uniform(far), id = uniform(here[0]);
    const float ks = __uint_as_float(uniform(here[1])), lv = __uint_as_float(uniform(here[2])), rv = __uint_as_float(uniform(here[3]));
    load(k_at, v_at, coming);
    v_at = k_at;
    if (n + 4 >= table_at + S::kTable) fill(n);
    here = entry(n + 1);
    far = entry(n + 4)[0];
    if (working) {
      const u32x4* kf = bundle(n);
      const u32x4* vf = kf + F * 128;
#pragma unroll
      for (int i = 0; i < kRing; ++i) fetch(kf, i);
      const int first = A.group_at(n) * 32;
      const Group group{id, first, ks, lv, rv, id < 0 || A.hides(n, first, w_first, w_last), A.lo_at(n), A.hi_at(n)};
      Weights<NQ> weights;
      weights.hide(A, group, now, qs, pos);
      products(kf, vf, score(next), [&](int i) { weights.form(group, now, m, i * 8 * NQ / C, (i + 1) * 8 * NQ / C); });
      half8 pf[NQ];
      weights.settle(group, now, m, l, o, pf);
      products(vf, static_cast<const u32x4*>(nullptr), [&](int i, half8 v) {
#pragma unroll
        for (int t = 0; t < NQ; ++t) o[t][i] = mfma(v, pf[t], o[t][i]);
      }, [&](int i) { store(n + 1, ready, i * 4 * S::kPer / C, (i + 1) * 4 * S::kPer / C); });
    } else {
      store(n + 1, ready, 0, 4 * S::kPer);
    }
    __syncthreads();
  };
  if (from < to) {
    f32x4 even[NQ][2], odd[NQ][2];
    store(from - 1, one, 0, 4 * S::kPer);
    load(at[2], at[1], one);
    store(from, two, 0, 4 * S::kPer);
    v_at = at[2];
    here = entry(from);
    far = (uint32_t)at[3];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(bundle(from - 1), i);
    products(bundle(from - 1), static_cast<const u32x4*>(nullptr), score(even), [](int) {});
    __syncthreads();   // its keys' place is the next bundle's
    for (int n = from;;) {
      step(n, even, odd, one, two);
      if (++n >= to) break;
      step(n, odd, even, two, one);
      if (++n >= to) break;
    }
  }
  finish(o, m, l);
}

}  // namespace dl
