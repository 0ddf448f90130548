// The draft layer's attention over the 8-bit cache on gfx950
// (draft_layer_attend).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layer.h"

namespace {

using namespace dl;

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

struct AttendArgs {
  Batch b;
  Cache c;
  const uint16_t* q;
  int64_t ldq;
  int hq, group;           // group = hq / hkv
  float scale_log2;        // scale * log2(e)
  int window, sinks;
  uint16_t* out;
  float* lse;
  int target;              // work items per head that fill the card
  uint32_t* arrived;       // [kMaxSlots] zero between calls
  float* part;             // [slot] partial results
};

// ------------------------------------------------------------------ the work
// A sequence's rows for one kv head are its query heads' rows, token after
// token: row x = (x / group)-th new token, head x % group of the kv head's.
// Tiles of R such rows share each key and value that they load.  A tile's
// visible tokens, as groups of 32, are cut into `splits` parts where the batch
// has too few tiles to fill the card, each part a workgroup.
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kTargetBlocks = 512;      // workgroups that fill the card
constexpr int kMinSplitGroups = 4;      // least groups of 32 tokens a workgroup is split down to
constexpr int kMaxSlots = 2 * (kTargetBlocks + DL_MAX_HEADS);
constexpr int kJoinFloats = 8192;       // scratch of a tile's joining: a weight for each of its rows and parts
template <int R>
constexpr int kMaxSplits = kJoinFloats / R;
constexpr size_t kArrivedBytes = (kMaxSlots * sizeof(uint32_t) + 255) / 256 * 256;

struct Range {   // groups of 32 tokens a tile sees: first `ns` groups, then g0 .. g0 + n - ns - 1
  int ns, g0, n;
};

__device__ __forceinline__ Range visible(const AttendArgs& A, int p_first, int p_last) {
  Range r{0, 0, 0};
  const int cap = A.b.max_pages << A.c.page_shift;
  const int hi = (min(p_last + 1, cap) + 31) >> 5;   // groups up to the last visible token
  if (p_last < 0) return r;
  if (A.window > 0) {
    const int low = p_first - A.window + 1;
    if (low > 0) r.g0 = min(low >> 5, hi);
    r.ns = min((min(A.sinks, cap) + 31) >> 5, r.g0);
  }
  r.n = r.ns + hi - r.g0;
  return r;
}

struct Item {
  int seq, tile, split, splits;
  int slot;   // partial slot of split 0 (splits > 1)
};

// The batch's plan, computed by every wave from the lengths alone: parts of
// `chunk` groups such that the items per head come near A.target, which fills
// the card once (one a tile, and at most A.target more).
template <int R>
__device__ __forceinline__ bool find_work(const AttendArgs& A, int item, Item& w) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](const Seq& q) { return (int)(((int64_t)q.n * A.group + R - 1) / R); };
  auto groups_of = [&](const Seq& q) {   // of the tile that sees most
    if (q.n == 0) return 0;
    const int tokens = min(q.n, R / A.group + 2);
    return visible(A, q.len - tokens, q.len - 1).n;
  };
  float sum = 0.0f, all = 0.0f;
  for (int s = lane; s < A.b.n_seq; s += 64) {
    const Seq q = load_seq(A.b, s);
    sum += (float)tiles_of(q) * (float)groups_of(q);
    all += (float)tiles_of(q);
  }
  // 0.1% more than the sum, so that no rounding of it can bring more items than A.target and a tile each
  sum = wave_sum(sum) * 1.001f;
  all = wave_sum(all);
  const float spare = fmaxf((float)A.target - all, 0.125f * (float)A.target);
  const int chunk = max(kMinSplitGroups, (int)fminf(ceilf(sum / spare), 1e9f));
  int slot0 = 0;
  for (int base = 0; base < A.b.n_seq; base += 64) {
    const int s = base + lane;
    int tiles = 0, splits = 1;
    if (s < A.b.n_seq) {
      const Seq q = load_seq(A.b, s);
      tiles = tiles_of(q);
      splits = min(max(1, (groups_of(q) + chunk - 1) / chunk), kMaxSplits<R>);
    }
    const int items = tiles * splits, slots = splits > 1 ? items : 0;
    const int isum = wave_inclusive_sum(items), ssum = wave_inclusive_sum(slots);
    const int total = __builtin_amdgcn_readlane(isum, 63);
    if (item < total) {
      const int at = __builtin_ctzll(__ballot(isum > item));
      w.seq = base + at;
      w.splits = __builtin_amdgcn_readlane(splits, at);
      const int rest = item - (__builtin_amdgcn_readlane(isum, at) - __builtin_amdgcn_readlane(items, at));
      w.tile = rest / w.splits;
      w.split = rest % w.splits;
      w.slot = slot0 + __builtin_amdgcn_readlane(ssum, at) - __builtin_amdgcn_readlane(slots, at) + rest - w.split;
      return true;
    }
    item -= total;
    slot0 += __builtin_amdgcn_readlane(ssum, 63);
  }
  return false;
}

// --------------------------------------------------------------- conversions
// Eight code bytes (value + 128) as fp16: 0x6400 | u is 1024 + u, and
// subtracting 1152 leaves the signed code exactly.
__device__ __forceinline__ half8 codes_to_half(uint32_t a, uint32_t b) {
  const half2v off = {(_Float16)1152.0f, (_Float16)1152.0f};
  u32x4 w;
  const uint32_t src[2] = {a, b};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, src[i], 0x04010400u)) - off);
    w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, src[i], 0x04030402u)) - off);
  }
  return __builtin_bit_cast(half8, w);
}

__device__ __forceinline__ f32x4 mfma(half8 a, half8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A row's query fragments, lane (hi, lo) holding elements 64 f + 16 hi ..
// + 15 of the tile's row lo, as fp16 scaled by 2^-e so that the row's largest
// element is in [2^14, 2^15).  Returns scale_log2 * 2^e.  A zero row keeps 1;
// an infinite or NaN element makes its own row NaN and no other.
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
  return __builtin_ldexpf(scale_log2, e);
}

// Online softmax of one row: weights are 2^(x - m) with x = z log2(e) +
// log2(value scale), so that a weight times a value code is the value's whole
// share, whatever its page's scale, and m near the running maximum of x; l sums
// the weights over the value scales again.  m is set kHead below the maximum and
// moves only when some x exceeds it by more than kHead + kSlack: the sums need
// no rescaling in most steps, weights stay below 2^15 (fp16's largest is just
// under 2^16), and one keeps its 11 bits down to 2^-21 of the largest.
constexpr float kHead = 7.0f, kSlack = 8.0f;
constexpr float kLowest = -1e30f;   // m before the first visible token; finite, so no inf - inf arises

// --------------------------------------------------------------- split parts
// Partial results pass between workgroups, perhaps on different XCDs, through
// memory written and read with agent-scope accesses (sc1): written through to where
// every XCD sees it and read past stale copies, without flushing a cache (with an
// agent-scope release fence, which writes the XCD's L2 back, one row over
// 131,072 tokens took 108 us instead of 58, a windowed batch of 32 199 instead of 63).
constexpr int kAgentScope = 16;   // sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, 0x7FFFFFFF, 0x00027000);
}
__device__ __forceinline__ void publish4(__amdgpu_buffer_rsrc_t b, int at, f32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, at * 4, 0, kAgentScope);
}
__device__ __forceinline__ void publish2(__amdgpu_buffer_rsrc_t b, int at, float x, float y) {
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(x), __float_as_uint(y)}, b, at * 4, 0, kAgentScope);
}
__device__ __forceinline__ f32x4 published4(__amdgpu_buffer_rsrc_t b, int at) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at * 4, 0, kAgentScope));
}
__device__ __forceinline__ float2 published2(__amdgpu_buffer_rsrc_t b, int at) {
  const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(b, at * 4, 0, kAgentScope);
  return float2{__uint_as_float(x[0]), __uint_as_float(x[1])};
}

// A part is R x D sums and R x (reference, sum of weights).
template <int D, int R>
constexpr int kPartFloats = R * (D + 2);

__device__ __forceinline__ void write_lse(const AttendArgs& A, size_t row, float ref, float sum) {
  if (A.lse) A.lse[row] = sum == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
}

// The last of a tile's parts to arrive joins them all, in the parts' order, so
// the result does not depend on which one that is.  Every part's stores have
// reached memory (vmcnt 0 in each wave, then the barrier) before its workgroup
// is counted.  `parts`: part 0 of this tile and head; part v is at v * step
// floats.  `lds`: kJoinFloats and four a thread.
template <int D, int R, int kThreads>
__device__ __forceinline__ void join_parts(const AttendArgs& A, const Item& w, const Seq& q, int x0, int rows, int head,
                                           __amdgpu_buffer_rsrc_t parts, int step, float* lds) {
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    uint32_t* count = A.arrived + w.slot * A.c.hkv + head;
    const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = before == (uint32_t)w.splits - 1;
    if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  auto row_of = [&](int r) {
    const int x = x0 + r;
    return (size_t)(q.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
  };
  // a wave a row, a lane a part: the parts' shares of the row
  for (int r = tid >> 6; r < rows; r += kThreads / 64) {
    float top = kLowest;
    for (int v = lane; v < w.splits; v += 64) {
      const float2 s = published2(parts, v * step + R * D + r * 2);
      top = fmaxf(top, s.x);
      lds[r * w.splits + v] = s.x;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    float sum = 0.0f;
    for (int v = lane; v < w.splits; v += 64) {
      const float share = __builtin_amdgcn_exp2f(lds[r * w.splits + v] - top);
      sum += share * published2(parts, v * step + R * D + r * 2).y;
      lds[r * w.splits + v] = share;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int v = lane; v < w.splits; v += 64) lds[r * w.splits + v] *= inv;
    if (lane == 0) write_lse(A, row_of(r), top, sum);
  }
  __syncthreads();
  // four elements of a row a thread; threads that are left over take turns at the parts
  const int items = rows * (D / 4), turns = max(1, kThreads / items);
  float* turned = lds + kJoinFloats;
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int i = turns > 1 ? tid % items : i0 + tid, turn = turns > 1 ? tid / items : 0;
    const bool busy = i < items && turn < turns;
    const int r = i / (D / 4), at = r * D + i % (D / 4) * 4;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    if (busy) {
#pragma unroll 8
      for (int v = turn; v < w.splits; v += turns) y += lds[r * w.splits + v] * published4(parts, v * step + at);
    }
    if (turns > 1) {
      if (busy && turn > 0) *reinterpret_cast<f32x4*>(turned + tid * 4) = y;
      __syncthreads();
      if (busy && turn == 0)
        for (int k = 1; k < turns; ++k) y += *reinterpret_cast<const f32x4*>(turned + (tid + k * items) * 4);
    }
    if (busy && turn == 0)
      *reinterpret_cast<u32x2*>(A.out + row_of(r) * D + i % (D / 4) * 4) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
  }
}

// ------------------------------------------------------- few rows: streaming
// R = 16 MT rows against a stream of groups of 32 tokens.  Each wave takes
// every kWaves-th group of its workgroup's part, straight from global memory
// into the fragments (each load instruction 1 KiB without gaps), so nothing is
// shared until the waves' results are joined.  S^T = K Q^T puts a row's
// weights into the lanes and order that the next product takes its columns in
// (O^T = V^T P^T), so they never leave their registers.
template <int F>
struct Bytes {   // a lane's codes of one group
  u32x4 k[F], v[F];
};

template <int D, int MT>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 3) void attend_stream_kernel(AttendArgs A) {
  constexpr int R = 16 * MT, F = D / 32, C = D / 16;
  constexpr int kRow = D + 4;
  constexpr bool kAhead = D * MT <= 256;   // beyond, a second group's bytes do not fit the registers
  __shared__ __align__(16) union {
    float o[kWaves][16][kRow];
    float join[kJoinFloats + 4 * kThreads];
  } lds;
  __shared__ float m_lds[kWaves][16], l_lds[kWaves][16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Item w;
  if (!find_work<R>(A, blockIdx.x / A.c.hkv, w)) return;
  const Seq q = load_seq(A.b, w.seq);
  const int x0 = w.tile * R, rows = min(R, q.n * A.group - x0);
  const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;

  half8 qf[MT][F];
  float qs[MT], m[MT], l[MT];
  int pos[MT];
  f32x4 o[MT][C];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int x = x0 + t * 16 + lo;
    const bool valid = t * 16 + lo < rows;
    pos[t] = valid ? q.begin + x / A.group : -1;
    const uint16_t* row = A.q + (int64_t)(q.row0 + x / A.group) * A.ldq + (head * A.group + x % A.group) * D;
    qs[t] = load_query<D>(row, valid, A.scale_log2, qf[t]);
    m[t] = kLowest;
    l[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const Range see = visible(A, p_first, p_last);
  const int from = (int)((int64_t)see.n * w.split / w.splits), to = (int)((int64_t)see.n * (w.split + 1) / w.splits);
  const size_t page_bytes = (size_t)D << A.c.page_shift;
  for (int base = from + wave; base < to; base += 64 * kWaves) {
    // lane i: page and scales of the wave's i-th group from here
    const int n_mine = base + lane * kWaves, g_mine = n_mine < see.ns ? n_mine : n_mine - see.ns + see.g0;
    const int id_mine = n_mine < to ? page_id(A.b, A.c.n_pages, w.seq, g_mine >> (A.c.page_shift - 5)) : -1;
    const size_t at_mine = (size_t)max(id_mine, 0) * A.c.hkv + head;
    const float ks_mine = A.c.ks[at_mine], vs_mine = fmaxf(A.c.vs[at_mine], kMinScale);
    const int count = min(64, (to - base + kWaves - 1) / kWaves);
    auto group_at = [&](int i) {
      const int n = base + i * kWaves;
      return n < see.ns ? n : n - see.ns + see.g0;
    };
    auto load = [&](int i, Bytes<F>& w) {   // a page that is not there: page 0's bytes, which step() hides
      const size_t off = ((size_t)max(__builtin_amdgcn_readlane(id_mine, i), 0) * A.c.hkv + head) * page_bytes +
                         (size_t)(group_at(i) & ((1 << (A.c.page_shift - 5)) - 1)) * 32 * D;
      const u32x4* kc = reinterpret_cast<const u32x4*>(A.c.k + off) + lane;
      const u32x4* vc = reinterpret_cast<const u32x4*>(A.c.v + off) + lane;
#pragma unroll
      for (int f = 0; f < F; ++f) w.k[f] = __builtin_nontemporal_load(kc + f * 64);
#pragma unroll
      for (int f = 0; f < F; ++f) w.v[f] = __builtin_nontemporal_load(vc + f * 64);
    };
    auto step = [&](int i, const Bytes<F>& w) {
      const int g = group_at(i), id = __builtin_amdgcn_readlane(id_mine, i);
      const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks_mine), i));
      const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs_mine), i));
      f32x4 s[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t) s[t][0] = s[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const half8 a = codes_to_half(w.k[f][0], w.k[f][1]), b = codes_to_half(w.k[f][2], w.k[f][3]);
        const int tt = f / (D / 64), c = f % (D / 64);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          s[t][tt] = mfma(a, qf[t][2 * c], s[t][tt]);
          s[t][tt] = mfma(b, qf[t][2 * c + 1], s[t][tt]);
        }
      }
      const float lv = __builtin_amdgcn_logf(vs), rv = __builtin_amdgcn_rcpf(vs);
      const int tok = g * 32 + hi * 4;
      const bool edge = id < 0 || g * 32 + 31 > p_first ||
                        (A.window > 0 && g * 32 <= p_last - A.window && g * 32 + 31 >= A.sinks);
      half8 pf[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const float c = ks * qs[t];
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s[t][j >> 2][j & 3] * c;
        if (edge) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = tok + (j >> 2) * 16 + (j & 3);
            const bool seen = id >= 0 && at <= pos[t] && (A.window == 0 || at > pos[t] - A.window || at < A.sinks);
            x[j] = seen ? x[j] : -INFINITY;
          }
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
        top += lv;
        if (__any(top > m[t] + (kHead + kSlack))) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float next = fmaxf(m[t], top - kHead), down = __builtin_amdgcn_exp2f(m[t] - next);
          m[t] = next;
          l[t] *= down;
#pragma unroll
          for (int cc = 0; cc < C; ++cc) o[t][cc] *= down;
        }
        const float shift = lv - m[t];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = __builtin_amdgcn_exp2f(x[j] + shift);
          sum += p;
          pf[t][j] = (_Float16)p;
        }
        l[t] = fmaf(sum, rv, l[t]);
      }
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const half8 a = codes_to_half(w.v[f][0], w.v[f][1]), b = codes_to_half(w.v[f][2], w.v[f][3]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          o[t][2 * f] = mfma(a, pf[t], o[t][2 * f]);
          o[t][2 * f + 1] = mfma(b, pf[t], o[t][2 * f + 1]);
        }
      }
    };
    if constexpr (kAhead) {
      // one group's loads are under way while the one before is worked on
      Bytes<F> even, odd;
      load(0, even);
      for (int i = 0; i < count; i += 2) {
        if (i + 1 < count) load(i + 1, odd);
        step(i, even);
        if (i + 1 >= count) break;
        if (i + 2 < count) load(i + 2, even);
        step(i + 1, odd);
      }
    } else {
      for (int i = 0; i < count; ++i) {
        Bytes<F> w;
        load(i, w);
        step(i, w);
      }
    }
  }

  // Join the waves, 16 rows at a time, then either the result or this part's
  // share of it.
  const __amdgpu_buffer_rsrc_t parts = part_buffer(A.part + (size_t)(w.slot * A.c.hkv + head) * kPartFloats<D, R>);
  const int step = A.c.hkv * kPartFloats<D, R>, mine = w.split * step;
  for (int t = 0; t < MT; ++t) {
    if (t * 16 >= rows) break;
    if (t) __syncthreads();
#pragma unroll
    for (int tt = 0; tt < MT; ++tt)
      if (tt == t) {
        float sum = l[tt];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (hi == 0) {
          m_lds[wave][lo] = m[tt];
          l_lds[wave][lo] = sum;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) *reinterpret_cast<f32x4*>(&lds.o[wave][lo][c * 16 + hi * 4]) = o[tt][c];
      }
    __syncthreads();
    const int r = tid >> 4, x = x0 + t * 16 + r;
    if (t * 16 + r < rows) {
      float top = m_lds[0][r], sum = 0.0f, share[kWaves];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) top = fmaxf(top, m_lds[v][r]);
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        share[v] = __builtin_amdgcn_exp2f(m_lds[v][r] - top);
        sum += l_lds[v][r] * share[v];
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const size_t to_row = (size_t)(q.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
#pragma unroll
      for (int e = (tid & 15) * 4; e < D; e += 64) {
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) y += share[v] * *reinterpret_cast<const f32x4*>(&lds.o[v][r][e]);
        if (w.splits == 1) {
          y *= inv;
          *reinterpret_cast<u32x2*>(A.out + to_row * D + e) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
        } else {
          publish4(parts, mine + (t * 16 + r) * D + e, y);
        }
      }
      if ((tid & 15) == 0) {
        if (w.splits > 1)
          publish2(parts, mine + R * D + (t * 16 + r) * 2, top, sum);
        else
          write_lse(A, to_row, top, sum);
      }
    }
  }
  if (w.splits == 1) return;

  __syncthreads();   // lds becomes join_parts' scratch
  join_parts<D, R, kThreads>(A, w, q, x0, rows, head, parts, step, &lds.join[0]);
}

// -------------------------------------------------------- many rows: shared
// R = 16 NQ W rows: each wave holds NQ tiles of 16 rows, and the workgroup's
// waves share the key and value fragments, converted to fp16 once, through
// LDS.  Steps of G groups alternate between two stages: while one is worked on,
// the next one's codes are converted into the other and the one after that is
// on its way from memory in registers; one barrier a step.
template <int D, int NQ, int W, int G>
struct Shared {
  static constexpr int R = 16 * NQ * W, F = D / 32, kThreads = 64 * W;
  static constexpr int kUnits = G * 2 * F;                 // KiB of codes a step: keys, then values
  static constexpr int kPer = kUnits / W;                  // of them a wave's
  static constexpr int kStage = kUnits * 2 * 64;           // 16-byte fragments a stage
  static constexpr size_t kLds = std::max(2 * (size_t)kStage * 16, (kJoinFloats + 4 * kThreads) * sizeof(float));
  static_assert(kUnits % W == 0, "every wave carries as many codes");
};

template <int D, int NQ, int W, int G>
__global__ __launch_bounds__(64 * W, 2) void attend_shared_kernel(AttendArgs A) {
  using S = Shared<D, NQ, W, G>;
  constexpr int R = S::R, F = S::F, C = D / 16;
  extern __shared__ __align__(16) u32x4 stage[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Item w;
  if (!find_work<R>(A, blockIdx.x / A.c.hkv, w)) return;
  const Seq q = load_seq(A.b, w.seq);
  w.tile = (int)(((int64_t)q.n * A.group + R - 1) / R) - 1 - w.tile;   // the tiles that see most first
  const int x0 = w.tile * R, rows = min(R, q.n * A.group - x0);
  const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;
  // this wave's own rows; none of them: it only carries codes
  const int mine0 = wave * 16 * NQ;
  const int w_first = q.begin + (x0 + mine0) / A.group, w_last = q.begin + (x0 + min(rows, mine0 + 16 * NQ) - 1) / A.group;
  const bool working = mine0 < rows;

  half8 qf[NQ][F];
  float qs[NQ], m[NQ], l[NQ];
  int pos[NQ];
  f32x4 o[NQ][C];
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int r = mine0 + t * 16 + lo, x = x0 + r;
    const bool valid = r < rows;
    pos[t] = valid ? q.begin + x / A.group : -1;
    const uint16_t* row = A.q + (int64_t)(q.row0 + x / A.group) * A.ldq + (head * A.group + x % A.group) * D;
    qs[t] = load_query<D>(row, valid, A.scale_log2, qf[t]);
    m[t] = kLowest;
    l[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) o[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const Range see = visible(A, p_first, p_last);
  const int from = (int)((int64_t)see.n * w.split / w.splits), to = (int)((int64_t)see.n * (w.split + 1) / w.splits);
  const size_t page_bytes = (size_t)D << A.c.page_shift;
  const int in_page = (1 << (A.c.page_shift - 5)) - 1;
  // lane i: page and scales of the i-th group from `base`, 64 at a time; the
  // loads run up to two steps ahead of the work, so theirs are kept apart
  int id_load = -1, id_work = -1, base_load = from - 64, base_work = from - 64;
  float ks_work = 0.0f, vs_work = 0.0f;
  auto group_at = [&](int n) { return n < see.ns ? n : n - see.ns + see.g0; };
  auto page_of = [&](int n) { return n < to ? page_id(A.b, A.c.n_pages, w.seq, group_at(n) >> (A.c.page_shift - 5)) : -1; };
  u32x4 raw[S::kPer];
  auto load = [&](int n0) {   // groups n0 .. n0 + G - 1; one that is not there: page 0's bytes, hidden later
    if (n0 - base_load >= 64) {
      base_load = n0;
      id_load = page_of(n0 + lane);
    }
#pragma unroll
    for (int u = 0; u < S::kPer; ++u) {
      const int unit = u * W + wave, g = unit / (2 * F), f = unit % F;
      const bool key = unit / F % 2 == 0;
      const int id = max(__builtin_amdgcn_readlane(id_load, n0 - base_load + g), 0);
      const size_t off = ((size_t)id * A.c.hkv + head) * page_bytes + (size_t)(group_at(n0 + g) & in_page) * 32 * D;
      raw[u] = *(reinterpret_cast<const u32x4*>((key ? A.c.k : A.c.v) + off) + f * 64 + lane);
    }
  };
  auto store = [&](int which) {
#pragma unroll
    for (int u = 0; u < S::kPer; ++u) {
      u32x4* at = stage + which * S::kStage + (u * W + wave) * 128 + lane;
      at[0] = __builtin_bit_cast(u32x4, codes_to_half(raw[u][0], raw[u][1]));
      at[64] = __builtin_bit_cast(u32x4, codes_to_half(raw[u][2], raw[u][3]));
    }
  };
  if (from < to) {
    load(from);
    store(0);
    if (from + G < to) load(from + G);
    __syncthreads();
  }
  for (int n0 = from, which = 0; n0 < to; n0 += G, which ^= 1) {
    if (n0 - base_work >= 64) {
      base_work = n0;
      id_work = page_of(n0 + lane);
      const size_t at = (size_t)max(id_work, 0) * A.c.hkv + head;
      ks_work = A.c.ks[at];
      vs_work = fmaxf(A.c.vs[at], kMinScale);
    }
    if (n0 + G < to) {
      store(which ^ 1);
      if (n0 + 2 * G < to) load(n0 + 2 * G);
    }
    if (working) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (G > 1 && n0 + g >= to) break;
        const int i = n0 + g - base_work, first = group_at(n0 + g) * 32;
        const u32x4* kf = stage + which * S::kStage + g * F * 256 + lane;
        const u32x4* vf = kf + F * 128;
        const int id = __builtin_amdgcn_readlane(id_work, i);
        const float ks = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks_work), i));
        const float vs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs_work), i));
        f32x4 s[NQ][2];
#pragma unroll
        for (int t = 0; t < NQ; ++t) s[t][0] = s[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const half8 a = __builtin_bit_cast(half8, kf[(f * 2 + h) * 64]);
#pragma unroll
            for (int t = 0; t < NQ; ++t) s[t][f / (D / 64)] = mfma(a, qf[t][f % (D / 64) * 2 + h], s[t][f / (D / 64)]);
          }
        const float lv = __builtin_amdgcn_logf(vs), rv = __builtin_amdgcn_rcpf(vs);
        const bool edge = id < 0 || first + 31 > w_first ||
                          (A.window > 0 && first <= w_last - A.window && first + 31 >= A.sinks);
        half8 pf[NQ];
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          float c = ks * qs[t];
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = s[t][j >> 2][j & 3];
          if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int at = first + hi * 4 + (j >> 2) * 16 + (j & 3);
              const bool seen = id >= 0 && at <= pos[t] && (A.window == 0 || at > pos[t] - A.window || at < A.sinks);
              x[j] = seen ? x[j] * c : -INFINITY;
            }
            c = 1.0f;
          }
          float top = x[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
          top = fmaf(top, c, lv);
          if (__any(top > m[t] + (kHead + kSlack))) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float next = fmaxf(m[t], top - kHead), down = __builtin_amdgcn_exp2f(m[t] - next);
            m[t] = next;
            l[t] *= down;
#pragma unroll
            for (int cc = 0; cc < C; ++cc) o[t][cc] *= down;
          }
          const float shift = lv - m[t];
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float p = __builtin_amdgcn_exp2f(fmaf(x[j], c, shift));
            sum += p;
            pf[t][j] = (_Float16)p;
          }
          l[t] = fmaf(sum, rv, l[t]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const half8 a = __builtin_bit_cast(half8, vf[c * 64]);
#pragma unroll
          for (int t = 0; t < NQ; ++t) o[t][c] = mfma(a, pf[t], o[t][c]);
        }
      }
    }
    __syncthreads();
  }

  const __amdgpu_buffer_rsrc_t parts = part_buffer(A.part + (size_t)(w.slot * A.c.hkv + head) * kPartFloats<D, R>);
  const int step = A.c.hkv * kPartFloats<D, R>, mine = w.split * step;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int r = mine0 + t * 16 + lo, x = x0 + r;
    float sum = l[t];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (r >= rows) continue;
    if (w.splits == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const size_t to_row = (size_t)(q.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const f32x4 y = o[t][c] * inv;
        *reinterpret_cast<u32x2*>(A.out + to_row * D + c * 16 + hi * 4) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
      }
      if (hi == 0) write_lse(A, to_row, m[t], sum);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) publish4(parts, mine + r * D + c * 16 + hi * 4, o[t][c]);
      if (hi == 0) publish2(parts, mine + R * D + r * 2, m[t], sum);
    }
  }
  if (w.splits == 1) return;
  __syncthreads();   // the stages become join_parts' scratch
  join_parts<D, R, S::kThreads>(A, w, q, x0, rows, head, parts, step, reinterpret_cast<float*>(stage));
}

// ------------------------------------------------------------------- launch
// The launch's kernel, by the rows that an average sequence has for one kv head.
struct Plan {
  int rows;      // a tile's
  bool shared;   // attend_shared_kernel (else the streaming one)
};
Plan plan_for(int T, int n_seq, int hq, int hkv, int D) {
  const int64_t rows = ((int64_t)T * (hq / hkv) + n_seq - 1) / n_seq;
  if (rows <= 16) return {16, false};
  if (rows <= 64) return {64, true};
  return {128, true};
}

int target_items(int hkv) { return std::max(1, kTargetBlocks / hkv); }

size_t workspace_bytes(int T, int n_seq, int hq, int hkv, int D) {
  const size_t slots = 2 * (size_t)target_items(hkv) * hkv;
  return kArrivedBytes + slots * plan_for(T, n_seq, hq, hkv, D).rows * (D + 2) * sizeof(float);
}

template <int D, int NQ, int W, int G>
hipError_t launch_shared(const AttendArgs& A, dim3 grid, hipStream_t s) {
  using S = Shared<D, NQ, W, G>;
  static bool attr_set = false;
  if (!attr_set) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&attend_shared_kernel<D, NQ, W, G>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)S::kLds);
    if (e != hipSuccess) return e;
    attr_set = true;
  }
  hipLaunchKernelGGL((attend_shared_kernel<D, NQ, W, G>), grid, dim3(S::kThreads), S::kLds, s, A);
  return hipSuccess;
}

template <int D>
int launch(const AttendArgs& A, const Plan& plan, hipStream_t s) {
  const int64_t rows = (int64_t)A.b.T * A.group;
  const int R = plan.rows;
  // tiles: sum over the sequences of ceil(rows / R), each with a row of its own
  const int64_t tiles = std::min<int64_t>((rows + (int64_t)A.b.n_seq * (R - 1)) / R, rows);
  const int64_t grid = (tiles + A.target) * A.c.hkv;
  if (grid > 0x7FFFFFFF) return dh::fail(DH_EUNSUP, "attend: too many rows for one launch");
  const dim3 g((unsigned)grid);
  constexpr int G = D == 256 ? 1 : 2;
  hipError_t e = hipSuccess;
  if (!plan.shared)
    hipLaunchKernelGGL((attend_stream_kernel<D, 1>), g, dim3(kThreads), 0, s, A);
  else if (R == 64)
    e = launch_shared<D, 1, 4, G>(A, g, s);
  else if constexpr (D == 256)
    e = launch_shared<D, 1, 8, 1>(A, g, s);
  else
    e = launch_shared<D, 2, 4, G>(A, g, s);
  if (e != hipSuccess) return dh::fail(DH_EHIP, "attend kernel: %s", hipGetErrorString(e));
  return launched("attend kernel");
}

}  // namespace

extern "C" {

int draft_layer_workspace_bytes(int T, int n_seq, int hq, int hkv, int D, size_t* bytes) {
  if (!bytes) return dh::fail(DH_EINVAL, "workspace_bytes: null pointer");
  int rc = check_heads("workspace_bytes", hq, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows("workspace_bytes", T, n_seq))) return rc;
  *bytes = workspace_bytes(T, n_seq, hq, hkv, D);
  return dh::ok();
}

int draft_layer_attend(const void* q, int64_t ldq, const uint8_t* k_codes, const uint8_t* v_codes,
                       const float* k_scale, const float* v_scale, int n_pages, int page, const int32_t* q_start,
                       const int32_t* kv_len, const int32_t* table, int n_seq, int max_pages, int T, int hq,
                       int hkv, int D, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                       size_t workspace_bytes_given, void* stream) {
  const char* who = "attend";
  int rc = check_heads(who, hq, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows(who, T, n_seq))) return rc;
  AttendArgs A{};
  A.b = Batch{q_start, kv_len, table, n_seq, max_pages, T};
  A.c = Cache{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes), const_cast<float*>(k_scale),
              const_cast<float*>(v_scale), n_pages, page_shift_of(page), hkv};
  if ((rc = check_cache(who, A.c, page, A.b))) return rc;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return dh::fail(DH_EINVAL, "attend: scale must be finite and > 0");
  if (window < 0 || sinks < 0) return dh::fail(DH_EINVAL, "attend: window and sinks must be >= 0 (got %d, %d)", window, sinks);
  if (T == 0) return dh::ok();
  if ((rc = check_stride(who, "q", q, ldq, (int64_t)hq * D))) return rc;
  if (!out || !aligned(out, 16)) return dh::fail(DH_EINVAL, "attend: out must be a 16-byte aligned pointer");
  if (lse && !aligned(lse, 4)) return dh::fail(DH_EINVAL, "attend: lse must be 4-byte aligned");
  if (!workspace || !aligned(workspace, 16)) return dh::fail(DH_EINVAL, "attend: workspace must be a 16-byte aligned pointer");
  const size_t need = workspace_bytes(T, n_seq, hq, hkv, D);
  if (workspace_bytes_given < need)
    return dh::fail(DH_EINVAL, "attend: workspace of %zu bytes is below the %zu needed", workspace_bytes_given, need);
  A.q = static_cast<const uint16_t*>(q);
  A.ldq = ldq;
  A.hq = hq;
  A.group = hq / hkv;
  A.scale_log2 = scale * 1.44269504088896f;
  A.window = window < DL_MAX_POSITIONS ? window : 0;   // past every position: no window
  A.sinks = std::min(sinks, DL_MAX_POSITIONS);
  A.out = static_cast<uint16_t*>(out);
  A.lse = lse;
  A.target = target_items(hkv);
  A.arrived = static_cast<uint32_t*>(workspace);
  A.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kArrivedBytes);
  const Plan R = plan_for(T, n_seq, hq, hkv, D);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  switch (D) {
    case 64: return launch<64>(A, R, st);
    case 128: return launch<128>(A, R, st);
    default: return launch<256>(A, R, st);
  }
}

}  // extern "C"
