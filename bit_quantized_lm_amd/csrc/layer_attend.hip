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
  int target;              // workgroups a head that fill the card
  int min_run, alone;      // least groups of a part or run; most of a tile that is not worth splitting
  uint32_t* arrived;       // [kMaxSlots] zero between calls
  float* part;             // [slot] partial results
};

// ------------------------------------------------------------------ the work
// A sequence's rows for one kv head are its query heads' rows, token after
// token: row x = (x / group)-th new token, head x % group of the kv head's.
// Tiles of R such rows share each key and value that they load.
//
// How the tiles become workgroups goes by their number against the `target` that
// fills the card:
//   twice the target or more, or up to the target and short or much the same
//     length, or a prompt whose first tiles see so much less than its last that
//     those set the pace: a tile a workgroup, the sequences in the batch's order,
//     in the shared kernel a sequence's tiles from the one that sees most;
//   a quarter of the target or fewer: each tile cut into equal parts of about the
//     same length for all, a part a workgroup;
//   else the tiles' visible tokens, as groups of 32, are laid end to end and cut
//     into equal runs, one a workgroup, so that all end together whatever the
//     lengths; a run may hold the end of one tile, whole tiles and the start of
//     another, which costs it a beginning and an end each.
// A tile of several parts is joined by the last of them (join_parts).  64 slots
// over 0.95 GB of mixed lengths (64 tiles a head, target 64): 158 us in runs, 180 a
// tile a workgroup.  A windowed batch of equal lengths (32, 32): 54.6 us in runs,
// 49.5 by tiles.  72 slots (7, 64): 34 us in runs, 29 in parts.  A prompt of 512
// rows (20, 64): 34 us in runs, 23 by tiles; of 2,048 (80, 64): 94 in runs, 67.
// From twice the target on the longest tile is not looked at: one sequence of
// 131,072 tokens among 126 of 500 (8 kv heads) takes 82 us in runs, among 127 of
// them 966, a workgroup a head walking it alone.
constexpr int kMaxBlocks = 512;          // most workgroups that a plan takes to fill the card
constexpr int kMaxSlots = 2 * (kMaxBlocks + DL_MAX_HEADS);
// Pairs of a row and a part that a tile's joining holds in LDS: what bounds the
// parts.  Few rows leave room for their parts at 32 KiB, more take 64.
template <int R>
constexpr int kJoinPairs = R <= 16 ? 4096 : 8192;
template <int R>
constexpr int kMaxParts = kJoinPairs<R> / R;
template <int R, int kThreads>
constexpr int kJoinFloats = 2 * kJoinPairs<R> + 4 * kThreads;
constexpr size_t kArrivedBytes = DL_WORKSPACE_ZERO_BYTES;
static_assert(kArrivedBytes >= kMaxSlots * sizeof(uint32_t) && kArrivedBytes % 256 == 0, "a counter a slot, the parts aligned");

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

// A part of a tile: from .. to of the `of` that the plan counts for it (groups,
// of which every tile has at least 1, so that one that sees nothing is visited
// too, or parts).
struct Segment {
  Seq q;
  int seq, tile;
  int from, to, of;
  int parts, part;   // the tile's parts, and which this is
  int first_run;     // the run that holds part 0
};

// The plan, which every wave computes alike from the lengths, and the walk
// through one run's segments.
template <int R>
class Walk {
 public:
  // Run (or tile) `run` of a head; false where there is none.
  __device__ __forceinline__ bool begin(const AttendArgs& A, int run) {
    const int lane = threadIdx.x & 63;
    float groups = 0.0f, real = 0.0f, tiles = 0.0f, most = 0.0f;   // real: with the tiles that see less than the last
    for (int s = lane; s < A.b.n_seq; s += 64) {
      const Seq q = load_seq(A.b, s);
      const int t = tiles_of(A, q), g = groups_of(A, q);
      if (s < 64) seq_ = q, tiles_ = t, groups_ = g;
      groups += (float)t * (float)g;
      real += (float)t * 0.5f * (float)(g + (t > 0 ? first_groups_of(A, q) : 0));
      tiles += (float)t;
      most = fmaxf(most, (float)g);
    }
    groups = wave_sum(groups);
    real = wave_sum(real);
    tiles = wave_sum(tiles);
    most = wave_max(most);
    const float target = (float)A.target;
    by_tile_ = true;
    run_ = run;
    const bool short_or_even = most <= (float)A.alone || most * target <= 1.25f * groups;
    if (tiles >= 2.0f * target || (tiles <= target && short_or_even) || fmaxf(most * target, 1.15f * real) < groups) {
      chunk_ = INT32_MAX;
      return true;
    }
    if (tiles * 4.0f <= target) {
      // the items are at most a tile's rounding up each more than groups / chunk
      const float chunk = fmaxf(groups * 1.001f / (target - tiles), most / (float)(kMaxParts<R> - 1));
      chunk_ = max(A.min_run, (int)fminf(ceilf(chunk), 1e9f));
      return true;
    }
    by_tile_ = false;
    // lengths are counted in units of 2^shift groups, so that their sum fits 32 bits
    shift_ = max(0, (int)((__float_as_uint(groups) >> 23) & 255u) - 127 - 28);
    const float unit = __builtin_ldexpf(1.0f, -shift_);
    // 0.1% more than the mean: float sums may fall short; tiles: each may be rounded up to a unit
    const float mean = (groups * unit * 1.001f + (shift_ ? tiles : 0.0f)) / target;
    per_ = max(max(A.min_run >> min(shift_, 8), 1), (int)ceilf(fmaxf(mean, most * unit / (float)(kMaxParts<R> - 3))));
    at_ = run * per_;
    end_ = at_ + per_;
    return run < A.target;
  }

  // The next segment; false past the run's (or the batch's) last.
  __device__ __forceinline__ bool next(const AttendArgs& A, Segment& g) {
    if (!by_tile_ && at_ >= end_) return false;
    const int lane = threadIdx.x & 63;
    int at = by_tile_ ? run_ : at_;
    for (int base = 0; base < A.b.n_seq; base += 64) {
      Seq q = seq_;
      int tiles = tiles_, groups = groups_;   // 0 past the last sequence
      if (base > 0) {
        tiles = groups = 0;
        if (base + lane < A.b.n_seq) {
          q = load_seq(A.b, base + lane);
          tiles = tiles_of(A, q);
          groups = groups_of(A, q);
        }
      }
      // a tile's parts, or its length
      const int each = by_tile_ ? groups / chunk_ + (groups % chunk_ != 0) : (groups + (1 << shift_) - 1) >> shift_;
      const int mine = tiles * each, sum = wave_inclusive_sum(mine);
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (at < total) {
        const int i = __builtin_ctzll(__ballot(sum > at));
        const int start = __builtin_amdgcn_readlane(sum, i) - __builtin_amdgcn_readlane(mine, i);
        g.seq = base + i;
        g.q.row0 = __builtin_amdgcn_readlane(q.row0, i);
        g.q.n = __builtin_amdgcn_readlane(q.n, i);
        g.q.len = __builtin_amdgcn_readlane(q.len, i);
        g.q.begin = g.q.len - g.q.n;
        g.of = __builtin_amdgcn_readlane(each, i);
        g.tile = (at - start) / g.of;
        g.from = at - start - g.tile * g.of;
        if (by_tile_) {
          g.to = g.from + 1;
          g.parts = g.of;
          g.part = g.from;
          g.first_run = run_ - g.part;
          by_tile_ = false;   // the only one
          at_ = end_ = 0;
          return true;
        }
        g.to = min(g.of, g.from + end_ - at_);
        const int tile_at = at_ - g.from;   // where the tile starts
        g.first_run = tile_at / per_;
        g.parts = (tile_at + g.of - 1) / per_ - g.first_run + 1;
        g.part = run_ - g.first_run;
        at_ += g.to - g.from;
        return true;
      }
      at -= total;
    }
    return false;
  }

 private:
  Seq seq_{};                    // sequence `lane`
  int tiles_ = 0, groups_ = 0;   // its tiles, and what one sees at most
  bool by_tile_;                 // a tile, or one of its parts of up to chunk_ groups, a workgroup
  int chunk_, run_;
  int shift_ = 0, per_ = 0, at_ = 0, end_ = 0;   // runs of per_ units of 2^shift_ groups: this one's

  static __device__ __forceinline__ int tiles_of(const AttendArgs& A, const Seq& q) {
    return (int)(((int64_t)q.n * A.group + R - 1) / R);
  }
  static __device__ __forceinline__ int groups_of(const AttendArgs& A, const Seq& q) {
    const int tokens = min(q.n, R / A.group + 2);   // a tile's, at most
    return q.n == 0 ? 0 : max(1, visible(A, q.len - tokens, q.len - 1).n);
  }
  static __device__ __forceinline__ int first_groups_of(const AttendArgs& A, const Seq& q) {
    return max(1, visible(A, q.begin, q.begin + min(q.n, R / A.group + 1) - 1).n);
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

// A run has a slot for the part of a tile that began in an earlier run (2 run)
// and one for the tile that it begins and does not end (2 run + 1): part v of a
// tile that begins in run f is in slot 2f + 1 or, v > 0, 2 (f + v).
struct Parts {
  __amdgpu_buffer_rsrc_t buffer;   // slot 2f of this head
  int step;                        // floats from a slot to the next
  __device__ __forceinline__ int at(int v) const { return max(2 * v, 1) * step; }
};
template <int D, int R>
__device__ __forceinline__ Parts parts_of(const AttendArgs& A, const Segment& g, int head) {
  return {part_buffer(A.part + ((size_t)2 * g.first_run * A.c.hkv + head) * kPartFloats<D, R>), A.c.hkv * kPartFloats<D, R>};
}

// The last of a tile's parts to arrive joins them all, in the parts' order, so
// the result does not depend on which one that is.  Every part's stores have
// reached memory (vmcnt 0 in each wave, then the barrier) before its workgroup
// is counted.  The published data come from beyond the L2, a microsecond or two
// away, so as many loads as the registers allow are under way together.
template <int D, int R, int kThreads>
__device__ __forceinline__ void join_parts(const AttendArgs& A, const Segment& w, const Seq& q, int x0, int rows, int head,
                                           const Parts& parts, float* lds) {
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    uint32_t* count = A.arrived + (2 * w.first_run + 1) * A.c.hkv + head;
    const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = before == (uint32_t)w.parts - 1;
    if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  auto row_of = [&](int r) {
    const int x = x0 + r;
    return (size_t)(q.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
  };
  // every (row, part)'s reference and sum of weights
  float* ref = lds;
  float* sums = lds + kJoinPairs<R>;
  const int n = w.parts, pairs = rows * n;
#pragma unroll 4
  for (int i = tid; i < pairs; i += kThreads) {
    const float2 s = published2(parts.buffer, parts.at(i % n) + R * D + i / n * 2);
    ref[i] = s.x;
    sums[i] = s.y;
  }
  __syncthreads();
  // the parts' shares of each row, in ref's place: few parts a thread a row, many a wave a row
  if (n <= 16) {
    if (tid < rows) {
      float top = kLowest, sum = 0.0f;
      for (int v = 0; v < n; ++v) top = fmaxf(top, ref[tid * n + v]);
      for (int v = 0; v < n; ++v) sum = fmaf(__builtin_amdgcn_exp2f(ref[tid * n + v] - top), sums[tid * n + v], sum);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int v = 0; v < n; ++v) ref[tid * n + v] = inv * __builtin_amdgcn_exp2f(ref[tid * n + v] - top);
      write_lse(A, row_of(tid), top, sum);
    }
  } else {
    for (int r = tid >> 6; r < rows; r += kThreads / 64) {
      float top = kLowest, sum = 0.0f;
      for (int v = lane; v < n; v += 64) top = fmaxf(top, ref[r * n + v]);
      top = wave_max(top);
      for (int v = lane; v < n; v += 64) {
        const float share = __builtin_amdgcn_exp2f(ref[r * n + v] - top);
        sum = fmaf(share, sums[r * n + v], sum);
        ref[r * n + v] = share;
      }
      sum = wave_sum(sum);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int v = lane; v < n; v += 64) ref[r * n + v] *= inv;
      if (lane == 0) write_lse(A, row_of(r), top, sum);
    }
  }
  __syncthreads();
  const int items = rows * (D / 4);   // four elements of a row each
  auto put = [&](int i, f32x4 y) {
    *reinterpret_cast<u32x2*>(A.out + row_of(i / (D / 4)) * D + i % (D / 4) * 4) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
  };
  // y of items i0 + k * kThreads over parts v0, v0 + by, ...: kItems x kParts loads under way together
  auto gather = [&](auto items_at_once, auto parts_at_once, int i0, int v0, int by, auto& y) {
    constexpr int kItems = decltype(items_at_once)::value, kParts = decltype(parts_at_once)::value;
    for (; v0 < n; v0 += by * kParts) {
      f32x4 x[kItems][kParts];
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int v = 0; v < kParts; ++v)   // past the end: the last item or part once more, with no share
          x[k][v] = published4(parts.buffer, parts.at(min(v0 + v * by, n - 1)) + min(i0 + k * kThreads, items - 1) * 4);
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int v = 0; v < kParts; ++v)
          y[k] += (v0 + v * by < n ? ref[min(i0 + k * kThreads, items - 1) / (D / 4) * n + min(v0 + v * by, n - 1)] : 0.0f) * x[k][v];
    }
  };
  using std::integral_constant;
  if (items <= kThreads) {
    // one item a thread; threads that are left over take turns at the parts
    const int turns = kThreads / items, i = tid % items, turn = tid / items;
    float* turned = lds + 2 * kJoinPairs<R>;
    f32x4 y[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
    if (turn < turns) gather(integral_constant<int, 1>(), integral_constant<int, 16>(), i, turn, turns, y);
    if (turn > 0) *reinterpret_cast<f32x4*>(turned + tid * 4) = y[0];
    __syncthreads();
    if (turn == 0) {
      for (int k = 1; k < turns; ++k) y[0] += *reinterpret_cast<const f32x4*>(turned + (i + k * items) * 4);
      put(i, y[0]);
    }
    return;
  }
  constexpr int kItems = 4;
  for (int i0 = tid; i0 < items; i0 += kThreads * kItems) {
    f32x4 y[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) y[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    gather(integral_constant<int, kItems>(), integral_constant<int, 4>(), i0, 0, 1, y);
#pragma unroll
    for (int k = 0; k < kItems; ++k)
      if (i0 + k * kThreads < items) put(i0 + k * kThreads, y[k]);
  }
}

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

// Whether some row at p_first .. p_last does not see some of the tokens first .. first + 31.
__device__ __forceinline__ bool hides(const AttendArgs& A, int first, int p_first, int p_last) {
  return first + 31 > p_first || (A.window > 0 && first <= p_last - A.window && first + 31 >= A.sinks);
}

// What is common to a group's scores: where its tokens are and its scales.
struct Group {
  int id, first;       // page (-1: nothing there), position of token 0
  float ks, lv, rv;    // key scale, log2(value scale), 1 / (value scale)
  bool edge;           // some row does not see some of its tokens
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

  __device__ __forceinline__ void hide(const AttendArgs& A, const Group& g, f32x4 (&x)[N][2], const float (&qs)[N], const int (&pos)[N]) {
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
        const bool seen = (g.id >= 0) & (at <= pos[t]) & ((A.window == 0) | (at > pos[t] - A.window) | (at < A.sinks));
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

template <int D, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attend_stream_kernel(AttendArgs A) {
  constexpr int R = 16, F = D / 32, C = D / 16, kThreads = 64 * W;
  __shared__ __align__(16) union {
    float o[W][R][D + 4];
    float join[kJoinFloats<R, kThreads>];
  } lds;
  __shared__ float m_lds[W][R], l_lds[W][R];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Walk<R> walk;
  if (!walk.begin(A, blockIdx.x / A.c.hkv)) return;
  for (Segment w; walk.next(A, w);) {
    const Seq q = w.q;
    const int x0 = w.tile * R, rows = min(R, q.n * A.group - x0);
    const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;
    const Range see = visible(A, p_first, p_last);
    const int from = (int)((int64_t)see.n * w.from / w.of), to = (int)((int64_t)see.n * w.to / w.of);
    const size_t page_bytes = (size_t)D << A.c.page_shift;

    // lane i: page and scales of the wave's i-th group from `base`, 64 at a time
    int base = from + wave, id_mine;
    PageScales mine_scales;
    auto group_at = [&](int n) { return n < see.ns ? n : n - see.ns + see.g0; };
    auto look = [&] {
      const int n = base + lane * W;
      id_mine = n < to ? page_id(A.b, A.c.n_pages, w.seq, group_at(n) >> (A.c.page_shift - 5)) : -1;
      const size_t at = (size_t)max(id_mine, 0) * A.c.hkv + head;
      mine_scales = page_scales(A.c.ks[at], A.c.vs[at]);   // of one that is not there page 0's, which step() hides
    };
    auto load = [&](int i, Bytes<F>& b) {   // of a group that is not there page 0's bytes, which step() hides
      const size_t off = ((size_t)max(__builtin_amdgcn_readlane(id_mine, i), 0) * A.c.hkv + head) * page_bytes +
                         (size_t)(group_at(base + i * W) & ((1 << (A.c.page_shift - 5)) - 1)) * 32 * D;
#pragma unroll
      for (int f = 0; f < F; ++f) b.k[f] = load_codes<kOnce>(A.c.k + off, f);
#pragma unroll
      for (int f = 0; f < F; ++f) b.v[f] = load_codes<kOnce>(A.c.v + off, f);
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
      const int x = x0 + lo;
      pos[0] = lo < rows ? q.begin + x / A.group : -1;
      const uint16_t* row = A.q + (int64_t)(q.row0 + x / A.group) * A.ldq + (head * A.group + x % A.group) * D;
      qs[0] = load_query<D>(row, lo < rows, A.scale_log2, qf);
#pragma unroll
      for (int c = 0; c < C; ++c) o[0][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto step = [&](int i, const Bytes<F>& b) {
      const int first = group_at(base + i * W) * 32, id = __builtin_amdgcn_readlane(id_mine, i);
      const Group group{id, first, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.ks), i)),
                        __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.lv), i)),
                        __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine_scales.rv), i)),
                        id < 0 || hides(A, first, p_first, p_last)};
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

    // join the waves; then either the result or this part's share of it
    const Parts parts = parts_of<D, R>(A, w, head);
    const int mine = parts.at(w.part);
    __syncthreads();   // lds: the segment before this one
    float sum_mine = l[0];
    sum_mine += __shfl_xor(sum_mine, 16);
    sum_mine += __shfl_xor(sum_mine, 32);
    if (hi == 0) {
      m_lds[wave][lo] = m[0];
      l_lds[wave][lo] = sum_mine;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) *reinterpret_cast<f32x4*>(&lds.o[wave][lo][c * 16 + hi * 4]) = o[0][c];
    __syncthreads();
    const int r = tid / (4 * W), x = x0 + r;   // 4 W threads a row
    if (r < rows) {
      float top = m_lds[0][r], sum = 0.0f, share[W];
#pragma unroll
      for (int v = 1; v < W; ++v) top = fmaxf(top, m_lds[v][r]);
#pragma unroll
      for (int v = 0; v < W; ++v) {
        share[v] = __builtin_amdgcn_exp2f(m_lds[v][r] - top);
        sum += l_lds[v][r] * share[v];
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const size_t to_row = (size_t)(q.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
#pragma unroll
      for (int e = tid % (4 * W) * 4; e < D; e += 16 * W) {
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < W; ++v) y += share[v] * *reinterpret_cast<const f32x4*>(&lds.o[v][r][e]);
        if (w.parts == 1) {
          y *= inv;
          *reinterpret_cast<u32x2*>(A.out + to_row * D + e) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
        } else {
          publish4(parts.buffer, mine + r * D + e, y);
        }
      }
      if (tid % (4 * W) == 0) {
        if (w.parts > 1)
          publish2(parts.buffer, mine + R * D + r * 2, top, sum);
        else
          write_lse(A, to_row, top, sum);
      }
    }
    if (w.parts == 1) continue;
    __syncthreads();   // lds becomes join_parts' scratch
    join_parts<D, R, kThreads>(A, w, q, x0, rows, head, parts, &lds.join[0]);
  }
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
  static constexpr size_t kLds = std::max((2 * (size_t)kBundle + kTable) * 16, kJoinFloats<R, kThreads> * sizeof(float));
  static_assert(2 * F % W == 0, "every wave carries as many codes");
};

template <int D, int NQ, int W>
__global__ __launch_bounds__(64 * W, 2) void attend_shared_kernel(AttendArgs A) {
  using S = Shared<D, NQ, W>;
  constexpr int R = S::R, F = S::F, C = D / 16;
  extern __shared__ __align__(16) u32x4 stage[];
  u32x4* table = stage + 2 * S::kBundle;   // number in the code arrays, key scale, log2 and reciprocal of the value scale
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Walk<R> walk;
  if (!walk.begin(A, blockIdx.x / A.c.hkv)) return;
  for (Segment w; walk.next(A, w);) {
    const Seq q = w.q;
    w.tile = (int)(((int64_t)q.n * A.group + R - 1) / R) - 1 - w.tile;   // the tiles that see most first
    const int x0 = w.tile * R, rows = min(R, q.n * A.group - x0);
    const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;
    // this wave's own rows; none of them: it only carries codes
    const int mine0 = wave * 16 * NQ;
    const int w_first = q.begin + (x0 + mine0) / A.group, w_last = q.begin + (x0 + min(rows, mine0 + 16 * NQ) - 1) / A.group;
    const bool working = mine0 < rows;

    const Range see = visible(A, p_first, p_last);
    const int from = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.from / w.of));
    const int to = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.to / w.of));
    const int in_page = (1 << (A.c.page_shift - 5)) - 1;
    auto group_at = [&](int n) { return n < see.ns ? n : n - see.ns + see.g0; };
    int table_at = 0;   // group of the table's first entry
    auto fill = [&](int n) {
      const int i = max(n + tid, from), g = group_at(i);
      const int id = i < to ? page_id(A.b, A.c.n_pages, w.seq, g >> (A.c.page_shift - 5)) : -1;
      const size_t at = (size_t)max(id, 0) * A.c.hkv + head;
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
        const int first = group_at(n) * 32;
        const Group group{id, first, ks, lv, rv, id < 0 || hides(A, first, w_first, w_last)};
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

    const Parts parts = parts_of<D, R>(A, w, head);
    const int mine = parts.at(w.part);
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const int r = mine0 + t * 16 + lo, x = x0 + r;
      float sum = l[t];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (r >= rows) continue;
      if (w.parts == 1) {
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
        for (int c = 0; c < C; ++c) publish4(parts.buffer, mine + r * D + c * 16 + hi * 4, o[t][c]);
        if (hi == 0) publish2(parts.buffer, mine + R * D + r * 2, m[t], sum);
      }
    }
    if (w.parts == 1) continue;
    __syncthreads();   // the stages become join_parts' scratch
    join_parts<D, R, S::kThreads>(A, w, q, x0, rows, head, parts, reinterpret_cast<float*>(stage));
    __syncthreads();   // and the next segment's stages
  }
}

// ------------------------------------------------------------------- launch
// The launch's kernel, by the rows that an average sequence has for one kv head
// (those without rows count; one prompt of 2,048 rows and 63 single tokens over 6,000,
// 225 us in tiles of 128, take 66 and 126 apart; one of 100 rows with them, 207 in
// tiles of 16, 13 and 126), and for few rows by the tiles: under 64 of them, which are split anyway, eight
// waves a workgroup leave half the parts to join (4 sequences of 8,000 tokens, 2 kv
// heads: 13.8 us instead of 16.2; 16 of 4,000, 8 heads: 36 instead of 31.7 with
// four); heads of 256 hold too many registers for it, and for two workgroups a CU:
// split for the 256 that run at once, one sequence of 60,000 tokens and 2 kv heads
// takes 40.5 us and 16 of 16,000 take 37.8; split for 512, 65.0 and 50.5 (four of
// 2,000 and 8 kv heads lose: 15.3 against 14.8).
struct Plan {
  int rows;      // a tile's
  int waves;     // of the streaming kernel's workgroup; 0: attend_shared_kernel
  int blocks;    // workgroups that fill the card: those that 256 CUs hold at once
  int min_run;   // least groups of a part: one a wave, or as many steps as its beginning takes
  int alone;     // most groups of a tile that joining parts would not make faster (4 us and more)
};
constexpr int kStreamRows = 16, kSmallRows = 64;   // most rows a sequence of the streaming kernel and of tiles of 64
Plan plan_of(int64_t rows, int n_seq, int hkv, int D) {
  if (rows <= kStreamRows) return D == 256 ? Plan{16, 4, 256, 4, 18} : (int64_t)n_seq * hkv < 64 ? Plan{16, 8, 256, 8, 36} : Plan{16, 4, 512, 4, 18};
  if (rows <= kSmallRows) return {64, 0, 512, 10, 14};
  return {128, 0, D == 256 ? 256 : 512, 30, 32};
}
Plan plan_for(int T, int n_seq, int hq, int hkv, int D) {
  return plan_of(((int64_t)T * (hq / hkv) + n_seq - 1) / n_seq, n_seq, hkv, D);
}

int target_items(int blocks, int hkv) { return std::max(1, blocks / hkv); }

size_t workspace_bytes(const Plan& p, int hkv, int D) {
  const size_t slots = 2 * (size_t)target_items(p.blocks, hkv) * hkv;
  return kArrivedBytes + slots * p.rows * (D + 2) * sizeof(float);
}

// What any call of up to T rows of up to n_seq sequences needs: fewer sequences
// have more rows each, up to all T in one, and any fewer, so every plan up to that
// one's is within reach (few rows: more sequences take no fewer workgroups).
size_t workspace_bound(int T, int n_seq, int hq, int hkv, int D) {
  const int64_t most = (int64_t)T * (hq / hkv);
  size_t bytes = workspace_bytes(plan_of(0, n_seq, hkv, D), hkv, D);
  if (most > kStreamRows) bytes = std::max(bytes, workspace_bytes(plan_of(kSmallRows, n_seq, hkv, D), hkv, D));
  if (most > kSmallRows) bytes = std::max(bytes, workspace_bytes(plan_of(kSmallRows + 1, n_seq, hkv, D), hkv, D));
  return bytes;
}

template <int D, int NQ, int W>
hipError_t launch_shared(const AttendArgs& A, dim3 grid, hipStream_t s) {
  using S = Shared<D, NQ, W>;
  static dh::OncePerDevice once;
  const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&attend_shared_kernel<D, NQ, W>), S::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_shared_kernel<D, NQ, W>), grid, dim3(S::kThreads), S::kLds, s, A);
  return hipSuccess;
}

template <int D>
int launch(const AttendArgs& A, const Plan& plan, hipStream_t s) {
  const int64_t rows = (int64_t)A.b.T * A.group;
  const int R = plan.rows;
  // tiles: sum over the sequences of ceil(rows / R), each with a row of its own
  const int64_t tiles = std::min<int64_t>((rows + (int64_t)A.b.n_seq * (R - 1)) / R, rows);
  const int64_t grid = std::max<int64_t>(tiles, A.target) * A.c.hkv;   // a tile a workgroup, or A.target runs a head
  if (grid > 0x7FFFFFFF) return dh::fail(DH_EUNSUP, "attend: too many rows for one launch");
  const dim3 g((unsigned)grid);
  hipError_t e = hipSuccess;
  if (plan.waves == 4) {
    hipLaunchKernelGGL((attend_stream_kernel<D, 4>), g, dim3(256), 0, s, A);
  } else if (plan.waves == 8) {
    if constexpr (D < 256) hipLaunchKernelGGL((attend_stream_kernel<D, 8>), g, dim3(512), 0, s, A);
  } else if (R == 64)
    e = launch_shared<D, 1, 4>(A, g, s);
  else if constexpr (D == 256)
    e = launch_shared<D, 1, 8>(A, g, s);
  else
    e = launch_shared<D, 2, 4>(A, g, s);
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
  *bytes = workspace_bound(T, n_seq, hq, hkv, D);
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
  const Plan plan = plan_for(T, n_seq, hq, hkv, D);
  const size_t need = workspace_bytes(plan, hkv, D);
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
  A.target = target_items(plan.blocks, hkv);
  A.min_run = plan.min_run;
  A.alone = plan.alone;
  A.arrived = static_cast<uint32_t*>(workspace);
  A.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kArrivedBytes);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  switch (D) {
    case 64: return launch<64>(A, plan, st);
    case 128: return launch<128>(A, plan, st);
    default: return launch<256>(A, plan, st);
  }
}

}  // extern "C"
