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
  uint32_t* arrived;       // [kMaxSlots] zero between calls
  float* part;             // [slot] partial results
};

// ------------------------------------------------------------------ the work
// A sequence's rows for one kv head are its query heads' rows, token after
// token: row x = (x / group)-th new token, head x % group of the kv head's.
// Tiles of R such rows share each key and value that they load.
//
// Where the batch has at least twice the tiles that fill the card, a workgroup
// takes one tile.  Where it has fewer, the tiles' visible tokens, as groups of
// 32, are laid end to end and cut into equal runs, one a workgroup, so that the
// card is filled and all end together whatever the lengths; a run may hold the
// end of one tile, whole tiles and the start of another.  A tile that several
// runs hold parts of is joined by the last of them (join_parts).  Cut by tiles
// instead, 64 slots over 0.95 GB of mixed lengths waited for the longest: 180 us.
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMinRun = 4;               // least groups of a run
constexpr int kMaxBlocks = 768;          // most workgroups that a plan takes to fill the card
constexpr int kMaxSlots = 2 * (kMaxBlocks + DL_MAX_HEADS);
// Pairs of a row and a part that a tile's joining holds in LDS: what bounds the
// parts.  Few rows leave room for their parts at 32 KiB, more take 64.
template <int R>
constexpr int kJoinPairs = R <= 16 ? 4096 : 8192;
template <int R>
constexpr int kMaxParts = kJoinPairs<R> / R;
template <int R, int kThreads>
constexpr int kJoinFloats = 2 * kJoinPairs<R> + 4 * kThreads;
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

// A part of a tile: groups from .. to - 1 of the `of` that the plan counts for
// it (the most that a tile of the sequence sees; at least 1, so that tiles that
// see nothing are visited too).
struct Segment {
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
    float groups = 0.0f, tiles = 0.0f, most = 0.0f;
    for (int s = lane; s < A.b.n_seq; s += 64) {
      const Seq q = load_seq(A.b, s);
      const int t = tiles_of(A, q), g = groups_of(A, q);
      if (s < 64) tiles_ = t, groups_ = g;
      groups += (float)t * (float)g;
      tiles += (float)t;
      most = fmaxf(most, (float)g);
    }
    groups = wave_sum(groups);
    tiles = wave_sum(tiles);
    most = wave_max(most);
    whole_ = tiles >= 2.0f * (float)A.target;
    // lengths are counted in units of 2^shift groups, so that their sum fits 32 bits
    shift_ = max(0, (int)((__float_as_uint(groups) >> 23) & 255u) - 127 - 28);
    const float unit = __builtin_ldexpf(1.0f, -shift_);
    // 0.1% more than the mean: float sums may fall short; tiles: each may be rounded up to a unit
    const float mean = (groups * unit * 1.001f + (shift_ ? tiles : 0.0f)) / (float)A.target;
    per_ = max(kMinRun >> min(shift_, 2), (int)ceilf(fmaxf(mean, most * unit / (float)(kMaxParts<R> - 3))));
    run_ = run;
    at_ = whole_ ? run : run * per_;
    end_ = at_ + (whole_ ? 1 : per_);
    return whole_ || run < A.target;
  }

  // The next segment; false past the run's (or the batch's) last.
  __device__ __forceinline__ bool next(const AttendArgs& A, Segment& g) {
    if (at_ >= end_) return false;
    const int lane = threadIdx.x & 63;
    int at = at_, before = 0;   // `before`: units of the sequences passed
    for (int base = 0; base < A.b.n_seq; base += 64) {
      int tiles = tiles_, groups = groups_;
      if (A.b.n_seq > 64 && base > 0) {
        tiles = groups = 0;
        if (base + lane < A.b.n_seq) {
          const Seq q = load_seq(A.b, base + lane);
          tiles = tiles_of(A, q);
          groups = groups_of(A, q);
        }
      } else if (lane >= A.b.n_seq) {
        tiles = groups = 0;
      }
      const int units = (groups + (1 << shift_) - 1) >> shift_;
      const int mine = whole_ ? tiles : tiles * units, sum = wave_inclusive_sum(mine);
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (at < total) {
        const int i = __builtin_ctzll(__ballot(sum > at));
        const int start = __builtin_amdgcn_readlane(sum, i) - __builtin_amdgcn_readlane(mine, i);
        g.seq = base + i;
        if (whole_) {
          g.tile = at - start;
          g.from = 0;
          g.to = g.of = 1;
          g.parts = 1;
          g.part = g.first_run = 0;
          at_ = end_;
          return true;
        }
        g.of = __builtin_amdgcn_readlane(units, i);
        g.tile = (at - start) / g.of;
        g.from = at - start - g.tile * g.of;
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
  int tiles_ = 0, groups_ = 0;   // of sequence `lane`
  bool whole_;                   // a tile a workgroup
  int shift_, per_, run_, at_, end_;

  static __device__ __forceinline__ int tiles_of(const AttendArgs& A, const Seq& q) {
    return (int)(((int64_t)q.n * A.group + R - 1) / R);
  }
  static __device__ __forceinline__ int groups_of(const AttendArgs& A, const Seq& q) {
    const int tokens = min(q.n, R / A.group + 2);   // a tile's, at most
    return q.n == 0 ? 0 : max(1, visible(A, q.len - tokens, q.len - 1).n);
  }
};

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
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 128 ? 2 : 3) void attend_stream_kernel(AttendArgs A) {
  constexpr int R = 16 * MT, F = D / 32, C = D / 16;
  constexpr int kRow = D + 4;
  constexpr bool kAhead = D * MT <= 256;   // beyond, a second group's bytes do not fit the registers
  __shared__ __align__(16) union {
    float o[kWaves][16][kRow];
    float join[kJoinFloats<R, kThreads>];
  } lds;
  __shared__ float m_lds[kWaves][16], l_lds[kWaves][16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Walk<R> walk;
  if (!walk.begin(A, blockIdx.x / A.c.hkv)) return;
  for (Segment w; walk.next(A, w);) {
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
  const int from = (int)((int64_t)see.n * w.from / w.of), to = (int)((int64_t)see.n * w.to / w.of);
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
  const Parts parts = parts_of<D, R>(A, w, head);
  const int mine = parts.at(w.part);
  for (int t = 0; t < MT; ++t) {
    if (t * 16 >= rows) break;
    __syncthreads();   // lds: the rows or the segment before this one
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
        if (w.parts == 1) {
          y *= inv;
          *reinterpret_cast<u32x2*>(A.out + to_row * D + e) = u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
        } else {
          publish4(parts.buffer, mine + (t * 16 + r) * D + e, y);
        }
      }
      if ((tid & 15) == 0) {
        if (w.parts > 1)
          publish2(parts.buffer, mine + R * D + (t * 16 + r) * 2, top, sum);
        else
          write_lse(A, to_row, top, sum);
      }
    }
  }
  if (w.parts == 1) continue;

  __syncthreads();   // lds becomes join_parts' scratch
  join_parts<D, R, kThreads>(A, w, q, x0, rows, head, parts, &lds.join[0]);
  }
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
  static constexpr size_t kLds = std::max(2 * (size_t)kStage * 16, kJoinFloats<R, kThreads> * sizeof(float));
  static_assert(kUnits % W == 0, "every wave carries as many codes");
};

// Four of a group's fragments out of LDS.  What follows stays behind the reads
// (only arithmetic may pass), so that they are under way while the four before
// them are used: left to itself the compiler reads one, waits, uses it and reads
// the next.
__device__ __forceinline__ void read4(half8 (&to)[4], const u32x4* at) {
#pragma unroll
  for (int i = 0; i < 4; ++i) to[i] = __builtin_bit_cast(half8, at[i * 64]);
  __builtin_amdgcn_sched_barrier(0x16);
}

template <int D, int NQ, int W, int G>
__global__ __launch_bounds__(64 * W, 2) void attend_shared_kernel(AttendArgs A) {
  using S = Shared<D, NQ, W, G>;
  constexpr int R = S::R, F = S::F, C = D / 16;
  extern __shared__ __align__(16) u32x4 stage[];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Walk<R> walk;
  if (!walk.begin(A, blockIdx.x / A.c.hkv)) return;
  for (Segment w; walk.next(A, w);) {
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
  const int from = (int)((int64_t)see.n * w.from / w.of), to = (int)((int64_t)see.n * w.to / w.of);
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
      // waited for here, once in 64 groups: a use further down would wait for
      // the codes too that are loaded in between, in every step
      __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt 0
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
        half8 now[4], next[4];
        read4(now, kf);
#pragma unroll
        for (int c = 0; c < C / 4; ++c) {
          read4(next, c + 1 < C / 4 ? kf + (c + 1) * 256 : vf);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < NQ; ++t) {
              const int n = c * 4 + i, tt = n / (D / 32);
              s[t][tt] = mfma(now[i], qf[t][n % (D / 32)], s[t][tt]);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) now[i] = next[i];
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
        for (int c = 0; c < C / 4; ++c) {
          if (c + 1 < C / 4) read4(next, vf + (c + 1) * 256);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < NQ; ++t) o[t][c * 4 + i] = mfma(now[i], pf[t], o[t][c * 4 + i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) now[i] = next[i];
        }
      }
    }
    __syncthreads();
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
// The launch's kernel, by the rows that an average sequence has for one kv head.
struct Plan {
  int rows;      // a tile's
  bool shared;   // attend_shared_kernel (else the streaming one)
  int blocks;    // workgroups that fill the card: those that 256 CUs hold at once
};
Plan plan_for(int T, int n_seq, int hq, int hkv, int D) {
  const int64_t rows = ((int64_t)T * (hq / hkv) + n_seq - 1) / n_seq;
  if (rows <= 16) return {16, false, 512};
  if (rows <= 64) return {64, true, 512};
  return {128, true, D == 256 ? 256 : 512};
}

int target_items(int blocks, int hkv) { return std::max(1, blocks / hkv); }

size_t workspace_bytes(const Plan& p, int hkv, int D) {
  const size_t slots = 2 * (size_t)target_items(p.blocks, hkv) * hkv;
  return kArrivedBytes + slots * p.rows * (D + 2) * sizeof(float);
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
  const int64_t grid = std::max<int64_t>(tiles, A.target) * A.c.hkv;   // a tile a workgroup, or A.target runs a head
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
  *bytes = workspace_bytes(plan_for(T, n_seq, hq, hkv, D), hkv, D);
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
