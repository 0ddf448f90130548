// The draft layer's attention over the 8-bit cache on gfx950
// (draft_layer_attend).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attend_tile.h"

namespace {

using namespace dl;

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

__device__ __forceinline__ Range visible(const AttendArgs& A, int p_first, int p_last) {
  Range r{0, 0, 0, 0};
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

// ---------------------------------------------------------------- the kernels
template <int D, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attend_stream_kernel(AttendArgs A) {
  constexpr int R = 16, C = D / 16, kThreads = 64 * W;
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
    auto place = [&](int r, int& pos) {
      const int x = x0 + r;
      pos = r < rows ? q.begin + x / A.group : -1;
      return A.q + (int64_t)(q.row0 + x / A.group) * A.ldq + (head * A.group + x % A.group) * D;
    };
    const Tokens<false> tokens{A.b, A.c, w.seq, head, see, A.window, A.sinks};
    stream_tile<D, W, kOnce>(tokens, from, to, rows, p_first, p_last, A.scale_log2, place, [&](const f32x4 (&o)[1][C], const float (&m)[1], const float (&l)[1]) {
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
      if (w.parts == 1) return;
      __syncthreads();   // lds becomes join_parts' scratch
      join_parts<D, R, kThreads>(A, w, q, x0, rows, head, parts, &lds.join[0]);
    });
  }
}

template <int D, int NQ, int W>
__global__ __launch_bounds__(64 * W, 2) void attend_shared_kernel(AttendArgs A) {
  using S = Shared<D, NQ, W>;
  constexpr int R = S::R, C = D / 16;
  extern __shared__ __align__(16) u32x4 stage[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int head = blockIdx.x % A.c.hkv;
  Walk<R> walk;
  if (!walk.begin(A, blockIdx.x / A.c.hkv)) return;
  for (Segment w; walk.next(A, w);) {
    const Seq q = w.q;
    w.tile = (int)(((int64_t)q.n * A.group + R - 1) / R) - 1 - w.tile;   // the tiles that see most first
    const int x0 = w.tile * R, rows = min(R, q.n * A.group - x0);
    const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;
    // this wave's own rows
    const int mine0 = wave * 16 * NQ;
    const int w_first = q.begin + (x0 + mine0) / A.group, w_last = q.begin + (x0 + min(rows, mine0 + 16 * NQ) - 1) / A.group;

    const Range see = visible(A, p_first, p_last);
    const int from = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.from / w.of));
    const int to = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.to / w.of));
    auto place = [&](int r, int& pos) {
      const int x = x0 + r;
      pos = r < rows ? q.begin + x / A.group : -1;
      return A.q + (int64_t)(q.row0 + x / A.group) * A.ldq + (head * A.group + x % A.group) * D;
    };
    const Tokens<false> tokens{A.b, A.c, w.seq, head, see, A.window, A.sinks};
    shared_tile<D, NQ, W>(tokens, from, to, rows, w_first, w_last, A.scale_log2, place, stage, [&](const f32x4 (&o)[NQ][C], const float (&m)[NQ], const float (&l)[NQ]) {
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
      if (w.parts == 1) return;
      __syncthreads();   // the stages become join_parts' scratch
      join_parts<D, R, S::kThreads>(A, w, q, x0, rows, head, parts, reinterpret_cast<float*>(stage));
      __syncthreads();   // and the next segment's stages
    });
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
  constexpr size_t kLds = std::max(S::kLds, kJoinFloats<S::R, S::kThreads> * sizeof(float));
  static dh::OncePerDevice once;
  const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&attend_shared_kernel<D, NQ, W>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_shared_kernel<D, NQ, W>), grid, dim3(S::kThreads), kLds, s, A);
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
