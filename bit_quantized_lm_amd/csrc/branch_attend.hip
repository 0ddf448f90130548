// Attention of a batch whose sequences share prefixes, over the 8-bit cache, on
// gfx950 (draft_branch_attend).
//
// A group's rows against its prefix, and each sequence's rows against its own
// tokens, are two kinds of items of one launch.  Both leave partial results (sums
// of values, reference and sum of the weights, fp32); a second launch joins a row's
// parts of both kinds.  The members' rows follow each other in memory, so a
// prefix's tiles are packed from all of them as if they were one sequence's, and
// each key and value of the prefix is loaded once for 16, 64 or 128 of them.
#include <algorithm>
#include <cmath>

#include "../../include/draftbranch.h"
#include "attend_tile.h"

namespace {

using namespace dl;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kNoLimit = DL_MAX_POSITIONS;

struct Parts {        // of one kind of items
  float* o;           // [hkv][rows + runs * tile rows][D]
  float2* ml;         // [hkv][rows + runs * tile rows] reference, sum of weights
};

struct BranchArgs {
  Batch b;
  Cache c;
  const int32_t *group_start, *prefix_len;
  int n_groups;
  const uint16_t* q;
  int64_t ldq;
  int hq, group;      // group = hq / hkv
  float scale_log2;   // scale * log2(e)
  int window, sinks;
  uint16_t* out;
  float* lse;
  int runs;           // workgroups a head
  int min_run;        // least units of a run
  int prefix_rows, own_rows;     // of a tile
  int prefix_cost, own_cost;     // units of a group of 32 tokens against a tile
  int64_t rows;       // T * group: rows of a kv head
  Parts prefix, own;
  int32_t* plan;      // units of a run, and from [4] on first unit and units a tile of each item
};

// ------------------------------------------------------------------ the work
// Items: the groups' prefixes, then the sequences' own tokens.  An item's tiles
// cost as many units as the last of them has groups of 32 tokens, times what such a
// group costs; all tiles' units are laid end to end and cut into equal runs, one a
// workgroup.  A run may hold the end of one tile, whole ones and the start of
// another; what it has of a tile is a part.  Row x of a kv head (token row * group +
// head) has its part from run r at place x + r * (rows of a tile): runs that share a
// tile stand that far apart, and two parts never meet.  So no part needs a number,
// and nothing has to be cleared or counted.
struct Item {
  int seq;               // whose table row names the pages
  int row0, n;           // token rows
  int lo, hi;            // tokens at positions lo .. hi - 1
  int p_first, p_last;   // the rows' positions
  int tiles, units;      // units of a tile
};

struct Segment {
  Item item;
  bool prefix;
  int tile, from, to, of, run;
};

__device__ __forceinline__ Range visible(const BranchArgs& A, const Item& t, int p_first, int p_last) {
  Range r{t.lo >> 5, 0, t.lo >> 5, 0};
  const int cap = A.b.max_pages << A.c.page_shift, end = min(min(t.hi, p_last + 1), cap);
  if (end <= t.lo) return r;
  const int top = (end + 31) >> 5;
  if (A.window > 0) {
    const int low = p_first - A.window + 1;
    if (low > t.lo) r.g0 = min(low >> 5, top);
    r.ns = min(max(((min(A.sinks, cap) + 31) >> 5) - r.s0, 0), r.g0 - r.s0);
  }
  r.n = r.ns + top - r.g0;
  return r;
}

__device__ __forceinline__ int prefix_of_group(const BranchArgs& A, int g) { return min(max(A.prefix_len[g], 0), kNoLimit); }

// First and past-the-last sequence of group g.
__device__ __forceinline__ int2 members(const BranchArgs& A, int g) {
  const int a = min(max(A.group_start[g], 0), A.b.n_seq), b = min(A.group_start[g + 1], A.b.n_seq);
  return int2{a, max(a, b)};
}

// The group that sequence s (its own in each lane) is of, or -1.
__device__ __forceinline__ int group_of(const BranchArgs& A, int s) {
  int g = -1;
  if (A.n_groups < 64) {
    const int lane = threadIdx.x & 63, mine = A.group_start[min(lane, A.n_groups)];
    for (int i = 0; i <= A.n_groups; ++i) g += __builtin_amdgcn_readlane(mine, i) <= s;
  } else {   // the last that starts at or before s
    int lo = 0, hi = A.n_groups + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (A.group_start[mid] <= s)
        lo = mid + 1;
      else
        hi = mid;
    }
    g = lo - 1;
  }
  return g < A.n_groups ? g : -1;
}

class Walk {
 public:
  __device__ __forceinline__ void begin(const BranchArgs& A, int run) {
    const int lane = threadIdx.x & 63;
    run_ = run;
    // whether some row does not see the whole of its prefix: only then do the positions of a prefix's rows matter
    placed_ = A.window > 0;
    for (int base = 0; base < A.b.n_seq && !placed_; base += 64) {
      const Item t = own_item(A, min(base + lane, A.b.n_seq - 1));
      placed_ = __any(t.n > 0 && t.p_first + 1 < t.lo);
    }
    float sum = 0.0f;
    for (int base = 0; base < items(A); base += 64) {
      const Item t = item_at(A, base + lane);
      if (base == 0) first_ = t;
      sum += (float)t.tiles * (float)t.units;
    }
    sum = wave_sum(sum);
    // units are counted in 2^shift, so that their sum fits 32 bits
    shift_ = max(0, (int)((__float_as_uint(sum) >> 23) & 255u) - 127 - 27);
    int total = 0;
    for (int base = 0; base < items(A); base += 64) {
      const Item t = base == 0 ? first_ : item_at(A, base + lane);
      total += __builtin_amdgcn_readlane(wave_inclusive_sum(t.tiles * scaled(t.units)), 63);
    }
    per_ = max(max(1, A.min_run >> shift_), (total + A.runs - 1) / A.runs);
    at_ = run * per_;
    end_ = at_ + per_;
  }

  // The plan, for the launch that joins the parts.
  __device__ __forceinline__ void write(const BranchArgs& A) const {
    const int lane = threadIdx.x & 63;
    if (lane == 0) A.plan[0] = per_;
    int before = 0;
    for (int base = 0; base < items(A); base += 64) {
      const Item t = base == 0 ? first_ : item_at(A, base + lane);
      const int each = scaled(t.units), sum = wave_inclusive_sum(t.tiles * each);
      if (base + lane < items(A)) {
        A.plan[4 + 2 * (base + lane)] = before + sum - t.tiles * each;
        A.plan[5 + 2 * (base + lane)] = each;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
  }

  // The run's next segment; false past its last.
  __device__ __forceinline__ bool next(const BranchArgs& A, Segment& g) {
    if (at_ >= end_) return false;
    const int lane = threadIdx.x & 63;
    int at = at_;
    for (int base = 0; base < items(A); base += 64) {
      const Item t = base == 0 ? first_ : item_at(A, base + lane);
      const int each = scaled(t.units), mine = t.tiles * each, sum = wave_inclusive_sum(mine);
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (at < total) {
        const int i = __builtin_ctzll(__ballot(sum > at));
        auto of = [&](int x) { return __builtin_amdgcn_readlane(x, i); };
        g.item = Item{of(t.seq), of(t.row0), of(t.n), of(t.lo), of(t.hi), of(t.p_first), of(t.p_last), of(t.tiles), of(t.units)};
        g.prefix = base + i < A.n_groups;
        g.of = of(each);
        const int start = of(sum) - of(mine);
        g.tile = (at - start) / g.of;
        g.from = at - start - g.tile * g.of;
        g.to = min(g.of, g.from + end_ - at_);
        g.run = run_;
        at_ += g.to - g.from;
        return true;
      }
      at -= total;
    }
    at_ = end_;
    return false;
  }

  __device__ __forceinline__ bool placed() const { return placed_; }

 private:
  Item first_;    // item `lane`
  bool placed_;
  int shift_, per_, run_, at_, end_;

  static __device__ __forceinline__ int items(const BranchArgs& A) { return A.n_groups + A.b.n_seq; }
  __device__ __forceinline__ int scaled(int units) const { return (units + (1 << shift_) - 1) >> shift_; }

  static __device__ __forceinline__ Item own_item(const BranchArgs& A, int s) {
    Item t;
    const Seq q = load_seq(A.b, s);
    const int g = group_of(A, s);
    t.seq = s;
    t.row0 = q.row0;
    t.n = q.n;
    t.lo = g < 0 ? 0 : prefix_of_group(A, max(g, 0));
    t.hi = kNoLimit;
    t.p_first = q.begin;
    t.p_last = q.len - 1;
    // a tile's rows at most, from the last on: how much it sees
    const int rows = min(q.n, A.own_rows / A.group + 2);
    t.tiles = (int)(((int64_t)q.n * A.group + A.own_rows - 1) / A.own_rows);
    t.units = max(visible(A, t, q.len - rows, q.len - 1).n, A.window > 0 ? 1 : 0) * A.own_cost;   // a window may hide all from the last tile alone
    return t;
  }

  __device__ __forceinline__ Item prefix_item(const BranchArgs& A, int g) const {
    Item t;
    const int2 m = members(A, g);
    t.seq = min(m.x, A.b.n_seq - 1);
    t.row0 = min(max(A.b.q_start[m.x], 0), A.b.T);
    t.n = max(min(A.b.q_start[m.y], A.b.T) - t.row0, 0);
    t.lo = 0;
    t.hi = prefix_of_group(A, g);
    t.p_first = t.p_last = kNoLimit;   // behind the prefix
    if (placed_) {
      t.p_last = -1;
      for (int s = m.x; s < m.y; ++s) {
        const Seq q = load_seq(A.b, s);
        if (q.n == 0) continue;
        t.p_first = min(t.p_first, q.begin);
        t.p_last = max(t.p_last, q.len - 1);
      }
    }
    t.tiles = (int)(((int64_t)t.n * A.group + A.prefix_rows - 1) / A.prefix_rows);
    t.units = visible(A, t, t.p_first, t.p_last).n * A.prefix_cost;
    return t;
  }

  __device__ __forceinline__ Item item_at(const BranchArgs& A, int i) const {
    Item t = own_item(A, min(max(i - A.n_groups, 0), A.b.n_seq - 1));   // every lane: group_of is the wave's
    if (i < A.n_groups) t = prefix_item(A, i);
    if (i >= items(A)) t.tiles = t.units = 0;
    return t;
  }
};

// ----------------------------------------------------------------- the parts
template <int D, int R>
struct Tile {
  static constexpr bool kStream = R == 16;
  static constexpr int kPer = kStream ? 1 : R / (16 * kWaves);   // tiles of 16 rows a wave
  static constexpr size_t kJoin = (size_t)kWaves * R * (D + 4 + 2) * 4;   // a wave's sums, references and sums of weights
  static constexpr size_t kLds = kStream ? kJoin : Shared<D, kPer, kWaves>::kLds;
};

template <int D, int R, bool kPrefix>
__device__ __forceinline__ void attend_part(const BranchArgs& A, const Segment& w, bool placed, int head, u32x4* stage) {
  constexpr int C = D / 16;
  const Item& t = w.item;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  const int x0 = w.tile * R, rows = (int)min((int64_t)R, (int64_t)t.n * A.group - x0);
  // positions of rows a .. b of the tile: a sequence's follow each other, a group's are anywhere among its own
  auto first_of = [&](int a) { return kPrefix ? t.p_first : t.p_first + (x0 + a) / A.group; };
  auto last_of = [&](int b) { return kPrefix ? t.p_last : t.p_first + (x0 + b) / A.group; };
  const Range see = visible(A, t, first_of(0), last_of(rows - 1));
  const int from = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.from / w.of));
  const int to = __builtin_amdgcn_readfirstlane((int)((int64_t)see.n * w.to / w.of));
  auto place = [&](int r, int& pos) {
    const int x = x0 + r, row = t.row0 + x / A.group;
    pos = -1;
    if (r < rows) {
      if (!kPrefix) {
        pos = t.p_first + x / A.group;
      } else if (!placed) {
        pos = kNoLimit;
      } else {   // the row's sequence: the last that starts at or before it
        int a = t.seq, b = A.b.n_seq;
        while (b - a > 1) {
          const int mid = (a + b) >> 1;
          if (A.b.q_start[mid] <= row)
            a = mid;
          else
            b = mid;
        }
        const Seq q = load_seq(A.b, a);
        pos = q.begin + row - q.row0;
      }
    }
    return A.q + (int64_t)row * A.ldq + (head * A.group + x % A.group) * D;
  };
  const Tokens<true> tokens{A.b, A.c, t.seq, head, see, A.window, A.sinks, t.lo, t.hi};
  const Parts& to_parts = kPrefix ? A.prefix : A.own;
  const size_t part_row = (size_t)head * (A.rows + (int64_t)A.runs * R) + (size_t)t.row0 * A.group + x0 + (size_t)w.run * R;
  __syncthreads();   // the LDS: the segment before this one
  if constexpr (Tile<D, R>::kStream) {
    // a prefix's codes are read by its other tiles too
    stream_tile<D, kWaves, kPrefix ? 0 : kOnce>(tokens, from, to, rows, first_of(0), last_of(rows - 1), A.scale_log2, place,
                                                [&](const f32x4 (&o)[1][C], const float (&m)[1], const float (&l)[1]) {
      float* sums = reinterpret_cast<float*>(stage);                 // [kWaves][R][D + 4]
      float* ref = sums + kWaves * R * (D + 4);                      // [kWaves][R]
      float* weight = ref + kWaves * R;
      float sum = l[0];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (hi == 0) {
        ref[wave * R + lo] = m[0];
        weight[wave * R + lo] = sum;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) *reinterpret_cast<f32x4*>(sums + (wave * R + lo) * (D + 4) + c * 16 + hi * 4) = o[0][c];
      __syncthreads();
      const int r = tid / (4 * kWaves);   // 16 threads a row
      if (r < rows) {
        float top = ref[r], all = 0.0f, share[kWaves];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) top = fmaxf(top, ref[v * R + r]);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          share[v] = __builtin_amdgcn_exp2f(ref[v * R + r] - top);
          all += weight[v * R + r] * share[v];
        }
#pragma unroll
        for (int e = tid % 16 * 4; e < D; e += 64) {
          f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int v = 0; v < kWaves; ++v) y += share[v] * *reinterpret_cast<const f32x4*>(sums + (v * R + r) * (D + 4) + e);
          *reinterpret_cast<f32x4*>(to_parts.o + (part_row + r) * D + e) = y;
        }
        if (tid % 16 == 0) to_parts.ml[part_row + r] = float2{top, all};
      }
    });
  } else {
    constexpr int N = Tile<D, R>::kPer;
    const int mine0 = wave * 16 * N;
    shared_tile<D, N, kWaves>(tokens, from, to, rows, first_of(mine0), last_of(min(rows, mine0 + 16 * N) - 1), A.scale_log2, place, stage,
                              [&](const f32x4 (&o)[N][C], const float (&m)[N], const float (&l)[N]) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int r = mine0 + u * 16 + lo;
        float sum = l[u];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (r >= rows) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) *reinterpret_cast<f32x4*>(to_parts.o + (part_row + r) * D + c * 16 + hi * 4) = o[u][c];
        if (hi == 0) to_parts.ml[part_row + r] = float2{m[u], sum};
      }
    });
  }
}

template <int D, int RP, int RS>
__global__ __launch_bounds__(kThreads, D == 256 && RS == 16 ? 1 : 2) void branch_parts_kernel(BranchArgs A) {
  extern __shared__ __align__(16) u32x4 stage[];
  const int head = blockIdx.x % A.c.hkv;
  Walk walk;
  walk.begin(A, blockIdx.x / A.c.hkv);
  if (blockIdx.x == 0 && threadIdx.x < 64) walk.write(A);
  for (Segment w; walk.next(A, w);) {
    if (w.prefix)
      attend_part<D, RP, true>(A, w, walk.placed(), head, stage);
    else
      attend_part<D, RS, false>(A, w, false, head, stage);
  }
}

// ---------------------------------------------------------------- the joining
// A row of one query head: W waves take turns at its parts.
template <int D, int W>
__global__ __launch_bounds__(kThreads) void branch_join_kernel(BranchArgs A) {
  constexpr int E = D / 64;   // elements a lane
  __shared__ float sums[kWaves][D], refs[kWaves], weights[kWaves];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int turn = wave % W;
  const int64_t i = (int64_t)blockIdx.x * (kWaves / W) + wave / W;
  const int r = (int)(i / A.hq), h = (int)(i % A.hq), head = h / A.group;
  // the row's sequence: the last that starts at or before it, 64 a look
  int s = -1;
  for (int base = 0; base < A.b.n_seq; base += 64) {
    const int before = __popcll(__ballot(base + lane < A.b.n_seq && A.b.q_start[min(base + lane, A.b.n_seq - 1)] <= r));
    s += before;
    if (before < 64) break;
  }
  const Seq q = load_seq(A.b, max(s, 0));
  const bool there = s >= 0 && r < A.b.T && r >= q.row0 && r < q.row0 + q.n;
  if (W == 1 && !there) return;   // more waves: all of them or none
  const int g = __builtin_amdgcn_readfirstlane(group_of(A, s));
  const int64_t x = (int64_t)r * A.group + h % A.group;
  const int per = A.plan[0];
  auto parts_of = [&](int item, int row0, int rows, int R, int& first) {
    if (r < row0 || r >= row0 + rows) return 0;   // groups and sequences that do not fit each other
    const int units = A.plan[5 + 2 * item], at = A.plan[4 + 2 * item] + (int)((x - (int64_t)row0 * A.group) / R) * units;
    first = at / per;
    return units == 0 ? 0 : (at + units - 1) / per - first + 1;
  };
  int first_prefix = 0, first_own = 0, n_prefix = 0, n_own = 0;
  if (there) {
    if (g >= 0) {
      const int2 m = members(A, g);
      const int row0 = min(max(A.b.q_start[m.x], 0), A.b.T);
      n_prefix = parts_of(g, row0, min(A.b.q_start[m.y], A.b.T) - row0, A.prefix_rows, first_prefix);
    }
    n_own = parts_of(A.n_groups + s, q.row0, q.n, A.own_rows, first_own);
  }
  const int n = n_prefix + n_own;
  const size_t prefix_at = (size_t)head * (A.rows + (int64_t)A.runs * A.prefix_rows) + x + (size_t)first_prefix * A.prefix_rows;
  const size_t own_at = (size_t)head * (A.rows + (int64_t)A.runs * A.own_rows) + x + (size_t)first_own * A.own_rows;
  float top = kLowest, sum = 0.0f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.0f;
  for (int base = turn; base < n; base += 64 * W) {
    // lane k: part base + k W
    const int k = base + lane * W;
    const bool of_prefix = k < n_prefix;
    const size_t at = of_prefix ? prefix_at + (size_t)k * A.prefix_rows : own_at + (size_t)(k - n_prefix) * A.own_rows;
    float2 ml = {kLowest, 0.0f};
    if (k < n) ml = (of_prefix ? A.prefix.ml : A.own.ml)[at];
    const float next = fmaxf(top, wave_max(ml.x)), share = __builtin_amdgcn_exp2f(ml.x - next), down = __builtin_amdgcn_exp2f(top - next);
    sum = sum * down + wave_sum(k < n ? share * ml.y : 0.0f);
    top = next;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= down;
    const int count = min(64, (n - base + W - 1) / W);
    for (int j0 = 0; j0 < count; j0 += 8) {   // eight parts' loads under way together; past the last, that once more with no share
      float x[8][E], w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at_j = min(j0 + j, count - 1), kj = base + at_j * W;
        const float* o = kj < n_prefix ? A.prefix.o + (prefix_at + (size_t)kj * A.prefix_rows) * D : A.own.o + (own_at + (size_t)(kj - n_prefix) * A.own_rows) * D;
        w[j] = j0 + j < count ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(share), at_j)) : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][e] = o[lane * E + e];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(w[j], x[j][e], y[e]);
    }
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = y[e];
    if (lane == 0) refs[wave] = top, weights[wave] = sum;
    __syncthreads();
    if (turn > 0 || !there) return;
    float all = refs[wave];
#pragma unroll
    for (int v = 1; v < W; ++v) all = fmaxf(all, refs[wave + v]);
    sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float share = __builtin_amdgcn_exp2f(refs[wave + v] - all);
      sum = fmaf(share, weights[wave + v], sum);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = fmaf(share, sums[wave + v][lane * E + e], y[e]);
    }
    top = all;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* to = A.out + ((size_t)r * A.hq + h) * D + lane * E;
  if constexpr (E == 1) {
    *to = (uint16_t)bf16_pair(y[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(to + e) = bf16_pair(y[e] * inv, y[e + 1] * inv);
  }
  if (lane == 0 && A.lse) A.lse[(size_t)r * A.hq + h] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
}

// ------------------------------------------------------------------- launch
// Tiles by the rows that an average group (and an average sequence) has for one
// kv head.
int tile_rows(int64_t rows, int D) { return rows <= 16 ? 16 : rows <= 64 || D == 256 ? 64 : 128; }
int runs_of(int hkv, int D) { return std::max(1, (D == 256 ? 256 : 512) / hkv); }
// What 32 tokens cost a tile, as a multiple of what they cost one of 16 rows.
int cost_of(int rows) { return rows == 16 ? 1 : rows == 64 ? 2 : 4; }

constexpr size_t kAlign = 256;
size_t rounded(size_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }
size_t plan_bytes(int64_t items) { return rounded((4 + 2 * items) * 4); }
size_t parts_rows(int64_t rows, int hkv, int D, int R) { return (size_t)hkv * (rows + (int64_t)runs_of(hkv, D) * R); }
size_t workspace_bytes(int64_t rows, int64_t items, int hkv, int D, int RP, int RS) {
  size_t bytes = plan_bytes(items);
  for (int R : {RP, RS}) bytes += rounded(parts_rows(rows, hkv, D, R) * D * 4) + rounded(parts_rows(rows, hkv, D, R) * 8);
  return bytes;
}

template <int D, int RP, int RS>
int launch_parts(const BranchArgs& A, hipStream_t s) {
  constexpr size_t kLds = std::max(Tile<D, RP>::kLds, Tile<D, RS>::kLds);
  static dh::OncePerDevice once;
  const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&branch_parts_kernel<D, RP, RS>), kLds);
  if (e != hipSuccess) return dh::fail(DH_EHIP, "branch_parts_kernel: %s", hipGetErrorString(e));
  hipLaunchKernelGGL((branch_parts_kernel<D, RP, RS>), dim3((unsigned)(A.runs * A.c.hkv)), dim3(kThreads), kLds, s, A);
  return launched("branch_parts_kernel");
}

template <int D>
int launch(const BranchArgs& A, hipStream_t s) {
  int rc;
  if (A.prefix_rows == 16)
    rc = launch_parts<D, 16, 16>(A, s);
  else if (A.prefix_rows == 64)
    rc = A.own_rows == 16 ? launch_parts<D, 64, 16>(A, s) : launch_parts<D, 64, 64>(A, s);
  else if constexpr (D == 256)
    return dh::fail(DH_EUNSUP, "attend: no tile of %d rows", A.prefix_rows);
  else
    rc = A.own_rows == 16 ? launch_parts<D, 128, 16>(A, s) : A.own_rows == 64 ? launch_parts<D, 128, 64>(A, s) : launch_parts<D, 128, 128>(A, s);
  if (rc) return rc;
  const int64_t rows = (int64_t)A.b.T * A.hq;
  if (rows <= 2048)
    hipLaunchKernelGGL((branch_join_kernel<D, kWaves>), dim3((unsigned)rows), dim3(kThreads), 0, s, A);
  else
    hipLaunchKernelGGL((branch_join_kernel<D, 1>), dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kThreads), 0, s, A);
  return launched("branch_join_kernel");
}

}  // namespace

extern "C" {

int draft_branch_attend_workspace_bytes(int T, int n_seq, int hq, int hkv, int D, size_t* bytes) {
  if (!bytes) return dh::fail(DH_EINVAL, "attend_workspace_bytes: null pointer");
  int rc = check_heads("attend_workspace_bytes", hq, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows("attend_workspace_bytes", T, n_seq))) return rc;
  // fewer sequences or groups have more rows each, up to all T in one
  const int64_t rows = (int64_t)T * (hq / hkv);
  const int R = tile_rows(rows, D);
  *bytes = workspace_bytes(rows, 2 * (int64_t)n_seq, hkv, D, R, R);
  return dh::ok();
}

int draft_branch_attend(const void* q, int64_t ldq, const uint8_t* k_codes, const uint8_t* v_codes,
                        const float* k_scale, const float* v_scale, int n_pages, int page, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* table, int n_seq, int max_pages,
                        const int32_t* group_start, const int32_t* prefix_len, int n_groups, int T, int hq, int hkv,
                        int D, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes_given, void* stream) {
  const char* who = "attend";
  int rc = check_heads(who, hq, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows(who, T, n_seq))) return rc;
  BranchArgs A{};
  A.b = Batch{q_start, kv_len, table, n_seq, max_pages, T};
  A.c = Cache{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes), const_cast<float*>(k_scale),
              const_cast<float*>(v_scale), n_pages, page_shift_of(page), hkv};
  if ((rc = check_cache(who, A.c, page, A.b))) return rc;
  if (n_groups < 1 || n_groups > n_seq) return dh::fail(DH_ESHAPE, "attend: n_groups must be in 1..n_seq (got %d of %d)", n_groups, n_seq);
  if (!group_start || !prefix_len) return dh::fail(DH_EINVAL, "attend: null pointer");
  if (!aligned(group_start, 4) || !aligned(prefix_len, 4)) return dh::fail(DH_EINVAL, "attend: group_start and prefix_len must be 4-byte aligned");
  if (!(scale > 0.0f) || !std::isfinite(scale)) return dh::fail(DH_EINVAL, "attend: scale must be finite and > 0");
  if (window < 0 || sinks < 0) return dh::fail(DH_EINVAL, "attend: window and sinks must be >= 0 (got %d, %d)", window, sinks);
  if (T == 0) return dh::ok();
  if ((rc = check_stride(who, "q", q, ldq, (int64_t)hq * D))) return rc;
  if (!out || !aligned(out, 16)) return dh::fail(DH_EINVAL, "attend: out must be a 16-byte aligned pointer");
  if (lse && !aligned(lse, 4)) return dh::fail(DH_EINVAL, "attend: lse must be 4-byte aligned");
  if (!workspace || !aligned(workspace, 16)) return dh::fail(DH_EINVAL, "attend: workspace must be a 16-byte aligned pointer");
  A.group = hq / hkv;
  A.rows = (int64_t)T * A.group;
  A.prefix_rows = tile_rows((A.rows + n_groups - 1) / n_groups, D);
  A.own_rows = tile_rows((A.rows + n_seq - 1) / n_seq, D);
  const size_t need = workspace_bytes(A.rows, (int64_t)n_groups + n_seq, hkv, D, A.prefix_rows, A.own_rows);
  if (workspace_bytes_given < need)
    return dh::fail(DH_EINVAL, "attend: workspace of %zu bytes is below the %zu needed", workspace_bytes_given, need);
  A.group_start = group_start;
  A.prefix_len = prefix_len;
  A.n_groups = n_groups;
  A.q = static_cast<const uint16_t*>(q);
  A.ldq = ldq;
  A.hq = hq;
  A.scale_log2 = scale * 1.44269504088896f;
  A.window = window < DL_MAX_POSITIONS ? window : 0;   // past every position: no window
  A.sinks = std::min(sinks, DL_MAX_POSITIONS);
  A.out = static_cast<uint16_t*>(out);
  A.lse = lse;
  A.runs = runs_of(hkv, D);
  A.min_run = 8;
  A.prefix_cost = cost_of(A.prefix_rows);
  A.own_cost = cost_of(A.own_rows);
  unsigned char* at = static_cast<unsigned char*>(workspace);
  auto take = [&](size_t bytes) {
    unsigned char* p = at;
    at += rounded(bytes);
    return p;
  };
  A.plan = reinterpret_cast<int32_t*>(take(plan_bytes((int64_t)n_groups + n_seq)));
  for (Parts* p : {&A.prefix, &A.own}) {
    const size_t rows = parts_rows(A.rows, hkv, D, p == &A.prefix ? A.prefix_rows : A.own_rows);
    p->o = reinterpret_cast<float*>(take(rows * D * 4));
    p->ml = reinterpret_cast<float2*>(take(rows * 8));
  }
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  switch (D) {
    case 64: return launch<64>(A, st);
    case 128: return launch<128>(A, st);
    default: return launch<256>(A, st);
  }
}

}  // extern "C"
