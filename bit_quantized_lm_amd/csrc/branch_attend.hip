// Attention of a batch whose sequences share prefixes, over the 8-bit cache, on
// gfx950 (draft_branch_attend).
//
// A group's rows against its prefix, and each sequence's rows against its own
// tokens, are two kinds of items of one launch.  Both leave partial results (sums
// of values, reference and sum of the weights, fp32); a second launch joins a row's
// parts.  The members' rows follow each other in memory, so a prefix's tiles are
// packed from all of them as if they were one sequence's, and each key and value of
// the prefix is loaded once for up to 128 of them.
#include <algorithm>
#include <cmath>

#include "../../include/draftbranch.h"
#include "attend_tile.h"

namespace {

using namespace dl;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kNoLimit = DL_MAX_POSITIONS;
constexpr int kStreamRows = 16, kSmallRows = 64;

// Partial results of one kind of items and of tiles: row x of a head from run r at
// place x + r * (rows of a tile).  Runs that share a tile stand that far apart, so two
// parts never meet: no part needs a number, and nothing has to be cleared or counted.
struct Parts {
  float* o;           // [hkv][places][D]
  float2* ml;         // [hkv][places] reference, sum of weights
};
enum Line { kShared, kStream };   // tiles of a workgroup, tiles of a wave

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
  int64_t places[2];  // a head's, by line
  Parts prefix[2], own[2];
  int32_t* plan;      // left by the first launch for the second: units of a run by line, then 8 numbers an item
};

// ------------------------------------------------------------------ the work
// Items: the sequences' own tokens, then the groups' prefixes.  An item's rows (query
// heads of one kv head, token after token) are cut into tiles of H = 128 (heads of
// 256: 64) and a rest; up to 16 rows are one wave's (stream_tile), up to 64 and up to
// H a workgroup's (shared_tile), whatever the other items have.  Where the members of
// a group have H rows each on average, sharing saves no time (such tiles are bound by
// the matrix units) and joining costs some, so the prefix's tokens are the
// sequences' own then (16 prompts of 112 rows over 6,000 tokens: 345 us so, 517 apart).
//
// All tiles of a line are laid end to end, each as long as it is thought to take, and
// cut into equal runs: a workgroup's, or a wave's, which walks its own segments and
// waits for no other.  A run may hold the end of one tile, whole ones and the start of
// another; what it has of a tile is a part.  The workgroups are divided between the
// lines by what the lines take.
struct Item {
  int seq, lead;         // whose table rows name the pages of the own and of the shared tokens
  int row0, n;           // token rows
  int split;             // positions below are the shared ones
  int sees;              // 1: the own tokens, 2: the shared ones
  int p_first, p_last;   // the rows' positions
  int groups;            // of 32 tokens that a tile sees at most
};

// Lengths of tiles in units of about 0.1 us of a workgroup (of a wave, for the
// stream): what a tile's beginning and end take, and what a group of 32 tokens
// takes: on a full card a tile of 128 rows with heads of 128 takes 1.2 us a group.
template <int D>
struct Cost {
  static constexpr int kRows = D == 256 ? 64 : 128;     // H
  static __host__ __device__ constexpr int per_group(int rows) {
    return std::max(1, (rows <= kStreamRows ? 16 : rows <= kSmallRows ? 7 : 12) * D / 128);
  }
  static __host__ __device__ constexpr int begin(int rows) { return rows <= kStreamRows ? 40 : 50; }
  static __device__ __forceinline__ int of(int rows, int groups) { return groups == 0 ? 0 : begin(rows) + groups * per_group(rows); }
};

// An item's tiles: `full` ones of H rows, then one of `rest`.
template <int D>
struct Shape {
  int full, rest, each, last;    // tiles and their units
  __device__ __forceinline__ Shape(int64_t rows, int groups, int shift) {
    constexpr int H = Cost<D>::kRows;
    full = (int)(rows / H);
    rest = (int)(rows % H);
    auto scaled = [&](int units) { return (int)(((int64_t)units + (1 << shift) - 1) >> shift); };
    each = scaled(Cost<D>::of(H, groups));
    last = rest == 0 ? 0 : scaled(Cost<D>::of(rest, groups));
    if (groups == 0) full = rest = 0;
  }
  __device__ __forceinline__ bool streams() const { return rest <= kStreamRows; }
  __device__ __forceinline__ int units(Line line) const {
    return line == kStream ? (streams() ? last : 0) : full * each + (streams() ? 0 : last);
  }
};

__device__ __forceinline__ Range visible(const BranchArgs& A, int lo, int hi, int p_first, int p_last) {
  Range r{lo >> 5, 0, lo >> 5, 0};
  const int cap = A.b.max_pages << A.c.page_shift, end = min(min(hi, p_last + 1), cap);
  if (end <= lo) return r;
  const int top = (end + 31) >> 5;
  if (A.window > 0) {
    const int low = p_first - A.window + 1;
    if (low > lo) r.g0 = min(low >> 5, top);
    r.ns = min(max(((min(A.sinks, cap) + 31) >> 5) - r.s0, 0), r.g0 - r.s0);
  }
  r.n = r.ns + top - r.g0;
  return r;
}
__device__ __forceinline__ Range visible_own(const BranchArgs& A, const Item& t, int p_first, int p_last) {
  return t.sees & 1 ? visible(A, t.split, kNoLimit, p_first, p_last) : Range{};
}
__device__ __forceinline__ Range visible_shared(const BranchArgs& A, const Item& t, int p_first, int p_last) {
  return t.sees & 2 ? visible(A, 0, t.split, p_first, p_last) : Range{};
}

// The group that sequence s (its own in each lane; every lane calls it) is of, or -1.
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

struct Members {
  int first, last;    // sequences first .. last - 1
  int row0, n;        // token rows
  int prefix;
  bool whole;         // its prefix's tokens count as the sequences' own
};
template <int D>
__device__ __forceinline__ Members members_of(const BranchArgs& A, int g) {
  Members r;
  r.first = min(max(A.group_start[g], 0), A.b.n_seq);
  r.last = max(r.first, min(A.group_start[g + 1], A.b.n_seq));
  r.row0 = min(max(A.b.q_start[r.first], 0), A.b.T);
  r.n = max(min(A.b.q_start[r.last], A.b.T) - r.row0, 0);
  r.prefix = min(max(A.prefix_len[g], 0), kNoLimit);
  r.whole = (int64_t)r.n * A.group >= (int64_t)Cost<D>::kRows * (r.last - r.first);
  return r;
}

__device__ __forceinline__ void write_lse(float* lse, size_t row, float ref, float sum) {
  if (lse) lse[row] = sum == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
}

struct Segment {
  Item item;
  Line line;
  int tile, from, to, of, run;
};

template <int D>
class Walk {
 public:
  // The plan, which every wave computes alike from the lengths.
  __device__ __forceinline__ void begin(const BranchArgs& A) {
    const int lane = threadIdx.x & 63;
    // whether some row does not see the whole of its prefix: only then do the positions of a prefix's rows matter
    placed_ = A.window > 0;
    for (int base = 0; base < A.b.n_seq; base += 64) {
      const Item t = own_item(A, base + lane);
      if (base == 0) first_ = t;
      placed_ |= __any(t.n > 0 && t.p_first + 1 < t.split) != 0;
    }
    if (lane >= A.b.n_seq && lane < items(A)) first_ = prefix_item(A, lane - A.b.n_seq);
    float sum[2] = {0.0f, 0.0f};
    for (int base = 0; base < items(A); base += 64) {
      const Item t = block(A, base);
      const Shape<D> s(rows_of(A, t), t.groups, 0);
      sum[kShared] += (float)s.full * (float)s.each + (s.streams() ? 0.0f : (float)s.last);
      sum[kStream] += s.streams() ? (float)s.last : 0.0f;
    }
    sum[0] = wave_sum(sum[0]);
    sum[1] = wave_sum(sum[1]);
    // lengths are counted in 2^shift units, so that their sums fit 32 bits
    shift_ = max(0, (int)((__float_as_uint(fmaxf(sum[0], sum[1])) >> 23) & 255u) - 127 - 27);
    int total[2] = {0, 0};
    for (int base = 0; base < items(A); base += 64) {
      const Item t = block(A, base);
      const Shape<D> s(rows_of(A, t), t.groups, shift_);
      for (int l = 0; l < 2; ++l) total[l] += __builtin_amdgcn_readlane(wave_inclusive_sum(s.units((Line)l)), 63);
    }
    const float by_wave = sum[kStream] * (1.0f / kWaves);
    shared_ = sum[kShared] == 0.0f ? 0 : by_wave == 0.0f ? A.runs
              : min(max((int)(A.runs * (sum[kShared] / (sum[kShared] + by_wave)) + 0.5f), 1), A.runs - 1);
    shared_ = __builtin_amdgcn_readfirstlane(shared_);
    const int runs[2] = {max(shared_, 1), max((A.runs - shared_) * kWaves, 1)};
    // a part shorter than four groups' time costs more to begin and to join than it saves
    for (int l = 0; l < 2; ++l) {
      const int rows = l == kStream ? kStreamRows : kSmallRows;
      per_[l] = max(max((Cost<D>::begin(rows) + 4 * Cost<D>::per_group(rows)) >> shift_, 1), (total[l] + runs[l] - 1) / runs[l]);
    }
  }

  // Workgroup `number` of a head: which line it works on, and which run of it this wave has.
  __device__ __forceinline__ Line take(int number) {
    const Line line = number < shared_ ? kShared : kStream;
    run_ = line == kShared ? number : (number - shared_) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    at_ = run_ * per_[line];
    end_ = at_ + per_[line];
    return line;
  }

  // What the launch that joins the parts has to know.
  __device__ __forceinline__ void write(const BranchArgs& A) const {
    const int lane = threadIdx.x & 63;
    if (lane == 0) *reinterpret_cast<int4*>(A.plan) = int4{per_[0], per_[1], shift_, 0};
    int before[2] = {0, 0};
    for (int base = 0; base < items(A); base += 64) {
      const Item t = block(A, base);
      const Shape<D> s(rows_of(A, t), t.groups, shift_);
      int at[2];
      for (int l = 0; l < 2; ++l) {
        const int mine = s.units((Line)l), sum = wave_inclusive_sum(mine);
        at[l] = before[l] + sum - mine;
        before[l] += __builtin_amdgcn_readlane(sum, 63);
      }
      if (base + lane < items(A)) {
        int4* to = reinterpret_cast<int4*>(A.plan + 8 + 8 * (base + lane));
        to[0] = int4{at[0], at[1], t.groups, t.n};
        to[1] = int4{t.row0, t.split == 0 || t.sees == 3, 0, 0};
      }
    }
  }

  // The run's next segment; false past its last.
  __device__ __forceinline__ bool next(const BranchArgs& A, Line line, Segment& g) {
    if (at_ >= end_) return false;
    const int lane = threadIdx.x & 63;
    int at = at_;
    for (int base = 0; base < items(A); base += 64) {
      const Item t = block(A, base);
      const Shape<D> s(rows_of(A, t), t.groups, shift_);
      const int mine = s.units(line), sum = wave_inclusive_sum(mine);
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (at < total) {
        const int i = __builtin_ctzll(__ballot(sum > at));
        auto of = [&](int x) { return __builtin_amdgcn_readlane(x, i); };
        g.item = Item{of(t.seq), of(t.lead), of(t.row0), of(t.n), of(t.split), of(t.sees), of(t.p_first), of(t.p_last), of(t.groups)};
        const int full = of(s.full), each = of(s.each), last = of(s.last);
        at -= of(sum) - of(mine);
        g.line = line;
        g.run = run_;
        g.tile = line == kStream ? full : min(at / each, full);
        g.of = g.tile < full ? each : last;
        g.from = at - (line == kStream ? 0 : g.tile * each);
        g.to = min(g.of, g.from + end_ - at_);
        at_ += g.to - g.from;
        return true;
      }
      at -= total;
    }
    at_ = end_;
    return false;
  }

  __device__ __forceinline__ bool placed() const { return placed_; }

  static __device__ __forceinline__ int64_t rows_of(const BranchArgs& A, const Item& t) { return (int64_t)t.n * A.group; }

 private:
  Item first_;    // item `lane`
  bool placed_;
  int shift_, per_[2], shared_, run_, at_, end_;   // shared_: workgroups a head of the shared line

  static __device__ __forceinline__ int items(const BranchArgs& A) { return A.n_groups + A.b.n_seq; }

  static __device__ __forceinline__ Item own_item(const BranchArgs& A, int i) {
    Item t;
    const int s = min(i, A.b.n_seq - 1);
    const Seq q = load_seq(A.b, s);
    const int g = group_of(A, s);
    const Members group = members_of<D>(A, max(g, 0));
    t.seq = s;
    t.lead = min(group.first, A.b.n_seq - 1);
    t.row0 = q.row0;
    t.n = i < A.b.n_seq ? q.n : 0;
    t.split = g < 0 ? 0 : group.prefix;
    t.sees = g >= 0 && group.whole ? 3 : 1;
    t.p_first = q.begin;
    t.p_last = q.len - 1;
    // the last tile's rows at most: what they see is the longest; a window may hide all from that tile alone
    const int first = q.len - min(q.n, Cost<D>::kRows / A.group + 2);
    t.groups = q.n == 0 ? 0 : max(visible_own(A, t, first, t.p_last).n + visible_shared(A, t, first, t.p_last).n, A.window > 0 ? 1 : 0);
    return t;
  }

  __device__ __forceinline__ Item prefix_item(const BranchArgs& A, int g) const {
    Item t;
    const Members group = members_of<D>(A, g);
    t.seq = t.lead = min(group.first, A.b.n_seq - 1);
    t.row0 = group.row0;
    t.n = group.whole ? 0 : group.n;
    t.split = group.prefix;
    t.sees = 2;
    t.p_first = t.p_last = kNoLimit;   // behind the prefix
    if (placed_) {
      t.p_last = -1;
      for (int s = group.first; s < group.last; ++s) {
        const Seq q = load_seq(A.b, s);
        if (q.n == 0) continue;
        t.p_first = min(t.p_first, q.begin);
        t.p_last = max(t.p_last, q.len - 1);
      }
    }
    t.groups = visible_shared(A, t, t.p_first, t.p_last).n;
    return t;
  }

  // Items base .. base + 63, one a lane; those past the last have no rows.
  __device__ __forceinline__ Item block(const BranchArgs& A, int base) const {
    if (base == 0) return first_;
    const int i = base + (threadIdx.x & 63);
    Item t = own_item(A, i);   // in every lane: group_of is the wave's
    if (i >= A.b.n_seq && i < items(A)) t = prefix_item(A, i - A.b.n_seq);
    return t;
  }
};

// ----------------------------------------------------------------- the parts
template <int D, int R>
__device__ __forceinline__ void attend_part(const BranchArgs& A, const Segment& w, bool placed, int head, u32x4* stage) {
  constexpr int C = D / 16;
  const Item& t = w.item;
  const bool prefix = t.sees == 2;
  const int lane = threadIdx.x & 63, hi = lane >> 4, lo = lane & 15;
  const int x0 = w.tile * Cost<D>::kRows, rows = (int)min((int64_t)R, (int64_t)t.n * A.group - x0);
  // positions of rows a .. b of the tile: a sequence's follow each other, a group's are anywhere among its own
  auto first_of = [&](int a) { return prefix ? t.p_first : t.p_first + (x0 + a) / A.group; };
  auto last_of = [&](int b) { return prefix ? t.p_last : t.p_first + (x0 + b) / A.group; };
  const Range own = visible_own(A, t, first_of(0), last_of(rows - 1)), shared = visible_shared(A, t, first_of(0), last_of(rows - 1));
  const int n = own.n + shared.n;
  const int from = __builtin_amdgcn_readfirstlane((int)((int64_t)n * w.from / w.of));
  const int to = __builtin_amdgcn_readfirstlane((int)((int64_t)n * w.to / w.of));
  auto place = [&](int r, int& pos) {
    const int x = x0 + r, row = t.row0 + x / A.group;
    pos = -1;
    if (r < rows) {
      if (!prefix) {
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
  const Tokens<true> tokens{A.b, A.c, t.seq, head, own, A.window, A.sinks, shared, t.lead, t.split};
  // a tile's only part of rows that have no prefix apart is the result
  const bool done = w.from == 0 && w.to == w.of && (t.sees == 3 || (t.sees == 1 && t.split == 0));
  const Parts& to_parts = (prefix ? A.prefix : A.own)[w.line];
  const size_t part_row = (size_t)head * A.places[w.line] + (size_t)t.row0 * A.group + x0 + (size_t)w.run * (R == kStreamRows ? R : Cost<D>::kRows);
  auto put = [&](int r, const f32x4 (&o)[C], float ref, float sum) {   // row r, a lane's elements
    if (r >= rows) return;
    if (done) {
      const int x = x0 + r;
      const size_t row = (size_t)(t.row0 + x / A.group) * A.hq + head * A.group + x % A.group;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int c = 0; c < C; ++c)
        *reinterpret_cast<u32x2*>(A.out + row * D + c * 16 + hi * 4) = u32x2{bf16_pair(o[c][0] * inv, o[c][1] * inv), bf16_pair(o[c][2] * inv, o[c][3] * inv)};
      if (hi == 0) write_lse(A.lse, row, ref, sum);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) *reinterpret_cast<f32x4*>(to_parts.o + (part_row + r) * D + c * 16 + hi * 4) = o[c];
      if (hi == 0) to_parts.ml[part_row + r] = float2{ref, sum};
    }
  };
  if constexpr (R == kStreamRows) {
    stream_tile<D, 1, kOnce>(tokens, from, to, rows, first_of(0), last_of(rows - 1), A.scale_log2, place,
                             [&](const f32x4 (&o)[1][C], const float (&m)[1], const float (&l)[1]) {
      float sum = l[0];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      put(lo, o[0], m[0], sum);
    });
  } else {
    constexpr int N = R / (16 * kWaves);
    const int mine0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 16 * N;
    __syncthreads();   // the LDS: the segment before this one
    shared_tile<D, N, kWaves>(tokens, from, to, rows, first_of(mine0), last_of(min(rows, mine0 + 16 * N) - 1), A.scale_log2, place, stage,
                              [&](const f32x4 (&o)[N][C], const float (&m)[N], const float (&l)[N]) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        float sum = l[u];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        put(mine0 + u * 16 + lo, o[u], m[u], sum);
      }
    });
  }
}

template <int D>
constexpr size_t kLds = std::max(Shared<D, 1, kWaves>::kLds, Shared<D, Cost<D>::kRows / (16 * kWaves), kWaves>::kLds);

template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void branch_parts_kernel(BranchArgs A) {
  extern __shared__ __align__(16) u32x4 stage[];
  const int head = blockIdx.x % A.c.hkv;
  Walk<D> walk;
  walk.begin(A);
  if (blockIdx.x == 0 && threadIdx.x < 64) walk.write(A);
  const Line line = walk.take(blockIdx.x / A.c.hkv);
  for (Segment w; walk.next(A, line, w);) {
    if (line == kStream) {
      attend_part<D, kStreamRows>(A, w, walk.placed(), head, stage);
    } else {
      constexpr int H = Cost<D>::kRows;
      if (H == kSmallRows || Walk<D>::rows_of(A, w.item) - (int64_t)w.tile * H <= kSmallRows)
        attend_part<D, kSmallRows>(A, w, walk.placed(), head, stage);
      else
        attend_part<D, H>(A, w, walk.placed(), head, stage);
    }
  }
}

// ---------------------------------------------------------------- the joining
// A row of one query head: W waves take turns at its parts.
template <int D, int W>
__global__ __launch_bounds__(kThreads) void branch_join_kernel(BranchArgs A) {
  constexpr int E = D / 64, H = Cost<D>::kRows;   // elements a lane
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
  const int g = __builtin_amdgcn_readfirstlane(group_of(A, s));
  const Seq q = load_seq(A.b, max(s, 0));
  if (s < 0 || r >= A.b.T || r < q.row0 || r >= q.row0 + q.n) return;   // all waves of a row, which are a workgroup's, or the one
  const int64_t x = (int64_t)r * A.group + h % A.group;
  const int4 plan = *reinterpret_cast<const int4*>(A.plan);
  // an item's parts of this row: where the first is, how far apart they are, how many
  struct Run {
    const float* o;
    const float2* ml;
    int step, n;
    bool alone;
  };
  auto parts_of = [&](int item, const Parts (&all)[2]) {
    const int4* of = reinterpret_cast<const int4*>(A.plan + 8 + 8 * item);
    const int4 a = of[0], b = of[1];
    Run p{nullptr, nullptr, 0, 0, b.y != 0};
    const int64_t y = x - (int64_t)b.x * A.group, rows = (int64_t)a.w * A.group;
    if (y < 0 || y >= rows || a.z == 0) return p;   // nothing to see, or groups and sequences that do not fit each other
    const Shape<D> shape(rows, a.z, plan.z);
    const int tile = min((int)(y / H), shape.full);
    const Line line = tile == shape.full && shape.streams() ? kStream : kShared;
    const int length = tile < shape.full ? shape.each : shape.last, at = line == kStream ? a.y : a.x + tile * shape.each;
    const int per = line == kStream ? plan.y : plan.x, first = at / per;
    p.step = line == kStream ? kStreamRows : H;
    p.n = (at + length - 1) / per - first + 1;
    const size_t place = (size_t)head * A.places[line] + x + (size_t)first * p.step;
    p.o = all[line].o + place * D;
    p.ml = all[line].ml + place;
    return p;
  };
  const Run own = parts_of(s, A.own);
  Run prefix{nullptr, nullptr, 0, 0, false};
  if (g >= 0) prefix = parts_of(A.b.n_seq + g, A.prefix);
  if (own.alone && own.n == 1) return;   // the result already
  const int n = prefix.n + own.n;
  float top = kLowest, sum = 0.0f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.0f;
  for (int base = turn; base < n; base += 64 * W) {
    // lane k: part base + k W
    const int k = base + lane * W;
    float2 ml = {kLowest, 0.0f};
    if (k < n) ml = k < prefix.n ? prefix.ml[(size_t)k * prefix.step] : own.ml[(size_t)(k - prefix.n) * own.step];
    const float next = fmaxf(top, wave_max(ml.x)), share = __builtin_amdgcn_exp2f(ml.x - next), down = __builtin_amdgcn_exp2f(top - next);
    sum = sum * down + wave_sum(k < n ? share * ml.y : 0.0f);
    top = next;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= down;
    const int count = min(64, (n - base + W - 1) / W);
    for (int j0 = 0; j0 < count; j0 += 8) {   // eight parts' loads under way together; past the last, that once more with no share
      float v[8][E], by[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at_j = min(j0 + j, count - 1), kj = base + at_j * W;
        const float* o = kj < prefix.n ? prefix.o + (size_t)kj * prefix.step * D : own.o + (size_t)(kj - prefix.n) * own.step * D;
        by[j] = j0 + j < count ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(share), at_j)) : 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = o[lane * E + e];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(by[j], v[j][e], y[e]);
    }
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = y[e];
    if (lane == 0) refs[wave] = top, weights[wave] = sum;
    __syncthreads();
    if (turn > 0) return;
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
  const size_t row = (size_t)r * A.hq + h;
  uint16_t* to = A.out + row * D + lane * E;
  if constexpr (E == 1) {
    *to = (uint16_t)bf16_pair(y[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(to + e) = bf16_pair(y[e] * inv, y[e + 1] * inv);
  }
  if (lane == 0) write_lse(A.lse, row, top, sum);
}

// ------------------------------------------------------------------- launch
// Workgroups that run at once, by head; two at least, so that both lines have one.
int runs_of(int hkv, int D) { return std::max(2, (D == 256 ? 256 : 512) / hkv); }
int rows_of_tall(int D) { return D == 256 ? 64 : 128; }

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t plan_bytes(int64_t items) { return rounded((8 + 8 * items) * 4); }
// Places of a line: the rows, and a tile's height a run.
int64_t places_of(int64_t rows, int hkv, int D, int line) {
  if (line == kStream) return rows + (int64_t)runs_of(hkv, D) * kWaves * kStreamRows;
  return rows <= kStreamRows ? 0 : rows + (int64_t)runs_of(hkv, D) * rows_of_tall(D);   // no tile has more than 16 rows
}
size_t sums_bytes(int64_t places, int hkv, int D) { return rounded((size_t)places * hkv * D * 4); }
size_t refs_bytes(int64_t places, int hkv) { return rounded((size_t)places * hkv * 8); }
size_t workspace_bytes(int64_t rows, int64_t items, int hkv, int D) {
  size_t bytes = plan_bytes(items);
  for (int line = 0; line < 2; ++line) {
    const int64_t places = places_of(rows, hkv, D, line);
    bytes += 2 * (sums_bytes(places, hkv, D) + refs_bytes(places, hkv));
  }
  return bytes;
}

template <int D>
int launch(const BranchArgs& A, hipStream_t s) {
  static dh::OncePerDevice once;
  const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&branch_parts_kernel<D>), kLds<D>);
  if (e != hipSuccess) return dh::fail(DH_EHIP, "branch_parts_kernel: %s", hipGetErrorString(e));
  hipLaunchKernelGGL((branch_parts_kernel<D>), dim3((unsigned)(A.runs * A.c.hkv)), dim3(kThreads), kLds<D>, s, A);
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
  *bytes = workspace_bytes((int64_t)T * (hq / hkv), 2 * (int64_t)n_seq, hkv, D);
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
  const int64_t rows = (int64_t)T * A.group, items = (int64_t)n_groups + n_seq;
  const size_t need = workspace_bytes(rows, items, hkv, D);
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
  unsigned char* at = static_cast<unsigned char*>(workspace);
  auto take = [&](size_t bytes) {
    unsigned char* p = at;
    at += bytes;
    return p;
  };
  A.plan = reinterpret_cast<int32_t*>(take(plan_bytes(items)));
  for (int line = 0; line < 2; ++line) {
    A.places[line] = places_of(rows, hkv, D, line);
    for (Parts* p : {&A.prefix[line], &A.own[line]}) {
      p->o = reinterpret_cast<float*>(take(sums_bytes(A.places[line], hkv, D)));
      p->ml = reinterpret_cast<float2*>(take(refs_bytes(A.places[line], hkv)));
    }
  }
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  switch (D) {
    case 64: return launch<64>(A, st);
    case 128: return launch<128>(A, st);
    default: return launch<256>(A, st);
  }
}

}  // extern "C"
