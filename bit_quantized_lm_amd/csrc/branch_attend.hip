// Attention of a batch whose sequences share prefixes, over the 8-bit cache, on
// gfx950 (draft_branch_attend).
//
// A group's rows against its prefix, and each sequence's rows against its own
// tokens, are two kinds of items of one launch.  Both leave partial results (sums
// of values, reference and sum of the weights, fp32); a second launch joins a row's
// parts.  The members' rows follow each other in memory, so a prefix's tiles are
// packed from all of them as if they were one sequence's, and each key and value of
// the prefix is loaded once for up to 128 of them.  Which tile or part a workgroup
// takes is computed on the device, from the lengths.  Short contexts take one launch
// that shares nothing (branch_short_kernel).
//
// 40 heads on 8 of 128: 64 samples of a prompt of 8,192 tokens 39 us, 16 sequences of
// 9 slots over four prefixes of up to 20,000 53, 16 prompts of 112 rows over 6,000
// tokens 266 (834 TFLOP/s).  Of the first two's 34 and 47 us on the card before the
// joining (8), a workgroup's tiles take 19 and 31; the rest begins (start 0.4, plan 2.9,
// segment and its setup 2) and leaves (2), and the last workgroups end 5 after most.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/draftbranch.h"
#include "attend_tile.h"
#include "branch_cost.h"

namespace {

using namespace dl;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kNoLimit = DL_MAX_POSITIONS;

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
  int32_t* plan;      // a Plan, then a Record an item
};

// ------------------------------------------------------------------ the work
// Items: the sequences' own tokens, then the groups' prefixes.  An item's rows (query
// heads of one kv head, token after token) are cut into tiles of H = 128 (heads of
// 256: 64) and a rest; up to 16 rows are one wave's (stream_tile), up to 64 and up to
// H a workgroup's (shared_tile), whatever the other items have.  Where the members of
// a group have H rows each on average, sharing saves no time (such tiles are bound by
// the matrix units) and joining costs some, so the prefix's tokens are the
// sequences' own then.  Heads of 128, 40 on 8, us so and apart: 16 prompts of 112 rows
// over 2,048, 6,144 and 20,480 tokens 121, 273, 805 and 135, 288, 845; of 300 rows down
// to 15, 160, 360, 1,081 and 199, 400, 1,088.  By the average, so a group of one prompt
// and many single tokens has each of them read the prefix: 2,000 rows and 15 of one 183,
// 335, 921 and 213, 372, 919, but 600 and 15 of one 72, 118, 315 and 70, 115, 278, and
// 4 of 112 and 12 of one 58, 103, 256 and 56, 91, 223.
//
// All tiles of a line are laid end to end, each as long as it is thought to take, and
// cut into equal runs: a workgroup's, or a wave's, which walks its own segments and
// waits for no other.  A run may hold the end of one tile, whole ones and the start of
// another; what it has of a tile is a part.  The workgroups are divided between the
// lines by what the lines take.
struct Item {
  int groups;            // of 32 tokens that a tile sees at most
  int n, row0;           // token rows
  int sees;              // 1: the own tokens, 2: the shared ones
  int split;             // positions below are the shared ones
  int of;                // the sequence's group, -1: none
  int seq, lead;         // whose table rows name the pages of the own and of the shared tokens
  int p_first, p_last;   // the rows' positions
};

// An item's tiles: `full` ones of H rows, then one of `rest`, and their units, of
// 2^shift (whole: 1 for the stream's).  A tile's first units are its beginning, `pad`
// of them: its groups are in the others.
template <int D>
struct Shape {
  int full, rest, each, last, whole, shift;
  __device__ __forceinline__ Shape(int rows, int groups, int shift_, int whole_) : whole(whole_), shift(shift_) {
    constexpr int H = Cost<D>::kRows;
    if (groups == 0) rows = 0;
    full = rows / H;
    rest = rows % H;
    each = scaled(Cost<D>::of(H, max(groups, 1)));
    last = rest == 0 ? 0 : whole && streams() ? 1 : scaled(Cost<D>::of(rest, groups));
  }
  __device__ __forceinline__ int scaled(int units) const { return (units + (1 << shift) - 1) >> shift; }
  __device__ __forceinline__ bool streams() const { return Cost<D>::kStreams && rest <= kStreamRows; }
  __device__ __forceinline__ int units(Line line) const {
    return line == kStream ? (streams() ? last : 0) : full * each + (streams() ? 0 : last);
  }
  // Of tile t of a line's
  __device__ __forceinline__ int length(int t) const { return t < full ? each : last; }
  __device__ __forceinline__ int pad(Line line, int t) const {
    return line == kStream && whole ? 0 : min(Cost<D>::begin(line == kStream ? kStreamRows : kSmallRows) >> shift, length(t) - 1);
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

struct Members {
  int first, last;    // sequences first .. last - 1
  int row0, n;        // token rows
  int prefix;
  bool whole;         // its prefix's tokens count as the sequences' own
};
// A group from its entries of the lists; rows_before(s) is q_start[s].
template <int D, class Rows>
__device__ __forceinline__ Members members_of(const BranchArgs& A, int2 group, int prefix, const Rows rows_before) {
  Members r;
  r.first = min(max(group.x, 0), A.b.n_seq);
  r.last = max(r.first, min(group.y, A.b.n_seq));
  r.row0 = min(max(rows_before(r.first), 0), A.b.T);
  r.n = max(min(rows_before(r.last), A.b.T) - r.row0, 0);
  r.prefix = min(max(prefix, 0), kNoLimit);
  r.whole = (int64_t)r.n * A.group >= (int64_t)Cost<D>::kRows * (r.last - r.first);
  return r;
}

__device__ __forceinline__ void write_lse(float* lse, size_t row, float ref, float sum) {
  if (lse) lse[row] = sum == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
}

// Sequence s with the group that it is of (g < 0: none).
template <int D>
__device__ __forceinline__ Item own_item(const BranchArgs& A, int s, const Seq& q, int g, const Members& group) {
  Item t;
  t.n = q.n;
  t.row0 = q.row0;
  t.sees = g >= 0 && group.whole ? 3 : 1;
  t.split = g < 0 ? 0 : group.prefix;
  t.of = g;
  t.seq = s;
  t.lead = min(group.first, A.b.n_seq - 1);
  t.p_first = q.begin;
  t.p_last = q.len - 1;
  // the last tile's rows at most: what they see is the longest; a window may hide all from that tile alone
  const int first = q.len - min(q.n, Cost<D>::kRows / A.group + 2);
  t.groups = q.n == 0 ? 0 : max(visible_own(A, t, first, t.p_last).n + visible_shared(A, t, first, t.p_last).n, A.window > 0 ? 1 : 0);
  return t;
}

// A group whose rows are at p_first .. p_last.
__device__ __forceinline__ Item prefix_item(const BranchArgs& A, const Members& group, int p_first, int p_last) {
  Item t;
  t.n = group.whole ? 0 : group.n;
  t.row0 = group.row0;
  t.sees = 2;
  t.split = group.prefix;
  t.of = -1;
  t.seq = t.lead = min(group.first, A.b.n_seq - 1);
  t.p_first = p_first;
  t.p_last = p_last;
  t.groups = visible_shared(A, t, p_first, p_last).n;
  return t;
}

// Whether the row at p_first does not see the whole of its prefix: only where some
// row does not, or has a window, do the positions of a prefix's rows matter.
__device__ __forceinline__ bool inside_prefix(const Item& t) { return t.n > 0 && t.p_first + 1 < t.split; }

// ------------------------------------------------------------------ the plan
// What every part and the joining go by, from the lengths.
struct Plan {
  int per[2];    // units of a run, by line
  int more;      // of the shared line's first `half` runs; the others have as many less
  int half;
  int shift;     // units are 2^shift, so that their sums fit 32 bits
  int whole;     // the stream's tiles are a wave each
  int shared;    // workgroups a head of the shared line
  int placed;    // the positions of a prefix's rows matter
};
struct Record {
  int at[2];     // first unit, by line
  Item item;
};
static_assert(sizeof(Plan) == 32 && sizeof(Record) == 48, "both are read 16 bytes at a time");

struct Sums {    // of all items' tiles, in units
  float units[2] = {0.0f, 0.0f}, tiles = 0.0f, longest = 0.0f;   // the last two: the stream's
  template <int D>
  __device__ __forceinline__ void add(const Shape<D>& s) {
    const float stream = (float)s.units(kStream);
    units[kShared] += (float)s.full * (float)s.each + (s.streams() ? 0.0f : (float)s.last);   // may be past 32 bits
    units[kStream] += stream;
    tiles += stream > 0.0f ? 1.0f : 0.0f;
    longest = fmaxf(longest, stream);
  }
};

// The lines' shares of the workgroups: by their work; or a wave a tile for the
// stream, where both lines end as soon so.  Nothing ends before a part of four groups.
template <int D>
__device__ __forceinline__ void divide(const BranchArgs& A, const Sums& sum, Plan& p) {
  const float shared = sum.units[kShared], stream = sum.units[kStream], runs = (float)A.runs;
  const float even = (shared + stream * (1.0f / kWaves)) / runs;
  const float end = fmaxf(even, (float)Cost<D>::of(kSmallRows, 4)) + (float)Cost<D>::begin(kStreamRows) * 0.5f;
  const float rest = runs - ceilf(sum.tiles * (1.0f / kWaves));
  p.whole = stream > 0.0f && sum.longest <= end && shared <= rest * end && rest >= 0.0f;
  p.shared = (int)(p.whole ? rest : stream == 0.0f ? runs : shared == 0.0f ? 0.0f : fminf(fmaxf(rintf(shared / even), 1.0f), runs - 1.0f));
  p.shift = max(0, (int)((__float_as_uint(fmaxf(shared, stream)) >> 23) & 255u) - 127 - 27);
}

// Two workgroups share a CU, and the one that came first is served first: of two
// equal ones of 220 groups it ended after 232 us, the other after 283.  So on long
// runs (100 us and more) those that come first, blocks 0 .. 255, have a share more:
// 16 prompts of 112 rows over 6,000 tokens took 284 us with even runs, 274 so (0.2:
// 282, 0.25: 287); on short ones it costs (16 slots of 9: 59.0 us, 61.5 with 0.08).
constexpr float kFirst = 0.15f;
// First unit of run r.
__device__ __forceinline__ int start_of(int r, int per, int more, int half) { return r * per + more * min(r, 2 * half - r); }
// A part of fewer than four groups costs more to begin and to join than it saves.
template <int D>
__device__ __forceinline__ void cut(const BranchArgs& A, int shared_units, int stream_units, Plan& p) {
  const int waves = max(A.runs - p.shared, 1) * kWaves;
  const int least = max((4 * Cost<D>::per_group(kSmallRows)) >> p.shift, 1);
  p.half = A.runs >> 1;
  const float even = (float)shared_units / (float)max(p.shared, 1), first = (float)(2 * min(p.half, p.shared) - p.shared);
  const bool full = even * (float)(1 << p.shift) >= 1000.0f;
  // 0.1% more than the mean: float quotients may fall short
  p.per[kShared] = max(least, (int)(1.001f * even / (1.0f + (full ? kFirst * first / (float)max(p.shared, 1) : 0.0f))) + 2);
  p.more = full ? (int)(kFirst * (float)p.per[kShared]) : 0;
  p.per[kStream] = p.whole ? 1 : max(max((4 * Cost<D>::per_group(kStreamRows)) >> p.shift, 1), (stream_units + waves - 1) / waves);
}

// LDS accesses before stay before those after, in a wave that is alone with them.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Up to 64 sequences and groups: one wave, a sequence and a group a lane, the
// lists' entries passed between the lanes.  Every workgroup makes the plan for itself.
constexpr int kSmall = 64;
template <int D>
__device__ __forceinline__ void make_plan(const BranchArgs& A, int (&first)[kSmall], int (&last)[kSmall], Plan* plan, Record* records) {
  const int lane = threadIdx.x & 63, s = min(lane, A.b.n_seq - 1), g = min(lane, A.n_groups - 1);
  const int start = A.b.q_start[s], end = A.b.q_start[s + 1], length = A.b.kv_len[s];
  const int2 group{A.group_start[g], A.group_start[g + 1]};
  const int prefix = A.prefix_len[g];
  const int all_rows = __builtin_amdgcn_readlane(end, A.b.n_seq - 1), all_seqs = __builtin_amdgcn_readlane(group.y, A.n_groups - 1);
  auto rows_before = [&](int i) {
    const int there = __shfl(start, i);   // by every lane: none is another's source else
    return i < A.b.n_seq ? there : all_rows;
  };
  Seq q;
  q.row0 = min(max(start, 0), A.b.T);
  q.n = max(min(end, A.b.T) - q.row0, 0);
  q.len = min(max(length, 0), DL_MAX_POSITIONS);
  q.begin = q.len - q.n;
  int of = -1;
  for (int i = 0; i < A.n_groups; ++i) of += __builtin_amdgcn_readlane(group.x, i) <= s;
  of = all_seqs <= s ? -1 : of;
  const int from = max(of, 0);
  const int group_prefix = __shfl(prefix, from);
  const Members mine = members_of<D>(A, int2{__shfl(group.x, from), __shfl(group.y, from)}, group_prefix, rows_before);
  const Members members = members_of<D>(A, group, prefix, rows_before);
  Item own = own_item<D>(A, s, q, of, mine);
  if (lane >= A.b.n_seq) own.n = 0;
  Plan p{};
  p.placed = A.window > 0 || __any(inside_prefix(own));
  int p_first = kNoLimit, p_last = kNoLimit;   // behind every prefix
  if (p.placed) {
    first[lane] = kNoLimit;
    last[lane] = -1;
    wave_fence();
    if (own.n > 0 && of >= 0) {
      atomicMin(&first[of], q.begin);
      atomicMax(&last[of], q.len - 1);
    }
    wave_fence();
    p_first = first[g];
    p_last = last[g];
  }
  Item shared = prefix_item(A, members, p_first, p_last);
  if (lane >= A.n_groups) shared.n = 0;
  const int own_rows = own.n * A.group, shared_rows = shared.n * A.group;   // up to 2^30
  Sums sum;
  sum.add(Shape<D>(own_rows, own.groups, 0, 0));
  sum.add(Shape<D>(shared_rows, shared.groups, 0, 0));
  for (float& x : sum.units) x = wave_sum(x);
  sum.tiles = wave_sum(sum.tiles);
  sum.longest = wave_max(sum.longest);
  divide<D>(A, sum, p);
  const Shape<D> a(own_rows, own.groups, p.shift, p.whole), b(shared_rows, shared.groups, p.shift, p.whole);
  Record r[2] = {{{0, 0}, own}, {{0, 0}, shared}};
  int total[2];
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    const int x = a.units((Line)l), y = b.units((Line)l), to_x = wave_inclusive_sum(x), to_y = wave_inclusive_sum(y);
    const int before = __builtin_amdgcn_readlane(to_x, 63);
    r[0].at[l] = to_x - x;
    r[1].at[l] = before + to_y - y;
    total[l] = before + __builtin_amdgcn_readlane(to_y, 63);
  }
  cut<D>(A, total[kShared], total[kStream], p);
  if (lane < A.b.n_seq) records[lane] = r[0];
  if (lane < A.n_groups) records[A.b.n_seq + lane] = r[1];
  if (lane == 0) *plan = p;
}

// More: a launch of its own makes it, one workgroup.
constexpr int kPlanThreads = 1024;
template <int D>
__global__ __launch_bounds__(kPlanThreads) void branch_plan_kernel(BranchArgs A) {
  __shared__ int first[DL_MAX_SEQS], last[DL_MAX_SEQS];   // positions of a group's rows
  __shared__ float sums[4][kPlanThreads / 64];
  __shared__ int totals[2][kPlanThreads / 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, items = A.b.n_seq + A.n_groups;
  Plan* plan = reinterpret_cast<Plan*>(A.plan);
  Record* records = reinterpret_cast<Record*>(plan + 1);
  auto rows_before = [&](int i) { return A.b.q_start[i]; };
  auto members = [&](int g) { return members_of<D>(A, int2{A.group_start[g], A.group_start[g + 1]}, A.prefix_len[g], rows_before); };
  for (int g = tid; g < A.n_groups; g += kPlanThreads) first[g] = kNoLimit, last[g] = -1;
  __syncthreads();
  Sums sum;
  bool inside = false;
  for (int s = tid; s < A.b.n_seq; s += kPlanThreads) {
    int g = 0;   // groups that start at or before s
    for (int end = A.n_groups + 1; g < end;) {
      const int mid = (g + end) >> 1;
      if (A.group_start[mid] <= s)
        g = mid + 1;
      else
        end = mid;
    }
    g = g - 1 < A.n_groups ? g - 1 : -1;
    const Seq q = load_seq(A.b, s);
    const Item t = own_item<D>(A, s, q, g, members(max(g, 0)));
    inside |= inside_prefix(t);
    if (g >= 0 && q.n > 0) {
      atomicMin(&first[g], q.begin);
      atomicMax(&last[g], q.len - 1);
    }
    sum.add(Shape<D>(t.n * A.group, t.groups, 0, 0));
    records[s].item = t;
  }
  Plan p{};
  p.placed = __syncthreads_or(inside) || A.window > 0;
  for (int g = tid; g < A.n_groups; g += kPlanThreads) {
    const Item t = prefix_item(A, members(g), p.placed ? first[g] : kNoLimit, p.placed ? last[g] : kNoLimit);
    sum.add(Shape<D>(t.n * A.group, t.groups, 0, 0));
    records[A.b.n_seq + g].item = t;
  }
  const float of_wave[4] = {wave_sum(sum.units[0]), wave_sum(sum.units[1]), wave_sum(sum.tiles), wave_max(sum.longest)};
  if (lane == 0)
    for (int i = 0; i < 4; ++i) sums[i][wave] = of_wave[i];
  __syncthreads();
  sum = Sums{};
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    sum.units[0] += sums[0][w];
    sum.units[1] += sums[1][w];
    sum.tiles += sums[2][w];
    sum.longest = fmaxf(sum.longest, sums[3][w]);
  }
  divide<D>(A, sum, p);
  int before[2] = {0, 0};
  for (int base = 0; base < items; base += kPlanThreads) {
    const int i = base + tid;
    const Shape<D> s(i < items ? records[i].item.n * A.group : 0, i < items ? records[i].item.groups : 0, p.shift, p.whole);
    int to[2], mine[2];
    __syncthreads();
    for (int l = 0; l < 2; ++l) {
      mine[l] = s.units((Line)l);
      to[l] = wave_inclusive_sum(mine[l]);
      if (lane == 63) totals[l][wave] = to[l];
    }
    __syncthreads();
    for (int l = 0; l < 2; ++l) {
      int all = 0, here = 0;
      for (int w = 0; w < kPlanThreads / 64; ++w) {
        here += w < wave ? totals[l][w] : 0;
        all += totals[l][w];
      }
      if (i < items) records[i].at[l] = before[l] + here + to[l] - mine[l];
      before[l] += all;
    }
  }
  cut<D>(A, before[kShared], before[kStream], p);
  if (tid == 0) *plan = p;
}

// The last of n ascending numbers that is at most x, by the whole wave: 64 at a look.
template <class At>
__device__ __forceinline__ int last_up_to(int n, int x, const At at) {
  const int lane = threadIdx.x & 63;
  int from = 0;
  for (int span = n; span > 1;) {
    const int step = (span + 63) >> 6;
    const bool is = lane * step < span && at(from + min(lane * step, span - 1)) <= x;
    const int up_to = (int)__popcll(__ballot(is));   // 0 where not even the first is
    from += max(up_to - 1, 0) * step;
    span = min(step, n - from);
  }
  return from;
}

struct Segment {
  Item item;
  Line line;
  int tile, from, to, of, run;
};

// The walk through one run's segments.
template <int D>
class Walk {
 public:
  // Workgroup `number` of a head works on one line, and each wave of the stream's has a run of its own.
  __device__ __forceinline__ Walk(const Plan& p, int number) {
    auto of = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    const int shared = of(p.shared);
    line_ = number < shared ? kShared : kStream;
    shift_ = of(p.shift);
    whole_ = of(p.whole);
    run_ = line_ == kShared ? number : (number - shared) * kWaves + of(threadIdx.x >> 6);
    const int per = of(p.per[line_]), more = line_ == kShared ? of(p.more) : 0, half = of(p.half);
    at_ = start_of(run_, per, more, half);
    end_ = start_of(run_ + 1, per, more, half);
  }
  __device__ __forceinline__ Line line() const { return line_; }

  // The run's next segment; false past its last.
  __device__ __forceinline__ bool next(const BranchArgs& A, const Record* records, Segment& g) {
    while (at_ < end_) {
      const Record* r = records + last_up_to(A.b.n_seq + A.n_groups, at_, [&](int i) { return records[i].at[line_]; });
      auto of = [&](int x) { return __builtin_amdgcn_readfirstlane(x); };
      const Item& t = r->item;
      g.item = Item{of(t.groups), of(t.n), of(t.row0), of(t.sees), of(t.split), of(t.of), of(t.seq), of(t.lead), of(t.p_first), of(t.p_last)};
      const Shape<D> s(g.item.n * A.group, g.item.groups, shift_, whole_);
      const int at = at_ - of(r->at[line_]);
      if (at >= s.units(line_)) return false;   // past the last item's
      g.line = line_;
      g.run = run_;
      g.tile = line_ == kStream ? s.full : min(at / s.each, s.full);
      const int in_tile = at - (line_ == kStream ? 0 : g.tile * s.each), pad = s.pad(line_, g.tile), length = s.length(g.tile);
      const int to = min(length, in_tile + end_ - at_);
      at_ += to - in_tile;
      g.of = length - pad;
      g.from = max(in_tile - pad, 0);
      g.to = to - pad;
      if (g.to > 0) return true;   // else the run ends in the tile's beginning
    }
    return false;
  }

 private:
  Line line_;
  int shift_, whole_, run_, at_, end_;
};

// ----------------------------------------------------------------- the parts
template <int D, int R>
__device__ __forceinline__ void attend_part(const BranchArgs& A, const Segment& w, bool placed, int head, u32x4* stage) {
  constexpr int C = D / 16;
  const Item& t = w.item;
  const bool prefix = t.sees == 2;
  const int lane = threadIdx.x & 63, hi = lane >> 4, lo = lane & 15;
  const int x0 = w.tile * Cost<D>::kRows, rows = min(R, t.n * A.group - x0);
  // positions of rows a .. b of the tile: a sequence's follow each other, a group's are anywhere among its own
  auto first_of = [&](int a) { return prefix ? t.p_first : t.p_first + (x0 + a) / A.group; };
  auto last_of = [&](int b) { return prefix ? t.p_last : t.p_first + (x0 + b) / A.group; };
  const Range own = visible_own(A, t, first_of(0), last_of(rows - 1)), shared = visible_shared(A, t, first_of(0), last_of(rows - 1));
  const int n = own.n + shared.n;
  // unit u's group: a float division is monotone too, so parts meet, and the ends are exact
  auto group_at = [&](int u) { return u == w.of ? n : min(n, (int)((float)n * ((float)u / (float)w.of))); };
  const int from = __builtin_amdgcn_readfirstlane(group_at(w.from)), to = __builtin_amdgcn_readfirstlane(group_at(w.to));
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

template <int D, bool kSmallBatch>
__global__ __launch_bounds__(kThreads, 2) void branch_parts_kernel(BranchArgs A) {
  extern __shared__ __align__(16) u32x4 stage[];
  __shared__ Plan plan_here;
  __shared__ Record records_here[kSmallBatch ? 2 * kSmall : 1];
  __shared__ int first[kSmallBatch ? kSmall : 1], last[kSmallBatch ? kSmall : 1];   // positions of a group's rows
  const Plan* plan = reinterpret_cast<const Plan*>(A.plan);
  const Record* records = reinterpret_cast<const Record*>(plan + 1);
  if constexpr (kSmallBatch) {
    if (threadIdx.x < 64) make_plan<D>(A, first, last, &plan_here, records_here);
    __syncthreads();
    if (blockIdx.x == 0) {   // for the launch that joins the parts
      for (int i = threadIdx.x; i < (A.b.n_seq + A.n_groups) * (int)(sizeof(Record) / 4); i += kThreads)
        A.plan[sizeof(Plan) / 4 + i] = reinterpret_cast<const int*>(records_here)[i];
      if (threadIdx.x < sizeof(Plan) / 4) A.plan[threadIdx.x] = reinterpret_cast<const int*>(&plan_here)[threadIdx.x];
    }
  }
  const int head = blockIdx.x % A.c.hkv;
  const Plan& p = kSmallBatch ? plan_here : *plan;
  const bool placed = __builtin_amdgcn_readfirstlane(p.placed);
  Walk<D> walk(p, blockIdx.x / A.c.hkv);
  for (Segment w; walk.next(A, kSmallBatch ? records_here : records, w);) {
    constexpr int H = Cost<D>::kRows;
    if (Cost<D>::kStreams && walk.line() == kStream) {
      if constexpr (Cost<D>::kStreams) attend_part<D, kStreamRows>(A, w, placed, head, stage);
    } else {
      if (H == kSmallRows || w.item.n * A.group - w.tile * H <= kSmallRows)
        attend_part<D, kSmallRows>(A, w, placed, head, stage);
      else
        attend_part<D, H>(A, w, placed, head, stage);
    }
  }
}

// ---------------------------------------------------------------- the joining
// D / 8 lanes a row of one query head, so that a pass takes four heads of 128 (16 prompts
// 263 us; with D / 4 lanes and half as many rows a pass 269, the other sizes the same).
// With few rows W waves take turns at a row's parts; with many (W = 1) a wave has `heads`
// query heads of a token row, because finding the parts takes longer than joining them.
template <int D, int W>
__global__ __launch_bounds__(kThreads) void branch_join_kernel(BranchArgs A, int heads) {
  constexpr int L = D / 8, P = 64 / L, H = Cost<D>::kRows;   // lanes a row, rows a pass
  __shared__ f32x4 sums[W][2][64];
  __shared__ float2 refs[W][P];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, l = lane % L;
  const int turn = wave % W, chunks = (A.hq + heads - 1) / heads;
  const int64_t unit = (int64_t)blockIdx.x * (kWaves / W) + wave / W;
  const int r = (int)(unit / chunks), h0 = (int)(unit % chunks) * heads;
  if (r >= A.b.T) return;   // W > 1: all waves, a workgroup has one unit
  const Plan plan = *reinterpret_cast<const Plan*>(A.plan);
  const Record* records = reinterpret_cast<const Record*>(A.plan + sizeof(Plan) / 4);
  // the row's sequence and its records: of up to 64 items each lane has one, loaded at once
  Record own_record, prefix_record;
  if (const int items = A.b.n_seq + A.n_groups; items <= 64) {
    const int start = A.b.q_start[min(lane, A.b.n_seq - 1)];
    const Record mine = records[min(lane, items - 1)];
    auto of_lane = [&](int i, Record& to) {
      const int* from = reinterpret_cast<const int*>(&mine);
#pragma unroll
      for (int k = 0; k < (int)(sizeof(Record) / 4); ++k) reinterpret_cast<int*>(&to)[k] = __builtin_amdgcn_readlane(from[k], i);
    };
    const int up_to = (int)__popcll(__ballot(lane < A.b.n_seq && start <= r));
    of_lane(max(up_to - 1, 0), own_record);
    of_lane(A.b.n_seq + max(own_record.item.of, 0), prefix_record);
  } else {
    const int s = __builtin_amdgcn_readfirstlane(last_up_to(A.b.n_seq, r, [&](int i) { return A.b.q_start[i]; }));
    own_record = records[s];
    prefix_record = records[A.b.n_seq + max(own_record.item.of, 0)];
  }
  if (r < own_record.item.row0 || r >= own_record.item.row0 + own_record.item.n) return;
  // an item's parts of a row: where the first is, how far apart they are, how many
  struct Run {
    const float* o;
    const float2* ml;
    int step, n;
  };
  // The run that has a unit: fewer than 2^12 runs, so the quotient from a reciprocal is at most one off.
  const int units[3] = {plan.per[kStream], plan.per[kShared] + plan.more, plan.per[kShared] - plan.more}, before = plan.half * units[1];
  const float inverse[3] = {1.0f / (float)units[0], 1.0f / (float)units[1], 1.0f / (float)units[2]};
  auto run_at = [&](Line line, int unit) {
    const bool stream = line == kStream, rest = !stream && unit >= before;
    const int d = stream ? units[0] : rest ? units[2] : units[1], x = rest ? unit - before : unit;
    int q = (int)((float)x * (stream ? inverse[0] : rest ? inverse[2] : inverse[1]));
    const int r = x - q * d;
    q += (r >= d) - (r < 0);
    return rest ? plan.half + q : q;
  };
  auto parts_of = [&](const Record& rec, const Parts (&all)[2], int head, int in_group) {
    constexpr Line any = Cost<D>::kStreams ? kStream : kShared;   // of which there are places
    Run p{all[any].o, all[any].ml, 0, 0};
    const int x = r * A.group + in_group, y = x - rec.item.row0 * A.group, rows = rec.item.n * A.group;
    if (y < 0 || y >= rows || rec.item.groups == 0) return p;   // nothing to see, or groups and sequences that do not fit each other
    const Shape<D> shape(rows, rec.item.groups, plan.shift, plan.whole);
    const int tile = min(y / H, shape.full);
    const Line line = tile == shape.full && shape.streams() ? kStream : kShared;
    const int at = line == kStream ? rec.at[kStream] : rec.at[kShared] + tile * shape.each;
    const int first = run_at(line, at + shape.pad(line, tile));
    p.step = line == kStream ? kStreamRows : H;
    p.n = run_at(line, at + shape.length(tile) - 1) - first + 1;
    const size_t place = (size_t)head * A.places[line] + x + (size_t)first * p.step;
    p.o = all[line].o + place * D;
    p.ml = all[line].ml + place;
    return p;
  };
  const bool alone = own_record.item.split == 0 || own_record.item.sees == 3;
  int head = (h0 + lane / L) / A.group, in_group = (h0 + lane / L) % A.group;
  for (int pass = h0; pass < min(A.hq, h0 + heads); pass += P) {
    const int h = pass + lane / L;   // past the last head: the last one's places
    const Run own = parts_of(own_record, A.own, min(head, A.c.hkv - 1), in_group);
    Run prefix{own.o, own.ml, 0, 0};
    if (own_record.item.of >= 0 && !alone) prefix = parts_of(prefix_record, A.prefix, min(head, A.c.hkv - 1), in_group);
    for (in_group += P; in_group >= A.group; ++head) in_group -= A.group;
    const bool done = h >= min(A.hq, h0 + heads) || (alone && own.n == 1);   // or the result already
    const int n = done ? 0 : prefix.n + own.n, most = (int)wave_max((uint32_t)n);
    if (W == 1 && __all(done)) continue;
    float top = kLowest, sum = 0.0f;
    f32x4 y[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};   // four elements of each half
    for (int base = turn; base < most; base += L * W) {
      // lane i of a row: part base + i W
      const int part = base + l * W;
      float2 ml = {kLowest, 0.0f};
      if (part < n) ml = part < prefix.n ? prefix.ml[part * prefix.step] : own.ml[(part - prefix.n) * own.step];
      float next = ml.x;
#pragma unroll
      for (int i = 1; i < L; i *= 2) next = fmaxf(next, __shfl_xor(next, i));
      next = fmaxf(next, top);
      const float share = part < n ? __builtin_amdgcn_exp2f(ml.x - next) : 0.0f, down = __builtin_amdgcn_exp2f(top - next);
      float weight = share * ml.y;
#pragma unroll
      for (int i = 1; i < L; i *= 2) weight += __shfl_xor(weight, i);
      sum = fmaf(sum, down, weight);
      top = next;
      y[0] *= down;
      y[1] *= down;
      const int count = min(L, (most - base + W - 1) / W);
      auto add = [&](auto at_once, int j0) {   // past a row's last part, that once more with no share
        constexpr int K = decltype(at_once)::value;
        f32x4 v[K][2];
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int at = max(min(base + (j0 + j) * W, n - 1), 0);
          const bool of_prefix = at < prefix.n;   // a run's distance is below 2^28 floats
          const float* o = (of_prefix ? prefix.o : own.o) + (of_prefix ? at : at - prefix.n) * (of_prefix ? prefix.step : own.step) * D + l * 4;
          v[j][0] = *reinterpret_cast<const f32x4*>(o);
          v[j][1] = *reinterpret_cast<const f32x4*>(o + D / 2);
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const float by = __shfl(share, lane - l + min(j0 + j, L - 1));
          const float w = j0 + j < L ? by : 0.0f;
          y[0] += w * v[j][0];
          y[1] += w * v[j][1];
        }
      };
      int j = 0;
      for (; j + 4 < count; j += 4) add(std::integral_constant<int, 4>{}, j);
      if (j + 2 < count)
        add(std::integral_constant<int, 4>{}, j);
      else if (j < count)
        add(std::integral_constant<int, 2>{}, j);
    }
    if constexpr (W > 1) {   // one pass
      sums[wave][0][lane] = y[0];
      sums[wave][1][lane] = y[1];
      if (l == 0) refs[wave][lane / L] = float2{top, sum};
      __syncthreads();
      if (turn > 0) return;
#pragma unroll
      for (int v = 1; v < W; ++v) {
        const float2 other = refs[v][lane / L];
        const float next = fmaxf(top, other.x), down = __builtin_amdgcn_exp2f(top - next), share = __builtin_amdgcn_exp2f(other.x - next);
        y[0] = down * y[0] + share * sums[v][0][lane];
        y[1] = down * y[1] + share * sums[v][1][lane];
        sum = fmaf(sum, down, share * other.y);
        top = next;
      }
    }
    if (done) continue;
    if (n == 0) y[0] = y[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};   // what was loaded for it is another row's
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const size_t row = (size_t)r * A.hq + h;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<u32x2*>(A.out + row * D + i * (D / 2) + l * 4) = u32x2{bf16_pair(y[i][0] * inv, y[i][1] * inv), bf16_pair(y[i][2] * inv, y[i][3] * inv)};
    if (l == 0) write_lse(A.lse, row, top, sum);
  }
}

// ------------------------------------------------------------------ short ones
// Contexts that are short by the table's width or the window, and few rows: a tile of
// 16 rows a workgroup, whose waves take turns at what it sees, the prefix's tokens and
// its own.  Nothing is shared but through the caches, nothing planned or joined, in one
// launch (3 us of the host's time, and 5 of the card's).  Heads of 128, 40 on 8, one row of
// each of 4 sequences over 500, 1,000, 2,000 and 4,000 tokens: 8.3, 10.1, 14.0 and
// 21.6 us so, 15.8, 16.0, 16.7 and 18.0 planned; 9 rows of each of 16: 16.3, 20.3,
// 28.4 and 46.0, planned 30.8, 33.6, 38.4 and 44.2; 100 of each of 4, 1,032 tiles:
// 32.4, 40.8, 56.5 and 90.9, planned 42.9, 47.5, 57.3 and 72.5.  Heads of 256, 16 on
// 2, one row of each of 4 over 500, 1,000 and 2,000: 11.4, 16.2 and 25.0, planned 17.7,
// 17.9 and 17.8.
template <int D>
constexpr int kShortWaves = D == 256 ? 4 : 8;   // heads of 256: a wave a SIMD
template <int D>
constexpr size_t kShortLds = (size_t)kShortWaves<D> * kStreamRows * (D + 4 + 2) * 4;   // a wave's sums, references and sums of weights

template <int D>
__global__ __launch_bounds__(64 * kShortWaves<D>, D == 256 ? 1 : 2) void branch_short_kernel(BranchArgs A) {
  extern __shared__ __align__(16) u32x4 stage[];
  constexpr int C = D / 16, W = kShortWaves<D>, R = kStreamRows;
  const int head = blockIdx.x % A.c.hkv, tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, hi = lane >> 4, lo = lane & 15;
  int s, tile;
  if (!find_item(A.b, blockIdx.x / A.c.hkv, [&](const Seq& q) { return (q.n * A.group + R - 1) / R; }, s, tile)) return;
  const Seq q = load_seq(A.b, s);
  const int g = __builtin_amdgcn_readfirstlane(A.group_start[0] <= s ? last_up_to(A.n_groups + 1, s, [&](int i) { return A.group_start[i]; }) : -1);
  const bool grouped = g >= 0 && g < A.n_groups;
  Item t{};
  t.sees = grouped ? 3 : 1;
  t.split = grouped ? min(max(A.prefix_len[g], 0), kNoLimit) : 0;
  const int lead = grouped ? min(max(A.group_start[g], 0), A.b.n_seq - 1) : s;
  const int x0 = tile * R, rows = min(R, q.n * A.group - x0);
  const int p_first = q.begin + x0 / A.group, p_last = q.begin + (x0 + rows - 1) / A.group;
  const Range own = visible_own(A, t, p_first, p_last), shared = visible_shared(A, t, p_first, p_last);
  auto place = [&](int r, int& pos) {
    const int x = x0 + r, row = q.row0 + x / A.group;
    pos = r < rows ? q.begin + x / A.group : -1;
    return A.q + (int64_t)row * A.ldq + (head * A.group + x % A.group) * D;
  };
  const Tokens<true> tokens{A.b, A.c, s, head, own, A.window, A.sinks, shared, lead, t.split};
  stream_tile<D, W, 0>(tokens, 0, own.n + shared.n, rows, p_first, p_last, A.scale_log2, place,
                       [&](const f32x4 (&o)[1][C], const float (&m)[1], const float (&l)[1]) {
    float* sums = reinterpret_cast<float*>(stage);   // [W][R][D + 4]
    float* ref = sums + W * R * (D + 4);              // [W][R]
    float* weight = ref + W * R;
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
    const int r = tid / (4 * W);   // 4 W threads a row
    if (r >= rows) return;
    float top = ref[r], all = 0.0f, share[W];
#pragma unroll
    for (int v = 1; v < W; ++v) top = fmaxf(top, ref[v * R + r]);
#pragma unroll
    for (int v = 0; v < W; ++v) {
      share[v] = __builtin_amdgcn_exp2f(ref[v * R + r] - top);
      all = fmaf(weight[v * R + r], share[v], all);
    }
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    const size_t row = (size_t)(q.row0 + (x0 + r) / A.group) * A.hq + head * A.group + (x0 + r) % A.group;
#pragma unroll
    for (int e = tid % (4 * W) * 4; e < D; e += 16 * W) {
      f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < W; ++v) y += share[v] * *reinterpret_cast<const f32x4*>(sums + (v * R + r) * (D + 4) + e);
      *reinterpret_cast<u32x2*>(A.out + row * D + e) = u32x2{bf16_pair(y[0] * inv, y[1] * inv), bf16_pair(y[2] * inv, y[3] * inv)};
    }
    if (tid % (4 * W) == 0) write_lse(A.lse, row, top, all);
  });
}

// ------------------------------------------------------------------- launch
// Workgroups that run at once, by head; two at least, so that both lines have one.
int runs_of(int hkv) { return std::max(2, 512 / hkv); }
bool streams(int D) { return D != 256; }
int rows_of_tall(int D) { return D == 256 ? 64 : 128; }

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t plan_bytes(int64_t items) { return rounded(sizeof(Plan) + items * sizeof(Record)); }
// Places of a line: the rows, and a tile's height a run.
int64_t places_of(int64_t rows, int hkv, int D, int line) {
  if (line == kStream) return streams(D) ? rows + (int64_t)runs_of(hkv) * kWaves * kStreamRows : 0;
  return streams(D) && rows <= kStreamRows ? 0 : rows + (int64_t)runs_of(hkv) * rows_of_tall(D);   // no tile has more than 16 rows
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

template <int D, bool kSmallBatch>
int launch_parts(const BranchArgs& A, hipStream_t s) {
  static dh::OncePerDevice once;
  const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&branch_parts_kernel<D, kSmallBatch>), kLds<D>);
  if (e != hipSuccess) return dh::fail(DH_EHIP, "branch_parts_kernel: %s", hipGetErrorString(e));
  if (!kSmallBatch) hipLaunchKernelGGL((branch_plan_kernel<D>), dim3(1), dim3(kPlanThreads), 0, s, A);
  hipLaunchKernelGGL((branch_parts_kernel<D, kSmallBatch>), dim3((unsigned)(A.runs * A.c.hkv)), dim3(kThreads), kLds<D>, s, A);
  return launched("branch_parts_kernel");
}

template <int D>
int launch(const BranchArgs& A, hipStream_t s) {
  const int64_t room = (int64_t)A.b.max_pages << A.c.page_shift, seen = A.window > 0 ? std::min<int64_t>(room, (int64_t)A.window + A.sinks) : room;
  if (seen <= short_tokens(D, short_tiles(A.b.T, A.b.n_seq, A.hq, A.c.hkv))) {
    const int64_t tiles = ((int64_t)A.b.T * A.group / kStreamRows + A.b.n_seq) * A.c.hkv;   // at least as many as there are
    static dh::OncePerDevice once;
    const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&branch_short_kernel<D>), kShortLds<D>);
    if (e != hipSuccess) return dh::fail(DH_EHIP, "branch_short_kernel: %s", hipGetErrorString(e));
    hipLaunchKernelGGL(branch_short_kernel<D>, dim3((unsigned)tiles), dim3(64 * kShortWaves<D>), kShortLds<D>, s, A);
    return launched("branch_short_kernel");
  }
  const int rc = A.b.n_seq <= kSmall && A.n_groups <= kSmall ? launch_parts<D, true>(A, s) : launch_parts<D, false>(A, s);
  if (rc) return rc;
  constexpr int P = 512 / D;   // rows a pass
  const int64_t rows = (int64_t)A.b.T * A.hq;
  if (rows <= 1024 * P) {
    const int64_t units = A.b.T * (int64_t)((A.hq + P - 1) / P);
    hipLaunchKernelGGL((branch_join_kernel<D, kWaves>), dim3((unsigned)units), dim3(kThreads), 0, s, A, P);
  } else {   // up to 8192 waves, a card's
    const int passes = (int)std::min<int64_t>((rows + 8192 * P - 1) / (8192 * P), (A.hq + P - 1) / P);
    const int64_t units = A.b.T * (int64_t)((A.hq + passes * P - 1) / (passes * P));
    hipLaunchKernelGGL((branch_join_kernel<D, 1>), dim3((unsigned)((units + kWaves - 1) / kWaves)), dim3(kThreads), 0, s, A, passes * P);
  }
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
  // a second launch finds the parts by the plan that the first one leaves in the workspace, and by the row starts
  const Span written[] = {{workspace, need}, {out, (size_t)T * hq * D * 2}, {lse, lse ? (size_t)T * hq * 4 : 0}};
  const Span lists[] = {{q_start, ((size_t)n_seq + 1) * 4}, {kv_len, (size_t)n_seq * 4}, {table, (size_t)n_seq * max_pages * 4},
                        {group_start, ((size_t)n_groups + 1) * 4}, {prefix_len, (size_t)n_groups * 4}};
  for (int w = 0; w < 3; ++w) {
    if (overlap(written[w], written[(w + 1) % 3])) return dh::fail(DH_EINVAL, "attend: out, lse and the workspace must not overlap each other");
    for (const Span& l : lists)
      if (overlap(written[w], l)) return dh::fail(DH_EINVAL, "attend: out, lse and the workspace must not overlap the batch or the groups");
  }
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
  A.runs = runs_of(hkv);
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
