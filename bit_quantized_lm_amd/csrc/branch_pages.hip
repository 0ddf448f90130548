// The pages of several branches on gfx950: the next batch's table from the
// present one, and the pool drawn together (draft_branch_fork,
// draft_branch_compact).
//
// All is decided on the device, since the lengths are there: the host knows
// none of them, waits for nothing, and a call can be captured.  Free pages are
// given out by rank (the r-th free page to the r-th entry that asks), which needs
// two sums over everything before an entry: the entries that ask in the rows
// before it, and the free pages below an id.  The first launch makes both, a
// number a row and a number a chunk of 2,048 pages; in the second every workgroup
// sums the few numbers before its own place, so no workgroup waits for another.
#include <algorithm>

#include "../../include/draftbranch.h"
#include "layer.h"

namespace {

using namespace dl;

constexpr int kThreads = 256;
constexpr int kChunk = 2048;         // pages a count is made of: eight a thread
constexpr int kSlice = 16 << 10;     // bytes of a page that a workgroup copies: four loads of 16 bytes a thread

struct PoolArgs {
  uint8_t *k, *v;
  float *ks, *vs;
  int n_pages, hkv, n_chunks;
  int64_t page_bytes;   // of one page's keys, all heads
  int slices;           // of a page's keys and values
  const int32_t* uses;
  const int32_t* table;
  int32_t* uses_out;
  int32_t* table_out;
  int32_t* status;
  int rows, wide;       // present table
  int32_t* counts;      // [n_chunks] free pages (fork) or pages in use (compact)
};

struct ForkArgs {
  PoolArgs p;
  const int32_t *kv_len, *parents, *need;
  int n_new, page_shift;
  int32_t* asked;       // [n_new] free pages that a row takes, and kEldest
};

struct CompactArgs {
  PoolArgs p;
  int32_t *src, *dst;   // [n_pages / 2 + 1] the moves
  int32_t* number;      // [n_pages] of a page that moves: which move
};

// ---------------------------------------------------------------- block sums
// Sum over the workgroup of the threads before this one; `total` of all.
__device__ __forceinline__ int block_before(int x, int& total, int* lds) {
  const int wave = threadIdx.x >> 6, sum = wave_inclusive_sum(x);
  if ((threadIdx.x & 63) == 63) lds[wave] = sum;
  __syncthreads();
  int before = sum - x;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    before += w < wave ? lds[w] : 0;
    total += lds[w];
  }
  __syncthreads();
  return before;
}
__device__ __forceinline__ int block_sum(int x, int* lds) {
  int total;
  block_before(x, total, lds);
  return total;
}

// The thread's eight counts of uses from its chunk (pages past the pool: `none`).
struct Eight {
  int32_t u[8];
};
__device__ __forceinline__ Eight load_uses(const PoolArgs& A, int chunk, int none) {
  Eight e;
  const int first = chunk * kChunk + threadIdx.x * 8;
  if ((reinterpret_cast<uintptr_t>(A.uses) & 15) == 0 && first + 8 <= A.n_pages) {
    const int4* at = reinterpret_cast<const int4*>(A.uses + first);
    const int4 a = at[0], b = at[1];
    e = Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e.u[i] = first + i < A.n_pages ? A.uses[first + i] : none;
  }
  return e;
}

// A chunk's part of the first launch: the copy of its counts, and how many of
// its pages are free (or in use).
template <bool kFree>
__device__ __forceinline__ void survey_chunk(const PoolArgs& A, int chunk, int* lds) {
  const Eight e = load_uses(A, chunk, kFree ? 1 : 0);
  const int first = chunk * kChunk + threadIdx.x * 8;
  int n = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (first + i < A.n_pages) A.uses_out[first + i] = max(e.u[i], 0);
    n += kFree ? e.u[i] <= 0 : e.u[i] > 0;
  }
  n = block_sum(n, lds);
  if (threadIdx.x == 0) A.counts[chunk] = n;
}

// ---------------------------------------------------------------------- fork
constexpr int kEldest = 1 << 30;   // the first row with its parent
struct Row {
  int parent, len, full, last;
  bool eldest;              // the first row with its parent
  const int32_t* old;       // the parent's entries
};

__device__ __forceinline__ Row row_of(const ForkArgs& A, int s, bool eldest) {
  Row r;
  const int p = A.parents[s], page = 1 << A.page_shift, cap = A.p.wide << A.page_shift;
  const bool has = (unsigned)p < (unsigned)A.p.rows;
  r.parent = has ? p : -1;
  r.old = A.p.table + (size_t)(has ? p : 0) * A.p.wide;
  r.len = has ? min(max(A.kv_len[p], 0), cap) : 0;
  r.full = r.len >> A.page_shift;
  r.last = (int)(((int64_t)min(max(A.need[s], r.len), cap) + page - 1) >> A.page_shift);
  r.eldest = eldest;
  return r;
}

// The page that the parent's entry j names, or -1.
__device__ __forceinline__ int named(const ForkArgs& A, const Row& r, int j) {
  if (r.parent < 0 || j >= A.p.wide) return -1;
  const int id = r.old[j];
  return (unsigned)id < (unsigned)A.p.n_pages ? id : -1;
}
__device__ __forceinline__ bool stays(const ForkArgs& A, const Row& r, int id) { return r.eldest && id >= 0 && A.p.uses[id] == 1; }

__global__ __launch_bounds__(kThreads) void fork_survey_kernel(ForkArgs A) {
  __shared__ int lds[kThreads / 64];
  if ((int)blockIdx.x < A.p.n_chunks) {
    survey_chunk<true>(A.p, blockIdx.x, lds);
    if (blockIdx.x == 0 && threadIdx.x < 2) A.p.status[threadIdx.x] = 0;
    return;
  }
  const int s = blockIdx.x - A.p.n_chunks;
  const int p = A.parents[s];
  const bool has = (unsigned)p < (unsigned)A.p.rows;
  int before = 0;
  for (int i = threadIdx.x; has && i < s; i += kThreads) before |= A.parents[i] == p;
  const bool eldest = !__syncthreads_or(before) && has;
  const Row r = row_of(A, s, eldest);
  int n = 0;
  for (int j = r.full + threadIdx.x; j < r.last; j += kThreads) n += !stays(A, r, named(A, r, j));
  n = block_sum(n, lds);
  if (threadIdx.x == 0) A.asked[s] = n | (eldest ? kEldest : 0);
}

// The free pages of ranks rank .. rank + n - 1 (n at most kThreads) to list[0 ..
// n - 1]: the chunks that hold them by the sums of the chunks' counts, then those
// chunks' pages themselves.
struct Finder {
  int sums[kThreads / 64], start[kThreads], first, last, list[kThreads];
};
struct Counted {   // of the first kThreads chunks: the thread's, the free pages before it, and in all of them
  int c, begin, total;
};
__device__ __forceinline__ void free_pages(const PoolArgs& A, const Counted& head, int rank, int n, Finder& f) {
  const int tid = threadIdx.x;
  int at = 0;
  for (int base = 0; base < A.n_chunks && at < rank + n; base += kThreads) {
    int c = head.c, begin = head.begin, total = head.total;
    if (base > 0) {
      c = base + tid < A.n_chunks ? A.counts[base + tid] : 0;
      begin = at + block_before(c, total, f.sums);
    }
    f.start[tid] = begin;
    if (tid == 0) f.first = kThreads, f.last = -1;
    __syncthreads();
    if (begin < rank + n && begin + c > rank) {
      atomicMin(&f.first, tid);
      atomicMax(&f.last, tid);
    }
    __syncthreads();
    const int first = f.first, last = f.last;
    for (int i = first; i <= last; ++i) {
      const Eight e = load_uses(A, base + i, 1);
      int mine = 0, all;
#pragma unroll
      for (int k = 0; k < 8; ++k) mine += e.u[k] <= 0;
      int r = f.start[i] + block_before(mine, all, f.sums) - rank;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e.u[k] <= 0) {
          if ((unsigned)r < (unsigned)n) f.list[r] = (base + i) * kChunk + tid * 8 + k;
          ++r;
        }
    }
    at += total;
    __syncthreads();
  }
}

// Part `slice` of page `from` over page `to`; scales with the first.  kOnce: past the
// caches, for pages that nobody reads soon (3,400 pages, 505 MB in and out: 104.4 us so,
// 113.1 through them, 108.2 with the stores alone past them).
template <bool kOnce>
__device__ __forceinline__ void copy_page(const PoolArgs& A, int from, int to, int slice) {
  const int64_t units = A.page_bytes / 16, all = 2 * units;   // keys, then values
  const int64_t a = all * slice / A.slices, b = all * (slice + 1) / A.slices;
  auto at = [&](int page, int64_t u) {
    return reinterpret_cast<u32x4*>((u < units ? A.k : A.v) + (size_t)page * A.page_bytes) + (u < units ? u : u - units);
  };
  for (int64_t u0 = a + threadIdx.x; u0 < b; u0 += 4 * kThreads) {
    u32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (u0 + i * kThreads < b) x[i] = kOnce ? __builtin_nontemporal_load(at(from, u0 + i * kThreads)) : *at(from, u0 + i * kThreads);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (u0 + i * kThreads < b) {
        if (kOnce)
          __builtin_nontemporal_store(x[i], at(to, u0 + i * kThreads));
        else
          *at(to, u0 + i * kThreads) = x[i];
      }
  }
  if (slice == 0)
    for (int h = threadIdx.x; h < A.hkv; h += kThreads) {
      A.ks[(size_t)to * A.hkv + h] = A.ks[(size_t)from * A.hkv + h];
      A.vs[(size_t)to * A.hkv + h] = A.vs[(size_t)from * A.hkv + h];
    }
}

// Grid: n_new * slices workgroups for the new rows (the first of a row writes
// its entries, all copy their part of its page), then one for each present row.
__global__ __launch_bounds__(kThreads) void fork_kernel(ForkArgs A) {
  __shared__ Finder f;
  const int tid = threadIdx.x, made = A.n_new * A.p.slices;
  const bool old_row = (int)blockIdx.x >= made;
  const int s = old_row ? 0 : blockIdx.x / A.p.slices, slice = old_row ? 0 : blockIdx.x % A.p.slices;
  Row r{};
  int partial = -1;   // the page whose tokens have to be copied
  if (old_row) {
    const int p = blockIdx.x - made;
    int has_heir = 0;
    for (int i = tid; i < A.n_new; i += kThreads) has_heir |= A.parents[i] == p;
    if (__syncthreads_or(has_heir)) return;
    r.old = A.p.table + (size_t)p * A.p.wide;
    r.parent = p;
  } else {
    r = row_of(A, s, (A.asked[s] & kEldest) != 0);
    if (r.len & ((1 << A.page_shift) - 1)) {
      partial = named(A, r, r.full);
      if (stays(A, r, partial)) partial = -1;
    }
    if (slice > 0 && partial < 0) return;
  }
  // what is free, what is asked for, and by the rows before this one
  Counted head;
  int free = 0, asked = 0, before = 0;
  head.c = tid < A.p.n_chunks ? A.p.counts[tid] : 0;
  for (int i = kThreads + tid; i < A.p.n_chunks; i += kThreads) free += A.p.counts[i];
  for (int i = tid; i < A.n_new; i += kThreads) {
    const int n = A.asked[i] & ~kEldest;
    asked += n;
    before += i < s ? n : 0;
  }
  __shared__ int4 of_wave[kThreads / 64];
  const int up_to = wave_inclusive_sum(head.c);
  free = wave_inclusive_sum(free);
  asked = wave_inclusive_sum(asked);
  before = wave_inclusive_sum(before);
  if ((tid & 63) == 63) of_wave[tid >> 6] = int4{up_to, free, asked, before};
  __syncthreads();
  head.begin = up_to - head.c;
  head.total = free = asked = before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    const int4 x = of_wave[w];
    head.begin += w < tid >> 6 ? x.x : 0;
    head.total += x.x;
    free += x.y;
    asked += x.z;
    before += x.w;
  }
  free += head.total;
  const bool done = asked <= free;
  if (blockIdx.x == 0 && tid == 0) {
    atomicAdd(A.p.status, done ? free - asked : free);
    A.p.status[1] = max(asked - free, 0);
  }
  int freed = 0, to = -1;   // to: where the partial page goes, the first that the row takes
  auto give_up = [&](int id) { freed += atomicSub(A.p.uses_out + id, 1) == 1; };
  if (old_row) {
    if (done)
      for (int j = tid; j < A.p.wide; j += kThreads)
        if (const int id = named(A, r, j); id >= 0) give_up(id);
  } else if (slice == 0) {
    int rank = before;
    for (int j0 = 0; j0 < A.p.wide; j0 += kThreads) {
      const int j = j0 + tid, id = named(A, r, j);
      const bool asks = j >= r.full && j < r.last, keeps = asks && stays(A, r, id), takes = asks && !keeps;
      int entry = j < r.full || keeps ? id : -1, n = 0;
      if (j0 < r.last && j0 + kThreads > r.full) {
        const int at = block_before(takes && done, n, f.sums);
        if (n > 0) {
          free_pages(A.p, head, rank, n, f);
          // an id is looked at before it is written through: counts that change meanwhile fault nothing
          if (takes) entry = (unsigned)f.list[at] < (unsigned)A.p.n_pages ? f.list[at] : -1;
          if (rank == before) to = f.list[0];
          __syncthreads();
        }
        rank += n;
      }
      if (j >= A.p.wide) continue;
      A.p.table_out[(size_t)s * A.p.wide + j] = done ? entry : -1;
      if (!done) continue;
      // the eldest takes over what its parent's entries counted for
      if (entry >= 0 && (takes || !r.eldest)) atomicAdd(A.p.uses_out + entry, 1);
      if (r.eldest && id >= 0 && j >= r.full && !keeps) give_up(id);
    }
  }
  if (!old_row && partial >= 0 && done) {
    if (slice > 0) {
      free_pages(A.p, head, before, 1, f);
      to = f.list[0];
    }
    if ((unsigned)to < (unsigned)A.p.n_pages) copy_page<false>(A.p, partial, to, slice);
  }
  freed = wave_inclusive_sum(freed);
  if ((tid & 63) == 63 && freed > 0) atomicAdd(A.p.status, freed);
}

// All of it, of one chunk and few rows: every workgroup counts and gives out for
// itself, in LDS; the first makes the table and the counts, the others copy pages.  A
// launch less is 3 us of the host's time: 32 rows of 8 sequences over 1,500 tokens, 880
// entries in both tables, take 12.5 us in a loop of calls, 16.0 in two launches.  On the
// card 6.4 and 12.1 (8.5 where the workgroups without a page to copy count too); 1,760
// entries 11.2 and 14.2, 3,600 19.1 and 21.3, 4,480 13.9 and 11.9, 8,448 26.9 and 21.5.
constexpr int kFewRows = kThreads, kFewEntries = 4096;
constexpr int kFewTaken = 8;   // entries that a first row's own thread goes through; of more all threads do

__global__ __launch_bounds__(kThreads) void fork_chunk_kernel(ForkArgs A) {
  __shared__ int uses[kChunk], counts[kChunk], first[kThreads], takes_from[kThreads], many[kThreads], n_many, lds[kThreads / 64];
  __shared__ int16_t list[kChunk];   // the free pages
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {   // nothing to copy: the parent's tokens end with a page
    const int parent = A.parents[(blockIdx.x - 1) / A.p.slices];
    if ((unsigned)parent >= (unsigned)A.p.rows || (A.kv_len[parent] & ((1 << A.page_shift) - 1)) == 0) return;
  }
  const Eight e = load_uses(A.p, 0, 1);
  const int p = tid < A.n_new ? A.parents[tid] : -1;
  const bool has = (unsigned)p < (unsigned)A.p.rows;
  int mine = 0, free, asked;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uses[tid * 8 + k] = e.u[k];
    counts[tid * 8 + k] = max(e.u[k], 0);
    mine += e.u[k] <= 0;
  }
  first[tid] = kThreads;
  if (tid == 0) n_many = 0;
  int at = block_before(mine, free, lds);   // its barriers are first's and uses' too
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e.u[k] <= 0) list[at++] = tid * 8 + k;
  if (has) atomicMin(&first[p], tid);
  __syncthreads();
  auto kept = [&](bool eldest, int id) { return eldest && id >= 0 && uses[id] == 1; };
  Row r{};
  int n = 0;
  if (tid < A.n_new) {
    r = row_of(A, tid, has && first[p] == tid);
    n = r.last - r.full;
    if (r.eldest && n > kFewTaken)
      many[atomicAdd(&n_many, 1)] = tid;
    else
      for (int j = r.full; r.eldest && j < r.last; ++j) n -= kept(true, named(A, r, j));
  }
  __syncthreads();
  for (int i = 0; i < n_many; ++i) {
    const Row row = row_of(A, many[i], true);
    int stay = 0;
    for (int j = row.full + tid; j < row.last; j += kThreads) stay += kept(true, named(A, row, j));
    stay = block_sum(stay, lds);
    if (tid == many[i]) n -= stay;
  }
  takes_from[tid] = block_before(n, asked, lds);
  __syncthreads();
  const bool done = asked <= free;
  if (blockIdx.x > 0) {
    const int s = (blockIdx.x - 1) / A.p.slices, parent = A.parents[s];
    const Row row = row_of(A, s, (unsigned)parent < (unsigned)A.p.rows && first[parent] == s);
    if (!done || !(row.len & ((1 << A.page_shift) - 1))) return;
    const int from = named(A, row, row.full);
    if (from >= 0 && !kept(row.eldest, from)) copy_page<false>(A.p, from, list[takes_from[s]], (blockIdx.x - 1) % A.p.slices);
    return;
  }
  const int wide = A.p.wide;
  for (int i = tid; i < A.n_new * wide; i += kThreads) {
    const int s = i / wide, j = i % wide, parent = A.parents[s];
    const Row row = row_of(A, s, (unsigned)parent < (unsigned)A.p.rows && first[parent] == s);
    const bool asks = j >= row.full && j < row.last;
    if (done && asks && row.eldest) continue;   // below, in order
    const int id = named(A, row, j), entry = j < row.full ? id : asks && done ? list[takes_from[s] + j - row.full] : -1;
    A.p.table_out[i] = done ? entry : -1;
    if (!done) continue;
    if (entry >= 0 && !row.eldest) atomicAdd(&counts[entry], 1);
    if (row.eldest && id >= 0 && j >= row.last) atomicSub(&counts[id], 1);
  }
  if (done) {
    auto put = [&](int s, int j, int id, int taken) {   // taken: -1 where the entry stays
      A.p.table_out[(size_t)s * wide + j] = taken < 0 ? id : taken;
      if (taken < 0) return;
      atomicAdd(&counts[taken], 1);
      if (id >= 0) atomicSub(&counts[id], 1);
    };
    if (r.eldest && r.last - r.full <= kFewTaken) {
      int next = takes_from[tid];
      for (int j = r.full; j < r.last; ++j) {
        const int id = named(A, r, j);
        put(tid, j, id, kept(true, id) ? -1 : list[next++]);
      }
    }
    for (int i = 0; i < n_many; ++i) {
      const Row row = row_of(A, many[i], true);
      int next = takes_from[many[i]];
      for (int j0 = row.full; j0 < row.last; j0 += kThreads) {
        const int j = j0 + tid, id = j < row.last ? named(A, row, j) : -1;
        const bool takes = j < row.last && !kept(true, id);
        int all;
        const int rank = block_before(takes, all, lds);
        if (j < row.last) put(many[i], j, id, takes ? list[next + rank] : -1);
        next += all;
      }
    }
    for (int i = tid; i < A.p.rows * wide; i += kThreads)   // of sequences that no row goes on from
      if (first[i / wide] == kThreads)
        if (const int id = A.p.table[i]; (unsigned)id < (unsigned)A.p.n_pages) atomicSub(&counts[id], 1);
  }
  __syncthreads();
  int left = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = tid * 8 + k;
    if (i >= A.p.n_pages) continue;
    A.p.uses_out[i] = counts[i];
    left += counts[i] <= 0;
  }
  left = block_sum(left, lds);
  if (tid == 0) {
    A.p.status[0] = left;
    A.p.status[1] = max(asked - free, 0);
  }
}

// ------------------------------------------------------------------- compact
// A pool of one chunk is numbered by every workgroup that moves pages, in LDS, in the
// one launch; a larger one by launches of their own (a launch is 3 us of the host's
// time: a third of 700 pages of 64 tokens on 8 heads of 128, 18.8 us in three, 12.3 in
// one; four chunks counted by every workgroup that numbers them, without the first
// launch, cost what that one takes: 116 us for 8,192 pages, 113 in three).
__global__ __launch_bounds__(kThreads) void compact_survey_kernel(CompactArgs A) {
  __shared__ int lds[kThreads / 64];
  survey_chunk<false>(A.p, blockIdx.x, lds);
}

// Numbers the moves: page i in use behind the first `used` is move (pages in use
// before it) - (those among the first `used`), a free one before them takes move
// (free pages before it).
__global__ __launch_bounds__(kThreads) void compact_number_kernel(CompactArgs A) {
  __shared__ int lds[kThreads / 64];
  const int tid = threadIdx.x, chunk = blockIdx.x;
  int used = 0, before = 0;
  for (int i = tid; i < A.p.n_chunks; i += kThreads) {
    const int n = A.p.counts[i];
    used += n;
    before += i < chunk ? n : 0;
  }
  used = block_sum(used, lds);
  before = block_sum(before, lds);
  // pages in use among the first `used`: whole chunks, and a part of one
  const int part = used / kChunk;
  int front = 0;
  for (int i = tid; i < part; i += kThreads) front += A.p.counts[i];
  if (part < A.p.n_chunks) {
    const Eight e = load_uses(A.p, part, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) front += e.u[i] > 0 && part * kChunk + tid * 8 + i < used;
  }
  front = block_sum(front, lds);
  if (chunk == 0 && tid == 0) {
    A.p.status[0] = used;
    A.p.status[1] = used - front;
  }
  const Eight e = load_uses(A.p, chunk, 0);
  int mine = 0, all;
#pragma unroll
  for (int i = 0; i < 8; ++i) mine += e.u[i] > 0;
  int rank = before + block_before(mine, all, lds);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = chunk * kChunk + tid * 8 + k;
    const bool taken = e.u[k] > 0;
    if (taken && i >= used) {
      A.src[rank - front] = i;
      A.number[i] = rank - front;
    } else if (!taken && i < used) {
      A.dst[i - rank] = i;
    }
    rank += taken;
  }
}

// Grid: `movers` workgroups that take turns at the moves' parts, then those for
// the table's entries.
__global__ __launch_bounds__(kThreads) void compact_move_kernel(CompactArgs A, int movers) {
  const int tid = threadIdx.x, used = A.p.status[0], moves = A.p.status[1];
  if ((int)blockIdx.x < movers) {
    const int64_t parts = (int64_t)moves * A.p.slices;
    for (int64_t i = blockIdx.x; i < parts; i += movers) {
      const int m = (int)(i / A.p.slices), slice = (int)(i % A.p.slices), from = A.src[m], to = A.dst[m];
      if ((unsigned)from >= (unsigned)A.p.n_pages || (unsigned)to >= (unsigned)A.p.n_pages) continue;
      copy_page<true>(A.p, from, to, slice);
      if (slice == 0 && tid == 0) {
        A.p.uses_out[to] = A.p.uses[from];
        A.p.uses_out[from] = 0;
      }
    }
    return;
  }
  const int64_t entries = (int64_t)A.p.rows * A.p.wide;
  for (int64_t i = (int64_t)(blockIdx.x - movers) * kThreads + tid; i < entries; i += (int64_t)(gridDim.x - movers) * kThreads) {
    int id = A.p.table[i];
    if (id >= used && id < A.p.n_pages && A.p.uses[id] > 0) id = A.dst[A.number[id]];
    A.p.table_out[i] = id;
  }
}

// All of it, of one chunk.  Grid as the one above; the first workgroup for the
// table's entries writes counts and status too.
__global__ __launch_bounds__(kThreads) void compact_chunk_kernel(CompactArgs A, int movers) {
  __shared__ int lds[kThreads / 64];
  __shared__ int16_t src[kChunk / 2 + 1], dst[kChunk / 2 + 1], number[kChunk];
  const int tid = threadIdx.x;
  const Eight e = load_uses(A.p, 0, 0);
  int mine = 0, used;
#pragma unroll
  for (int k = 0; k < 8; ++k) mine += e.u[k] > 0;
  const int before = block_before(mine, used, lds);
  int front = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) front += e.u[k] > 0 && tid * 8 + k < used;
  front = block_sum(front, lds);
  int rank = before;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = tid * 8 + k;
    const bool taken = e.u[k] > 0;
    number[i] = -1;
    if (taken && i >= used)
      src[rank - front] = i, number[i] = rank - front;
    else if (!taken && i < used)
      dst[i - rank] = i;
    rank += taken;
  }
  __syncthreads();
  const int moves = used - front;
  if ((int)blockIdx.x < movers) {
    for (int i = blockIdx.x; i < moves * A.p.slices; i += movers) copy_page<true>(A.p, src[i / A.p.slices], dst[i / A.p.slices], i % A.p.slices);
    return;
  }
  if ((int)blockIdx.x == movers) {
    rank = before;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = tid * 8 + k;
      const bool taken = e.u[k] > 0;
      if (i < A.p.n_pages) A.p.uses_out[i] = i >= used ? 0 : taken ? e.u[k] : A.p.uses[src[i - rank]];
      rank += taken;
    }
    if (tid == 0) {
      A.p.status[0] = used;
      A.p.status[1] = moves;
    }
  }
  const int64_t entries = (int64_t)A.p.rows * A.p.wide;
  for (int64_t i = (int64_t)(blockIdx.x - movers) * kThreads + tid; i < entries; i += (int64_t)(gridDim.x - movers) * kThreads) {
    int id = A.p.table[i];
    if ((unsigned)id < (unsigned)A.p.n_pages && number[id] >= 0) id = dst[number[id]];
    A.p.table_out[i] = id;
  }
}

// -------------------------------------------------------------------- checks
size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
int chunks_of(int n_pages) { return (n_pages + kChunk - 1) / kChunk; }
size_t counts_bytes(int n_pages) { return rounded((size_t)chunks_of(n_pages) * 4); }
size_t moves_bytes(int n_pages) { return rounded(((size_t)n_pages / 2 + 1) * 4); }
size_t fork_bytes(int n_pages, int n_new) { return counts_bytes(n_pages) + (size_t)n_new * 4; }
size_t compact_bytes(int n_pages) { return counts_bytes(n_pages) + 2 * moves_bytes(n_pages) + (size_t)n_pages * 4; }

int check_pool(const char* who, int n_pages, int rows, const char* rows_name) {
  if (n_pages < 1 || n_pages > DB_MAX_PAGES)
    return dh::fail(DH_ESHAPE, "%s: n_pages must be in 1..%d (got %d)", who, DB_MAX_PAGES, n_pages);
  if (rows < 1 || rows > DL_MAX_SEQS) return dh::fail(DH_ESHAPE, "%s: %s must be in 1..%d (got %d)", who, rows_name, DL_MAX_SEQS, rows);
  return DH_OK;
}

// What fork and compact have in common; `made` is the new table's rows, `lists` what else is read.
int check_pages(const char* who, PoolArgs& A, int page, int D, int made, const char* rows_name, const Span (&lists)[3], void* workspace,
                size_t given, size_t need) {
  int rc = check_heads(who, A.hkv, A.hkv, D);
  if (rc) return rc;
  if ((rc = check_pool(who, A.n_pages, A.rows, rows_name))) return rc;
  // the table stands in for the row starts and lengths, which these calls do not have
  const Batch b{A.table, A.table, A.table, A.rows, A.wide, 0};
  if ((rc = check_cache(who, Cache{A.k, A.v, A.ks, A.vs, A.n_pages, page_shift_of(page), A.hkv}, page, b))) return rc;
  if (!A.uses || !A.uses_out || !A.table_out || !A.status) return dh::fail(DH_EINVAL, "%s: null pointer", who);
  if (!aligned(A.uses, 4) || !aligned(A.uses_out, 4) || !aligned(A.table_out, 4) || !aligned(A.status, 4))
    return dh::fail(DH_EINVAL, "%s: counts, tables and status must be 4-byte aligned", who);
  const size_t counts = (size_t)A.n_pages * 4, old = (size_t)A.rows * A.wide * 4, made_bytes = (size_t)made * A.wide * 4;
  // the kernels go by what they have left in them, and by the inputs, in more than one launch
  const Span present[] = {{A.uses, counts}, {A.table, old}, lists[0], lists[1], lists[2]}, out[] = {{A.uses_out, counts}, {A.table_out, made_bytes}, {A.status, 8}};
  for (int o = 0; o < 3; ++o) {
    for (const Span& i : present)
      if (overlap(out[o], i)) return dh::fail(DH_EINVAL, "%s: the new counts, table and status must not overlap the inputs", who);
    if (overlap(out[o], out[(o + 1) % 3])) return dh::fail(DH_EINVAL, "%s: the new counts, table and status must not overlap each other", who);
  }
  if (!workspace || !aligned(workspace, 16)) return dh::fail(DH_EINVAL, "%s: workspace must be a 16-byte aligned pointer", who);
  if (given < need) return dh::fail(DH_EINVAL, "%s: workspace of %zu bytes is below the %zu needed", who, given, need);
  A.page_bytes = (int64_t)A.hkv * page * D;
  // so it is with the workspace, and pages are written while all of them are read
  const size_t codes = (size_t)A.n_pages * A.page_bytes, scales = (size_t)A.n_pages * A.hkv * 4;
  const Span scratch{workspace, need}, pool[] = {{A.k, codes}, {A.v, codes}, {A.ks, scales}, {A.vs, scales}, scratch};
  for (const Span& p : pool) {
    if (&p != &pool[4] && overlap(p, scratch)) return dh::fail(DH_EINVAL, "%s: the workspace must not overlap the cache", who);
    for (const Span& i : present)
      if (overlap(p, i)) return dh::fail(DH_EINVAL, "%s: the counts, table and lists must not overlap the cache or the workspace", who);
    for (const Span& o : out)
      if (overlap(p, o)) return dh::fail(DH_EINVAL, "%s: the new counts, table and status must not overlap the cache or the workspace", who);
  }
  A.n_chunks = chunks_of(A.n_pages);
  A.slices = (int)std::min<int64_t>(std::max<int64_t>(2 * A.page_bytes / kSlice, 1), 128);
  A.counts = static_cast<int32_t*>(workspace);
  return DH_OK;
}

}  // namespace

extern "C" {

int draft_branch_pages_workspace_bytes(int n_pages, int n_new, size_t* bytes) {
  if (!bytes) return dh::fail(DH_EINVAL, "pages_workspace_bytes: null pointer");
  const int rc = check_pool("pages_workspace_bytes", n_pages, n_new, "n_new");
  if (rc) return rc;
  *bytes = std::max(fork_bytes(n_pages, n_new), compact_bytes(n_pages));
  return dh::ok();
}

int draft_branch_fork(uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page, int hkv,
                      int D, const int32_t* uses, const int32_t* table, const int32_t* kv_len, int n_seq,
                      const int32_t* parents, const int32_t* need, int n_new, int max_pages, int32_t* uses_out,
                      int32_t* table_out, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "fork";
  ForkArgs A{};
  A.p = PoolArgs{k_codes, v_codes, k_scale, v_scale, n_pages, hkv, 0, 0, 0, uses, table, uses_out, table_out, status, n_seq, max_pages, nullptr};
  int rc = check_pool(who, n_pages, n_new, "n_new");
  if (rc) return rc;
  if ((int64_t)n_new * max_pages > INT32_MAX)   // the entries that ask are counted in 32 bits
    return dh::fail(DH_ESHAPE, "fork: n_new * max_pages must be below 2^31 (got %d * %d)", n_new, max_pages);
  const Span lists[3] = {{kv_len, (size_t)std::max(n_seq, 0) * 4}, {parents, (size_t)n_new * 4}, {need, (size_t)n_new * 4}};
  if ((rc = check_pages(who, A.p, page, D, n_new, "n_seq", lists, workspace, workspace_bytes, fork_bytes(n_pages, n_new)))) return rc;
  if (!kv_len || !parents || !need) return dh::fail(DH_EINVAL, "fork: null pointer");
  if (!aligned(kv_len, 4) || !aligned(parents, 4) || !aligned(need, 4))
    return dh::fail(DH_EINVAL, "fork: kv_len, parents and need must be 4-byte aligned");
  A.kv_len = kv_len;
  A.parents = parents;
  A.need = need;
  A.n_new = n_new;
  A.page_shift = page_shift_of(page);
  A.asked = A.p.counts + counts_bytes(n_pages) / 4;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (A.p.n_chunks == 1 && n_new <= kFewRows && n_seq <= kFewRows && (int64_t)(n_new + n_seq) * max_pages <= kFewEntries) {
    hipLaunchKernelGGL(fork_chunk_kernel, dim3(1 + n_new * A.p.slices), dim3(kThreads), 0, st, A);
    return launched("fork_chunk_kernel");
  }
  hipLaunchKernelGGL(fork_survey_kernel, dim3(A.p.n_chunks + n_new), dim3(kThreads), 0, st, A);
  hipLaunchKernelGGL(fork_kernel, dim3(n_new * A.p.slices + n_seq), dim3(kThreads), 0, st, A);
  return launched("fork_kernel");
}

int draft_branch_compact(uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page,
                         int hkv, int D, const int32_t* uses, const int32_t* table, int n_rows, int max_pages,
                         int32_t* uses_out, int32_t* table_out, int32_t* status, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const char* who = "compact";
  CompactArgs A{};
  A.p = PoolArgs{k_codes, v_codes, k_scale, v_scale, n_pages, hkv, 0, 0, 0, uses, table, uses_out, table_out, status, n_rows, max_pages, nullptr};
  const int rc = check_pages(who, A.p, page, D, n_rows, "n_rows", {}, workspace, workspace_bytes, compact_bytes(n_pages));
  if (rc) return rc;
  A.src = A.p.counts + counts_bytes(n_pages) / 4;
  A.dst = A.src + moves_bytes(n_pages) / 4;
  A.number = A.dst + moves_bytes(n_pages) / 4;
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  // eight rounds of a card's workgroups, so that those that get on faster take more (3,400
  // pages: 2,048 workgroups 104.5 us, 4,096 100.9, 8,192 96.7, 16,384 93.4, 32,768 95.5); one round where each numbers
  // the moves for itself; a move at most for every second page
  const int64_t parts = std::max<int64_t>((int64_t)(n_pages / 2) * A.p.slices, 1);
  const int movers = (int)std::min<int64_t>(A.p.n_chunks == 1 ? 2048 : 16384, parts);
  const int entries = (int)std::min<int64_t>(256, ((int64_t)n_rows * max_pages + kThreads - 1) / kThreads);
  if (A.p.n_chunks == 1) {
    hipLaunchKernelGGL(compact_chunk_kernel, dim3(movers + entries), dim3(kThreads), 0, st, A, movers);
    return launched("compact_chunk_kernel");
  }
  hipLaunchKernelGGL(compact_survey_kernel, dim3(A.p.n_chunks), dim3(kThreads), 0, st, A);
  hipLaunchKernelGGL(compact_number_kernel, dim3(A.p.n_chunks), dim3(kThreads), 0, st, A);
  hipLaunchKernelGGL(compact_move_kernel, dim3(movers + entries), dim3(kThreads), 0, st, A, movers);
  return launched("compact_move_kernel");
}

}  // extern "C"
