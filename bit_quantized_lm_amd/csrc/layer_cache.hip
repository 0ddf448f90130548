// The draft layer's cache on gfx950: rotary positions, the 8-bit write and
// the reading back (draft_layer_append, draft_layer_read).
#include <algorithm>

#include "layer.h"

namespace {

using namespace dl;

struct AppendArgs {
  Batch b;
  Cache c;
  const uint16_t *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const u32x4* rope;   // [positions][rot/2] of (cos, sin), two an element
  int rot, interleaved, hq;
  uint16_t* q_out;
  int q_blocks;        // workgroups that rotate queries, before those that write pages
};

constexpr int kThreads = 256;

// Sixteen of a head's elements as two runs of eight, starting at d0 and d1:
// unit u < rot/16 holds eight rotary pairs ((d0 + i, d1 + i) in halves, or
// (2i, 2i + 1) of the sixteen from 16u interleaved), a later one sixteen
// elements that no rotation touches.
struct Place {
  int d0, d1;
  bool turned, halves;
};
__device__ __forceinline__ Place place_of(int u, int rot, bool interleaved) {
  Place p;
  p.turned = u * 16 < rot;
  p.halves = p.turned && !interleaved;
  p.d0 = p.halves ? 8 * u : 16 * u;
  p.d1 = p.halves ? 8 * u + rot / 2 : 16 * u + 8;
  return p;
}

struct Turn {   // cos and sin of a unit's eight pairs
  u32x4 cs[4];
};
__device__ __forceinline__ Turn load_turn(const u32x4* __restrict__ rope, int64_t position, int rot, int u) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) t.cs[i] = rope[position * (rot / 4) + 4 * u + i];
  return t;
}

struct Unit {
  float x[16];
};

// Each operation is rounded on its own (no fused multiply-add), so that the
// result is what the documented fp32 steps give, bit for bit.
__device__ __forceinline__ Unit make_unit(u32x4 a, u32x4 b, const Turn& turn, const Place& p) {
#pragma clang fp contract(off)
  Unit r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = bf16_lo(a[i]);
    r.x[2 * i + 1] = bf16_hi(a[i]);
    r.x[8 + 2 * i] = bf16_lo(b[i]);
    r.x[8 + 2 * i + 1] = bf16_hi(b[i]);
  }
  auto turn_pair = [&](float& xa, float& xb, int i) {
#pragma clang fp contract(off)
    const float c = __uint_as_float(turn.cs[i / 2][i % 2 * 2]), s = __uint_as_float(turn.cs[i / 2][i % 2 * 2 + 1]);
    const float ac = xa * c, bs = xb * s, bc = xb * c, as = xa * s;
    xa = ac - bs;
    xb = bc + as;
  };
  if (p.halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[i], r.x[8 + i], i);
  } else if (p.turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[2 * i], r.x[2 * i + 1], i);
  }
  return r;
}

__device__ __forceinline__ u32x4 load8(const uint16_t* at) { return *reinterpret_cast<const u32x4*>(at); }

__device__ __forceinline__ u32x4 pack8(const float* x) {
  return u32x4{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
}

__device__ __forceinline__ uint32_t code_of(float x, float inv) {
#pragma clang fp contract(off)
  const float c = fminf(fmaxf(__builtin_rintf(x * inv), -127.0f), 127.0f);
  return (uint32_t)((int)c + 128);
}

__device__ __forceinline__ uint32_t again(uint32_t code, float ratio) {
#pragma clang fp contract(off)
  return (uint32_t)((int)__builtin_rintf((float)((int)code - 128) * ratio) + 128);
}

// Rotates the queries, a row a wave: a lane keeps one unit's cosines and sines
// for all heads of the row (64/U heads a turn of the wave).
template <int D>
__device__ __forceinline__ void rotate_queries(const AppendArgs& A) {
  constexpr int U = D / 16;
  const int lane = threadIdx.x & 63, u = lane % U, r = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (r >= A.b.T) return;
  // the row's sequence: the last that starts at or before it, 64 a look
  int s = -1;
  for (int base = 0; base < A.b.n_seq; base += 64) {
    const int before = __popcll(__ballot(base + lane < A.b.n_seq && A.b.q_start[min(base + lane, A.b.n_seq - 1)] <= r));
    s += before;
    if (before < 64) break;
  }
  const Seq q = load_seq(A.b, max(s, 0));
  const int last = (A.b.max_pages << A.c.page_shift) - 1, position = min(max(q.begin + r - q.row0, 0), last);
  const Place p = place_of(u, A.rot, A.interleaved);
  const Turn turn = p.turned ? load_turn(A.rope, position, A.rot, u) : Turn{};
  const uint16_t* in = A.q + r * A.ldq;
  uint16_t* out = A.q_out + (size_t)r * A.hq * D;
#pragma unroll 4
  for (int h = lane / U; h < A.hq; h += 64 / U) {
    const Unit x = make_unit(load8(in + h * D + p.d0), load8(in + h * D + p.d1), turn, p);
    *reinterpret_cast<u32x4*>(out + h * D + p.d0) = pack8(x.x);
    *reinterpret_cast<u32x4*>(out + h * D + p.d1) = pack8(x.x + 8);
  }
}

// One (page, head) of keys or values: the scale from the new values' largest
// magnitude, the new codes in LDS in the fragment order, then its 16-byte units
// out of LDS.  The page has one writer, so an older token's code is re-rounded
// here without a race, and only where the scale rose.  Values that a thread has
// read for the scale it keeps for the codes, as far as its registers go; a
// larger page's are read again.
//
// largest() gives the largest magnitude's bits: magnitudes compare as integers,
// infinity above all numbers and NaN above it, so none is lost on the way. A page
// that takes one of them gets the scale NaN, whatever the codes: its tokens' values
// are NaN from then on, and no number is made of what is none.
struct Page {
  const uint16_t* x;   // token 0's head (tokens before t0 are not there)
  int64_t ld;
  int p0, t0, t1;      // position of token 0; new tokens
};

// Keys: a unit of a token a thread and turn.
template <int D>
struct KeyCodes {
  static constexpr int kKept = 2;
  Unit kept[kKept];
  __device__ __forceinline__ Unit unit(const AppendArgs& A, const Page& g, int i) const {
    const int t = g.t0 + i / (D / 16), u = i % (D / 16);
    const Place p = place_of(u, A.rot, A.interleaved);
    const uint16_t* at = g.x + t * g.ld;
    return make_unit(load8(at + p.d0), load8(at + p.d1), p.turned ? load_turn(A.rope, g.p0 + t, A.rot, u) : Turn{}, p);
  }
  __device__ __forceinline__ uint32_t largest(const AppendArgs& A, const Page& g) {
    const int units = (g.t1 - g.t0) * (D / 16);
    uint32_t top = 0u;
    auto take = [&](const Unit& x) {
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x.x[j]) & 0x7FFFFFFFu);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < units) take(kept[k] = unit(A, g, i));
    }
    for (int i = threadIdx.x + kKept * kThreads; i < units; i += kThreads) take(unit(A, g, i));
    return top;
  }
  __device__ __forceinline__ void write(const AppendArgs& A, const Page& g, float inv, uint8_t* lds) const {
    const int units = (g.t1 - g.t0) * (D / 16);
    auto put = [&](const Unit& x, int i) {
      const int t = g.t0 + i / (D / 16);
      const Place p = place_of(i % (D / 16), A.rot, A.interleaved);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j >> 2] |= code_of(x.x[j], inv) << (8 * (j & 3));
      auto at = [&](int e) {
        return lds + t / 32 * 32 * D + ((t % 32 / 16 * (D / 64) + e / 64) * 64 + e % 64 / 16 * 16 + t % 16) * 16 + e % 16;
      };
      *reinterpret_cast<u32x2*>(at(p.d0)) = u32x2{w[0], w[1]};
      *reinterpret_cast<u32x2*>(at(p.d1)) = u32x2{w[2], w[3]};
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < units) put(kept[k], i);
    }
    for (int i = threadIdx.x + kKept * kThreads; i < units; i += kThreads) put(unit(A, g, i), i);
  }
  // token of byte j of the fragment order's unit i
  static __device__ __forceinline__ int token(int i, int) { return i / (2 * D) * 32 + i % (2 * D) / 64 / (D / 64) * 16 + (i & 15); }
};

// Values: eight elements of four tokens a thread and turn, whose codes stand in
// fours of one element in the fragment order.
template <int D>
struct ValueCodes {
  static constexpr int kKept = 2;
  struct Four {
    u32x4 x[4];
  };
  Four kept[kKept];
  static __device__ __forceinline__ int quads(const Page& g) { return ((g.t1 - 1) / 4 - g.t0 / 4 + 1) * (D / 8); }
  __device__ __forceinline__ Four four(const Page& g, int i) const {
    const int t = (g.t0 / 4 + i / (D / 8)) * 4, e = i % (D / 8) * 8;
    Four f;
#pragma unroll
    for (int k = 0; k < 4; ++k) f.x[k] = t + k >= g.t0 && t + k < g.t1 ? load8(g.x + (t + k) * g.ld + e) : u32x4{0u, 0u, 0u, 0u};
    return f;
  }
  __device__ __forceinline__ uint32_t largest(const AppendArgs&, const Page& g) {
    const int n = quads(g);
    uint32_t top = 0u;
    auto take = [&](const Four& f) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(f.x[k][j] & 0x7FFFu, f.x[k][j] >> 16 & 0x7FFFu));
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < n) take(kept[k] = four(g, i));
    }
    for (int i = threadIdx.x + kKept * kThreads; i < n; i += kThreads) take(four(g, i));
    return top << 16;
  }
  __device__ __forceinline__ void write(const AppendArgs&, const Page& g, float inv, uint8_t* lds) const {
    const int n = quads(g);
    auto put = [&](const Four& f, int i) {
      const int t = (g.t0 / 4 + i / (D / 8)) * 4, e0 = i % (D / 8) * 8;
      uint8_t* at = lds + t / 32 * 32 * D + ((e0 / 32 * 4 + t % 16 / 4) * 16 + e0 % 16) * 16 + e0 % 32 / 16 * 8 + t % 32 / 16 * 4;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) w |= code_of(j % 2 ? bf16_hi(f.x[k][j / 2]) : bf16_lo(f.x[k][j / 2]), inv) << (8 * k);
        *reinterpret_cast<uint32_t*>(at + j * 16) = w;
      }
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = threadIdx.x + k * kThreads;
      if (i < n) put(kept[k], i);
    }
    for (int i = threadIdx.x + kKept * kThreads; i < n; i += kThreads) put(four(g, i), i);
  }
  static __device__ __forceinline__ int token(int i, int j) { return i / (2 * D) * 32 + i % 64 / 16 * 4 + j % 8 / 4 * 16 + j % 4; }
};

template <int D, class Codes>
__device__ __forceinline__ void write_page(const AppendArgs& A, int s, int page_no, int head, const uint16_t* x, int64_t ld,
                                           uint8_t* codes_base, float* scale_base, uint8_t* lds) {
#pragma clang fp contract(off)
  __shared__ uint32_t wave_top[kThreads / 64];
  const int tid = threadIdx.x, page = 1 << A.c.page_shift;
  const int id = page_id(A.b, A.c.n_pages, s, page_no);
  if (id < 0) return;
  const Seq q = load_seq(A.b, s);
  Page g;
  g.p0 = page_no << A.c.page_shift;
  g.t0 = max(q.begin - g.p0, 0);
  g.t1 = min(q.len - g.p0, page);
  g.x = x + ((int64_t)q.row0 + g.p0 - q.begin) * ld + head * D;
  g.ld = ld;
  float* scale = scale_base + (size_t)id * A.c.hkv + head;
  u32x4* codes = reinterpret_cast<u32x4*>(codes_base + ((size_t)id * A.c.hkv + head) * ((size_t)page * D));
  Codes values;
  uint32_t top = wave_max(values.largest(A, g));
  if ((tid & 63) == 0) wave_top[tid >> 6] = top;
  const float before = *scale;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = max(top, wave_top[w]);
  float step = fmaxf(__uint_as_float(top) / 127.0f, kMinScale);
  if (g.t0 > 0) step = fmaxf(step, before);
  if (top >= kNotFinite || (g.t0 > 0 && (__float_as_uint(before) & 0x7FFFFFFFu) >= kNotFinite)) step = __builtin_nanf("");
  const float ratio = before / step;
  const bool raised = g.t0 > 0 && step > before;
  values.write(A, g, 1.0f / step, lds);
  __syncthreads();
  if (tid == 0) *scale = step;
  const u32x4* made = reinterpret_cast<const u32x4*>(lds);
  for (int i = tid; i < page * (D / 16); i += kThreads) {
    const int first = Codes::token(i, 0), last = Codes::token(i, 15);
    if (first >= g.t0 && last < g.t1) {
      codes[i] = made[i];
      continue;
    }
    if (first >= g.t1 || (last < g.t0 && !raised)) continue;
    u32x4 w = codes[i];
    const u32x4 n = made[i];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int t = Codes::token(i, j);
      uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 255u;
      if (t >= g.t0 && t < g.t1)
        c = (n[j >> 2] >> (8 * (j & 3))) & 255u;
      else if (raised && t < g.t0)
        c = again(c, ratio);
      w[j >> 2] = (w[j >> 2] & ~(255u << (8 * (j & 3)))) | c << (8 * (j & 3));
    }
    codes[i] = w;
  }
}

// Grid: q_blocks workgroups for the queries, then one per (page that a new
// token touches, head, keys or values).  Bound by memory: prompts of four
// sequences, 287 MB in and out, 58 us (5.0 TB/s against 4.8 for a large copy); one
// token 5.3 us, a launch and its chain of loads (lengths, page, old scale).  Where
// every call raises the old scales, so that older codes are re-rounded, the times are
// the same (56.2 and 56.3 us in a captured graph, one token 4.2 and 5.2).
template <int D>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs A) {
  extern __shared__ __align__(16) uint8_t lds[];
  if ((int)blockIdx.x < A.q_blocks) {
    rotate_queries<D>(A);
    return;
  }
  const int w = blockIdx.x - A.q_blocks, kind = w & 1, head = (w >> 1) % A.c.hkv;
  int s, j;
  const int shift = A.c.page_shift;
  auto pages = [&](const Seq& q) {
    const int end = min(q.len, A.b.max_pages << shift), first = max(q.begin, 0);
    return q.n > 0 && end > first ? ((end - 1) >> shift) - (first >> shift) + 1 : 0;
  };
  if (!find_item(A.b, (w >> 1) / A.c.hkv, pages, s, j)) return;
  s = __builtin_amdgcn_readfirstlane(s);
  j = __builtin_amdgcn_readfirstlane(j) + (max(load_seq(A.b, s).begin, 0) >> shift);
  if (kind == 0)
    write_page<D, KeyCodes<D>>(A, s, j, head, A.k, A.ldk, A.c.k, A.c.ks, lds);
  else
    write_page<D, ValueCodes<D>>(A, s, j, head, A.v, A.ldv, A.c.v, A.c.vs, lds);
}

struct ReadArgs {
  Batch b;
  Cache c;
  uint16_t *k_out, *v_out;
};

// Reading back: a wave takes one head's 32 tokens of one sequence (a group of
// the fragment order; its values pass through LDS, where they turn from eight
// tokens a lane into rows of one).  Bound by memory: eight long contexts, 371 MB
// in and out, 82 us (4.5 TB/s against 4.8 for a large copy).
template <int D>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs A) {
  __shared__ __align__(16) uint16_t lds[kThreads / 64][32][D + 8];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int hblocks = (A.c.hkv + kThreads / 64 - 1) / (kThreads / 64);
  const int head = blockIdx.x % hblocks * (kThreads / 64) + wave;
  int s, j;
  auto groups = [&](const Seq& q) { return q.n > 0 ? ((q.len - 1) >> 5) - (q.begin >> 5) + 1 : 0; };
  if (!find_item(A.b, blockIdx.x / hblocks, groups, s, j)) return;
  s = __builtin_amdgcn_readfirstlane(s);
  const Seq q = load_seq(A.b, s);
  const int g = __builtin_amdgcn_readfirstlane(j) + (q.begin >> 5);   // group of positions 32 g ..
  if (head < A.c.hkv) {
    const int page = 1 << A.c.page_shift;
    const int id = g < 0 ? -1 : page_id(A.b, A.c.n_pages, s, g >> (A.c.page_shift - 5));
    const size_t at = ((size_t)max(id, 0) * A.c.hkv + head);
    const size_t off = at * ((size_t)page * D) + (size_t)(max(g, 0) & ((page >> 5) - 1)) * 32 * D;
    const float ks = id < 0 ? 0.0f : A.c.ks[at], vs = id < 0 ? 0.0f : A.c.vs[at];
    const u32x4* kc = reinterpret_cast<const u32x4*>(A.c.k + off);
    const u32x4* vc = reinterpret_cast<const u32x4*>(A.c.v + off);
    const int hi = lane >> 4, lo = lane & 15;
    const int64_t row0 = (int64_t)q.row0 - q.begin + g * 32;   // row of the group's token 0
    const int t0 = max(q.begin - g * 32, 0), t1 = min(q.len - g * 32, 32);
    const u32x4 none = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
    const size_t ld = (size_t)A.c.hkv * D;
#pragma unroll
    for (int f = 0; f < D / 32; ++f) {
      const int t = f / (D / 64) * 16 + lo, e = f % (D / 64) * 64 + hi * 16;
      const u32x4 w = id < 0 ? none : kc[f * 64 + lane];
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = (float)((int)((w[i >> 2] >> (8 * (i & 3))) & 255u) - 128) * ks;
      if (t >= t0 && t < t1) {
        u32x4* out = reinterpret_cast<u32x4*>(A.k_out + (row0 + t) * ld + head * D + e);
        out[0] = pack8(x);
        out[1] = pack8(x + 8);
      }
    }
#pragma unroll
    for (int f = 0; f < D / 32; ++f) {
      const u32x4 w = id < 0 ? none : vc[f * 64 + lane];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = (float)((int)((w[i >> 2] >> (8 * (i & 3))) & 255u) - 128) * vs;
        lds[wave][(i & 7) / 4 * 16 + hi * 4 + (i & 3)][f * 32 + i / 8 * 16 + lo] = (uint16_t)bf16_pair(x, x);
      }
    }
    // the wave reads what it wrote itself
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
#pragma unroll
    for (int i = lane; i < 32 * (D / 8); i += 64) {
      const int t = i / (D / 8), e = i % (D / 8) * 8;
      if (t >= t0 && t < t1)
        *reinterpret_cast<u32x4*>(A.v_out + (row0 + t) * ld + head * D + e) = *reinterpret_cast<const u32x4*>(&lds[wave][t][e]);
    }
  }
}

}  // namespace

extern "C" {

int draft_layer_append(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                       const float* rope, int positions, int rot, int interleaved, uint8_t* k_codes,
                       uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page,
                       const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int n_seq,
                       int max_pages, int T, int hq, int hkv, int D, void* q_out, void* stream) {
  const char* who = "append";
  int rc = check_heads(who, hq, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows(who, T, n_seq))) return rc;
  AppendArgs A{};
  A.b = Batch{q_start, kv_len, table, n_seq, max_pages, T};
  A.c = Cache{k_codes, v_codes, k_scale, v_scale, n_pages, page_shift_of(page), hkv};
  if ((rc = check_cache(who, A.c, page, A.b))) return rc;
  if (rot < 0 || rot > D || rot % 16 != 0)
    return dh::fail(DH_ESHAPE, "append: rot must be a multiple of 16 in 0..D (got %d)", rot);
  if (rot > 0 && (!rope || !aligned(rope, 16))) return dh::fail(DH_EINVAL, "append: rope must be a 16-byte aligned pointer");
  if (rot > 0 && positions < max_pages * page)
    return dh::fail(DH_ESHAPE, "append: rope has %d positions, the table reaches %d", positions, max_pages * page);
  if (!q != !q_out) return dh::fail(DH_EINVAL, "append: q and q_out go together");
  if (T == 0) return dh::ok();
  if ((rc = check_stride(who, "k", k, ldk, (int64_t)hkv * D))) return rc;
  if ((rc = check_stride(who, "v", v, ldv, (int64_t)hkv * D))) return rc;
  if (q) {
    if ((rc = check_stride(who, "q", q, ldq, (int64_t)hq * D))) return rc;
    if (!aligned(q_out, 16)) return dh::fail(DH_EINVAL, "append: q_out must be 16-byte aligned");
    if (q == q_out && ldq != (int64_t)hq * D) return dh::fail(DH_EINVAL, "append: q_out may be q only where q has no gaps");
    A.q_blocks = (T + kThreads / 64 - 1) / (kThreads / 64);   // a row a wave
  }
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k);
  A.v = static_cast<const uint16_t*>(v);
  A.ldq = ldq;
  A.ldk = ldk;
  A.ldv = ldv;
  A.rope = reinterpret_cast<const u32x4*>(rope);
  A.rot = rot;
  A.interleaved = interleaved != 0;
  A.hq = hq;
  A.q_out = static_cast<uint16_t*>(q_out);
  // pages that hold a new token: at most one a token, and all but two of a
  // sequence's are full of them
  const int64_t pages = std::min<int64_t>(T, (int64_t)T / page + 2 * (int64_t)n_seq);
  const int64_t grid = A.q_blocks + pages * hkv * 2;
  if (grid > 0x7FFFFFFF) return dh::fail(DH_EUNSUP, "append: too many pages for one launch");
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const size_t lds = (size_t)page * D;
  switch (D) {
    case 64: hipLaunchKernelGGL(append_kernel<64>, dim3((unsigned)grid), dim3(kThreads), lds, st, A); break;
    case 128: hipLaunchKernelGGL(append_kernel<128>, dim3((unsigned)grid), dim3(kThreads), lds, st, A); break;
    default: {
      static dh::OncePerDevice once;   // 64 KiB and the wave maxima: above the default limit
      const hipError_t e = allow_lds(once, reinterpret_cast<const void*>(&append_kernel<256>), 256 * 256);
      if (e != hipSuccess) return dh::fail(DH_EHIP, "append_kernel: %s", hipGetErrorString(e));
      hipLaunchKernelGGL(append_kernel<256>, dim3((unsigned)grid), dim3(kThreads), lds, st, A);
    }
  }
  return launched("append_kernel");
}

int draft_layer_read(const uint8_t* k_codes, const uint8_t* v_codes, const float* k_scale, const float* v_scale,
                     int n_pages, int page, const int32_t* q_start, const int32_t* kv_len, const int32_t* table,
                     int n_seq, int max_pages, int T, int hkv, int D, void* k_out, void* v_out, void* stream) {
  const char* who = "read";
  int rc = check_heads(who, hkv, hkv, D);
  if (rc) return rc;
  if ((rc = check_rows(who, T, n_seq))) return rc;
  ReadArgs A{};
  A.b = Batch{q_start, kv_len, table, n_seq, max_pages, T};
  A.c = Cache{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes), const_cast<float*>(k_scale),
              const_cast<float*>(v_scale), n_pages, page_shift_of(page), hkv};
  if ((rc = check_cache(who, A.c, page, A.b))) return rc;
  if (T == 0) return dh::ok();
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
    return dh::fail(DH_EINVAL, "read: k_out and v_out must be 16-byte aligned pointers");
  A.k_out = static_cast<uint16_t*>(k_out);
  A.v_out = static_cast<uint16_t*>(v_out);
  const int64_t groups = std::min<int64_t>(T, (int64_t)T / 32 + 2 * (int64_t)n_seq);
  const int64_t grid = groups * ((hkv + 3) / 4);
  if (grid > 0x7FFFFFFF) return dh::fail(DH_EUNSUP, "read: too many rows for one launch");
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  switch (D) {
    case 64: hipLaunchKernelGGL(read_kernel<64>, dim3((unsigned)grid), dim3(kThreads), 0, st, A); break;
    case 128: hipLaunchKernelGGL(read_kernel<128>, dim3((unsigned)grid), dim3(kThreads), 0, st, A); break;
    default: hipLaunchKernelGGL(read_kernel<256>, dim3((unsigned)grid), dim3(kThreads), 0, st, A); break;
  }
  return launched("read_kernel");
}

}  // extern "C"
