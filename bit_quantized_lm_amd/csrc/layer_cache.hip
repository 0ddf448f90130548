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
  const u32x2* rope;   // [positions][rot/2] of (cos, sin)
  int rot, interleaved, hq;
  uint16_t* q_out;
  int q_blocks;        // workgroups that rotate queries, before those that write pages
};

constexpr int kThreads = 256;

// Sixteen of a head's elements as two runs of eight, starting at d0 and d1:
// unit u < rot/16 holds eight rotary pairs ((d0 + i, d1 + i) in halves, or
// (2i, 2i + 1) of the sixteen from 16u interleaved), a later one sixteen
// elements that no rotation touches.
struct Unit {
  float x[16];
  int d0, d1;
};

// Each operation is rounded on its own (no fused multiply-add), so that the
// result is what the documented fp32 steps give, bit for bit.
__device__ __forceinline__ Unit load_unit(const uint16_t* __restrict__ row, const u32x2* __restrict__ turn, int rot,
                                          bool interleaved, int u) {
#pragma clang fp contract(off)
  Unit r;
  const bool turned = u * 16 < rot;
  const bool halves = turned && !interleaved;
  r.d0 = halves ? 8 * u : 16 * u;
  r.d1 = halves ? 8 * u + rot / 2 : 16 * u + 8;
  const u32x4 a = *reinterpret_cast<const u32x4*>(row + r.d0);
  const u32x4 b = *reinterpret_cast<const u32x4*>(row + r.d1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = bf16_lo(a[i]);
    r.x[2 * i + 1] = bf16_hi(a[i]);
    r.x[8 + 2 * i] = bf16_lo(b[i]);
    r.x[8 + 2 * i + 1] = bf16_hi(b[i]);
  }
  auto turn_pair = [&](float& xa, float& xb, int i) {
#pragma clang fp contract(off)
    const u32x2 t = turn[8 * u + i];
    const float c = __uint_as_float(t[0]), s = __uint_as_float(t[1]);
    const float ac = xa * c, bs = xb * s, bc = xb * c, as = xa * s;
    xa = ac - bs;
    xb = bc + as;
  };
  if (halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[i], r.x[8 + i], i);
  } else if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(r.x[2 * i], r.x[2 * i + 1], i);
  }
  return r;
}

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

// Rotates the queries: one Unit a thread and step.
template <int D>
__device__ __forceinline__ void rotate_queries(const AppendArgs& A) {
  constexpr int U = D / 16;
  const int per_row = A.hq * U, half = A.rot / 2;
  const int64_t units = (int64_t)A.b.T * per_row;
  const int last = (A.b.max_pages << A.c.page_shift) - 1;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units; i += (int64_t)A.q_blocks * kThreads) {
    const int r = (int)(i / per_row), x = (int)(i % per_row), h = x / U, u = x % U;
    int s = 0;   // the row's sequence: the last that starts at or before it
    for (int lo = 0, hi = A.b.n_seq; hi - lo > 1;) {
      const int mid = (lo + hi) / 2;
      (A.b.q_start[mid] <= r ? lo : hi) = mid;
      s = lo;
    }
    const Seq q = load_seq(A.b, s);
    const int p = min(max(q.begin + r - q.row0, 0), last);
    const Unit t = load_unit(A.q + r * A.ldq + h * D, A.rope + (size_t)p * half, A.rot, A.interleaved, u);
    uint16_t* out = A.q_out + ((size_t)r * A.hq + h) * D;
    *reinterpret_cast<u32x4*>(out + t.d0) = pack8(t.x);
    *reinterpret_cast<u32x4*>(out + t.d1) = pack8(t.x + 8);
  }
}

// One (page, head) of keys or values: the scale from the new values' largest
// magnitude, the new codes in token order in LDS, then the 16-byte units of
// the fragment order out of LDS.  The page has one writer, so an older
// token's code is re-rounded here without a race, and only where the scale rose.
template <int D, bool kKeys>
__device__ __forceinline__ void write_page(const AppendArgs& A, int s, int page_no, int head, uint8_t* lds) {
#pragma clang fp contract(off)
  constexpr int U = D / 16;
  __shared__ float wave_max[kThreads / 64];
  const int tid = threadIdx.x, page = 1 << A.c.page_shift;
  const int id = page_id(A.b, A.c.n_pages, s, page_no);
  if (id < 0) return;
  const Seq q = load_seq(A.b, s);
  const int p0 = page_no << A.c.page_shift;
  const int t0 = max(q.begin - p0, 0), t1 = min(q.len - p0, page);   // new tokens of the page
  const uint16_t* x = kKeys ? A.k : A.v;
  const int64_t ld = kKeys ? A.ldk : A.ldv;
  const int half = A.rot / 2, rot = kKeys ? A.rot : 0;
  float* scale = (kKeys ? A.c.ks : A.c.vs) + (size_t)id * A.c.hkv + head;
  u32x4* codes = reinterpret_cast<u32x4*>((kKeys ? A.c.k : A.c.v) + ((size_t)id * A.c.hkv + head) * ((size_t)page * D));
  const int64_t row0 = (int64_t)q.row0 + p0 - q.begin;   // row of token 0 of the page
  auto unit = [&](int i) {
    const int t = t0 + i / U;
    return load_unit(x + (row0 + t) * ld + head * D, A.rope + (size_t)(p0 + t) * half, rot, A.interleaved, i % U);
  };
  const int units = (t1 - t0) * U;
  float top = 0.0f;
  for (int i = tid; i < units; i += kThreads) {
    const Unit r = unit(i);
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(r.x[j]));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((tid & 63) == 0) wave_max[tid >> 6] = top;
  const float before = *scale;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = fmaxf(top, wave_max[w]);
  float step = fmaxf(top / 127.0f, kMinScale);
  if (t0 > 0) step = fmaxf(step, before);
  const float inv = 1.0f / step, ratio = before / step;
  const bool raised = t0 > 0 && step > before;
  for (int i = tid; i < units; i += kThreads) {
    const Unit r = unit(i);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j >> 2] |= code_of(r.x[j], inv) << (8 * (j & 3));
    uint8_t* at = lds + (t0 + i / U) * D;
    *reinterpret_cast<u32x2*>(at + r.d0) = u32x2{w[0], w[1]};
    *reinterpret_cast<u32x2*>(at + r.d1) = u32x2{w[2], w[3]};
  }
  __syncthreads();
  if (tid == 0) *scale = step;
  // 16-byte units of the fragment order
  for (int i = tid; i < page * U; i += kThreads) {
    const int g = i / (2 * D), f = i % (2 * D) / 64, lane = i & 63, hi = lane >> 4, lo = lane & 15;
    if (kKeys) {
      const int t = g * 32 + f / (D / 64) * 16 + lo, e = f % (D / 64) * 64 + hi * 16;
      if (t >= t0 && t < t1) {
        codes[i] = *reinterpret_cast<const u32x4*>(lds + t * D + e);
      } else if (raised && t < t0) {
        u32x4 w = codes[i];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t c = again((w[j >> 2] >> (8 * (j & 3))) & 255u, ratio);
          w[j >> 2] = (w[j >> 2] & ~(255u << (8 * (j & 3)))) | c << (8 * (j & 3));
        }
        codes[i] = w;
      }
    } else {
      // tokens g*32 + hi*4 + {0..3, 16..19}, elements f*32 + lo and + 16
      const int tb = g * 32 + hi * 4, e = f * 32 + lo;
      if (tb >= t1 || (tb + 19 < t0 && !raised)) continue;
      const bool whole = tb >= t0 && tb + 19 < t1;
      u32x4 w = whole ? u32x4{0u, 0u, 0u, 0u} : codes[i];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = tb + (j & 7) / 4 * 16 + (j & 3);
        uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 255u;
        if (t >= t0 && t < t1)
          c = lds[t * D + e + j / 8 * 16];
        else if (raised && t < t0)
          c = again(c, ratio);
        w[j >> 2] = (w[j >> 2] & ~(255u << (8 * (j & 3)))) | c << (8 * (j & 3));
      }
      codes[i] = w;
    }
  }
}

// Grid: q_blocks workgroups for the queries, then one per (page that a new
// token touches, head, keys or values).
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
    write_page<D, true>(A, s, j, head, lds);
  else
    write_page<D, false>(A, s, j, head, lds);
}

struct ReadArgs {
  Batch b;
  Cache c;
  uint16_t *k_out, *v_out;
};

// Reading back: a wave takes one head's 32 tokens of one sequence (a group of
// the fragment order; its values pass through LDS, where they turn from eight
// tokens a lane into rows of one).
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
  if (rot > 0 && (!rope || !aligned(rope, 8))) return dh::fail(DH_EINVAL, "append: rope must be an 8-byte aligned pointer");
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
    const int64_t want = ((int64_t)T * hq * (D / 16) + kThreads - 1) / kThreads;
    A.q_blocks = (int)(want < 4096 ? want : 4096);
  }
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k);
  A.v = static_cast<const uint16_t*>(v);
  A.ldq = ldq;
  A.ldk = ldk;
  A.ldv = ldv;
  A.rope = reinterpret_cast<const u32x2*>(rope);
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
      static bool attr_set = false;   // 64 KiB and the wave maxima: above the default limit
      if (!attr_set) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&append_kernel<256>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, 256 * 256);
        if (e != hipSuccess) return dh::fail(DH_EHIP, "append_kernel: %s", hipGetErrorString(e));
        attr_set = true;
      }
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
