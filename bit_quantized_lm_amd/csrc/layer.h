// Shared by the draft layer's device translation units: the batch and cache
// descriptions, the walk from a work item to its sequence, bf16 conversions
// and the argument checks (not part of the public ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/draftlayer.h"
#include "common.h"

namespace dl {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kMinScale = 0x1p-40f;   // smallest scale of a page
constexpr uint32_t kNotFinite = 0x7F800000u;   // fp32 magnitudes from here on are infinity and NaN

struct Batch {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* table;
  int n_seq, max_pages, T;
};

struct Cache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int n_pages, page_shift, hkv;
};

// One sequence of a batch.  Rows are clamped to 0..T and the length to 0..2^30,
// so that no row index leaves the caller's arrays whatever they hold.
struct Seq {
  int row0, n;   // first row, rows
  int len;       // kv_len
  int begin;     // position of row 0 (negative where kv_len < n)
};

__device__ __forceinline__ Seq load_seq(const Batch& b, int s) {
  Seq q;
  q.row0 = min(max(b.q_start[s], 0), b.T);
  q.n = max(min(b.q_start[s + 1], b.T) - q.row0, 0);
  q.len = min(max(b.kv_len[s], 0), DL_MAX_POSITIONS);
  q.begin = q.len - q.n;
  return q;
}

// One step of a scan over the wave's lanes: `x` moved by the DPP control, 0
// where no lane stands there.
template <int kControl, int kRows>
__device__ __forceinline__ int moved(int x) {
  return __builtin_amdgcn_update_dpp(0, x, kControl, kRows, 0xf, false);
}

// Inclusive sums over the lanes: within rows of 16 (shifts by 1, 2, 4, 8), then
// row 0's and 2's last lane to the rows after them, then the lower half's.
__device__ __forceinline__ int wave_inclusive_sum(int x) {
  x += moved<0x111, 0xf>(x);
  x += moved<0x112, 0xf>(x);
  x += moved<0x114, 0xf>(x);
  x += moved<0x118, 0xf>(x);
  x += moved<0x142, 0xa>(x);
  x += moved<0x143, 0xc>(x);
  return x;
}

__device__ __forceinline__ float last_lane(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}

// The wave's sum, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
  x += __uint_as_float((uint32_t)moved<0x111, 0xf>((int)__float_as_uint(x)));
  x += __uint_as_float((uint32_t)moved<0x112, 0xf>((int)__float_as_uint(x)));
  x += __uint_as_float((uint32_t)moved<0x114, 0xf>((int)__float_as_uint(x)));
  x += __uint_as_float((uint32_t)moved<0x118, 0xf>((int)__float_as_uint(x)));
  x += __uint_as_float((uint32_t)moved<0x142, 0xa>((int)__float_as_uint(x)));
  x += __uint_as_float((uint32_t)moved<0x143, 0xc>((int)__float_as_uint(x)));
  return last_lane(x);
}

// The wave's maximum, in every lane; a lane that nothing moves to keeps its own.
template <int kControl, int kRows>
__device__ __forceinline__ float max_moved(float x) {
  const int v = (int)__float_as_uint(x);
  return fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(v, v, kControl, kRows, 0xf, false)));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, (uint32_t)moved<0x111, 0xf>((int)x));
  x = max(x, (uint32_t)moved<0x112, 0xf>((int)x));
  x = max(x, (uint32_t)moved<0x114, 0xf>((int)x));
  x = max(x, (uint32_t)moved<0x118, 0xf>((int)x));
  x = max(x, (uint32_t)moved<0x142, 0xa>((int)x));
  x = max(x, (uint32_t)moved<0x143, 0xc>((int)x));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ float wave_max(float x) {
  x = max_moved<0x111, 0xf>(x);
  x = max_moved<0x112, 0xf>(x);
  x = max_moved<0x114, 0xf>(x);
  x = max_moved<0x118, 0xf>(x);
  x = max_moved<0x142, 0xa>(x);
  x = max_moved<0x143, 0xc>(x);
  return last_lane(x);
}

// Work items are numbered over the sequences in order, count(sequence) each.
// Finds item `item`'s sequence and its number within it; false past the last.
// The whole wave calls it with one item and gets one answer: 64 sequences a
// step, so a batch costs its sequences' two loads and one scan, and the host
// needs none of the lengths.
template <class F>
__device__ __forceinline__ bool find_item(const Batch& b, int item, F&& count, int& seq, int& rest) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < b.n_seq; base += 64) {
    const int s = base + lane;
    const int c = s < b.n_seq ? count(load_seq(b, s)) : 0;
    const int sum = wave_inclusive_sum(c);
    const int total = __builtin_amdgcn_readlane(sum, 63);
    if (item < total) {
      const int at = __builtin_ctzll(__ballot(sum > item));
      seq = base + at;
      rest = item - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(c, at));
      return true;
    }
    item -= total;
  }
  return false;
}

// Page id of page j of sequence s, or -1 (no such page).
__device__ __forceinline__ int page_id(const Batch& b, int n_pages, int s, int j) {
  if (j < 0 || j >= b.max_pages) return -1;
  const int id = b.table[(size_t)s * b.max_pages + j];
  return (unsigned)id < (unsigned)n_pages ? id : -1;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 to a bf16 pair, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// ------------------------------------------------------------- host checks
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {   // none with nothing
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

inline int page_shift_of(int page) { return page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : page == 256 ? 8 : -1; }

inline int check_heads(const char* who, int hq, int hkv, int D) {
  if (hkv < 1 || hq < hkv || hq > DL_MAX_HEADS || hq % hkv != 0)
    return dh::fail(DH_ESHAPE, "%s: heads must be 1 <= hkv <= hq <= %d with hq a multiple of hkv (got hq %d, hkv %d)", who,
                    DL_MAX_HEADS, hq, hkv);
  if (D != 64 && D != 128 && D != 256) return dh::fail(DH_EUNSUP, "%s: D must be 64, 128 or 256 (got %d)", who, D);
  return DH_OK;
}

inline int check_rows(const char* who, int T, int n_seq) {
  if (T < 0 || T > DL_MAX_ROWS) return dh::fail(DH_ESHAPE, "%s: T must be in 0..%d (got %d)", who, DL_MAX_ROWS, T);
  if (n_seq < 1 || n_seq > DL_MAX_SEQS)
    return dh::fail(DH_ESHAPE, "%s: n_seq must be in 1..%d (got %d)", who, DL_MAX_SEQS, n_seq);
  return DH_OK;
}

inline int check_cache(const char* who, const Cache& c, int page, const Batch& b) {
  if (!c.k || !c.v || !c.ks || !c.vs || !b.q_start || !b.kv_len || !b.table)
    return dh::fail(DH_EINVAL, "%s: null pointer", who);
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return dh::fail(DH_EINVAL, "%s: codes must be 16-byte aligned", who);
  if (!aligned(c.ks, 4) || !aligned(c.vs, 4) || !aligned(b.q_start, 4) || !aligned(b.kv_len, 4) || !aligned(b.table, 4))
    return dh::fail(DH_EINVAL, "%s: scales, q_start, kv_len and table must be 4-byte aligned", who);
  if (c.page_shift < 0) return dh::fail(DH_EUNSUP, "%s: page must be 32, 64, 128 or 256 (got %d)", who, page);
  if (c.n_pages < 1) return dh::fail(DH_ESHAPE, "%s: n_pages must be >= 1 (got %d)", who, c.n_pages);
  if (b.max_pages < 1 || (int64_t)b.max_pages * page >= DL_MAX_POSITIONS)
    return dh::fail(DH_ESHAPE, "%s: max_pages must be >= 1 with max_pages * page < 2^30 (got %d pages of %d)", who,
                    b.max_pages, page);
  return DH_OK;
}

inline int check_stride(const char* who, const char* what, const void* p, int64_t ld, int64_t row) {
  if (!p) return dh::fail(DH_EINVAL, "%s: null pointer (%s)", who, what);
  if (!aligned(p, 16) || ld % 8 != 0) return dh::fail(DH_EINVAL, "%s: %s must be 16-byte aligned with a row stride that is a multiple of 8", who, what);
  if (ld < row) return dh::fail(DH_EINVAL, "%s: the row stride of %s is %lld, below its %lld elements", who, what, (long long)ld, (long long)row);
  return DH_OK;
}

// Lets `kernel` take `bytes` of dynamic LDS on the current device.
inline hipError_t allow_lds(dh::OncePerDevice& once, const void* kernel, size_t bytes) {
  int device = 0;
  const hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  return once.run(device, hipSuccess, [&] { return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
}

inline int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return dh::fail(DH_EHIP, "%s: %s", what, hipGetErrorString(e));
  return dh::ok();
}

}  // namespace dl
