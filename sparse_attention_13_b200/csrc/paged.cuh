// paged.cuh -- the paged key/value cache as the kernels see it (include/dsa.h,
// dsa_paged_kv and dsa_paged_batch after the host checks).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {

struct PagedArgs {
  void *k, *v;
  float *k_scale, *v_scale;
  int8_t* sum;
  float* sum_scale;
  int n_pages, n_kv;
  const int *cu_q, *sp, *bt;
  int B, max_pages, total_q, max_Lq, max_Lk;
  bool one;  // every sequence has one row (the contract then fixes cu_q: no loads for it)
};

// Loads of what earlier work in the stream wrote.  Not read-only loads: the
// kernels start before that work ends (programmatic dependent launch), and a
// read-only load may be moved ahead of the wait for it, or hit a stale line.
template <typename T>
__device__ __forceinline__ T ld_global(const T* p) {
  return *p;
}

// Row range of sequence b, clamped so that a batch that breaks its contract
// still names only rows of the tensors.
__device__ __forceinline__ void paged_rows(const PagedArgs& a, int b, int& r0, int& n) {
  if (a.one) { r0 = b; n = 1; return; }
  r0 = min(max(ld_global(a.cu_q + b), 0), a.total_q);
  n = min(max(ld_global(a.cu_q + b + 1) - r0, 0), min(a.max_Lq, a.total_q - r0));
}

// Sequence of a packed row: the last b with cu_q[b] <= row.
__device__ __forceinline__ int paged_seq(const PagedArgs& a, int row) {
  if (a.one) return row;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ld_global(a.cu_q + mid) <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// First packed row of sequence b.
__device__ __forceinline__ int paged_first(const PagedArgs& a, int b) { return a.one ? b : ld_global(a.cu_q + b); }

// Positions visible to the row: s < start_pos + i (+ 1 when inclusive).
__device__ __forceinline__ int paged_visible(const PagedArgs& a, int b, int i, int inclusive) {
  const long long t = static_cast<long long>(ld_global(a.sp + b)) + i + inclusive;
  return static_cast<int>(t < 0 ? 0 : (t > a.max_Lk ? a.max_Lk : t));
}

// Pool page of page j of sequence b, or -1 when there is none.
__device__ __forceinline__ int paged_page(const PagedArgs& a, int b, int j) {
  if (j < 0 || j >= a.max_pages) return -1;
  const int p = ld_global(a.bt + static_cast<int64_t>(b) * a.max_pages + j);
  return p >= 0 && p < a.n_pages ? p : -1;
}

// Blocks of work of a ragged batch in a row: block idx of the concatenation of
// count(b) blocks per sequence is block blk of sequence b.  The grid is then
// as large as the rows are in all, not as the longest sequence times the batch.
// All lanes of a warp call together; false beyond the last block.
template <typename Count>
__device__ __forceinline__ bool paged_block(const PagedArgs& a, int64_t idx, Count count, int& b, int& blk) {
  const int lane = threadIdx.x & 31;
  const int per = a.B <= 32 ? 1 : 4;  // sequences per lane (independent loads)
  int64_t base = 0;
  for (int s0 = 0; s0 < a.B; s0 += 32 * per) {
    int w[4] = {0, 0, 0, 0};
    int own = 0;  // (all counts together are below 2^31: the rows are)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s = s0 + per * lane + e;
      if (e < per && s < a.B) w[e] = count(s);
      own += w[e];
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, base + incl > idx);
    if (over) {
      const int f = __ffs(over) - 1;
      b = s0 + per * f;
      int left = static_cast<int>(idx - base) - __shfl_sync(0xffffffffu, incl - own, f);
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        const int x = __shfl_sync(0xffffffffu, w[e], f);
        if (e + 1 < per && b == s0 + per * f + e && x <= left) { left -= x; ++b; }
      }
      blk = left;
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two E4M3 codes (nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(x);
}

// The host checks shared by the paged entry points (null: no attention heads).
dsa_status check_paged_host(const char* who, const dsa_paged_kv* kv, const dsa_paged_batch* pb, PagedArgs* out);

}  // namespace dsa
