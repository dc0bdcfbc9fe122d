// paged.cu -- the paged key/value cache (include/dsa.h, dsa_paged_kv): host
// checks, the append kernel (rotation, 8-bit quantisation with a scale for
// each page and head, page summaries) and the page selection.
#include <algorithm>
#include <string>

#include "paged.cuh"

namespace dsa {

dsa_status check_paged_host(const char* who, const dsa_paged_kv* kv, const dsa_paged_batch* pb, PagedArgs* out) {
  const auto bad = [&](dsa_status st, const char* what) { return set_error(st, std::string(who) + ": " + what); };
  if (!kv || !pb) return bad(DSA_ERR_INVALID_ARG, "null cache or batch descriptor");
  if (!kv->k || !kv->v || !pb->cu_q || !pb->start_pos || !pb->block_table)
    return bad(DSA_ERR_INVALID_ARG, "null pointer in a descriptor");
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->k_scale) || !aligned16(kv->v_scale) ||
      !aligned16(kv->sum) || !aligned16(kv->sum_scale))
    return bad(DSA_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(pb->cu_q) | reinterpret_cast<uintptr_t>(pb->start_pos) |
       reinterpret_cast<uintptr_t>(pb->block_table)) & 3u)
    return bad(DSA_ERR_INVALID_ARG, "batch arrays must be 4-byte aligned");
  if (kv->n_pages < 1 || kv->n_kv < 1 || pb->B < 1 || pb->max_pages < 1 || pb->total_q < 1 || pb->max_Lq < 1 ||
      pb->max_Lk < 1)
    return bad(DSA_ERR_INVALID_ARG, "sizes must be positive");
  if (kv->page != 16 && kv->page != 32 && kv->page != 64 && kv->page != 128)
    return bad(DSA_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 tokens");
  if (kv->D != 64 && kv->D != 128) return bad(DSA_ERR_UNSUPPORTED, "D must be 64 or 128");
  if (kv->fmt != DSA_KV_BF16 && kv->fmt != DSA_KV_E4M3) return bad(DSA_ERR_UNSUPPORTED, "unknown cache format");
  if (kv->fmt == DSA_KV_E4M3 ? (!kv->k_scale || !kv->v_scale) : (kv->k_scale || kv->v_scale))
    return bad(DSA_ERR_INVALID_ARG, "an E4M3 cache needs both scales and a bf16 cache takes none");
  if (!kv->sum != !kv->sum_scale) return bad(DSA_ERR_INVALID_ARG, "summaries need both arrays");
  if (static_cast<long long>(kv->n_pages) * kv->n_kv > (1ll << 31) - 1 || kv->n_kv > 128)
    return bad(DSA_ERR_UNSUPPORTED, "too many pages or heads");
  if (pb->max_Lq > pb->total_q) return bad(DSA_ERR_INVALID_ARG, "max_Lq exceeds total_q");
  if (pb->max_Lk > (1 << 30)) return bad(DSA_ERR_UNSUPPORTED, "max_Lk too large");
  if (static_cast<long long>(pb->max_pages) * kv->page < pb->max_Lk)
    return bad(DSA_ERR_INVALID_ARG, "the block table does not cover max_Lk positions");
  if (out)
    *out = PagedArgs{kv->k, kv->v, kv->k_scale, kv->v_scale, kv->sum, kv->sum_scale, kv->n_pages, kv->n_kv,
                     pb->cu_q, pb->start_pos, pb->block_table, pb->B, pb->max_pages, pb->total_q, pb->max_Lq, pb->max_Lk,
                     pb->max_Lq == 1 && pb->total_q == pb->B};
  return DSA_OK;
}

namespace {

// ---------------------------------------------------------------- contract
__global__ void check_paged_kernel(const PagedArgs a, int page, int* bad) {
  const int b = blockIdx.x;
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], sp = a.sp[b];
  const long long end = static_cast<long long>(sp) + q1 - q0;
  bool ok = q1 >= q0 && q1 - q0 <= a.max_Lq && sp >= 0 && end <= a.max_Lk;
  if (b == 0) ok = ok && q0 == 0;
  if (b == a.B - 1) ok = ok && q1 == a.total_q;
  if (ok)
    for (long long j = threadIdx.x; j * page < end; j += blockDim.x) ok = ok && paged_page(a, b, static_cast<int>(j)) >= 0;
  if (__syncthreads_or(!ok) && threadIdx.x == 0) atomicAdd(bad, 1);
}

// ---------------------------------------------------------------- append
struct AppendParams {
  PagedArgs a;
  const dsa_bf16 *k, *v, *q;
  dsa_bf16* q_out;
  int64_t k_stride, v_stride, q_stride;
  const float *cos, *sin;
  int n_h, half, interleaved, n_pos;
  int touched;     // pages a sequence can touch
  int packed;      // ragged: blocks count the pages in all instead
  int64_t units;   // blocks of cache pages: every period-th; the others rotate q
  int period;
  int q_runs, q_heads;  // runs of heads a row is cut into, heads of a run
};

constexpr int kAppendThreads = 256;
constexpr float kMaxF32 = 3.402823466e38f;
constexpr float kMinTop = 3.8e-37f;  // 127 * (1 / amax) stays finite above it

// Rotates the eight columns of vector `vec` of a head's row (raw: the bf16
// columns, f: the same in f32) by the angles of position pos.  A pair's other
// half is in another lane of the row.  Products and sums are rounded one by one
// (no fused multiply-add), so that the result does not depend on the compiler.
__device__ __forceinline__ void rotate8(const uint4& raw, int vec, int pos, const AppendParams& p, float (&f)[8]) {
  const int64_t at = static_cast<int64_t>(pos) * p.half;
  const int c = 8 * vec;
  const bool turn = c < 2 * p.half;
  if (p.interleaved) {
    if (!turn) return;
    const float4 cs = ld_global(reinterpret_cast<const float4*>(p.cos + at + c / 2));
    const float4 sn = ld_global(reinterpret_cast<const float4*>(p.sin + at + c / 2));
    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = f[2 * i], w = f[2 * i + 1];
      f[2 * i] = __fsub_rn(__fmul_rn(u, cc[i]), __fmul_rn(w, ss[i]));
      f[2 * i + 1] = __fadd_rn(__fmul_rn(w, cc[i]), __fmul_rn(u, ss[i]));
    }
    return;
  }
  const bool low = c < p.half;
  const int lane = threadIdx.x & 31, src = !turn ? lane : lane + (low ? p.half / 8 : -p.half / 8);
  uint4 other;
  other.x = __shfl_sync(0xffffffffu, raw.x, src);
  other.y = __shfl_sync(0xffffffffu, raw.y, src);
  other.z = __shfl_sync(0xffffffffu, raw.z, src);
  other.w = __shfl_sync(0xffffffffu, raw.w, src);
  if (!turn) return;
  float o[8];
  bf16x8_to_f32(other, o);
  const int pair = low ? c : c - p.half;
  const float4* cs4 = reinterpret_cast<const float4*>(p.cos + at + pair);
  const float4* sn4 = reinterpret_cast<const float4*>(p.sin + at + pair);
  const float4 c0 = ld_global(cs4), c1 = ld_global(cs4 + 1), s0 = ld_global(sn4), s1 = ld_global(sn4 + 1);
  const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = low ? __fsub_rn(__fmul_rn(f[i], cc[i]), __fmul_rn(o[i], ss[i]))
               : __fadd_rn(__fmul_rn(f[i], cc[i]), __fmul_rn(o[i], ss[i]));
}

// Smallest power of two X with amax <= 448 X (448 = 1.75 * 2^8), at least 2^-100.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -100) + 127) << 23);
}

// Reduces a maximum over the block (all threads get it).
__device__ __forceinline__ float block_max(float x, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int i = 1; i < kAppendThreads / 32; ++i) x = fmaxf(x, red[i]);
  return x;
}

// One block per (sequence, touched page, head, K or V): every slot of that
// page and head has one owner, so the scale, the rescaled older codes and the
// summary need no atomics and no second pass over the new rows.  A thread owns
// 8 columns of every (256 / (D/8))-th slot, in registers from the load to the
// store.  Bound by memory for prompts (13,653 rows of 64 + 8 + 8 heads of 128,
// 8-bit pages: 108 us, 4.9 TB/s of the bytes that have to move; 75 us of it the
// queries) and by the chain of dependent loads for a decode step (64 rows: 11 us).
template <int D, int PAGE, bool F8>
__global__ void __launch_bounds__(kAppendThreads, PAGE * D > 8192 ? 2 : 3) paged_append_kernel(const AppendParams p) {
  constexpr int kVecs = D / 8;                    // threads per slot
  constexpr int kRows = kAppendThreads / kVecs;   // slots per step
  constexpr int kSteps = PAGE > kRows ? PAGE / kRows : 1;
  __shared__ float red[kAppendThreads / 32];
  __shared__ float part[kAppendThreads][9];
  pdl_trigger();
  pdl_wait();
  const int vec = threadIdx.x % kVecs, g = threadIdx.x / kVecs, c = vec * 8;

  // cache blocks (long chains of latencies) are spread among the query blocks
  // (streams), so that both kinds share every SM
  const int64_t turn_of = blockIdx.x / p.period;
  const bool cache = blockIdx.x % p.period == 0 && turn_of < p.units;
  if (!cache) {  // queries: a warp per row and run of heads
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes per head (two vectors each), heads per step
    const int lane = threadIdx.x & 31;
    const int64_t w = (blockIdx.x - min(p.units, turn_of + 1)) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = w / p.q_runs;
    if (row >= p.a.total_q) return;
    const int b = paged_seq(p.a, static_cast<int>(row));
    const int64_t pos = static_cast<int64_t>(ld_global(p.a.sp + b)) + row - paged_first(p.a, b);
    if (p.half && (pos < 0 || pos >= p.n_pos)) return;
    // the lane's two vectors: a rotating pair, or two neighbours behind the
    // rotated columns; the angles are read once for all heads
    const int i = lane % kLanes;
    const bool turn = 8 * i < p.half;
    const int c0 = !turn ? 16 * i : (p.interleaved ? 16 * i : 8 * i);
    const int c1 = turn && !p.interleaved ? c0 + p.half : c0 + 8;
    float cc[8], ss[8];
    if (turn) {
      const int64_t at = pos * p.half + 8 * i;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 x = ld_global(reinterpret_cast<const float4*>(p.cos + at) + v), y = ld_global(reinterpret_cast<const float4*>(p.sin + at) + v);
        cc[4 * v] = x.x; cc[4 * v + 1] = x.y; cc[4 * v + 2] = x.z; cc[4 * v + 3] = x.w;
        ss[4 * v] = y.x; ss[4 * v + 1] = y.y; ss[4 * v + 2] = y.z; ss[4 * v + 3] = y.w;
      }
    }
    const int h_end = min(p.n_h, static_cast<int>(w % p.q_runs + 1) * p.q_heads);
    // (the loads of a batch of heads come first: stores to q_out, which may be
    // q, would hold back the loads behind them)
    constexpr int kBatch = 4;
    for (int h0 = static_cast<int>(w % p.q_runs) * p.q_heads + lane / kLanes; h0 < h_end; h0 += kBatch * kHeads) {
      uint4 u0[kBatch], u1[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int h = h0 + k * kHeads;
        if (h < h_end) {
          const dsa_bf16* x = p.q + row * p.q_stride + h * D;
          u0[k] = *reinterpret_cast<const uint4*>(x + c0);
          u1[k] = *reinterpret_cast<const uint4*>(x + c1);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int h = h0 + k * kHeads;
        if (h >= h_end) break;
        if (turn) {
          uint32_t* w0 = &u0[k].x;
          uint32_t* w1 = &u1[k].x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // halves: word e of both vectors, (x[2e], x[2e+1]) and their
            // partners; interleaved: the pairs in word e of each vector
            const float a0 = __uint_as_float(w0[e] << 16), a1 = __uint_as_float(w0[e] & 0xffff0000u);
            const float b0 = __uint_as_float(w1[e] << 16), b1 = __uint_as_float(w1[e] & 0xffff0000u);
            if (p.interleaved) {
              w0[e] = pack_bf16(__fsub_rn(__fmul_rn(a0, cc[e]), __fmul_rn(a1, ss[e])), __fadd_rn(__fmul_rn(a1, cc[e]), __fmul_rn(a0, ss[e])));
              w1[e] = pack_bf16(__fsub_rn(__fmul_rn(b0, cc[e + 4]), __fmul_rn(b1, ss[e + 4])), __fadd_rn(__fmul_rn(b1, cc[e + 4]), __fmul_rn(b0, ss[e + 4])));
            } else {
              w0[e] = pack_bf16(__fsub_rn(__fmul_rn(a0, cc[2 * e]), __fmul_rn(b0, ss[2 * e])), __fsub_rn(__fmul_rn(a1, cc[2 * e + 1]), __fmul_rn(b1, ss[2 * e + 1])));
              w1[e] = pack_bf16(__fadd_rn(__fmul_rn(b0, cc[2 * e]), __fmul_rn(a0, ss[2 * e])), __fadd_rn(__fmul_rn(b1, cc[2 * e + 1]), __fmul_rn(a1, ss[2 * e + 1])));
            }
          }
        }
        dsa_bf16* y = p.q_out + (row * p.n_h + h) * D;
        *reinterpret_cast<uint4*>(y + c0) = u0[k];
        *reinterpret_cast<uint4*>(y + c1) = u1[k];
      }
    }
    return;
  }

  int u = static_cast<int>(turn_of);
  const bool is_v = u & 1;
  u >>= 1;
  const int head = u % p.a.n_kv;
  u /= p.a.n_kv;
  int tp = u % p.touched, b = u / p.touched;
  if (p.packed) {  // u counts the pages that the sequences really touch
    const bool some = paged_block(p.a, u, [&](int s) {
      int r, rows;
      paged_rows(p.a, s, r, rows);
      const int at = max(ld_global(p.a.sp + s), 0) % PAGE;
      return rows ? (at + rows - 1) / PAGE + 1 : 0;
    }, b, tp);
    if (!some) return;
  }
  int r0, n;
  paged_rows(p.a, b, r0, n);
  const int sp = ld_global(p.a.sp + b);
  if (n == 0 || sp < 0 || static_cast<long long>(sp) + n > p.a.max_Lk) return;
  const int j = sp / PAGE + tp;              // page of the sequence
  const int first = max(sp, j * PAGE), end = min(sp + n, (j + 1) * PAGE);
  if (first >= end) return;
  const int pg = paged_page(p.a, b, j);  // (used after the rows, whose loads need not wait for it)
  const int a0 = first - j * PAGE, a1 = end - j * PAGE;  // new slots of the page
  const bool whole = !is_v && a1 == PAGE && p.a.sum;

  // all rows of the thread are in flight before the first is used
  uint4 raw[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int slot = s * kRows + g;
    raw[s] = make_uint4(0, 0, 0, 0);
    if (slot >= a0 && slot < a1) {
      const int64_t row = r0 + (j * PAGE + slot - sp);
      raw[s] = ld_global(reinterpret_cast<const uint4*>((is_v ? p.v + row * p.v_stride : p.k + row * p.k_stride) + head * D + c));
    }
  }
  float f[kSteps][8];
  float amax = 0.f;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int slot = s * kRows + g;
    bf16x8_to_f32(raw[s], f[s]);
    if (!is_v && p.half) rotate8(raw[s], vec, j * PAGE + min(max(slot, a0), a1 - 1), p, f[s]);
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[s][i]) <= kMaxF32 ? fabsf(f[s][i]) : 0.f);
    }
  }

  if (pg < 0) return;
  const int64_t unit = static_cast<int64_t>(pg) * p.a.n_kv + head;
  const int64_t base = unit * PAGE * D;
  float scale = 1.f, ratio = 1.f;
  if constexpr (F8) {
    float* sc = (is_v ? p.a.v_scale : p.a.k_scale) + unit;
    scale = pow2_scale(block_max(amax, red));
    if (a0 > 0) {
      const float old = *sc;
      scale = fmaxf(scale, old);
      ratio = __fdiv_rn(old, scale);
    }
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *sc = scale;
  }

#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int slot = s * kRows + g;
    const bool fresh = slot >= a0 && slot < a1, older = slot < a0 && (whole || ratio != 1.f);
    if (!fresh && !older) continue;
    const int64_t at = base + static_cast<int64_t>(slot) * D + c;
    if constexpr (F8) {
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? p.a.v : p.a.k) + at);
      float mul = ratio;
      if (older) {
        const uint2 w = *dst;
        const uint32_t h[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = e4m3x2_to_f32(h[i]);
          f[s][2 * i] = x.x;
          f[s][2 * i + 1] = x.y;
        }
      } else {
        mul = __fdiv_rn(1.f, scale);  // a power of two: exact (at most 2^100)
      }
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = e4m3x2(f[s][2 * i] * mul, f[s][2 * i + 1] * mul);
        const float2 x = e4m3x2_to_f32(h[i]);
        f[s][2 * i] = x.x;  // the summary takes what the cache holds
        f[s][2 * i + 1] = x.y;
      }
      if (fresh || ratio != 1.f) *dst = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<dsa_bf16*>(is_v ? p.a.v : p.a.k) + at);
      uint4 w;
      if (older) w = *dst;
      else {
        w = make_uint4(pack_bf16(f[s][0], f[s][1]), pack_bf16(f[s][2], f[s][3]), pack_bf16(f[s][4], f[s][5]),
                       pack_bf16(f[s][6], f[s][7]));
        *dst = w;
      }
      bf16x8_to_f32(w, f[s]);
    }
  }
  if (!whole) return;

  // ---- summary of a page that is now complete: the sum over its slots by
  // halving (slot i + slot i + PAGE/2, ...).  The slots of a thread are g,
  // g + kRows, ...: the first levels are its own, the rest go through shared
  // memory in the same order.
#pragma unroll
  for (int h = kSteps / 2; h; h >>= 1)
#pragma unroll
    for (int s = 0; s < kSteps / 2; ++s)
      if (s < h)
#pragma unroll
        for (int i = 0; i < 8; ++i) f[s][i] = __fadd_rn(f[s][i], f[s + h][i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = f[0][i];
  __syncthreads();
  constexpr int kGroups = PAGE < kRows ? PAGE : kRows;
  const int col = threadIdx.x;  // a thread per column from here on
  float x = 0.f;
  if (col < D) {
    float v[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) v[i] = part[i * kVecs + col / 8][col % 8];
#pragma unroll
    for (int h = kGroups / 2; h; h >>= 1)
#pragma unroll
      for (int i = 0; i < kGroups / 2; ++i)
        if (i < h) v[i] = __fadd_rn(v[i], v[i + h]);
    x = __fmul_rn(v[0], scale);
  }
  bool fine = __syncthreads_and(fabsf(x) <= kMaxF32);
  const float top = block_max(fabsf(x), red);
  fine = fine && top >= kMinTop;
  if (col < D) {
    p.a.sum[unit * D + col] = fine ? static_cast<int8_t>(__float2int_rn(__fmul_rn(x, __fmul_rn(127.f, __frcp_rn(top))))) : 0;
    if (col == 0) p.a.sum_scale[unit] = fine ? __fmul_rn(__fmul_rn(top, 1.f / 127.f), 1.f / PAGE) : 0.f;
  }
}

template <int D, int PAGE>
cudaError_t launch_append(const AppendParams& p, bool f8, unsigned grid, cudaStream_t s) {
  return f8 ? launch_pdl(paged_append_kernel<D, PAGE, true>, dim3(grid), dim3(kAppendThreads), 0, s, p)
            : launch_pdl(paged_append_kernel<D, PAGE, false>, dim3(grid), dim3(kAppendThreads), 0, s, p);
}
template <int D>
cudaError_t launch_append(const AppendParams& p, int page, bool f8, unsigned grid, cudaStream_t s) {
  switch (page) {
    case 16: return launch_append<D, 16>(p, f8, grid, s);
    case 32: return launch_append<D, 32>(p, f8, grid, s);
    case 64: return launch_append<D, 64>(p, f8, grid, s);
    default: return launch_append<D, 128>(p, f8, grid, s);
  }
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 256;
constexpr int kSelMaxPages = 49152;  // one f32 key per visible page in shared memory

struct SelParams {
  PagedArgs a;
  const dsa_bf16* q;
  int n_h, page, shift, inclusive, n_sel, n_first, n_last;
  int ranks;                   // blocks of a decode row's cluster
  int key_stride;              // keys of a row in shared memory
  int32_t* sel;
};

// 8-bit codes of the pooled query of a row and head (the exact sum over the
// group, rounded once); one warp, D / 32 columns per lane.
template <int D>
__device__ __forceinline__ void pooled_query(const SelParams& p, int64_t row, int head, int8_t* qc) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31, G = p.n_h / p.a.n_kv;
  const dsa_bf16* x = p.q + (row * p.n_h + head * G) * D + lane * kCols;
  double acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.0;
#pragma unroll 4
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const uint32_t w = ld_global(reinterpret_cast<const uint32_t*>(x + h * D) + i);
      acc[2 * i] += static_cast<double>(__uint_as_float(w << 16));
      acc[2 * i + 1] += static_cast<double>(__uint_as_float(w & 0xffff0000u));
    }
  float f[kCols], amax = 0.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    f[i] = static_cast<float>(acc[i]);
    fine = fine && fabsf(f[i]) <= kMaxF32;
    amax = fmaxf(amax, fabsf(f[i]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  fine = __all_sync(0xffffffffu, fine) && amax >= kMinTop;
  const float inv = __fmul_rn(127.f, __frcp_rn(amax));
#pragma unroll
  for (int i = 0; i < kCols; ++i) qc[lane * kCols + i] = fine ? static_cast<int8_t>(__float2int_rn(__fmul_rn(f[i], inv))) : 0;
}

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A key halfway between lo and hi: first by value (float keys crowd around
// zero), later by key, so that the search ends whatever the values are.
__device__ __forceinline__ uint32_t key_between(uint32_t lo, uint32_t hi, int step) {
  uint32_t mid = lo + (hi - lo) / 2;
  if (step < 14 && hi < 0xff800000u && lo > 0x007fffffu) {
    const uint32_t m = float_key(0.5f * key_value(lo) + 0.5f * key_value(hi));
    if (m > lo && m < hi) mid = m;
  }
  return mid;
}

// Scores have to be finite: a product beyond f32's range, or a summary that no
// call wrote (NaN), must not look like a forced page.  Such scores become the
// largest or lowest finite one, NaN the lowest, and are looked for where that
// costs least: clamping every product took 16.3 us against 15.3 here (few rows)
// and 70.8 against 69.5 (eight rows to a block; 68.4 without any such care).
// Few rows: where the scales that a thread has seen sum to no more than this,
// its products are finite (a dot is at most 128 * 128 * 127).
constexpr float kFarScale = 1.6e32f;

constexpr uint32_t kForced = 0xffffffffu;  // above the key of every finite score (and the key of NaN)
constexpr uint32_t kLowest = 0x00800000u, kHighest = 0xff7fffffu;  // keys of the ends of the finite range

// Decode rows: one cluster per (row, head).  Each block scores a part of the
// row's pages and puts the keys into the first block's shared memory, which
// finds the n_sel-th largest key and writes the pages in order: a histogram of
// 1,024 equal steps of value, the keys of one step ranked against each other;
// or halving, where a step holds too many keys.  Bound by the chain of
// latencies (dependent loads, barriers): the work is split until the blocks
// fill the GPU (8 sequences x 8 heads x 3,125 pages: 14.3 us).
constexpr int kDecThreads = 512, kDecWarps = kDecThreads / 32;
constexpr int kBins = 1024, kRankMax = 256;
template <int D>
__global__ void __launch_bounds__(kDecThreads) page_topk_kernel(const SelParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int8_t qc[D];
  __shared__ int hist[kBins], counts[2][kDecWarps], scan[2][kDecWarps], pick[4];
  __shared__ uint32_t red[2][kDecWarps], cand[kRankMax];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = p.ranks;
  pdl_trigger();
  pdl_wait();
  const int64_t u = blockIdx.x / ranks;
  const int row = static_cast<int>(u / p.a.n_kv), head = static_cast<int>(u % p.a.n_kv);
  const int b = paged_seq(p.a, row);
  const int t = paged_visible(p.a, b, row - paged_first(p.a, b), p.inclusive);
  const int n = (t + p.page - 1) / p.page;
  int32_t* out = p.sel + u * p.n_sel;
  if (n <= p.n_sel) {  // the same for the whole cluster
    if (rank == 0)
      for (int e = tid; e < p.n_sel; e += kDecThreads) out[e] = e < n ? e : -1;
    return;
  }
  // D / 16 lanes per page, 16 bytes each: whole lines, and the dot over lanes.
  // The loads of a batch of pages are in flight before the first is used.
  constexpr int kLanes = D / 16, kPages = 32 / kLanes, kStep = kDecThreads / kLanes, kBatch = 4;
  const int part = (n + ranks - 1) / ranks, j1 = min(n, (rank + 1) * part);
  const uint32_t dst = mapa_shared(smem_u32(keys), 0);
  int pg[kBatch];
  const auto page_of = [&](int j) { return j < j1 && j >= p.n_first && j < n - p.n_last ? paged_page(p.a, b, j) : -1; };
  const int first = rank * part + warp * kPages + lane / kLanes;
#pragma unroll
  for (int e = 0; e < kBatch; ++e) pg[e] = page_of(first + e * kStep);
  if (warp == 0) pooled_query<D>(p, row, head, qc);
  if (rank == 0)
    for (int i = tid; i < kBins; i += kDecThreads) hist[i] = 0;
  if (ranks > 1) cluster_sync();  // the first block runs before its memory is written
  else __syncthreads();
  const int4 mine = *reinterpret_cast<const int4*>(qc + lane % kLanes * 16);
  float scales = 0.f;
  for (int j0 = first; j0 - lane / kLanes < j1; j0 += kBatch * kStep) {
    int4 w[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      w[e] = make_int4(0, 0, 0, 0);
      scale[e] = 0.f;
      if (pg[e] >= 0) {
        const int64_t unit = static_cast<int64_t>(pg[e]) * p.a.n_kv + head;
        w[e] = ld_global(reinterpret_cast<const int4*>(p.a.sum + unit * D) + lane % kLanes);
        scale[e] = ld_global(p.a.sum_scale + unit);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) pg[e] = page_of(j0 + (kBatch + e) * kStep);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) scales += fabsf(scale[e]);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int j = j0 + e * kStep;
      int dot = __dp4a(w[e].x, mine.x, __dp4a(w[e].y, mine.y, __dp4a(w[e].z, mine.z, __dp4a(w[e].w, mine.w, 0))));
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const bool scored = j >= p.n_first && j < n - p.n_last;
      // (a page outside the pool leaves the zeros: score 0)
      const uint32_t key = scored ? float_key(__fmul_rn(static_cast<float>(dot), scale[e])) : kForced;
      if (j < j1 && lane % kLanes == 0) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + 4u * j), "r"(key) : "memory");
    }
  }
  if (!(scales <= kFarScale) && lane % kLanes == 0)
    for (int j = first; j < j1; j += kStep) {
      if (j < p.n_first || j >= n - p.n_last) continue;
      uint32_t key;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(key) : "r"(dst + 4u * j) : "memory");
      key = key == kForced ? kLowest : min(max(key, kLowest), kHighest);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + 4u * j), "r"(key) : "memory");
    }
  if (ranks > 1) {
    cluster_sync();
    if (rank) return;
  } else {
    __syncthreads();
  }
  // ---- the n_sel-th largest key.  Each warp owns a run of 32 * per pages.
  const int per = (n + kDecThreads - 1) / kDecThreads, w0 = warp * per * 32 + lane;
  uint32_t low = kForced, high = 0u;
  for (int i = 0; i < per; ++i) {
    const uint32_t x = w0 + i * 32 < n ? keys[w0 + i * 32] : kForced;
    low = min(low, x);
    if (x != kForced) high = max(high, x);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) { red[0][warp] = low; red[1][warp] = high; }
  if (tid < 4) pick[tid] = 0;
  __syncthreads();
  low = __reduce_min_sync(0xffffffffu, red[0][lane % kDecWarps]);
  high = __reduce_max_sync(0xffffffffu, red[1][lane % kDecWarps]);
  uint32_t hi = high + 1u;  // fewer than n_sel keys are >= hi, at least n_sel are >= low
  int above = p.n_first + p.n_last;
  bool exact = above >= p.n_sel;  // exactly the keys >= low are taken
  if (exact) low = kForced;       // the forced pages alone
  const float v0 = key_value(low), gain = kBins / (key_value(high) - v0);
  if (!exact && high > low && gain > 0.f && gain < 1e30f) {
    const auto bin = [&](uint32_t key) { return min(kBins - 1, static_cast<int>((key_value(key) - v0) * gain)); };  // grows with the value
    for (int i = 0; i < per; ++i) {
      const uint32_t x = w0 + i * 32 < n ? keys[w0 + i * 32] : kForced;
      if (x != kForced) atomicAdd(&hist[bin(x)], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int run = above;
      for (int i = 0; i < kBins / 32; ++i) {  // 32 bins at a time, the highest in lane 0
        const int c = hist[kBins - 1 - (i * 32 + lane)];
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + incl >= p.n_sel);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            pick[0] = kBins - 1 - (i * 32 + lane);
            pick[1] = run + incl - c;  // keys above the bin
            pick[2] = c;
            pick[3] = 0;
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
    const int sel_bin = pick[0], in_bin = pick[2];
    if (in_bin <= kRankMax) {  // rank the bin's keys against each other
      for (int i = 0; i < per; ++i) {
        const uint32_t x = w0 + i * 32 < n ? keys[w0 + i * 32] : kForced;
        if (x != kForced && bin(x) == sel_bin) cand[atomicAdd(&pick[3], 1)] = x;  // any order
      }
      __syncthreads();
      above = pick[1];
      if (tid < in_bin) {
        int gt = 0, ge = 0;
        for (int i = 0; i < in_bin; ++i) { gt += cand[i] > cand[tid]; ge += cand[i] >= cand[tid]; }
        if (above + gt < p.n_sel && above + ge >= p.n_sel) {  // equal candidates write the same
          red[0][0] = cand[tid];
          counts[0][0] = above + gt;
          counts[0][1] = above + ge;
        }
      }
      __syncthreads();
      low = red[0][0];
      above = counts[0][0];
      exact = counts[0][1] == p.n_sel;
      hi = low + 1u;
    }
  }
  __syncthreads();
  for (int step = 0; !exact && hi - low > 1u; ++step) {
    const uint32_t mid = key_between(low, hi, step);
    int c = 0;
    for (int i = 0; i < per; ++i) c += w0 + i * 32 < n && keys[w0 + i * 32] >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) counts[step & 1][warp] = c;
    __syncthreads();
    c = __reduce_add_sync(0xffffffffu, lane < kDecWarps ? counts[step & 1][lane] : 0);
    if (c >= p.n_sel) {
      low = mid;
      exact = c == p.n_sel;
    } else {
      hi = mid;
      above = c;
    }
  }
  const int want = exact ? p.n_sel : p.n_sel - above;  // keys equal to low that are taken
  // ---- ordered output: keys above low, and the first `want` equal to it; the
  // warps count theirs, then write
  const auto is_gt = [&](int i, bool& eq) {
    const int j = w0 + i * 32;
    const uint32_t key = j < n ? keys[j] : 0u;
    eq = j < n && !exact && key == low;
    return j < n && (exact ? key >= low : key > low);
  };
  int at = 0, ties = 0;
  for (int i = 0; i < per; ++i) {
    bool eq;
    at += is_gt(i, eq);
    ties += eq;
  }
  at = __reduce_add_sync(0xffffffffu, at);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) { scan[0][warp] = at; scan[1][warp] = ties; }
  const bool some = at + ties > 0;
  __syncthreads();
  if (!some) return;
  at = __reduce_add_sync(0xffffffffu, lane < warp ? scan[0][lane] : 0);
  ties = __reduce_add_sync(0xffffffffu, lane < warp ? scan[1][lane] : 0);
  const unsigned lt = (1u << lane) - 1u;
  for (int i = 0; i < per; ++i) {
    bool eq;
    const bool gt = is_gt(i, eq);
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const int g0 = at + __popc(bg & lt), e0 = ties + __popc(be & lt);
    // (n_sel in all: the comparison with it is a bound, not a case)
    if (gt && g0 + min(e0, want) < p.n_sel) out[g0 + min(e0, want)] = w0 + i * 32;
    else if (eq && e0 < want && g0 + e0 < p.n_sel) out[g0 + e0] = w0 + i * 32;
    at += __popc(bg);
    ties += __popc(be);
  }
}

// D += A B^T for 16 x 32 and 8 x 32 signed bytes, whole numbers throughout.
__device__ __forceinline__ void mma_s8_16x8x32(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Many rows: one block per (eight rows of a sequence, head).  The scores of
// eight rows and sixteen pages are one small integer matrix product, with the
// columns permuted so that a lane's operands are 16 consecutive bytes; then a
// warp selects for each row from the scores in shared memory (forced pages:
// +inf).  Bound by instruction issue: about 1,700 per warp and row at 1,000
// pages, a third of them the scores (4,096 rows x 4 heads, 960 pages on
// average: 68 us; with dot products on the CUDA cores and halving it took 117).
constexpr int kSelRows = 8, kRowBins = 256;
template <int D>
__global__ void __launch_bounds__(kSelThreads) page_topk_rows_kernel(const SelParams p) {
  extern __shared__ __align__(16) float score[];  // [kSelRows][p.key_stride]
  __shared__ __align__(16) int8_t qc[kSelRows][D];
  __shared__ int hist[kSelRows][kRowBins];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int head = blockIdx.x % p.a.n_kv;
  int b, blk, r0, rows;
  const bool some = paged_block(p.a, blockIdx.x / p.a.n_kv, [&](int s) {
    paged_rows(p.a, s, r0, rows);
    return (rows + kSelRows - 1) / kSelRows;
  }, b, blk);
  if (!some) return;
  paged_rows(p.a, b, r0, rows);
  const int first = blk * kSelRows;
  const int nr = min(kSelRows, rows - first);
  if (nr <= 0) return;
  const auto pages_of = [&](int r) { return (paged_visible(p.a, b, first + r, p.inclusive) + p.page - 1) >> p.shift; };
  const int n_max = pages_of(nr - 1);
  const int n = warp < nr ? pages_of(warp) : 0;
  if (n_max > p.n_sel) {
    if (warp < nr) pooled_query<D>(p, r0 + first + warp, head, qc[warp]);
    __syncthreads();
    constexpr int kVecs = D / 64;  // 16-byte vectors of a lane, for a page or a row
    const int g = lane >> 2, tq = lane & 3;
    int4 q[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) q[v] = *reinterpret_cast<const int4*>(&qc[g][v * 64 + tq * 16]);
    int last[2];  // pages before the forced ones, of the lane's two rows
#pragma unroll
    for (int c = 0; c < 2; ++c) last[c] = pages_of(min(2 * tq + c, nr - 1)) - p.n_last;
#pragma unroll 2
    for (int j0 = warp * 16; j0 < n_max; j0 += 16 * (kSelThreads / 32)) {
      int4 s[2][kVecs];
      float scale[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + g + 8 * e, pg = j < n_max ? paged_page(p.a, b, j) : -1;
        const int64_t unit = static_cast<int64_t>(max(pg, 0)) * p.a.n_kv + head;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) s[e][v] = ld_global(reinterpret_cast<const int4*>(p.a.sum + unit * D + v * 64) + tq);
        scale[e] = pg >= 0 ? ld_global(p.a.sum_scale + unit) : 0.f;
      }
      int d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        mma_s8_16x8x32(d, s[0][v].x, s[1][v].x, s[0][v].y, s[1][v].y, q[v].x, q[v].y);
        mma_s8_16x8x32(d, s[0][v].z, s[1][v].z, s[0][v].w, s[1][v].w, q[v].z, q[v].w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + g + 8 * (e >> 1), c = e & 1;
        const float x = __fmul_rn(static_cast<float>(d[e]), scale[e >> 1]);
        if (j < n_max) score[(2 * tq + c) * p.key_stride + j] = j >= p.n_first && j < last[c] ? x : INFINITY;
      }
    }
    __syncthreads();
  }
  if (warp >= nr) return;
  int32_t* out = p.sel + ((static_cast<int64_t>(r0) + first + warp) * p.a.n_kv + head) * p.n_sel;
  if (n <= p.n_sel) {
    for (int e = lane; e < p.n_sel; e += 32) out[e] = e < n ? e : -1;
    return;
  }
  float* kr = score + warp * p.key_stride;
  const unsigned lt = (1u << lane) - 1u;
  int forced = p.n_first + p.n_last;
  float v_lo, v_hi;  // of the scores, which have to be finite
  for (bool clamped = false;; clamped = true) {
    v_lo = INFINITY;
    v_hi = -INFINITY;
    int odd = 0;  // +inf and NaN: the forced pages, and no others
    for (int j = lane; j < n; j += 32) {
      const float x = kr[j];
      v_lo = fminf(v_lo, x);
      if (x < INFINITY) v_hi = fmaxf(v_hi, x);
      else ++odd;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      v_lo = fminf(v_lo, __shfl_xor_sync(0xffffffffu, v_lo, o));
      v_hi = fmaxf(v_hi, __shfl_xor_sync(0xffffffffu, v_hi, o));
    }
    odd = __reduce_add_sync(0xffffffffu, odd);
    if (clamped || (odd == forced && v_lo > -INFINITY)) break;
    for (int j = p.n_first + lane; j < n - p.n_last; j += 32) kr[j] = fminf(fmaxf(kr[j], -kMaxF32), kMaxF32);
    __syncwarp();
  }
  // thr: the n_sel-th largest score; `above` scores are larger, and `want` of
  // those equal to it are taken (all of them when exact)
  float thr = INFINITY;
  int above = 0;
  bool done = forced >= p.n_sel, exact = done;
  const float gain = kRowBins / (v_hi - v_lo), off = -v_lo * gain;
  if (!done && v_hi > v_lo && gain > 0.f && gain < 1e30f && fabsf(off) < 1e30f) {
    // equal steps of value (forced pages in the last one): the step that holds
    // the n_sel-th largest score, and its scores (up to 32) ranked
    int* h = hist[warp];
    const auto bin = [&](float x) { return min(kRowBins - 1, static_cast<int>(fmaf(x, gain, off))); };  // grows with the value
#pragma unroll
    for (int i = 0; i < kRowBins / 32; ++i) h[i * 32 + lane] = 0;
    __syncwarp();
#pragma unroll 4
    for (int j = lane; j < n; j += 32) atomicAdd(&h[max(0, bin(kr[j]))], 1);
    __syncwarp();
    constexpr int kPer = kRowBins / 32;  // lane 0 holds the highest steps
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) { c[i] = h[kRowBins - 1 - (lane * kPer + i)]; sum += c[i]; }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, incl >= p.n_sel)) - 1;
    int run = incl - sum, pick = 0, in_bin = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (!found && run + c[i] >= p.n_sel) { found = true; pick = kRowBins - 1 - (lane * kPer + i); in_bin = c[i]; }
      if (!found) run += c[i];
    }
    pick = __shfl_sync(0xffffffffu, pick, src);
    in_bin = __shfl_sync(0xffffffffu, in_bin, src);
    run = __shfl_sync(0xffffffffu, run, src);
    if (in_bin <= 32) {
      int got = 0;
      __syncwarp();
#pragma unroll 4
      for (int j0 = 0; j0 < n; j0 += 32) {
        const float x = j0 + lane < n ? kr[j0 + lane] : 0.f;
        const bool in = j0 + lane < n && max(0, bin(x)) == pick;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (m) {
          if (in) h[got + __popc(m & lt)] = __float_as_int(x);
          got += __popc(m);
        }
      }
      __syncwarp();
      const float mine = lane < in_bin ? __int_as_float(h[lane]) : 0.f;
      int gt = 0, ge = 0;
      for (int i = 0; i < in_bin; ++i) {
        const float x = __int_as_float(h[i]);
        gt += x > mine;
        ge += x >= mine;
      }
      const bool is = lane < in_bin && run + gt < p.n_sel && run + ge >= p.n_sel;
      const int who = __ffs(__ballot_sync(0xffffffffu, is)) - 1;
      thr = __shfl_sync(0xffffffffu, mine, who);
      above = run + __shfl_sync(0xffffffffu, gt, who);
      exact = run + __shfl_sync(0xffffffffu, ge, who) == p.n_sel;
      done = true;
    }
  }
  if (!done) {  // halving: fewer than n_sel scores are >= hi's, at least n_sel >= lo's
    uint32_t lo = float_key(v_lo), hi = float_key(v_hi) + 1u;
    above = forced;
    for (int step = 0; !exact && hi - lo > 1u; ++step) {
      const uint32_t mid = key_between(lo, hi, step);
      const float v = key_value(mid);
      int c = 0;
      for (int j = lane; j < n; j += 32) c += kr[j] >= v;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= p.n_sel) {
        lo = mid;
        exact = c == p.n_sel;
      } else {
        hi = mid;
        above = c;
      }
    }
    thr = key_value(lo);
  }
  // ---- ordered output: lane i holds the bits of the taken pages 32 i .. of a
  // run of 1,024; equal scores are taken from the lowest page on
  int want = exact ? n : p.n_sel - above, at = 0;
  for (int base = 0; base < n; base += 1024) {
    unsigned gt = 0, eq = 0;
    const int words = min(32, (n - base + 31) / 32);
#pragma unroll 4
    for (int w = 0; w < words; ++w) {
      const int j = base + w * 32 + lane;
      const float x = j < n ? kr[j] : -INFINITY;
      const unsigned bg = __ballot_sync(0xffffffffu, j < n && x > thr), be = __ballot_sync(0xffffffffu, j < n && x == thr);
      if (lane == w) { gt = bg; eq = be; }
    }
    int ties = __popc(eq), tsum = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, tsum, o);
      if (lane >= o) tsum += y;
    }
    for (int drop = min(ties, max(0, tsum - want)); drop > 0; --drop) eq &= ~(0x80000000u >> __clz(eq));
    want -= __shfl_sync(0xffffffffu, tsum, 31);
    want = max(want, 0);
    unsigned bits = gt | eq;
    int cnt = __popc(bits), csum = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, csum, o);
      if (lane >= o) csum += y;
    }
    int to = at + csum - cnt;
    while (bits && to < p.n_sel) {  // (n_sel in all: a bound, not a case)
      out[to++] = base + lane * 32 + __ffs(bits) - 1;
      bits &= bits - 1;
    }
    at += __shfl_sync(0xffffffffu, csum, 31);
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_paged_append(const dsa_paged_kv* kv, const dsa_paged_batch* batch, const dsa_bf16* k,
                            int64_t k_row_stride, const dsa_bf16* v, int64_t v_row_stride, const float* cos,
                            const float* sin, int n_pos, int rot, int interleaved, const dsa_bf16* q,
                            int64_t q_row_stride, int n_h, dsa_bf16* q_out, void* stream) {
  AppendParams p{};
  dsa_status st = check_paged_host("dsa_paged_append", kv, batch, &p.a);
  if (st != DSA_OK) return st;
  if (!k || !v || !q != !q_out) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: null pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(cos) || !aligned16(sin))
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: pointers must be 16-byte aligned");
  const int64_t need = static_cast<int64_t>(kv->n_kv) * kv->D;
  if (k_row_stride < need || v_row_stride < need || (k_row_stride % 8) || (v_row_stride % 8))
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: row strides must cover the heads and be multiples of 8");
  if (q && (n_h < 1 || q_row_stride < static_cast<int64_t>(n_h) * kv->D || (q_row_stride % 8)))
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: bad n_h or query row stride");
  if (q && n_h > 1024) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_append: n_h too large");
  if (q == q_out && q && q_row_stride != static_cast<int64_t>(n_h) * kv->D)
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: in-place queries must be contiguous");
  if (rot < 0 || rot > kv->D || rot % 16) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_append: rot must be a multiple of 16, at most D");
  if (interleaved != 0 && interleaved != 1) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: interleaved is 0 or 1");
  if (rot && (!cos || !sin || n_pos < batch->max_Lk))
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_append: cos and sin must cover max_Lk positions");
  p.k = k; p.v = v; p.q = q; p.q_out = q_out;
  p.k_stride = k_row_stride; p.v_stride = v_row_stride; p.q_stride = q_row_stride;
  p.cos = cos; p.sin = sin; p.n_h = n_h; p.half = rot / 2; p.interleaved = interleaved; p.n_pos = n_pos;
  p.touched = (batch->max_Lq + kv->page - 2) / kv->page + 1;
  // A sequence of n rows touches at most n / page + 2 pages: in all no more
  // than this, however long the longest sequence is.
  const int64_t most = batch->total_q / kv->page + 2ll * std::min(batch->B, batch->total_q);
  p.packed = static_cast<int64_t>(batch->B) * p.touched > most;
  p.units = 2ll * kv->n_kv * (p.packed ? most : static_cast<int64_t>(batch->B) * p.touched);
  if (p.units > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_append: batch too large");
  // queries: long runs of heads reuse a row's angles; few rows are cut into
  // short runs so that some 2,000 warps share the work
  const int step = 512 / kv->D;  // heads of a warp's step
  const int steps = q ? (n_h + step - 1) / step : 1;
  const int per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, static_cast<int64_t>(batch->total_q) * steps / 2048)));
  p.q_heads = per * step;
  p.q_runs = q ? (n_h + p.q_heads - 1) / p.q_heads : 1;
  const int64_t q_blocks = q ? (static_cast<int64_t>(batch->total_q) * p.q_runs + kAppendThreads / 32 - 1) / (kAppendThreads / 32) : 0;
  const int64_t grid = p.units + q_blocks;
  p.period = static_cast<int>(std::min<int64_t>(1 << 20, grid / p.units));
  if (grid > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_append: batch too large");
  const cudaError_t e = kv->D == 64
      ? launch_append<64>(p, kv->page, kv->fmt == DSA_KV_E4M3, static_cast<unsigned>(grid), static_cast<cudaStream_t>(stream))
      : launch_append<128>(p, kv->page, kv->fmt == DSA_KV_E4M3, static_cast<unsigned>(grid), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_paged_append launch: ") + cudaGetErrorString(e));
  return DSA_OK;
}

dsa_status dsa_page_topk(const dsa_bf16* q, int n_h, const dsa_paged_kv* kv, const dsa_paged_batch* batch,
                         int inclusive, int n_sel, int n_first, int n_last, int32_t* sel, void* stream) {
  SelParams p{};
  dsa_status st = check_paged_host("dsa_page_topk", kv, batch, &p.a);
  if (st != DSA_OK) return st;
  if (!q || !sel || !kv->sum) return set_error(DSA_ERR_INVALID_ARG, "dsa_page_topk: null pointer, or a cache without summaries");
  if (!aligned16(q) || !aligned16(sel)) return set_error(DSA_ERR_INVALID_ARG, "dsa_page_topk: pointers must be 16-byte aligned");
  if (n_h < 1 || n_h % kv->n_kv) return set_error(DSA_ERR_INVALID_ARG, "dsa_page_topk: n_h must be a multiple of n_kv");
  if (n_h / kv->n_kv > 128) return set_error(DSA_ERR_UNSUPPORTED, "dsa_page_topk: more than 128 query heads per key/value head");
  if (inclusive != 0 && inclusive != 1) return set_error(DSA_ERR_INVALID_ARG, "dsa_page_topk: inclusive is 0 or 1");
  if (n_sel < 1 || n_first < 0 || n_last < 1 || static_cast<long long>(n_first) + n_last > n_sel)
    return set_error(DSA_ERR_INVALID_ARG, "dsa_page_topk: need n_first >= 0, n_last >= 1, n_first + n_last <= n_sel");
  const int max_n = (batch->max_Lk + kv->page - 1) / kv->page;
  if (n_sel > 1024 || max_n > kSelMaxPages)
    return set_error(DSA_ERR_UNSUPPORTED, "dsa_page_topk: n_sel <= 1024 and at most 49152 pages per sequence");
  p.q = q; p.n_h = n_h; p.page = kv->page; p.shift = kv->page == 16 ? 4 : kv->page == 32 ? 5 : kv->page == 64 ? 6 : 7; p.inclusive = inclusive; p.n_sel = n_sel; p.n_first = n_first; p.n_last = n_last;
  p.sel = sel;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool d64 = kv->D == 64;
  // Eight rows share a block when sequences have that many rows and the keys
  // of eight rows fit in shared memory; otherwise each row has a cluster.
  p.key_stride = (max_n + 31) / 32 * 32 + 4;  // (a lane's rows start in different banks)
  cudaError_t e;
  if (batch->max_Lq >= 4 && kSelRows * p.key_stride * 4 <= 200 * 1024) {
    const int64_t grid = (static_cast<int64_t>(batch->total_q) / kSelRows + std::min(batch->B, batch->total_q)) * kv->n_kv;
    if (grid > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_page_topk: too many rows");
    auto fn = d64 ? page_topk_rows_kernel<64> : page_topk_rows_kernel<128>;
    const int smem = kSelRows * p.key_stride * 4;
    e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem);
    if (e == cudaSuccess) e = launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kSelThreads), smem, s, p);
  } else {
    const int64_t units = static_cast<int64_t>(batch->total_q) * kv->n_kv;
    // 256 pages and more per block, at most two blocks per SM in all (at 8
    // sequences x 8 heads x 3,125 pages: 1, 2, 4, 8 blocks 23.5, 18.6, 14.8,
    // 22.8 us; eight no longer fit at once)
    p.ranks = 1;
    while (p.ranks < 8 && max_n > 256 * p.ranks && units * p.ranks * 2 <= 300) p.ranks *= 2;
    if (units * p.ranks > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_page_topk: too many rows");
    auto fn = d64 ? page_topk_kernel<64> : page_topk_kernel<128>;
    const int smem = p.key_stride * 4;
    e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * p.ranks));
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, fn, p);
  }
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_page_topk launch: ") + cudaGetErrorString(e));
  return DSA_OK;
}

dsa_status dsa_check_paged(const dsa_paged_kv* kv, const dsa_paged_batch* batch, int* bad_seqs, void* stream) {
  PagedArgs a{};
  dsa_status st = check_paged_host("dsa_check_paged", kv, batch, &a);
  if (st != DSA_OK) return st;
  if (!bad_seqs) return set_error(DSA_ERR_INVALID_ARG, "dsa_check_paged: null pointer");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(bad_seqs, 0, sizeof(int), s);
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_check_paged: ") + cudaGetErrorString(e));
  check_paged_kernel<<<static_cast<unsigned>(batch->B), 128, 0, s>>>(a, kv->page, bad_seqs);
  e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_check_paged launch: ") + cudaGetErrorString(e));
  return DSA_OK;
}

}  // extern "C"
