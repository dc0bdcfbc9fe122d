// paged_attn.cu -- attention over a paged key/value cache (include/dsa.h,
// dsa_paged_attn): all pages of a sequence, or the selected ones.
#include <algorithm>
#include <string>

#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;

struct PattnParams {
  PagedArgs a;
  const dsa_bf16* q;
  const int32_t* sel;
  int n_h, page, inclusive, n_sel;
  float scale;
  dsa_bf16* out;
  float* lse;
};

// One block per (row, key/value head); thread = key in the score step and
// thread = column in the value step.  Running maximum and sum per head.
template <int D, bool F8>
__global__ void __launch_bounds__(kTile) paged_attn_simple_kernel(const PattnParams p) {
  extern __shared__ float sm[];
  const int G = p.n_h / p.a.n_kv, tid = threadIdx.x;
  float* qf = sm;                 // [G][D]
  float* w = qf + G * D;          // [G][kTile]
  float* o = w + G * kTile;       // [G][D]
  float* ml = o + G * D;          // [G][3]: max, sum, factor
  __shared__ int unit_of[kTile], base_of[kTile];
  const int row = blockIdx.x / p.a.n_kv, head = blockIdx.x % p.a.n_kv;
  pdl_trigger();
  pdl_wait();
  const int b = paged_seq(p.a, row);
  const int t = paged_visible(p.a, b, row - __ldg(p.a.cu_q + b), p.inclusive);
  const int pages = (t + p.page - 1) / p.page;
  for (int e = tid; e < G * D; e += kTile) {
    qf[e] = __uint_as_float(static_cast<uint32_t>(p.q[(static_cast<int64_t>(row) * p.n_h + head * G) * D + e]) << 16) * p.scale;
    o[e] = 0.f;
  }
  for (int h = tid; h < G; h += kTile) { ml[3 * h] = -INFINITY; ml[3 * h + 1] = 0.f; }
  const int n_list = p.sel ? p.n_sel : pages;
  const int per = kTile / p.page;
  for (int l0 = 0; l0 < n_list; l0 += per) {
    __syncthreads();
    const int l = l0 + tid / p.page;
    int j = -1;
    if (l < n_list) j = p.sel ? __ldg(p.sel + (static_cast<int64_t>(row) * p.a.n_kv + head) * p.n_sel + l) : l;
    const int pg = j >= 0 && j < pages ? paged_page(p.a, b, j) : -1;
    const bool seen = pg >= 0 && j * p.page + tid % p.page < t;
    const int64_t unit = seen ? static_cast<int64_t>(pg) * p.a.n_kv + head : 0;
    unit_of[tid] = seen ? static_cast<int>(unit) : -1;
    const int64_t at = (unit * p.page + tid % p.page) * D;
    for (int h = 0; h < G; ++h) {
      float acc = 0.f;
      if (seen) {
        for (int c = 0; c < D; ++c) {
          float x;
          if constexpr (F8) x = e4m3x2_to_f32(static_cast<const uint8_t*>(p.a.k)[at + c]).x;
          else x = __uint_as_float(static_cast<uint32_t>(static_cast<const dsa_bf16*>(p.a.k)[at + c]) << 16);
          acc = fmaf(x, qf[h * D + c], acc);
        }
        if constexpr (F8) acc *= p.a.k_scale[unit];
      }
      w[h * kTile + tid] = seen ? acc : -INFINITY;
    }
    __syncthreads();
    for (int h = tid >> 5; h < G; h += kTile / 32) {
      const int lane = tid & 31;
      float m = -INFINITY;
      for (int e = lane; e < kTile; e += 32) m = fmaxf(m, w[h * kTile + e]);
      for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float mo = ml[3 * h], mn = fmaxf(mo, m), mu = mn == -INFINITY ? 0.f : mn;
      float sum = 0.f;
      for (int e = lane; e < kTile; e += 32) {
        const float x = expf(w[h * kTile + e] - mu);
        w[h * kTile + e] = x;
        sum += x;
      }
      for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      __syncwarp();
      if (lane == 0) {
        const float f = expf(mo - mu);
        ml[3 * h] = mn;
        ml[3 * h + 1] = ml[3 * h + 1] * f + sum;
        ml[3 * h + 2] = f;
      }
    }
    __syncthreads();
    if (tid < D)
      for (int h = 0; h < G; ++h) {
        float acc = o[h * D + tid] * ml[3 * h + 2];
        for (int e = 0; e < kTile; ++e) {
          if (unit_of[e] < 0) continue;
          const int64_t va = (static_cast<int64_t>(unit_of[e]) * p.page + e % p.page) * D + tid;
          float x;
          if constexpr (F8) x = e4m3x2_to_f32(static_cast<const uint8_t*>(p.a.v)[va]).x * p.a.v_scale[unit_of[e]];
          else x = __uint_as_float(static_cast<uint32_t>(static_cast<const dsa_bf16*>(p.a.v)[va]) << 16);
          acc = fmaf(w[h * kTile + e], x, acc);
        }
        o[h * D + tid] = acc;
      }
  }
  __syncthreads();
  if (tid < D)
    for (int h = 0; h < G; ++h) {
      const float l = ml[3 * h + 1];
      const int64_t r = static_cast<int64_t>(row) * p.n_h + head * G + h;
      const __nv_bfloat16 x = __float2bfloat16_rn(l == 0.f ? 0.f : o[h * D + tid] / l);
      p.out[r * D + tid] = *reinterpret_cast<const dsa_bf16*>(&x);
      if (p.lse && tid == 0) p.lse[r] = l == 0.f ? -INFINITY : ml[3 * h] + logf(l);
    }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_paged_attn_workspace(const dsa_paged_kv* kv, const dsa_paged_batch* batch, int n_h, int n_sel) {
  if (check_paged_host("dsa_paged_attn_workspace", kv, batch, nullptr) != DSA_OK || n_h < 1 || n_sel < 0) return 0;
  return 16;
}

dsa_status dsa_paged_attn(const dsa_bf16* q, int n_h, const dsa_paged_kv* kv, const dsa_paged_batch* batch,
                          int inclusive, const int32_t* sel, int n_sel, float scale, dsa_bf16* out, float* lse,
                          void* ws, size_t ws_bytes, void* stream) {
  PattnParams p{};
  dsa_status st = check_paged_host("dsa_paged_attn", kv, batch, &p.a);
  if (st != DSA_OK) return st;
  if (!q || !out) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: null pointer");
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned16(sel))
    return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: pointers must be 16-byte aligned");
  if (n_h < 1 || n_h % kv->n_kv) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: n_h must be a multiple of n_kv");
  if (n_h > 128) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_attn: n_h <= 128");
  if (inclusive != 0 && inclusive != 1) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: inclusive is 0 or 1");
  if (sel ? n_sel < 1 : n_sel != 0) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: n_sel goes with sel");
  if (n_sel > 1024) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_attn: n_sel <= 1024");
  if (!(scale > 0.f) || scale > 3.402823466e38f) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: scale must be positive and finite");
  if (!ws || !aligned16(ws) || ws_bytes < dsa_paged_attn_workspace(kv, batch, n_h, n_sel))
    return set_error(DSA_ERR_WORKSPACE, "dsa_paged_attn: workspace null, misaligned or too small");
  p.q = q; p.sel = sel; p.n_h = n_h; p.page = kv->page; p.inclusive = inclusive; p.n_sel = n_sel; p.scale = scale;
  p.out = out; p.lse = lse;
  const int G = n_h / kv->n_kv;
  const int smem = (2 * G * kv->D + G * kTile + 3 * G) * 4;
  const bool f8 = kv->fmt == DSA_KV_E4M3;
  auto fn = kv->D == 64 ? (f8 ? paged_attn_simple_kernel<64, true> : paged_attn_simple_kernel<64, false>)
                        : (f8 ? paged_attn_simple_kernel<128, true> : paged_attn_simple_kernel<128, false>);
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), smem);
  if (e == cudaSuccess)
    e = launch_pdl(fn, dim3(static_cast<unsigned>(batch->total_q * kv->n_kv)), dim3(kTile), smem, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_paged_attn launch: ") + cudaGetErrorString(e));
  return DSA_OK;
}

}  // extern "C"
