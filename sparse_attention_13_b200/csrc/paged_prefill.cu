// paged_prefill.cu -- attention of many rows of a sequence over all pages of
// its cache (prompts and chunks of prompts; dsa_paged_attn).
//
// Query rows on the 128 rows of the tensor-core tile: a tile holds TOK = 128/G
// consecutive tokens x the G heads that share a key/value head, a CTA works on
// two tiles in turn so that one's softmax runs under the other's products:
//     S[128 rows, 128 keys] = Q K^T,   O[128 rows, D] += P V
// S and O live in TMEM (all 512 columns); P overwrites S and is the A operand
// of the second product.  An 8-bit cache is widened to f16 (exact) on its way
// from a staging tile to the operand tile by four warps of their own; Q rows
// are scaled to f16 by a power of two per row: exact down to 2^-16 of the row's
// largest element, off by 2^-25 of it below.
//
// Bound by the softmax warps: 128 x 128 exponentials a tile are 1,024 cycles of
// the special-function unit, as long as the tile's two products, and the
// instructions around them take as long again.  4,096 rows x 64 heads at 16,384
// 8-bit tokens (heads of 128): 2.09 to 2.12 ms, 910 to 920 TFLOP/s, 57% of the
// measured cuBLAS rate.  When that was 2.0 ms, moving every fourth exponential to
// a polynomial made it slower (2.15 ms), as did polling instead of sleeping in
// the softmax warps (2.05 ms).
#include <algorithm>

#include "paged.cuh"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128, kHalf = 64;  // keys of a loaded tile, and of a step of the products and the softmax
constexpr int kMetas = 8;
constexpr int kStages = 2;     // staging tiles of an 8-bit cache
constexpr int kRing = 4;       // operand tiles: K, V, K, V
constexpr int kSoftWarps = 8, kConvWarp = 8, kTmaWarp = 12, kMmaWarp = 13;
constexpr int kThreads = 16 * 32;  // four warpgroups, for the register split (two warps idle)
// 65,536 registers: 128 a thread at launch; 2 x 128 x 208 + 2 x 128 x 48
constexpr int kSoftRegs = 208, kOtherRegs = 48;
// A row's reference exponent may lag its maximum until sixteen weights sum to
// more than kMostSum: rescaling O is rare, and no maximum is taken on the way.
// The f16 weights of an 8-bit cache are at most 2^16 and have steps of 2^-24:
// their reference lies kLift octaves below the maximum, so that weights keep 8
// bits down to 2^-24 of the row's largest and are off by 2^-33 of it below (many
// small weights behind a large one count).  The sums are kept in units of the
// maximum all the same: a V scale of 2^-100 adds its share to them.
template <bool F8> constexpr float kMostSum = F8 ? 32768.f : 4096.f;
template <bool F8> constexpr float kLift = F8 ? 8.f : 0.f;
constexpr float kUnlift = 1.f / 256.f;
// A score is rounded to f32 before it becomes the reference, but not inside the
// fused exponent score * k - reference.  Up to this reference the difference is
// at most 2^-8; beyond, the exponent takes the rounded score as well (at 2^28
// the difference is 16, and a weight of 2^16 after its own maximum), and the
// share of the V scales, which such a sum would swallow, is kept apart (off).
constexpr float kFarRef = 65536.f;

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The weights of a row over half a tile, 2^(score * k + add), rounded and packed two
// to a word in pk; sum: their f32 sum without the V scales, in units of the reference + kLift; high: the
// largest sum of sixteen.  GENERAL: columns from lim on are masked, and a V
// scale so small that it would flush the weights (thin: below vmax by 2^90)
// does not flush their share of the sum.  The other case has no branches, so
// that the 64 exponentials overlap.
template <bool F8, bool GENERAL>
__device__ __forceinline__ void tile_weights(uint32_t ts, const float4* mt, int shift, float cr, float mu, int lim,
                                             uint32_t (&pk)[32], float& sum, float& high) {
  sum = 0.f;
  high = 0.f;
  uint32_t sb[2][32];
  tmem_ld32<32>(ts, sb[0]);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    tmem_ld_wait();
    if (c == 0) tmem_ld32<32>(ts + 32, sb[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t* s = sb[c] + h * 16;
      float k = cr, add = -mu, inv = 1.f;
      bool thin = false;
      if constexpr (F8) {
        const float4 sc = mt[(c * 32 + h * 16) >> shift];
        k = cr * sc.x;
        add = sc.y - mu;
        inv = sc.z;
        thin = GENERAL && (sc.w == 1.f || sc.w == 3.f);
      }
      const int left = lim - (c * 32 + h * 16);
      const uint64_t kk = f32x2(k, k), aa = f32x2(add, add);
      uint64_t acc[2] = {0, 0};  // f32 zeros
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float2 x = f32x2_parts(fma_f32x2(f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), kk, aa));
        if (GENERAL) {
          x.x = e < left ? x.x : -INFINITY;
          x.y = e + 1 < left ? x.y : -INFINITY;
        }
        const float w0 = ex2_approx(x.x), w1 = ex2_approx(x.y);
        acc[e / 2 & 1] = add_f32x2(acc[e / 2 & 1], f32x2(w0, w1));
        pk[c * 16 + h * 8 + e / 2] = F8 ? pack_f16(w0, w1) : pack_bf16(w0, w1);
      }
      const float2 t = f32x2_parts(add_f32x2(acc[0], acc[1]));
      float part = t.x + t.y;
      high = fmaxf(high, part);
      if (thin) {
        part = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) part += e < left ? ex2_approx(fmaf(__uint_as_float(s[e]), k, -mu)) : 0.f;
        inv = kUnlift;
      }
      sum = F8 ? fmaf(part, inv, sum) : sum + part;
    }
  }
}

// O follows a new reference.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t to, float f) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32<32>(to + c * 32, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st32x32(to + c * 32, o);
  }
  tmem_st_wait();
}

// A row's state: reference exponent (ref + off; off is zero up to kFarRef) and
// the sum of 2^(score - reference - kLift).
struct RowState {
  float ref, off, l;
};

// Half a tile of rows whose scores are past kFarRef: maxima, O (the product of
// the half before has been added), weights (stored over the scores) and sum.
// Apart from tile_weights, whose ordinary halves it would slow down by 2 %.
template <int D, bool F8>
__device__ __forceinline__ RowState far_half(uint32_t ts, uint32_t to, const float4* mt, int shift, float cr, int lim, bool first, RowState row) {
  const auto scales = [&](int r) { return F8 ? mt[r * 16 >> shift] : make_float4(1.f, 0.f, 1.f, 0.f); };
  const auto load = [&](int r, float (&x)[16]) {  // scores of a run of 16 keys
    uint32_t s[16];
    tmem_ld32<16>(ts + r * 16, s);
    tmem_ld_wait();
    const float k = F8 ? cr * scales(r).x : cr;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = r * 16 + e < lim ? __fmul_rn(__uint_as_float(s[e]), k) : -INFINITY;
  };
  float x[16];
  // the largest bare score is the base, what the V scales add comes on top
  float next = row.ref;
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {
    load(r, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) next = fmaxf(next, x[e]);
  }
  const float was = row.ref == next ? row.off : row.off + (row.ref - next);  // the reference so far, from the new base
  const float mu = next == -INFINITY ? 0.f : next;
  float off = was;
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {
    load(r, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) off = fmaxf(off, __fadd_rn(__fsub_rn(x[e], mu), scales(r).y) - kLift<F8>);
  }
  const float f = off == was ? 1.f : ex2_approx(was - off);
  if (!first && __any_sync(0xffffffffu, f != 1.f)) scale_o<D>(to, f);
  float sum = 0.f;
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {  // (the weights of a run lie over scores that have been read)
    uint32_t pk[8];
    load(r, x);
    const float4 sc = scales(r);
    const bool thin = sc.w == 1.f || sc.w == 3.f;
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float d = __fsub_rn(x[e + i], mu);
        w[i] = ex2_approx(d + (sc.y - off));
        part += thin ? ex2_approx(d - off) : w[i];
      }
      pk[e / 2] = F8 ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]);
    }
    sum = fmaf(part, thin ? kUnlift : sc.z, sum);
    tmem_st32x8(ts + r * 8, pk);
  }
  return {next, off, fmaf(row.l, f, sum)};
}

template <int D, bool F8>
struct PreCfg {
  static constexpr int kSlabs = D / 64;               // operand slabs of 64 columns (128 bytes)
  static constexpr int kSlabBytes = kTile * 128;
  static constexpr int kEntry = kSlabs * kSlabBytes;  // an operand tile
  static constexpr int kStage = F8 ? kTile * D : 0;
  static constexpr int kMetaBytes = kMetas * 8 * 16;
  static constexpr int kSmem = 1024 + (2 + kRing) * kEntry + kStages * kStage + kMetaBytes +
                               8 * (2 * kRing + 2 * kStages + kMetas + 17) + 32;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Unit {
  int b, row0, rows, nq, kvh;     // first packed row, rows of the unit, Q tiles
  int t0, t1;                     // visible positions of the first and last row
  int lo, hi[2];                  // key tiles of each Q tile
};

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return h;
}
// Block id / n_kv of the batch: its sequence and number there; returns the
// sequence's last block, or -1 beyond the batch.
__device__ __forceinline__ int prefill_block(const PrefillParams& p, int64_t id, int& b, int& blk) {
  int r0, n;
  const auto blocks = [&](int s) {
    paged_rows(p.a, s, r0, n);
    return (n + 2 * p.tok - 1) / (2 * p.tok);
  };
  return paged_block(p.a, id / p.a.n_kv, blocks, b, blk) ? blocks(b) - 1 : -1;
}

// Adds the values of positions [s0, s1) that are not finite to a row's output
// (the tiles held zeros in their place, because other rows do not see them).
template <int D, bool F8>
__device__ __forceinline__ void add_nonfinite(const PrefillParams& p, int b, int kvh, int s0, int s1, float* part, dsa_bf16* out) {
  for (int s = s0; s < s1; ++s) {
    const int pg = paged_page(p.a, b, s / p.page);
    if (pg < 0) continue;
    const int64_t va = ((static_cast<int64_t>(pg) * p.a.n_kv + kvh) * p.page + s % p.page) * D;
    for (int c = 0; c < D; ++c) {
      float v;
      if constexpr (F8) v = e4m3x2_to_f32(static_cast<const uint8_t*>(p.a.v)[va + c]).x;
      else v = __uint_as_float(static_cast<uint32_t>(static_cast<const dsa_bf16*>(p.a.v)[va + c]) << 16);
      if (fabsf(v) <= 3.4e38f) continue;
      if (part) part[c] += v;
      else out[c] = static_cast<dsa_bf16>(pack_bf16(__uint_as_float(static_cast<uint32_t>(out[c]) << 16) + v, 0.f));
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  using C = PreCfg<D, F8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_smem = smem;
  uint8_t* ring = q_smem + 2 * C::kEntry;
  uint8_t* stage = ring + kRing * C::kEntry;
  float4* meta = reinterpret_cast<float4*>(stage + kStages * C::kStage);  // [kMetas][8] K scale, log2 V scale, kUnlift / V scale, flags
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(meta) + C::kMetaBytes);
  uint64_t *full = bars, *empty = full + kRing, *st_full = empty + kRing, *st_empty = st_full + kStages;
  uint64_t *meta_full = st_empty + kStages;
  uint64_t *s_full = meta_full + kMetas, *p_full = s_full + 4, *pv_done = p_full + 4, *o_full = pv_done + 4;  // [Q tile][half]
  uint64_t *q_full = o_full + 2, *v_fixed = q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_fixed + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* poison = abort_flag + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) { mbar_init(&full[i], F8 ? 4 : 1); mbar_init(&empty[i], 2); }
    for (int i = 0; i < kStages; ++i) { mbar_init(&st_full[i], 1); mbar_init(&st_empty[i], 4); }
    for (int i = 0; i < kMetas; ++i) mbar_init(&meta_full[i], 1);
    for (int i = 0; i < 4; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4); mbar_init(&pv_done[i], 1); }
    mbar_init(&o_full[0], 1);
    mbar_init(&o_full[1], 1);
    mbar_init(q_full, kSoftWarps);
    mbar_init(&v_fixed[0], 4);
    mbar_init(&v_fixed[1], 4);
    *abort_flag = 0;
    *poison = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(*tmem_slot)));
  pdl_trigger();
  pdl_wait();

  // the unit of this CTA
  Unit u;
  const int split = blockIdx.x % p.splits;
  const int64_t id = blockIdx.x / p.splits;
  {
    int r0 = 0, n = 0, blk = 0;
    u.kvh = static_cast<int>(id % p.a.n_kv);
    u.b = 0;
    const int last = prefill_block(p, id, u.b, blk);
    if (last >= 0) paged_rows(p.a, u.b, r0, n);
    const int first = (last - blk) * 2 * p.tok;  // late blocks first (they see the most keys)
    u.row0 = r0 + first;
    u.rows = last < 0 ? 0 : max(0, min(2 * p.tok, n - first));
    u.nq = u.rows > p.tok ? 2 : (u.rows > 0 ? 1 : 0);
    u.t0 = u.t1 = 0;
    u.lo = u.hi[0] = u.hi[1] = 0;
    if (u.rows > 0) {
      u.t0 = paged_visible(p.a, u.b, first, p.inclusive);
      u.t1 = paged_visible(p.a, u.b, first + u.rows - 1, p.inclusive);
      const int tq = paged_visible(p.a, u.b, first + min(u.rows, p.tok) - 1, p.inclusive);
      const int all = (u.t1 + kTile - 1) / kTile, one = (tq + kTile - 1) / kTile;
      u.lo = static_cast<int>(static_cast<int64_t>(all) * split / p.splits);
      u.hi[1] = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / p.splits);
      u.hi[0] = max(u.lo, min(u.hi[1], one));
      if (u.nq == 1) u.hi[1] = u.hi[0];
    }
  }
  const int n_tiles = u.hi[1] - u.lo, n0 = u.hi[0] - u.lo;  // tile 1 of Q never sees fewer keys than tile 0
  const int fix = max(u.lo, u.t0 / kTile) - u.lo;           // from this tile on, V slots need a look

  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kTmaWarp) {
    if (lane == 0) { tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
    const int per = 32 / p.ppt, n_vis = (u.t1 + p.page - 1) / p.page;
    const auto fetch = [&](int tile, int& pg, float& ks, float& vs) {
      const int j = tile * p.ppt + lane;
      pg = j < n_vis ? paged_page(p.a, u.b, j) : -1;
      ks = vs = 1.f;
      if (F8 && pg >= 0) {
        const int64_t at = static_cast<int64_t>(pg) * p.a.n_kv + u.kvh;
        ks = ld_global(p.a.k_scale + at);
        vs = ld_global(p.a.v_scale + at);
      }
    };
    float vmax = -INFINITY;  // largest log2 of a V scale so far
    int pg = -1, pn = -1;
    float ks = 1.f, vs = 1.f, kn = 1.f, vn = 1.f;
    if (n_tiles > 0) fetch(u.lo, pn, kn, vn);
    bool ok = true;
    int i = 0;
    for (; i < n_tiles && ok; ++i) {
      const int in = i % per;
      if (in == 0) {
        pg = pn; ks = kn; vs = vn;
        if (i + per < n_tiles) fetch(u.lo + i + per, pn, kn, vn);
      }
      const int src = in * p.ppt + lane % p.ppt;
      const int mp = __shfl_sync(0xffffffffu, pg, src);
      const float mk = __shfl_sync(0xffffffffu, ks, src), mv = __shfl_sync(0xffffffffu, vs, src);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int e = 2 * i + kv;
        constexpr int kDepth = F8 ? kStages : kRing;
        const int st = e % kDepth;
        uint64_t *fb = F8 ? &st_full[st] : &full[st], *eb = F8 ? &st_empty[st] : &empty[st];
        uint8_t* dst = F8 ? stage + st * C::kStage : ring + st * C::kEntry;
        ok = __all_sync(0xffffffffu, mbar_wait(eb, ((e / kDepth) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (F8 && kv == 0) {
          // w: 1 for a page whose V scale would flush the weights (thin), 2 more
          // where the tile has such a page
          const float lv = __log2f(mv);
          vmax = fmaxf(vmax, warp_max_f32(lv));
          const bool thin = lv < vmax - 90.f;
          const float w = (thin ? 1.f : 0.f) + (__any_sync(0xffffffffu, thin) ? 2.f : 0.f);
          if (lane < p.ppt) meta[i % kMetas * 8 + lane] = make_float4(mk, lv, __fdividef(kUnlift, mv), w);
          __syncwarp();
          if (lane == 0) mbar_arrive(&meta_full[i % kMetas]);
        }
        if (lane == 0) mbar_arrive_expect_tx(fb, F8 ? C::kStage : C::kEntry);
        __syncwarp();
        if (lane < p.ppt) {  // a slot without a page reads outside the pool: zeros
          const int page = mp >= 0 ? mp : p.a.n_pages;
          if constexpr (F8) {
            tma_load_4d(dst + lane * p.page * D, kv ? &tm_v : &tm_k, fb, 0, 0, u.kvh, page);
          } else {
#pragma unroll
            for (int c = 0; c < C::kSlabs; ++c)
              tma_load_4d(dst + c * C::kSlabBytes + lane * p.page * 128, kv ? &tm_v : &tm_k, fb, c * 64, 0, u.kvh, page);
          }
        }
      }
    }
    if (!ok && lane == 0) {  // let the loads in flight land
      constexpr int kDepth = F8 ? kStages : kRing;
      for (int st = 0; st < kDepth; ++st)
        for (int w = 0; w < 64 && 2 * i > st; ++w)
          if (mbar_try_wait(smem_u32(F8 ? &st_full[st] : &full[st]), ((2 * i - 1 - st) / kDepth) & 1)) break;
    }
  } else if (warp >= kMmaWarp && warp < kMmaWarp + 2) {
    // One warp per Q tile: while one sets up its next products, the other's run.
    const int q = warp - kMmaWarp;
    const int n_tiles_ = warp_uniform(n_tiles), nt = warp_uniform(q ? (u.nq > 1 ? n_tiles : 0) : n0);
    if (n_tiles_ > 0) {
      const bool lead = elect_one();
      const auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_spin(bar, parity, abort_flag)); };
      constexpr uint32_t fmt = F8 ? 0u : (1u << 7) | (1u << 10);
      constexpr uint32_t idesc_qk = (make_idesc_bf16(128, kHalf, 0, 0) & ~((1u << 7) | (1u << 10))) | fmt;
      constexpr uint32_t idesc_pv = (make_idesc_bf16(128, D, 0, 1) & ~((1u << 7) | (1u << 10))) | fmt;
      const uint32_t qb = smem_u32(q_smem);
      // descriptors differ in the start address alone (16-byte units, low bits)
      const uint64_t qd = make_smem_desc(qb, 16, 1024, kSwizzle128B);
      const uint64_t kd = make_smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
      const uint64_t vd = make_smem_desc(smem_u32(ring), C::kSlabBytes, 1024, kSwizzle128B);
      const auto qk = [&](int i, int h) {  // S of half h: its keys are rows 64 h on of the tile
        const uint64_t a0 = qd + q * (C::kEntry >> 4), b0 = kd + (2 * i % kRing) * (C::kEntry >> 4) + h * (kHalf * 128 >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (C::kSlabBytes >> 4) + (k & 3) * 2;
          umma_f16_ss_by(lead, tmem + q * 128 + h * kHalf, a0 + off, b0 + off, idesc_qk, k != 0);
        }
        umma_commit_by(lead, &s_full[2 * q + h]);
      };
      const auto pv = [&](int i, int h) {
        const uint64_t b0 = vd + ((2 * i + 1) % kRing) * (C::kEntry >> 4) + h * (kHalf * 128 >> 4);
#pragma unroll
        for (int k = 0; k < kHalf / 16; ++k)
          umma_f16_ts_by(lead, tmem + 256 + q * D, tmem + q * 128 + h * kHalf + k * 8, b0 + k * (2048 >> 4), idesc_pv, (i | h | k) != 0);
        umma_commit_by(lead, &pv_done[2 * q + h]);
      };
      const auto wait_tile = [&](int e) { return wait_all(&full[e % kRing], (e / kRing) & 1); };
      bool ok = wait_all(q_full, 0) && wait_tile(0);
      if (ok) {
        tc_fence_after();
        if (nt > 0) { qk(0, 0); qk(0, 1); }
        umma_commit_by(lead, &empty[0]);
      }
      // Each half of S is refilled as soon as its weights have been used, while
      // the softmax works on the other half.  Tiles that this Q tile does not
      // need are released all the same.
      for (int i = 0; i < n_tiles_ && ok; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i < nt) ok = ok && wait_all(&p_full[2 * q + h], i & 1);
          if (h == 0) ok = ok && (F8 ? wait_tile(2 * i + 1) : wait_all(&v_fixed[i & 1], (i >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (i < nt) pv(i, h);
          if (i + 1 < n_tiles_) {
            if (h == 0) {
              ok = wait_tile(2 * i + 2);
              tc_fence_after();
            }
            if (ok && i + 1 < nt) qk(i + 1, h);
          }
        }
        if (!ok) break;
        umma_commit_by(lead, &empty[(2 * i + 1) % kRing]);
        if (i + 1 < n_tiles_) umma_commit_by(lead, &empty[(2 * i + 2) % kRing]);
      }
      if (ok) umma_commit_by(lead, &o_full[q]);
    }
  } else if (warp < kTmaWarp) {
    // ---------------------------------------------------------------- 8-bit tiles to f16; V slots past the rows
    const int tid = threadIdx.x - kConvWarp * 32;
    bool ok = true;
    if constexpr (F8) {
      for (int e = 0; e < 2 * n_tiles && ok; ++e) {
        const int st = e % kStages, rg = e % kRing, i = e >> 1;
        ok = mbar_wait(&st_full[st], (e / kStages) & 1, abort_flag) && mbar_wait(&empty[rg], ((e / kRing) & 1) ^ 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // A thread widens the same 16 columns of every (128 / kChunks)-th row:
        // its place in the swizzled rows is fixed.  The upper slab's lanes
        // store their second chunk first, so that eight lanes cover all banks.
        constexpr int kChunks = D / 16, kRows = 128 / kChunks, kSteps = kTile / kRows, kBatch = 4;
        const int row0 = tid / kChunks, cc = tid % kChunks;
        const bool flip = cc & 4;
        const uint8_t* src = stage + st * C::kStage + tid * 16;
        uint8_t* d = ring + rg * C::kEntry + cc / 4 * C::kSlabBytes + row0 * 128;
        const int ch = cc % 4 * 2;
        uint8_t *d0 = d + (((ch + flip) ^ (row0 & 7)) << 4), *d1 = d + (((ch + 1 - flip) ^ (row0 & 7)) << 4);
        const int look = (e & 1) && i >= fix ? u.t0 - (u.lo + i) * kTile : kTile;  // rows from here on need a look
#pragma unroll
        for (int j0 = 0; j0 < kSteps; j0 += kBatch) {
          uint4 w[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) w[j] = *reinterpret_cast<const uint4*>(src + (j0 + j) * kRows * D);
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            const int row = row0 + (j0 + j) * kRows;
            if (row >= look) {
              const bool gone = (u.lo + i) * kTile + row >= u.t1;
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const uint32_t nan = __vcmpeq4(x[v] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                if (nan && !gone) *poison = 1;
                x[v] = gone ? 0u : x[v] & ~nan;
              }
            }
            const uint32_t a0 = flip ? x[2] : x[0], a1 = flip ? x[3] : x[1], b0 = flip ? x[0] : x[2], b1 = flip ? x[1] : x[3];
            *reinterpret_cast<uint4*>(d0 + (j0 + j) * kRows * 128) =
                make_uint4(f16x2_of_e4m3x2(a0 & 0xffffu), f16x2_of_e4m3x2(a0 >> 16), f16x2_of_e4m3x2(a1 & 0xffffu), f16x2_of_e4m3x2(a1 >> 16));
            *reinterpret_cast<uint4*>(d1 + (j0 + j) * kRows * 128) =
                make_uint4(f16x2_of_e4m3x2(b0 & 0xffffu), f16x2_of_e4m3x2(b0 >> 16), f16x2_of_e4m3x2(b1 & 0xffffu), f16x2_of_e4m3x2(b1 >> 16));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&st_empty[st]);
          mbar_arrive(&full[rg]);
        }
      }
    } else {
      for (int i = 0; i < n_tiles && ok; ++i) {  // every V tile passes here, so that the phases stay in step
        const int e = 2 * i + 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[e % kRing], (e / kRing) & 1, abort_flag));
        if (!ok) break;
        const int pos = (u.lo + i) * kTile + tid;
        if (i >= fix && pos >= u.t0) {
#pragma unroll
          for (int c = 0; c < C::kSlabs; ++c) {
            uint4* row = reinterpret_cast<uint4*>(ring + e % kRing * C::kEntry + c * C::kSlabBytes + tid * 128);
            for (int v = 0; v < 8; ++v) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (pos < u.t1) {
                w = row[v];
                uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t inf = __vcmpeq2(y[k] & 0x7f807f80u, 0x7f807f80u);
                  if (inf) *poison = 1;
                  y[k] &= ~inf;
                }
                w = make_uint4(y[0], y[1], y[2], y[3]);
              }
              row[v] = w;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_fixed[i & 1]);
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------------- softmax (thread = row) and output
    const int q = warp >> 2, m = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + q * 128 + lanes, to = tmem + 256 + q * D + lanes;
    const int tok = m / p.G, g = m - tok * p.G;
    const int row = q * p.tok + tok;               // row of the unit
    const bool live = tok < p.tok && row < u.rows;
    // (rows beyond the unit compute along with the last one and are not written)
    const int t = paged_visible(p.a, u.b, u.row0 - paged_first(p.a, u.b) + min(row, max(0, u.rows - 1)), p.inclusive);
    const int t_lo = __reduce_min_sync(0xffffffffu, t);
    const int64_t at = static_cast<int64_t>(u.row0 + row) * p.n_h + u.kvh * p.G + g;
    float cr = p.scale_log2;  // factor of the row's scores
    {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + at * D);
      uint8_t* dst = q_smem + q * C::kEntry + m * 128;
      float mul = 1.f;
      if constexpr (F8) {  // X = the power of two with 2^-1 X < amax <= X
        float amax = 0.f;
        for (int c = 0; c < D / 8; ++c) {
          float f[8];
          bf16x8_to_f32(live ? ld_global(src + c) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
        }
        const uint32_t w = __float_as_uint(fminf(amax, 3.3e38f));
        const int ex = min(max(static_cast<int>(w >> 23) - 127 + ((w & 0x7fffffu) ? 1 : 0), -100), 126);
        mul = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        cr *= __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      }
      for (int c = 0; c < D / 8; ++c) {
        uint4 w = live ? ld_global(src + c) : make_uint4(0, 0, 0, 0);
        if constexpr (F8) {
          float f[8];
          bf16x8_to_f32(w, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = fabsf(f[e]) <= 3.4e38f ? f[e] * mul : __int_as_float(0x7fffffff);
          w = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
        }
        *reinterpret_cast<uint4*>(dst + c / 8 * C::kSlabBytes + ((c % 8 ^ (m & 7)) << 4)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }

    float ref = -INFINITY, off = 0.f, l = 0.f;
    const int nt = q ? (u.nq > 1 ? n_tiles : 0) : n0;
    bool ok = true;
    bool thin = false;  // a page of the tile has a V scale far below the others'
    bool far = false;   // a row's reference is past kFarRef
    for (int g = 0; g < 2 * nt && ok; ++g) {
      const int i = g >> 1, h = g & 1;
      const int lim = t - (u.lo + i) * kTile - h * kHalf;  // keys of the half that the row sees
      const bool edge = t_lo - (u.lo + i) * kTile - h * kHalf < kHalf;
      if (F8 && h == 0) ok = mbar_wait(&meta_full[i % kMetas], (i / kMetas) & 1, abort_flag);
      ok = mbar_wait(&s_full[2 * q + h], i & 1, abort_flag) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t th = ts + h * kHalf;
      const float4* mt = meta + i % kMetas * 8 + (h ? kHalf >> p.shift : 0);  // (a page of 128: its only entry)
      if (F8 && h == 0) thin = mt[0].w >= 2.f;
      bool find = g == 0;  // (a row that sees no key of the first half sees none)
      uint32_t pk[32];
      float sum;
      for (int tries = 0; !far; tries = 1) {
        if (find) {  // the rows' maxima first
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32];
            tmem_ld32<32>(th + c * 32, s);
            tmem_ld_wait();
#pragma unroll
            for (int e0 = 0; e0 < 32; e0 += 16) {
              float part = -INFINITY;
#pragma unroll
              for (int e = e0; e < e0 + 16; ++e) part = fmaxf(part, c * 32 + e < lim ? __uint_as_float(s[e]) : -INFINITY);
              if constexpr (F8) {
                const float4 sc = mt[(c * 32 + e0) >> p.shift];
                part = part == -INFINITY ? part : fmaf(part, cr * sc.x, sc.y);
              } else {
                part *= cr;
              }
              top = fmaxf(top, part);
            }
          }
          const float next = fmaxf(ref, top - kLift<F8>);
          far = __any_sync(0xffffffffu, fabsf(next) > kFarRef && next != -INFINITY);
          if (far) break;
          const float f = next == ref ? 1.f : ex2_approx(ref - next);
          ref = next;
          l *= f;
          if (g > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // once the product of the half before has been added
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[2 * q + (h ^ 1)], ((g - 1) >> 1) & 1, abort_flag));
            tc_fence_after();
            scale_o<D>(to, f);
          }
        }
        // (all scores so far -inf: the first one that is not asks for the maxima)
        const float mu = ref == -INFINITY ? -1e38f : ref;
        float high;
        if (edge || thin) tile_weights<F8, true>(th, mt, p.shift, cr, mu, lim, pk, sum, high);
        else tile_weights<F8, false>(th, mt, p.shift, cr, mu, lim, pk, sum, high);
        // (once the maxima have been taken no exponent is above kLift + 2^-8: one more try at most)
        if (tries || !__any_sync(0xffffffffu, high > kMostSum<F8>)) break;
        find = true;
      }
      if (far) {
        if (g > 0) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[2 * q + (h ^ 1)], ((g - 1) >> 1) & 1, abort_flag));
        tc_fence_after();
        const RowState row = far_half<D, F8>(th, to, mt, p.shift, cr, lim, g == 0, {ref, off, l});
        ref = row.ref;
        off = row.off;
        l = row.l;
      } else {
        l += sum;
        tmem_st32x32(th, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * q + h]);
    }
    // ---- output
    if (ok && nt > 0) ok = mbar_wait(&o_full[q], 0, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && q < u.nq) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : (F8 ? kUnlift : 1.f) / l;
      const float ls = off + kLift<F8> + log2f(l);  // with ref: log2 of the row's sum (apart, since ref may swallow it)
      const int64_t part = ((id * p.splits + split) * 2 + q) * 128 + m;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32<32>(to + c * 32, o);
          tmem_ld_wait();
        }
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = nt > 0 && l != 0.f ? __uint_as_float(o[e]) * inv : 0.f;
        if (!live) continue;
        if (p.splits > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + c * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16(y[8 * e], y[8 * e + 1]), pack_bf16(y[8 * e + 2], y[8 * e + 3]),
                                pack_bf16(y[8 * e + 4], y[8 * e + 5]), pack_bf16(y[8 * e + 6], y[8 * e + 7]));
        }
      }
      if (live) {
        if (p.splits > 1) p.part_l[part] = l == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(ref, ls);
        else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (ref + ls) * 0.6931471805599453f;
        if (*poison)
          add_nonfinite<D, F8>(p, u.b, u.kvh, max(u.t0, u.lo * kTile), min(t, u.hi[1] * kTile), p.splits > 1 ? p.part_o + part * D : nullptr,
                               p.out + at * D);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, 1u);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of split rows: one block per (unit, Q tile, 128 / (D/4) rows).
template <int D>
__global__ void __launch_bounds__(128) paged_prefill_merge_kernel(const PrefillParams p) {
  constexpr int kVecs = D / 4, kRows = 128 / kVecs;
  pdl_trigger();
  pdl_wait();
  const int64_t tile = blockIdx.x / (128 / kRows), id = tile / 2;
  const int q = static_cast<int>(tile & 1), m = blockIdx.x % (128 / kRows) * kRows + threadIdx.x / kVecs, v = threadIdx.x % kVecs;
  const int kvh = static_cast<int>(id % p.a.n_kv);
  int b, blk, r0, n;
  const int last = prefill_block(p, id, b, blk);
  if (last < 0) return;
  paged_rows(p.a, b, r0, n);
  const int tok = m / p.G, row = (last - blk) * 2 * p.tok + q * p.tok + tok;
  if (tok >= p.tok || row >= n) return;
  const auto at = [&](int s) { return ((id * p.splits + s) * 2 + q) * 128 + m; };
  // sums 2^(x + y) of the parts: relative to the largest x, then to the largest of all
  float base = -INFINITY, top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) base = fmaxf(base, p.part_l[at(s)].x);
  if (base == -INFINITY) base = 0.f;
  const auto log_sum = [&](int s) { return p.part_l[at(s)].x - base + p.part_l[at(s)].y; };
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, log_sum(s));
  const float ref = top == -INFINITY ? 0.f : top;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float l2 = log_sum(s), w = exp2f(l2 - ref);
    sum += w;
    if (l2 == -INFINITY) continue;
    const float4 o = *reinterpret_cast<const float4*>(p.part_o + at(s) * D + v * 4);
    acc.x += w * o.x; acc.y += w * o.y; acc.z += w * o.z; acc.w += w * o.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t o = static_cast<int64_t>(r0 + row) * p.n_h + kvh * p.G + (m - tok * p.G);
  *reinterpret_cast<uint2*>(p.out + o * D + v * 4) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (v == 0 && p.lse) p.lse[o] = sum == 0.f ? -INFINITY : (base + (ref + log2f(sum))) * 0.6931471805599453f;
}

template <int D, bool F8>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const PrefillParams& p, cudaStream_t s) {
  using C = PreCfg<D, F8>;
  const int64_t units = p.blocks * p.a.n_kv;
  auto fn = paged_prefill_kernel<D, F8>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), C::kSmem);
  if (e == cudaSuccess) e = launch_pdl(fn, dim3(static_cast<unsigned>(units * p.splits)), dim3(kThreads), C::kSmem, s, k, v, p);
  if (e == cudaSuccess && p.splits > 1)
    e = launch_pdl(paged_prefill_merge_kernel<D>, dim3(static_cast<unsigned>(units * 2 * (128 / (512 / D)))), dim3(128), 0, s, p);
  return e;
}

}  // namespace

PrefillPlan paged_prefill_plan(const dsa_paged_kv* kv, const dsa_paged_batch* pb, int n_h) {
  PrefillPlan pl{};
  const int G = n_h / kv->n_kv;
  pl.tok = 128 / G;
  // a sequence of n rows has at most n / (2 tok) + 1 blocks
  pl.blocks = pb->total_q / (2 * pl.tok) + std::min(pb->B, pb->total_q);
  const int64_t units = pl.blocks * kv->n_kv;
  pl.units = units;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const int tiles = (pb->max_Lk + kTile - 1) / kTile;
  // Few units share the GPU in equal parts of their keys, of three tiles and more
  // (64 rows x 8 heads x 4 groups at up to 2,000 tokens: 28.2 us, in parts of one
  // tile 30.2, of eight 33.3; 8-bit 35.5, 36.1 and 42.5; at 500 and at 30,000
  // tokens, and with more rows, all three are equal).
  pl.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms / units, tiles / 3)));
  if (pl.splits > 1) {
    pl.o_bytes = static_cast<size_t>(units) * pl.splits * 256 * kv->D * 4;
    pl.l_bytes = static_cast<size_t>(units) * pl.splits * 256 * 8;
  }
  return pl;
}

cudaError_t paged_prefill_launch(const CUtensorMap& k, const CUtensorMap& v, int D, bool f8, const PrefillParams& p, cudaStream_t s) {
  return D == 64 ? (f8 ? launch<64, true>(k, v, p, s) : launch<64, false>(k, v, p, s))
                 : (f8 ? launch<128, true>(k, v, p, s) : launch<128, false>(k, v, p, s));
}

}  // namespace dsa
