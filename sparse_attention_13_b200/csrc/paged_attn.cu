// paged_attn.cu -- attention over a paged key/value cache (include/dsa.h,
// dsa_paged_attn): all pages of a sequence, or the selected ones.
//
// paged_attn_kernel puts KEYS on the 128 rows of the tensor-core tile and the
// few query heads that share them on the columns, so that a decode row wastes
// no tensor work on padding and the cache streams from HBM straight into the
// MMA's operands:
//     S^T[128 keys, N] = K . Q^T        A = K tile (K-major),  B = Q rows
//     O^T[D, N]       += V^T . P        A = V tile (MN-major), B = P rows
// An 8-bit cache is never widened.  E4M3 x E4M3 products are exact, and the
// 16-bit operands are split into two E4M3 terms, x = hi + lo / 32, which hold
// the 8 significant bits of a bf16 value down to 2^-15 of the largest (256), and
// steps of 2^-14 below: the columns are the heads' hi terms, then their lo
// terms, with an accumulator each (N = 2 heads).
#include <algorithm>
#include <string>

#include "paged.cuh"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;         // keys per tile
constexpr int kMaxCtas = 480;      // CTAs that may leave partial results
constexpr int kNoPage = 1 << 30;   // position of a slot that no page holds
// Weights over 8-bit pages are scaled to at most 256 and held in steps of 2^-14
// (two E4M3 terms).  The reference follows a tile whose largest weight is more
// than kFall octaves below it, so that many small weights behind a large one
// are not lost: no weight is off by more than 2^-14 of its tile's largest.  It
// stays within kFallMost octaves of the row's largest (O grows as it falls).
constexpr float kFall = 8.f, kFallMost = 40.f, kLowest = -110.f;  // (2^-118 is a factor of the output)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct PattnParams {
  PagedArgs a;
  const dsa_bf16* q;
  const int32_t* sel;
  int n_h, G, page, shift, ppt, inclusive, n_sel;  // shift: log2 page; ppt: pages per tile
  int Gx, R, hbs, max_rb;  // heads and rows of a unit, head blocks (sparse), row blocks (dense)
  int tpu, aligned;        // sparse: tiles per unit; CTAs take whole units
  float scale_log2;
  dsa_bf16* out;
  float* lse;
  float* part_o;           // [2 CTAs][NH][D]
  float2* part_l;          // [2 CTAs][NH]: log2 of a part's sum is x + y
  int2* meta;              // [units] first and last CTA of a split unit
  unsigned int* err;
};

// A unit is what one accumulator holds: R consecutive rows of a sequence (one
// row when pages are selected) x Gx heads of one key/value head.  A segment is
// a CTA's run of a unit's tiles.
struct Seg {
  int b, row0, nr, kvh, h0, nh, t0, t1;  // rows; heads; visible positions of the first and last row
  int lo, hi;                            // tiles
  int unit, slot;                        // slot -1: the whole unit, 1: its beginning, 0: a later part
  int last_cta;
};

// The tiles of all units in a row, cut into equal runs, one per CTA: equal
// work whatever the sequences' lengths.  Every role of a CTA walks its run by
// itself; all lanes of a warp call together.
template <bool SPARSE>
struct Walker {
  const PattnParams& p;
  long long pos, end, total;
  long long base, weight;  // dense: first tile and tiles of the current sequence
  int b, r0, n, nrb, tiles;
  // the unit that holds pos: its row or row block, head and head block, and
  // pos's tile in it (kept by counting: no divisions on the way)
  int at, kvh, hb, tile;

  __device__ __forceinline__ long long seq(int s, int& r, int& rows, int& blocks, int& t) const {
    paged_rows(p.a, s, r, rows);
    blocks = (rows + p.R - 1) / p.R;
    // (where CTAs take whole units, a unit counts as one)
    t = rows && !p.aligned ? max(1, (paged_visible(p.a, s, rows - 1, p.inclusive) + kTile - 1) / kTile) : 1;
    return static_cast<long long>(blocks) * p.a.n_kv * t;
  }

  __device__ __forceinline__ explicit Walker(const PattnParams& pp) : p(pp) {
    const long long c = blockIdx.x, C = gridDim.x;
    if constexpr (SPARSE) {
      const long long units = static_cast<long long>(p.a.total_q) * p.a.n_kv * p.hbs;
      total = units * p.tpu;
      pos = p.aligned ? units * c / C * p.tpu : total * c / C;
      end = p.aligned ? units * (c + 1) / C * p.tpu : total * (c + 1) / C;
      const long long u = pos / p.tpu;
      tile = static_cast<int>(pos - u * p.tpu);
      at = static_cast<int>(u % p.a.total_q);
      kvh = static_cast<int>(u / p.a.total_q) / p.hbs;
      hb = static_cast<int>(u / p.a.total_q) % p.hbs;
      b = -1;
    } else {
      const int lane = threadIdx.x & 31;
      // 128 sequences at a time, four per lane (independent loads)
      int r, rows, blocks, t;
      long long w[4];
      const auto load = [&](int s0) {
        long long sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = s0 + 4 * lane + e;
          w[e] = s < p.a.B ? seq(s, r, rows, blocks, t) : 0;
          sum += w[e];
        }
        return sum;
      };
      total = 0;
      long long sum = 0;
      for (int s0 = 0; s0 < p.a.B; s0 += 128) {
        sum = load(s0);
        long long all = sum;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        total += all;
      }
      pos = total * c / C;
      end = total * (c + 1) / C;
      base = 0;
      b = 0;
      for (int s0 = 0; s0 < p.a.B; s0 += 128) {  // the sequence that holds tile pos
        if (p.a.B > 128) sum = load(s0);
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, base + incl > pos);
        if (over) {
          const int f = __ffs(over) - 1;
          b = s0 + 4 * f;
          base += __shfl_sync(0xffffffffu, incl - sum, f);
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const long long x = __shfl_sync(0xffffffffu, w[e], f);
            if (b == s0 + 4 * f + e && base + x <= pos) { base += x; ++b; }
          }
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      weight = b < p.a.B ? seq(b, r0, n, nrb, tiles) : 0;
      if (weight) {
        const long long u = (pos - base) / tiles;
        tile = static_cast<int>(pos - base - u * tiles);
        at = static_cast<int>(u % nrb);
        kvh = static_cast<int>(u / nrb);
        hb = 0;
      }
    }
  }

  // (A run that begins past the own tiles of its unit begins with a segment that
  // has none.  The roles pass over it, so that barriers count those with tiles.)
  __device__ __forceinline__ bool next(Seg& s) {
    if (pos >= end) return false;
    int nominal;
    if constexpr (SPARSE) {
      nominal = p.tpu;
      s.unit = (kvh * p.hbs + hb) * p.a.total_q + at;
      s.row0 = at;
      if (b < 0) b = paged_seq(p.a, at);
      else if (p.a.one) b = at;
      else while (b + 1 < p.a.B && ld_global(p.a.cu_q + b + 1) <= at) ++b;
      s.nr = 1;
      s.t0 = s.t1 = paged_visible(p.a, b, at - paged_first(p.a, b), p.inclusive);
    } else {
      while (pos >= base + weight) {  // (tile, at, kvh and hb are zero here)
        base += weight;
        weight = seq(++b, r0, n, nrb, tiles);
      }
      nominal = tiles;
      s.unit = (b * p.a.n_kv + kvh) * p.max_rb + at;
      s.row0 = r0 + at * p.R;
      s.nr = min(p.R, n - at * p.R);
      s.t0 = paged_visible(p.a, b, at * p.R, p.inclusive);
      s.t1 = paged_visible(p.a, b, at * p.R + s.nr - 1, p.inclusive);
    }
    s.b = b;
    s.kvh = kvh;
    s.h0 = hb * p.Gx;
    s.nh = min(p.Gx, p.G - s.h0) * s.nr;
    s.lo = tile;
    s.hi = static_cast<int>(min(static_cast<long long>(nominal), tile + (end - pos)));
    s.slot = s.lo == 0 ? (s.hi == nominal ? -1 : 1) : 0;
    if (s.slot == 1) s.last_cta = static_cast<int>(((pos - s.lo + nominal) * gridDim.x - 1) / total);
    pos += s.hi - s.lo;
    tile = s.hi;
    if (tile == nominal) {  // the next unit: rows within a head, heads within a sequence
      tile = 0;
      if (++at == (SPARSE ? p.a.total_q : nrb)) {
        at = 0;
        if (SPARSE) b = -1;
        if (!SPARSE || ++hb == p.hbs) {
          hb = 0;
          if (++kvh == p.a.n_kv) kvh = 0;
        }
      }
    }
    // the unit's own tiles: earlier rows end earlier than the sequence, and a
    // list that is longer than the row's pages ends with its last valid entry
    int own;
    if constexpr (SPARSE) {
      own = nominal;
      const int n_vis = (s.t1 + p.page - 1) >> p.shift;
      if (n_vis < p.n_sel) {
        const int32_t* list = p.sel + (static_cast<int64_t>(s.row0) * p.a.n_kv + s.kvh) * p.n_sel;
        int l0 = (p.n_sel - 1) / 32 * 32, last = -1;
        for (; l0 >= 0 && last < 0; l0 -= 32) {
          const int l = l0 + (static_cast<int>(threadIdx.x) & 31);
          const int e = l < p.n_sel ? ld_global(list + l) : -1;
          const unsigned m = __ballot_sync(0xffffffffu, e >= 0 && e < n_vis);
          if (m) last = l0 + 31 - __clz(m);
        }
        own = last < 0 ? 1 : (last * p.page) / kTile + 1;
      }
      s.hi = min(s.hi, own);
    } else {
      own = max(1, (s.t1 + kTile - 1) / kTile);
      s.hi = p.aligned ? own : min(s.hi, own);
    }
    s.lo = min(s.lo, own);
    return true;
  }
};

template <int D, bool F8, int NH, bool SPARSE>
struct Cfg {
  // Heads per epilogue group of four warps.  Four groups of 8 for 32 heads of an
  // 8-bit cache (177 us against 194 for two of 16, 16 x 30,000 tokens x 4 heads,
  // before the references fell with the tiles; 183 since); a bf16 cache, with
  // half the work per weight, loses by it (162 against 157).
  static constexpr int kHG = NH < 16 || (F8 && NH == 32) ? 8 : 16;
  static constexpr int kGroups = NH / kHG;
  static constexpr int kEpiWarps = 4 * kGroups;
  static constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
  static constexpr int kThreads = 32 * (kEpiWarps + 2);
  static constexpr int kCtasPerSm = SPARSE && NH == 8 && F8 ? 3 : NH <= 16 ? 2 : 1;
  static constexpr int kElem = F8 ? 1 : 2;
  static constexpr int kN = F8 ? 2 * NH : (NH < 16 ? 16 : NH);  // MMA columns
  // Weights as two terms: always for an 8-bit cache; for a bf16 cache where
  // the second fits in columns that the tile has anyway (N >= 16).
  static constexpr bool kTwo = F8 || NH < 16;
  static constexpr int kRow = D * kElem;                        // bytes of a cached row
  static constexpr int kRowB = kRow < 128 ? kRow : 128;         // bytes of a row in a tile slab
  static constexpr int kSlabs = kRow / kRowB;
  static constexpr uint32_t kSwz = kRowB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr int kSlabBytes = kTile * kRowB;
  static constexpr int kEntry = kTile * kRow;                   // a K or V tile
  static constexpr int kQBytes = kN * kRow;
  static constexpr int kPBytes = kN * kTile * kElem;
  static constexpr int kRing = (kCtasPerSm == 3 ? 64 : kCtasPerSm == 2 ? 96 : 176) * 1024 / kEntry;  // entries: K, V, K, V, ...
  static constexpr int kMetas = kRing / 2 + 3;  // a slot is rewritten only after the PV of its tile
  static constexpr int kMetaBytes = kMetas * 8 * 16;
  static constexpr int kWmRow = F8 ? 2 * kHG : kHG;  // a warp's maxima of a tile: scores, what the V scales add
  static constexpr int kWm = kGroups * 2 * 4 * kWmRow;
  static constexpr int kTmemCols = 3 * kN <= 64 ? 64 : (3 * kN <= 128 ? 128 : 256);
  static constexpr int kSmem = 1024 + kRing * kEntry + kQBytes + 2 * kPBytes + kMetaBytes + kWm * 4 + 2 * NH * 4 +
                               4 * NH * 4 + kEpiWarps * 4 * kHG * 4 + 8 * (2 * kRing + kMetas + 8) + 64;
  static_assert(kSmem <= (kCtasPerSm == 3 ? 75 : kCtasPerSm == 2 ? 113 : 227) * 1024, "shared memory");
};

// Byte offset of row n, byte column c of a K-major operand slab with rows of
// ROWB bytes (swizzled in 16-byte chunks).
template <int ROWB>
__device__ __forceinline__ uint32_t op_off(int n, int c) {
  const int sw = ROWB == 128 ? (n & 7) : ((n >> 1) & 3);
  return n * ROWB + ((((c >> 4) ^ sw) << 4) | (c & 15));
}

// Warps 0 .. 4 groups - 1: softmax and output (thread = key in the scores,
// = column of D in the output); then one TMA warp and one MMA warp.  Bound by
// the cache's bytes for decode: the ring keeps 96 KB per CTA in flight (8
// sequences x 200,000 8-bit tokens x 8 heads of 128: 440 to 455 us, 6.2 to 6.4
// TB/s; 32 ragged sequences of up to 16,384 bf16 tokens x 4 heads: 130 to 133 us,
// 6.1 to 6.3 TB/s).  Bound by L2 where every row reads pages of its own (2,048
// rows x 8 heads x 32 pages of 64: 1,057 us, 8.1 TB/s), and by the softmax warps'
// chain (about 2,700 cycles a tile) where a tile has few bytes or many heads.
template <int D, bool F8, int NH, bool SPARSE>
__global__ void __launch_bounds__(Cfg<D, F8, NH, SPARSE>::kThreads, Cfg<D, F8, NH, SPARSE>::kCtasPerSm)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const PattnParams p) {
  using C = Cfg<D, F8, NH, SPARSE>;
  constexpr int HG = C::kHG, kRing = C::kRing, kMetas = C::kMetas;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint8_t* q_smem = ring + kRing * C::kEntry;
  uint8_t* p_smem = q_smem + C::kQBytes;
  int4* meta = reinterpret_cast<int4*>(p_smem + 2 * C::kPBytes);  // [kMetas][8] position, K scale, V scale
  float* wm = reinterpret_cast<float*>(meta + kMetas * 8);        // [group][2][4 warps][kWmRow]
  float* cq = wm + C::kWm;                                        // [2][NH] factor of a head's scores
  float* lsum = cq + 2 * NH;                                      // [4 warps][NH]
  float* bcast = lsum + 4 * NH;                                   // [warps][4][HG]
  uint64_t* bars = reinterpret_cast<uint64_t*>(bcast + C::kEpiWarps * 4 * HG);
  uint64_t *full = bars, *empty = full + kRing, *meta_full = empty + kRing;
  uint64_t *s_full = meta_full + kMetas, *p_full = s_full + 2, *pv_done = p_full + 2, *q_full = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* poison = abort_flag + 1;  // [2] a value that not every row of the unit sees is not finite

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < kMetas; ++i) mbar_init(&meta_full[i], 1);
    for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], C::kEpiWarps); mbar_init(&pv_done[i], 1); }
    mbar_init(q_full, C::kEpiWarps);
    *abort_flag = 0;
    poison[0] = poison[1] = 0;
    fence_barrier_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if constexpr (C::kN > NH && !F8)  // the padding rows of Q stay zero
    for (int i = threadIdx.x; i < C::kQBytes / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(q_smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(*tmem_slot)));
  const uint32_t tmem_o = tmem + 2 * C::kN;
  pdl_trigger();
  pdl_wait();

  Walker<SPARSE> walk(p);
  Seg s;
  if (warp == C::kTmaWarp) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) { tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
    const int per = 32 / p.ppt;  // tiles whose pages one load of the warp covers
    int it = 0;
    bool ok = true;
    // list entry, pool page and scales of the lane's page in a batch of tiles
    const auto fetch = [&](const Seg& g, int tile0, int& j, int& pg, float& ks, float& vs) {
      const int n_vis = (g.t1 + p.page - 1) >> p.shift, n_list = SPARSE ? p.n_sel : n_vis;
      const int l = tile0 * p.ppt + lane;
      j = -1;
      if (l < n_list) j = SPARSE ? ld_global(p.sel + (static_cast<int64_t>(g.row0) * p.a.n_kv + g.kvh) * p.n_sel + l) : l;
      pg = j >= 0 && j < n_vis ? paged_page(p.a, g.b, j) : -1;
      ks = vs = 0.f;
      if (F8 && pg >= 0) {
        const int64_t u = static_cast<int64_t>(pg) * p.a.n_kv + g.kvh;
        ks = ld_global(p.a.k_scale + u);
        vs = ld_global(p.a.v_scale + u);
      }
    };
    int j, pg, jn, pn, j2, p2;
    float ks, vs, kn, vn, k2, v2;
    Seg s2;
    bool more = walk.next(s2);
    if (more) fetch(s2, s2.lo, j2, p2, k2, v2);
    while (ok && more) {
      s = s2;
      jn = j2; pn = p2; kn = k2; vn = v2;
      // the next unit's first pages, while this one's tiles are loaded
      more = walk.next(s2);
      if (more) fetch(s2, s2.lo, j2, p2, k2, v2);
      for (int i = s.lo; i < s.hi; ++i, ++it) {
        const int in = (i - s.lo) % per;
        if (in == 0) {
          j = jn; pg = pn; ks = kn; vs = vn;
          if (i + per < s.hi) fetch(s, i + per, jn, pn, kn, vn);
        }
        const int src = in * p.ppt + lane % p.ppt;
        const int mj = __shfl_sync(0xffffffffu, j, src), mp = __shfl_sync(0xffffffffu, pg, src);
        const float mk = __shfl_sync(0xffffffffu, ks, src), mv = __shfl_sync(0xffffffffu, vs, src);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int e = 2 * it + kv, st = e % kRing;
          ok = ok && mbar_wait(&empty[st], ((e / kRing) & 1) ^ 1, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (kv == 0) {
            if (lane < p.ppt)
              meta[it % kMetas * 8 + lane] = make_int4(mp >= 0 ? mj * p.page : kNoPage, __float_as_int(mk), __float_as_int(mv), 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&meta_full[it % kMetas]);
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kEntry);
          __syncwarp();
          // a slot without a page reads outside the pool: zeros
          if (lane < p.ppt)
#pragma unroll
            for (int c = 0; c < C::kSlabs; ++c)
              tma_load_4d(ring + st * C::kEntry + c * C::kSlabBytes + lane * p.page * C::kRowB, kv ? &tm_v : &tm_k, &full[st],
                          c * (128 / C::kElem), 0, s.kvh, mp >= 0 ? mp : p.a.n_pages);
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) {  // let the loads in flight land
      for (int st = 0; st < kRing; ++st)
        for (int w = 0; w < 64 && 2 * it > st; ++w)
          if (mbar_try_wait(smem_u32(&full[st]), ((2 * it - 1 - st) / kRing) & 1)) break;
    }
  } else if (warp == C::kMmaWarp) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t idesc_qk = F8 ? make_idesc_f8(128, C::kN, 0, 0) : make_idesc_bf16(128, C::kN, 0, 0);
    constexpr uint32_t idesc_pv = F8 ? make_idesc_f8(128, C::kN, 1, 0) : make_idesc_bf16(128, C::kN, 1, 0);
    const bool lead = elect_one();
    const auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)); };
    // descriptors differ in the start address alone (16-byte units, low bits)
    const uint64_t qd = make_smem_desc(smem_u32(q_smem), 16, 8 * C::kRowB, C::kSwz);
    const uint64_t kd = make_smem_desc(smem_u32(ring), 16, 8 * C::kRowB, C::kSwz);
    // V is MN-major: D on the rows.  D = 64 fills only half of the 128 rows;
    // the second half repeats it (stride 0) and is not read.
    const uint64_t vd = make_smem_desc(smem_u32(ring), D == 128 ? C::kSlabBytes : 0, 8 * C::kRowB, C::kSwz);
    const uint64_t pd = make_smem_desc(smem_u32(p_smem), 16, 1024, kSwizzle128B);
    int it = 0, seg = 0;
    bool ok = true;
    const auto qk = [&](int t) {  // S(t) = K(t) Q^T
      const int e = 2 * t, st = e % kRing;
      if (!wait_all(&full[st], (e / kRing) & 1)) return false;
      tc_fence_after();
      const uint64_t k0 = kd + st * (C::kEntry >> 4);
#pragma unroll
      for (int k = 0; k < C::kRow / 32; ++k) {
        constexpr int kPer = C::kRowB / 32;
        const uint64_t ad = k0 + (k / kPer * (C::kSlabBytes >> 4) + k % kPer * 2);
        const uint64_t bd = qd + (k / kPer * (C::kN * C::kRowB >> 4) + k % kPer * 2);
        if constexpr (F8) umma_f8_ss_by(lead, tmem + (t & 1) * C::kN, ad, bd, idesc_qk, k != 0);
        else umma_f16_ss_by(lead, tmem + (t & 1) * C::kN, ad, bd, idesc_qk, k != 0);
      }
      umma_commit_by(lead, &empty[st]);
      umma_commit_by(lead, &s_full[t & 1]);
      return true;
    };
    while (ok && walk.next(s)) {
      const int n = warp_uniform(s.hi - s.lo);
      if (n == 0) continue;
      ok = wait_all(q_full, seg & 1) && qk(it);
      for (int i = 0; ok && i < n; ++i) {
        const int t = it + i;
        if (i + 1 < n && !qk(t + 1)) { ok = false; break; }
        const int e = 2 * t + 1, st = e % kRing;
        ok = wait_all(&p_full[t & 1], (t >> 1) & 1) && wait_all(&full[st], (e / kRing) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t v0 = vd + st * (C::kEntry >> 4), p0 = pd + (t & 1) * (C::kPBytes >> 4);
        constexpr int kKeys = 32 / C::kElem;  // keys per MMA
#pragma unroll
        for (int k = 0; k < kTile / kKeys; ++k) {
          const uint64_t ad = v0 + k * (kKeys * C::kRowB >> 4), bd = p0 + (k / 4 * (C::kN * 128 >> 4) + k % 4 * 2);
          if constexpr (F8) umma_f8_ss_by(lead, tmem_o, ad, bd, idesc_pv, (i | k) != 0);
          else umma_f16_ss_by(lead, tmem_o, ad, bd, idesc_pv, (i | k) != 0);
        }
        umma_commit_by(lead, &empty[st]);
        umma_commit_by(lead, &pv_done[t & 1]);
      }
      it += n;
      ++seg;
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int grp = warp >> 2, wq = warp & 3, key = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const int gh = grp * HG;  // first head of the group
    float* wmg = wm + grp * 2 * 4 * C::kWmRow;
    float* bc = bcast + warp * 4 * HG;  // per warp: references, weight factors, factors of the sums and of O
    int it = 0, seg = 0;
    bool ok = true;

    // Q rows of a segment as the MMA's B operand, 8 columns per thread: loaded
    // while the segment before is worked on, laid out when its QK are complete
    constexpr int kVecs = D / 8, kStep = C::kEpiWarps * 32 / kVecs, kQSteps = (NH + kStep - 1) / kStep;
    const int vec = threadIdx.x % kVecs;
    uint4 qw[kQSteps];
    const auto fetch_q = [&](const Seg& g) {
      const int heads = min(p.Gx, p.G - g.h0);
#pragma unroll
      for (int e = 0; e < kQSteps; ++e) {
        const int n = e * kStep + threadIdx.x / kVecs;
        qw[e] = make_uint4(0, 0, 0, 0);
        if (n < g.nh) {
          const int r = SPARSE ? 0 : n / heads;
          qw[e] = ld_global(reinterpret_cast<const uint4*>(
              p.q + (static_cast<int64_t>(g.row0 + r) * p.n_h + g.kvh * p.G + g.h0 + (n - r * heads)) * D + vec * 8));
        }
      }
    };
    const auto store_q = [&](int par) {
#pragma unroll
      for (int e = 0; e < kQSteps; ++e) {
        const int n = e * kStep + threadIdx.x / kVecs;
        const uint4 w = qw[e];
        if constexpr (F8) {
          float f[8], amax = 0.f;
          bf16x8_to_f32(w, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!(fabsf(f[i]) <= 3.4e38f)) f[i] = __int_as_float(0x7fffffff);  // the scores become NaN
            amax = fmaxf(amax, fabsf(f[i]));
          }
#pragma unroll
          for (int o = kVecs / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // X = the power of two with amax <= 256 X: hi rounds off at most 8
          const uint32_t u = __float_as_uint(amax);
          const int ex = max(static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) ? 1 : 0), -100);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = f[2 * i] * inv, b = f[2 * i + 1] * inv;
            hi[i] = e4m3x2(a, b);
            const float2 h = e4m3x2_to_f32(hi[i]);
            lo[i] = e4m3x2((a - h.x) * 32.f, (b - h.y) * 32.f);
          }
          if (n < NH) {
            *reinterpret_cast<uint2*>(q_smem + op_off<C::kRowB>(n, vec * 8)) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(q_smem + op_off<C::kRowB>(NH + n, vec * 8)) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            if (vec == 0) cq[par * NH + n] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * p.scale_log2;
          }
        } else {
          if (n < NH) *reinterpret_cast<uint4*>(q_smem + vec / 8 * (C::kN * 128) + op_off<128>(n, vec % 8 * 16)) = w;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };

    bool more;
    do more = walk.next(s); while (more && s.lo == s.hi);
    if (more) {
      fetch_q(s);
      store_q(0);
    }
    // this CTA's part of the unit in which its run begins, where it has none
    if (p.part_l && threadIdx.x < NH && !(more && s.slot == 0)) p.part_l[2ll * blockIdx.x * NH + threadIdx.x] = make_float2(-INFINITY, 0.f);
    while (ok && more) {
      const Seg cur = s;
      more = walk.next(s);
      if (more) fetch_q(s);
      // lane h (mod HG) keeps the reference exponents of head h: m of the
      // weights, m + mr of the weighted V scales (relative, because a large m
      // would swallow a scale's share), m + low the lowest that the latter may
      // fall to; every thread its keys' sums
      float m = -INFINITY, mr = -INFINITY, low = kLowest, l[HG];
#pragma unroll
      for (int h = 0; h < HG; ++h) l[h] = 0.f;
      const int heads = min(p.Gx, p.G - cur.h0);
      float c[HG];  // factors of the scores
      if constexpr (F8) {
        ok = mbar_wait(q_full, seg & 1, abort_flag);
#pragma unroll
        for (int h = 0; h < HG; ++h) c[h] = cq[(seg & 1) * NH + gh + h];
      }
      for (int i = cur.lo; i < cur.hi; ++i, ++it) {
        const int buf = it & 1;
        ok = mbar_wait(&meta_full[it % kMetas], (it / kMetas) & 1, abort_flag) && ok;
        const int4 mt = ok ? meta[it % kMetas * 8 + (key >> p.shift)] : make_int4(kNoPage, 0, 0, 0);
        const float ks = __int_as_float(mt.y), vs = __int_as_float(mt.z);
        const int pos = mt.x + (key & (p.page - 1)), past = pos - cur.t0;
        float x[HG];
        float lvs = 0.f;
        if constexpr (F8) lvs = __log2f(p.page == 16 ? vs : warp_max_f32(vs));  // (a warp's keys lie in one page, or in two of 16)
        ok = ok && mbar_wait(&s_full[buf], (it >> 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const uint32_t ts = tmem + buf * C::kN + lanes;
        if constexpr (F8) {
          uint32_t a[HG], b[HG];
          tmem_ld32<HG>(ts + gh, a);
          tmem_ld32<HG>(ts + NH + gh, b);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < HG; ++h) x[h] = __fmul_rn(fmaf(__uint_as_float(b[h]), 1.f / 32, __uint_as_float(a[h])), ks * c[h]);
        } else {
          uint32_t a[HG];
          tmem_ld32<HG>(ts + gh, a);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < HG; ++h) x[h] = __fmul_rn(__uint_as_float(a[h]), p.scale_log2);
        }
        const bool edge = __any_sync(0xffffffffu, past >= 0);
        if (edge) {
          // head row n sees this key from n = nmin on (rows see one position more each)
          const int nmin = past < 0 ? 0 : (past < cur.nr ? (past + 1) * heads : kNoPage);
#pragma unroll
          for (int h = 0; h < HG; ++h) x[h] = gh + h >= nmin ? x[h] : -INFINITY;
        }
        // ---- the tile's maximum per head, over the four warps
        {
          float* w = wmg + (buf * 4 + wq) * C::kWmRow;
          float r[HG];
#pragma unroll
          for (int h = 0; h < HG; ++h) r[h] = warp_max_f32(x[h]);
          if (lane == 0) {
#pragma unroll
            for (int h = 0; h < HG; h += 4) *reinterpret_cast<float4*>(w + h) = make_float4(r[h], r[h + 1], r[h + 2], r[h + 3]);
            if (F8) w[HG] = lvs;
          }
          if (F8 && p.page == 16) {  // per head: a page below the top score may weigh more
#pragma unroll
            for (int h = 0; h < HG; ++h) r[h] = warp_max_f32((x[h] - r[h]) + lvs);
            if (lane == 0) {
#pragma unroll
              for (int h = 0; h < HG; h += 4) *reinterpret_cast<float4*>(w + HG + h) = make_float4(r[h], r[h + 1], r[h + 2], r[h + 3]);
            }
          }
        }
        if (!named_bar_and(1 + grp, 128, ok)) { ok = false; break; }
        bool grew, grew_l;
        {
          const float* w = wmg + buf * 4 * C::kWmRow;
          const int h = lane % HG;
          float t = -INFINITY, tp = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) t = fmaxf(t, w[q * C::kWmRow + h]);
          const float mn = fmaxf(m, ceilf(t));
          const float mu = mn == -INFINITY ? 0.f : mn;
          if (F8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) tp = fmaxf(tp, (w[q * C::kWmRow + h] - mu) + w[q * C::kWmRow + HG + (p.page == 16 ? h : 0)]);
          }
          const float was = mr + (m - mu);
          float pr = 0.f;
          if (F8) {
            tp = ceilf(tp);
            pr = tp > was || (tp < was - kFall && tp > low) ? tp : was;
          }
          grew_l = __any_sync(0xffffffffu, mn > m);
          grew = F8 ? __any_sync(0xffffffffu, pr != was) : grew_l;
          if (lane < HG) {
            bc[lane] = mu;
            if (F8) bc[HG + lane] = ex2_approx(pr == -INFINITY ? 8.f : fminf(8.f - pr, 120.f));
            if (grew_l) bc[2 * HG + lane] = mn > m ? ex2_approx(m - mn) : 1.f;
            if (F8 && grew) bc[3 * HG + lane] = pr != was ? ex2_approx(was - pr) : 1.f;
          }
          if (F8) low = fmaxf(fmaxf(low + (m - mu), tp - kFallMost), kLowest);
          m = mn;
          mr = pr;
          __syncwarp();
        }
        if (grew_l) {
#pragma unroll
          for (int h = 0; h < HG; ++h) l[h] *= bc[2 * HG + h];
        }
        // ---- weights, as the MMA's B operand.  P(it - 2) has been read.
        if (it >= 2) ok = mbar_wait(&pv_done[buf], ((it - 2) >> 1) & 1, abort_flag) && ok;
        uint8_t* pb = p_smem + buf * C::kPBytes;
        // (all computed before the first store: byte stores may alias the factors)
        uint32_t code[HG];  // F8: a pair's hi codes, its lo codes above them; bf16: a pair's hi words, then the lo words
#pragma unroll
        for (int h = 0; h < HG; h += 2) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            w[e] = ex2_approx(x[h + e] - bc[h + e]);
            l[h + e] += w[e];
            if constexpr (F8) w[e] = w[e] * vs * bc[HG + h + e];  // (in this order no product overflows)
          }
          if constexpr (F8) {
            const uint32_t hi = e4m3x2(w[0], w[1]);
            const float2 back = e4m3x2_to_f32(hi);
            code[h / 2] = hi | e4m3x2((w[0] - back.x) * 32.f, (w[1] - back.y) * 32.f) << 16;
          } else {
            const uint32_t hi = pack_bf16(w[0], w[1]);
            code[h / 2] = hi;
            if constexpr (C::kTwo)
              code[HG / 2 + h / 2] = pack_bf16(w[0] - __uint_as_float(hi << 16), w[1] - __uint_as_float(hi & 0xffff0000u));
          }
        }
        if constexpr (F8) {
#pragma unroll
          for (int h = 0; h < HG; h += 2) {
            const uint32_t v = code[h / 2];
            pb[op_off<128>(gh + h, key)] = static_cast<uint8_t>(v);
            pb[op_off<128>(gh + h + 1, key)] = static_cast<uint8_t>(v >> 8);
            pb[op_off<128>(NH + gh + h, key)] = static_cast<uint8_t>(v >> 16);
            pb[op_off<128>(NH + gh + h + 1, key)] = static_cast<uint8_t>(v >> 24);
          }
        } else {
          uint8_t* dst = pb + (key >> 6) * (C::kN * 128);
#pragma unroll
          for (int t = 0; t < (C::kTwo ? 2 : 1); ++t)
#pragma unroll
            for (int h = 0; h < HG; h += 2) {
              const uint32_t v = code[t * (HG / 2) + h / 2];
              *reinterpret_cast<uint16_t*>(dst + op_off<128>(t * NH + gh + h, (key & 63) * 2)) = static_cast<uint16_t>(v);
              *reinterpret_cast<uint16_t*>(dst + op_off<128>(t * NH + gh + h + 1, (key & 63) * 2)) = static_cast<uint16_t>(v >> 16);
            }
        }
        // ---- O follows a new reference exponent
        if (grew && i > cur.lo) {  // the same for the whole group
          ok = mbar_wait(&pv_done[buf ^ 1], ((it - 1) >> 1) & 1, abort_flag) && ok;
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          if (wq * 32 < D) {
            const float* fo = bc + (F8 ? 3 : 2) * HG;
#pragma unroll
            for (int t = 0; t < (C::kTwo ? 2 : 1); ++t) {
              uint32_t o[HG];
              const uint32_t to = tmem_o + lanes + gh + t * NH;
              tmem_ld32<HG>(to, o);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < HG; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * fo[h]);
              if constexpr (HG == 8) tmem_st32x8(to, o);
              else tmem_st32x16(to, o);
            }
            tmem_st_wait();
          }
        }
        // ---- slots that no row of the unit sees hold anything: V = 0 there.
        // A slot that only later rows see must not reach the earlier ones
        // through 0 * inf: such values are set aside and added at the end.
        if (grp == 0 && edge && __any_sync(0xffffffffu, past >= 0 && mt.x != kNoPage)) {
          const int e = 2 * it + 1, st = e % kRing;
          ok = mbar_wait(&full[st], (e / kRing) & 1, abort_flag) && ok;
          if (ok && past >= 0 && mt.x != kNoPage) {
#pragma unroll
            for (int c = 0; c < C::kSlabs; ++c) {
              uint4* row = reinterpret_cast<uint4*>(ring + st * C::kEntry + c * C::kSlabBytes + key * C::kRowB);
              for (int v = 0; v < C::kRowB / 16; ++v) {
                uint4 w = row[v];
                uint32_t y[4] = {w.x, w.y, w.z, w.w};
                bool bad = pos >= cur.t1;
                if (!bad) {
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    const uint32_t gone = F8 ? __vcmpeq4(y[u] & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(y[u] & 0x7f807f80u, 0x7f807f80u);
                    y[u] &= ~gone;
                    bad = bad || gone != 0;
                  }
                  if (bad) poison[seg & 1] = 1;
                  if (bad) row[v] = make_uint4(y[0], y[1], y[2], y[3]);
                } else {
                  row[v] = make_uint4(0, 0, 0, 0);
                }
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // ---- the next segment's queries: every QK of this one is complete
      const int last = it - 1;
      if (more) store_q((seg + 1) & 1);

      // ---- output of the segment
#pragma unroll
      for (int h = 0; h < HG; ++h) {
#pragma unroll
        for (int o = 16; o; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
        if (lane == h) lsum[wq * NH + gh + h] = l[h];
      }
      if (ok) ok = mbar_wait(&pv_done[last & 1], (last >> 1) & 1, abort_flag);
      // the other flag's readers (the segment before) are done: every warp has
      // delivered weights of this segment, and none begins the next one before
      // the barrier below
      if (threadIdx.x == 0) poison[(seg & 1) ^ 1] = 0;
      if (!named_bar_and(1 + grp, 128, ok)) { ok = false; break; }
      tc_fence_after();
      float o[HG];
      if constexpr (C::kTwo) {
        uint32_t a[HG], b[HG];
        tmem_ld32<HG>(tmem_o + lanes + gh, a);
        tmem_ld32<HG>(tmem_o + lanes + NH + gh, b);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HG; ++h) o[h] = fmaf(__uint_as_float(b[h]), F8 ? 1.f / 32 : 1.f, __uint_as_float(a[h]));
      } else {
        uint32_t a[HG];
        tmem_ld32<HG>(tmem_o + lanes + gh, a);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HG; ++h) o[h] = __uint_as_float(a[h]);
      }
      tc_fence_before();
      // lane h: total, 1 / total and log2 of head h
      {
        const float* t = lsum + gh + lane % HG;
        const float sum = (t[0] + t[NH]) + (t[2 * NH] + t[3 * NH]);
        const float f = F8 ? ex2_approx((mr == -INFINITY ? 0.f : mr) - 8.f) : 1.f;
        if (lane < HG) bc[lane] = sum == 0.f ? 0.f : f / sum;
        if (wq == 0 && lane < HG && gh + lane < cur.nh) {
          const int n = gh + lane, r = SPARSE ? 0 : n / heads;
          if (cur.slot < 0) {
            if (p.lse) p.lse[static_cast<int64_t>(cur.row0 + r) * p.n_h + cur.kvh * p.G + cur.h0 + (n - r * heads)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
          } else {
            p.part_l[(2ll * blockIdx.x + cur.slot) * NH + n] = sum == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(m, log2f(sum));
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < HG; ++h) o[h] = bc[h] == 0.f ? 0.f : o[h] * bc[h];
      if (poison[seg & 1] && key < D) {  // values that are not finite, for the rows that see them
        for (int t = max(cur.t0, cur.lo * kTile); t < min(cur.t1, cur.hi * kTile); ++t) {
          const int pg = paged_page(p.a, cur.b, t / p.page);
          if (pg < 0) continue;
          const int64_t at = ((static_cast<int64_t>(pg) * p.a.n_kv + cur.kvh) * p.page + t % p.page) * D + key;
          float v;
          if constexpr (F8) v = e4m3x2_to_f32(static_cast<const uint8_t*>(p.a.v)[at]).x;
          else v = __uint_as_float(static_cast<uint32_t>(static_cast<const dsa_bf16*>(p.a.v)[at]) << 16);
          if (fabsf(v) <= 3.4e38f) continue;
#pragma unroll
          for (int h = 0; h < HG; ++h)
            if ((gh + h) / heads > t - cur.t0) o[h] += v;
        }
      }
      if (key < D) {
        if (cur.slot < 0) {
          int r = SPARSE ? 0 : gh / heads, g = gh - r * heads;
          dsa_bf16* dst = p.out + (static_cast<int64_t>(cur.row0) * p.n_h + cur.kvh * p.G + cur.h0) * D + key;
#pragma unroll
          for (int h = 0; h < HG; ++h) {
            const __nv_bfloat16 y = __float2bfloat16_rn(o[h]);
            if (gh + h < cur.nh) dst[(r * p.n_h + g) * D] = *reinterpret_cast<const dsa_bf16*>(&y);
            if (++g == heads) { g = 0; ++r; }
          }
        } else {
          float* dst = p.part_o + ((2ll * blockIdx.x + cur.slot) * NH + gh) * D + key;
#pragma unroll
          for (int h = 0; h < HG; ++h) dst[h * D] = o[h];
        }
      }
      if (threadIdx.x == 0 && cur.slot != 0 && p.meta) p.meta[cur.unit] = cur.slot < 0 ? make_int2(-1, -1) : make_int2(blockIdx.x, cur.last_cta);
      ++seg;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, 1u);
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of a unit that several CTAs worked on: each part is its
// normalised output, and its reference and log2 of its sum above that.  One block per (unit, head).
template <int D>
__global__ void __launch_bounds__(D) paged_attn_merge_kernel(const PattnParams p, int NH, int sparse) {
  pdl_trigger();
  pdl_wait();
  const int unit = blockIdx.x, n = blockIdx.y, d = threadIdx.x;
  int row0, nr, kvh, h0;
  if (sparse) {
    row0 = unit % p.a.total_q;
    nr = 1;
    const int rem = unit / p.a.total_q;
    kvh = rem / p.hbs;
    h0 = rem % p.hbs * p.Gx;
  } else {
    const int rb = unit % p.max_rb;
    const int rem = unit / p.max_rb;
    h0 = 0;
    kvh = rem % p.a.n_kv;
    int r0, rows;
    paged_rows(p.a, rem / p.a.n_kv, r0, rows);
    row0 = r0 + rb * p.R;
    nr = min(p.R, rows - rb * p.R);
  }
  const int heads = min(p.Gx, p.G - h0);
  if (nr <= 0 || n >= heads * nr) return;
  const int2 c = p.meta[unit];
  if (c.x < 0 || c.x >= kMaxCtas || c.y >= kMaxCtas) return;  // (anything may stand here after a call that gave up waiting)
  const auto slot = [&](int i) { return static_cast<int64_t>(2 * i + (i == c.x)) * NH + n; };
  float base = -INFINITY, top = -INFINITY;  // top relative to the largest x, since that may swallow y
  for (int i = c.x; i <= c.y; ++i) {
    const float2 x = p.part_l[slot(i)];
    if (x.x > base) { top += base - x.x; base = x.x; }
    top = fmaxf(top, (x.x - base) + x.y);  // (NaN for the empty parts before the first sum: passed over)
  }
  if (base == -INFINITY) base = 0.f;
  const float ref = top == -INFINITY ? 0.f : top;
  float acc = 0.f, sum = 0.f;
  for (int i = c.x; i <= c.y; ++i) {
    const float2 x = p.part_l[slot(i)];
    const float l2 = (x.x - base) + x.y;
    const float w = exp2f(l2 - ref);
    sum += w;
    if (l2 != -INFINITY) acc += w * p.part_o[slot(i) * D + d];
  }
  const int r = n / heads;
  const int64_t at = static_cast<int64_t>(row0 + r) * p.n_h + kvh * p.G + h0 + (n - r * heads);
  const __nv_bfloat16 y = __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
  p.out[at * D + d] = *reinterpret_cast<const dsa_bf16*>(&y);
  if (d == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (base + (ref + log2f(sum))) * kLn2;
}

// How a call is cut into units, and what it needs.
struct Plan {
  int NH, G, Gx, R, hbs, max_rb, tpu, aligned, grid, merge;
  long long units;
  size_t o_bytes, l_bytes, meta_bytes;
  size_t total() const { return o_bytes + l_bytes + meta_bytes; }
};

Plan make_plan(const dsa_paged_kv* kv, const dsa_paged_batch* pb, int n_h, int n_sel) {
  Plan pl{};
  const int G = n_h / kv->n_kv;
  pl.G = G;
  // columns of a unit: the group's heads, times a few rows when all pages are
  // read (32 columns at most then: use_prefill; selected pages take larger
  // groups in blocks of 32 heads)
  const long long want = n_sel ? G : static_cast<long long>(G) * pb->max_Lq;
  pl.NH = want <= 8 ? 8 : (want <= 16 ? 16 : 32);
  pl.Gx = std::min(G, pl.NH);
  pl.hbs = (G + pl.Gx - 1) / pl.Gx;
  pl.R = n_sel ? 1 : pl.NH / pl.Gx;
  pl.max_rb = n_sel ? 1 : (pb->max_Lq + pl.R - 1) / pl.R;
  pl.tpu = n_sel ? (n_sel * kv->page + kTile - 1) / kTile : (pb->max_Lk + kTile - 1) / kTile;
  pl.units = (n_sel ? static_cast<long long>(pb->total_q) : static_cast<long long>(pb->B) * pl.max_rb) * kv->n_kv * pl.hbs;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const int two = std::min(kMaxCtas, sms * (pl.NH <= 16 ? 2 : 1));
  // many units of selected 8-bit pages run three CTAs to an SM (latency-bound:
  // 1359 -> 1157 us for 16,384 units of 16 tiles)
  const int ctas = n_sel && pl.NH == 8 && kv->fmt == DSA_KV_E4M3 && pl.units >= 8ll * two ? std::min(kMaxCtas, sms * 3) : two;
  // Whole units per CTA and no merge: for units of a few tiles (1 x 8 heads x 500
  // tokens: 9.8 us whole, 10.4 us cut; 1,000 tokens 14.3 and 10.8), a few more
  // where the units occupy a third of the GPU (16 x 8 heads x 1,000 tokens: 15.5
  // and 17.6), and for many equal units of selected pages.
  pl.aligned = pl.tpu <= 4 || (pl.tpu <= 8 && pl.units * 3 >= ctas) || (n_sel && pl.units >= 8ll * ctas);
  pl.grid = static_cast<int>(std::min<long long>(ctas, pl.aligned ? pl.units : std::max(1ll, pl.units * pl.tpu / 2)));
  pl.merge = !pl.aligned && pl.grid > 1;
  if (pl.merge) {
    pl.o_bytes = static_cast<size_t>(2 * kMaxCtas) * pl.NH * kv->D * 4;
    pl.l_bytes = static_cast<size_t>(2 * kMaxCtas) * pl.NH * 8;
    pl.meta_bytes = static_cast<size_t>((pl.units + 1) / 2) * 16;
  }
  return pl;
}

template <int D, bool F8, int NH, bool SPARSE>
cudaError_t launch_attn(const CUtensorMap& k, const CUtensorMap& v, const PattnParams& p, const Plan& pl, cudaStream_t s) {
  using C = Cfg<D, F8, NH, SPARSE>;
  auto fn = paged_attn_kernel<D, F8, NH, SPARSE>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(fn), C::kSmem);
  if (e == cudaSuccess) e = launch_pdl(fn, dim3(pl.grid), dim3(C::kThreads), C::kSmem, s, k, v, p);
  if (e == cudaSuccess && pl.merge)
    e = launch_pdl(paged_attn_merge_kernel<D>, dim3(static_cast<unsigned>(pl.units), NH), dim3(D), 0, s, p, NH, SPARSE ? 1 : 0);
  return e;
}
template <int D, bool F8, int NH>
cudaError_t launch_attn(const CUtensorMap& k, const CUtensorMap& v, const PattnParams& p, const Plan& pl, cudaStream_t s) {
  return p.sel ? launch_attn<D, F8, NH, true>(k, v, p, pl, s) : launch_attn<D, F8, NH, false>(k, v, p, pl, s);
}
template <int D, bool F8>
cudaError_t launch_attn(const CUtensorMap& k, const CUtensorMap& v, const PattnParams& p, const Plan& pl, cudaStream_t s) {
  return pl.NH == 8 ? launch_attn<D, F8, 8>(k, v, p, pl, s)
                    : (pl.NH == 16 ? launch_attn<D, F8, 16>(k, v, p, pl, s) : launch_attn<D, F8, 32>(k, v, p, pl, s));
}

// Many rows that read all pages: query rows on the tile's rows.  The border is
// the most columns of the other kernel.  At 40, 64 and 128 columns (5, 8 and 16
// rows x 8 heads) that one, in several units, takes 156, 193 and 274 us against
// 194, 195 and 355 here for 16 sequences of up to 30,000 bf16 tokens (8-bit 182,
// 223 and 377 against 246, 248 and 455), but 42, 47 and 72 against 35, 35 and 36
// for 32 sequences of up to 2,000 (8-bit 46, 52 and 82 against 40, 42 and 44);
// for one sequence the two are equal.
bool use_prefill(const dsa_paged_kv* kv, const dsa_paged_batch* pb, int n_h, int n_sel) {
  return !n_sel && static_cast<long long>(n_h / kv->n_kv) * pb->max_Lq > 32;
}

// Tensor map of a pool: {columns, slots, heads, pages}, boxes of one page of one head.
bool pool_map(CUtensorMap* m, const dsa_paged_kv* kv, const void* base, bool swizzled) {
  const bool f8 = kv->fmt == DSA_KV_E4M3;
  const uint64_t e = f8 ? 1 : 2, D = static_cast<uint64_t>(kv->D);
  const uint32_t cols = static_cast<uint32_t>(std::min<uint64_t>(D, 128 / e));
  return encode_tiled_4d(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                         {D, static_cast<uint64_t>(kv->page), static_cast<uint64_t>(kv->n_kv), static_cast<uint64_t>(kv->n_pages)},
                         {D * e, D * e * kv->page, D * e * kv->page * kv->n_kv}, cols, static_cast<uint32_t>(kv->page),
                         !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : cols * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_paged_attn_workspace(const dsa_paged_kv* kv, const dsa_paged_batch* batch, int n_h, int n_sel) {
  if (check_paged_host("dsa_paged_attn_workspace", kv, batch, nullptr) != DSA_OK || n_h < 1 || n_h % kv->n_kv || n_sel < 0) return 0;
  if (n_h > 128) return 0;
  return std::max<size_t>(16, use_prefill(kv, batch, n_h, n_sel) ? paged_prefill_plan(kv, batch, n_h).total()
                                                                 : make_plan(kv, batch, n_h, n_sel).total());
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
  if (!(scale > 0.f) || scale > 1e30f) return set_error(DSA_ERR_INVALID_ARG, "dsa_paged_attn: scale must be positive and at most 1e30");
  if (!ws || !aligned16(ws) || ws_bytes < dsa_paged_attn_workspace(kv, batch, n_h, n_sel))
    return set_error(DSA_ERR_WORKSPACE, "dsa_paged_attn: workspace null, misaligned or too small");
  unsigned int* err = device_error_word();
  if (!err) return set_error(DSA_ERR_CUDA, "dsa_paged_attn: cannot find the device error word");
  const bool f8 = kv->fmt == DSA_KV_E4M3, many = use_prefill(kv, batch, n_h, n_sel);
  const int shift = kv->page == 16 ? 4 : (kv->page == 32 ? 5 : (kv->page == 64 ? 6 : 7));
  uint8_t* w = static_cast<uint8_t*>(ws);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap mk, mv;
  if (!pool_map(&mk, kv, kv->k, !(many && f8)) || !pool_map(&mv, kv, kv->v, !(many && f8)))
    return set_error(DSA_ERR_CUDA, "dsa_paged_attn: cuTensorMapEncodeTiled failed");
  cudaError_t e;
  if (many) {
    const PrefillPlan pl = paged_prefill_plan(kv, batch, n_h);
    if (pl.units * 256 > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_attn: batch too large");
    PrefillParams x{};
    x.a = p.a; x.q = q; x.n_h = n_h; x.G = n_h / kv->n_kv; x.page = kv->page; x.shift = shift; x.ppt = kTile / kv->page;
    x.inclusive = inclusive; x.tok = pl.tok; x.blocks = pl.blocks; x.splits = pl.splits; x.scale_log2 = scale * kLog2e;
    x.out = out; x.lse = lse; x.err = err;
    if (pl.splits > 1) {
      x.part_o = reinterpret_cast<float*>(w);
      x.part_l = reinterpret_cast<float2*>(w + pl.o_bytes);
    }
    e = paged_prefill_launch(mk, mv, kv->D, f8, x, s);
  } else {
    const Plan pl = make_plan(kv, batch, n_h, n_sel);
    if (pl.units > 2147483647ll) return set_error(DSA_ERR_UNSUPPORTED, "dsa_paged_attn: batch too large");
    p.q = q; p.sel = sel; p.n_h = n_h; p.G = pl.G; p.page = kv->page; p.shift = shift; p.ppt = kTile / kv->page;
    p.inclusive = inclusive; p.n_sel = n_sel; p.Gx = pl.Gx; p.R = pl.R; p.hbs = pl.hbs; p.max_rb = pl.max_rb; p.tpu = pl.tpu;
    p.aligned = pl.aligned; p.scale_log2 = scale * kLog2e; p.out = out; p.lse = lse; p.err = err;
    if (pl.merge) {
      p.part_o = reinterpret_cast<float*>(w);
      p.part_l = reinterpret_cast<float2*>(w + pl.o_bytes);
      p.meta = reinterpret_cast<int2*>(w + pl.o_bytes + pl.l_bytes);
    }
    e = kv->D == 64 ? (f8 ? launch_attn<64, true>(mk, mv, p, pl, s) : launch_attn<64, false>(mk, mv, p, pl, s))
                    : (f8 ? launch_attn<128, true>(mk, mv, p, pl, s) : launch_attn<128, false>(mk, mv, p, pl, s));
  }
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, std::string("dsa_paged_attn launch: ") + cudaGetErrorString(e));
  return DSA_OK;
}

}  // extern "C"
