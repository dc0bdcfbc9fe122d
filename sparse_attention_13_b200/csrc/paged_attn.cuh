// paged_attn.cuh -- what the two attention kernels over a paged cache share:
// keys on the tile's rows (paged_attn.cu: few rows, or selected pages) and
// query rows on the tile's rows (paged_prefill.cu: many rows, all pages).
#pragma once

#include "paged.cuh"

namespace dsa {

struct PrefillParams {
  PagedArgs a;
  const dsa_bf16* q;
  int n_h, G, page, shift, ppt, inclusive;  // shift: log2 page; ppt: pages per tile
  int tok, splits;                          // tokens of a Q tile, parts of the keys
  long long blocks;                         // blocks of two Q tiles of the batch, at most
  float scale_log2;
  dsa_bf16* out;
  float* lse;
  float* part_o;                            // [unit][split][2][128][D]
  float2* part_l;                           // [unit][split][2][128]: log2 of a part's sum is x + y
  unsigned int* err;
};

struct PrefillPlan {
  int tok, splits;
  long long blocks, units;
  size_t o_bytes, l_bytes;
  size_t total() const { return o_bytes + l_bytes; }
};

PrefillPlan paged_prefill_plan(const dsa_paged_kv* kv, const dsa_paged_batch* pb, int n_h);
cudaError_t paged_prefill_launch(const CUtensorMap& k, const CUtensorMap& v, int D, bool f8, const PrefillParams& p, cudaStream_t s);

}  // namespace dsa
