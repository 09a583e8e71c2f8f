// Shared by the chunk attention's kernels: their arguments and the reading of
// a sequence's place in the batch.  Not part of the C ABI.
#pragma once

#include "et_paged_attn.cuh"

namespace et {

struct ChunkArgs {
  PagedAttnArgs a;   // N: the most new rows of a sequence; kt, vt: the new keys and values; mask unused
  int rows;          // of q, the new keys and values and out
  long long qs, ks, vs;  // elements from row to row
  const int32_t *row_start;
};

// bf16 (et_chunk_attention_tc.cu): units of 128 or 256 (token, head) rows of a KV head, a block or several each
struct ChunkTcPlan {
  int S;      // parts of a unit's keys at most
  int shift;  // a unit: 1 << shift rows of a KV head, 128 or 256
  int tiles;  // units per KV head at most
  int whole;  // units that stay in one part: of up to 32 sequences those with the most keys, of more the first ones
  size_t ml_off, o_off;
};
ET_HIDDEN et_status chunk_tc_launch(const et_paged_cache *cache, const ChunkArgs &c, const ChunkTcPlan &p, void *ws,
                                    cudaStream_t stream);

namespace {

// New rows of sequence b: first row and count; count 0 = nothing to do.
__device__ __forceinline__ void chunk_rows(const ChunkArgs &c, int b, int &first, int &n, int &bad) {
  const int r0 = c.row_start[b], r1 = c.row_start[b + 1];
  first = r0;
  n = r1 - r0;
  if (r0 < 0 || r1 > c.rows || r1 < r0) {
    bad = 1;
    n = 0;
  } else if (n > c.a.N) {
    bad = 1;
    n = c.a.N;
  }
}

// A start that counts where row_start is wrong.  A sequence whose first row lies before an earlier one of them is left out: b's
// rows may be others', too.  Without such sequences no two have a row in common: the units fit the plan's count of them, and
// their sums fit 32 bits.
__device__ __forceinline__ int chunk_start(const ChunkArgs &c, int first) { return first >= 0 && first <= c.rows ? first : -1; }

}  // namespace
}  // namespace et
