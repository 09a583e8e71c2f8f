// Shared by the paged attention's kernels: their arguments, the merge of the
// chunks a prefix is split into, and small helpers.  Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>

#include "et_attn_internal.h"
#include "et_paged.cuh"
#include "et_tc.cuh"

namespace et {

struct PagedAttnArgs {
  int B, N, Hq, Hkv, G, P, max_blocks, W, max_prefix;
  float scale_log2;  // scale * log2(e)
  long long num_pages, page_stride;
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *prefix_len;
  const void *q, *kt, *vt;
  const unsigned long long *mask;
  void *out;
  float *lse;
  int32_t *dev_status;
};

// A call whose prefixes are split into chunks.
struct PagedSplitArgs {
  PagedAttnArgs a;
  int S, tiles_y;       // chunks, Hkv * row tiles
  int flat;             // blocks per row tile that share the whole batch; 0: S of each sequence
  int row_tiles;        // row tiles per KV head
  int box;              // rows per TMA box
  unsigned int *cnt;    // [B * tiles_y] arrival counters; null when the chunks need none (one, or a cluster)
  float2 *part_ml;      // [B * tiles_y][S][R] (maximum, sum)
  float4 *part_o;       // [B * tiles_y][S][R][D] fp32
  uint32_t page_magic, group_magic, group_shift;  // page_index, row_token
  long long wait_cycles;
};

// D = 128, many rows per KV head (et_paged_attention_tc.cu)
constexpr int kPtKeys = 128;  // keys per tile
constexpr int kPtRows = 64;   // query rows per block
constexpr int kPaMaxCluster = 8;  // chunks up to which a sequence's blocks form a cluster (the portable size)
// clusters of S blocks that the device runs at once (a property of the device, asked once)
ET_HIDDEN int paged_tc_clusters(int S, int sms);
// pages as [num_pages][Hkv][P][d] bytes; a box is `box` rows of one head of one page
ET_HIDDEN bool make_page_map(CUtensorMap *m, const void *base, const et_paged_cache *c, int box);
ET_HIDDEN et_status paged_tc_launch(const et_paged_cache *cache, const PagedSplitArgs &a, cudaStream_t stream);

namespace {

constexpr int kPaMaxSplits = 64;
// Weights lie at or below 2^kPaTop when a row's reference moves to its maximum, and the reference stays until one would
// pass 2^15, short of fp16's largest.  What lies 2^28 below the maximum is lost then (fp16's smallest value is 2^-24).
constexpr float kPaTop = 3.f, kPaSlack = 12.f;

// token -> page of its sequence, pages of 16 * p tokens, p <= 16: umulhi by ceil(2^32 / p) is exact below 2^28 units of 16
__device__ __forceinline__ int page_index(const PagedSplitArgs &a, int token) {
  const uint32_t u = (uint32_t)token >> 4;
  return (int)(a.page_magic ? __umulhi(u, a.page_magic) : u);
}
// row of a KV head's (token, head in group) rows -> token: with 2^k < G <= 2^(k + 1), umulhi by ceil(2^(32 + k) / G) and a
// shift by k are exact below 2^31 rows
__device__ __forceinline__ int row_token(const PagedSplitArgs &a, int row) {
  return (int)(a.group_magic ? __umulhi((uint32_t)row, a.group_magic) >> a.group_shift : (uint32_t)row);
}
// prefix length of sequence b as the kernels use it: -1 = no sequence here
__device__ __forceinline__ int paged_prefix(const PagedAttnArgs &a, int b, int &bad) {
  int L = a.prefix_len[b];
  const long long room = min((long long)a.max_prefix, (long long)a.max_blocks * a.P);
  if (L > room) {
    bad = 1;
    L = (int)room;
  }
  return L < 0 ? -1 : L;
}
// tiles that n tokens take, n < 2^31
__device__ __forceinline__ int tiles_of(int n, uint32_t tile) { return (int)(((uint32_t)n + tile - 1u) / tile); }
__device__ __forceinline__ float clamp_v_scale(float s) {
  return fminf(fmaxf(s, 1.f / (1ll << kScaleExp)), (float)(1ll << kScaleExp));  // NaN -> the smallest
}
__device__ __forceinline__ bool tree_keeps(const PagedAttnArgs &a, int b, int i, int tt) {
  if (!a.mask) return tt <= i;
  return (a.mask[((long long)b * a.N + i) * a.W + (tt >> 6)] >> (tt & 63)) & 1ull;
}

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float4 cl_ld_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// The rows of a tile's chunks, from the workspace, weighted by their maxima:
// run by the last block of the tile to arrive (NT threads, `sm` free shared
// memory).  Every load of a row's parts is in flight before any arithmetic.
template <int D, int R, int NT, typename Write>
__device__ __forceinline__ void merge_chunks(const PagedSplitArgs &ma, long long slot0, int chunks, int real,
                                             unsigned char *sm, Write write_row) {
  const int t = threadIdx.x;
  const long long base = slot0 * R;  // slot0: the first chunk's place in the workspace
  float2 *pair = reinterpret_cast<float2 *>(sm);  // [chunks][real]: (maximum, sum), then (weight, -)
  float2 *stat = pair + kPaMaxSplits * R;         // [real]: the row's maximum and sum
  for (int x = t; x < chunks * real; x += NT) {
    const int k = x / real, r = x - k * real;
    pair[x] = __ldcg(&ma.part_ml[base + (long long)k * R + r]);
  }
  __syncthreads();
  for (int r = t; r < real; r += NT) {
    float M = pair[r].x, sum = 0.f;
    for (int k = 1; k < chunks; ++k) M = fmaxf(M, pair[k * real + r].x);
    for (int k = 0; k < chunks; ++k) {
      const float w = ex2_fast(pair[k * real + r].x - M);
      sum = fmaf(pair[k * real + r].y, w, sum);
      pair[k * real + r].x = w;
    }
    stat[r] = make_float2(M, sum);
  }
  __syncthreads();
  constexpr int X = 4, K = 4;  // four cells' loads of four chunks
  for (int x0 = t; x0 < real * (D / 4); x0 += X * NT) {
    float4 v[X];
#pragma unroll
    for (int i = 0; i < X; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < chunks; k0 += K) {
      float4 y[X][K];
#pragma unroll
      for (int i = 0; i < X; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int x = x0 + i * NT, r = x / (D / 4), c = x - r * (D / 4);
          y[i][j] = x < real * (D / 4) && k0 + j < chunks
                        ? __ldcg(&ma.part_o[(base + (long long)(k0 + j) * R + r) * (D / 4) + c])
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int i = 0; i < X; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int x = x0 + i * NT, r = x / (D / 4);
          const float w = x < real * (D / 4) && k0 + j < chunks ? pair[(k0 + j) * real + r].x : 0.f;
          v[i].x = fmaf(y[i][j].x, w, v[i].x); v[i].y = fmaf(y[i][j].y, w, v[i].y);
          v[i].z = fmaf(y[i][j].z, w, v[i].z); v[i].w = fmaf(y[i][j].w, w, v[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < X; ++i) {
      const int x = x0 + i * NT, r = x / (D / 4), c = x - r * (D / 4);
      if (x < real * (D / 4)) write_row(r, c, v[i], stat[r].x, stat[r].y);
    }
  }
}

}  // namespace
}  // namespace et
