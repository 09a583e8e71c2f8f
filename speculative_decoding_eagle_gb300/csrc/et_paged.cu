// The paged 8-bit KV cache's bookkeeping and writer (EAGLE blog section 1.1:
// the accepted tokens of one verification forward are kept; EAGLE-2 article:
// the flattened tree's rows attend the prefix and their ancestors).
//
//  k_block_map      block tables and slot maps from the requests' lengths
//  k_commit_paged   accepted rows, or a prompt's, quantised into the pages
#include <cuda_bf16.h>

#include "et_paged.cuh"

namespace et {
namespace {

// ---------------------------------------------------------------------------
// block map
// ---------------------------------------------------------------------------
// Every returned page and every taken page has a place on one virtual stack,
// free_list[0..F) followed by the R returned pages in (request, block) order;
// the a-th taken page is entry F + R - 1 - a.  So two exclusive sums over the
// requests (pages returned, pages taken) say where each page goes, and each
// page is moved by one thread: no atomics, no order to depend on.
//
// One cluster does it all in place: every block reads all B lengths and forms
// the sums itself (a few KB out of L2, cheaper than sharing them), a cluster
// barrier lets the first write happen only after the last read, the pages and
// then (after a second barrier) the slots are dealt out over all threads.
// Latency-bound: three dependent rounds of loads between two barriers (32
// requests 5.5 us in a graph, 1024 with 128 new tokens each 13.3 us).
constexpr int kMapThreads = 1024;
constexpr int kMapMaxB = 4096;
constexpr int kMapCluster = 8;  // portable cluster size
constexpr int kMapBatch = 4;    // items a thread has in flight

struct MapArgs {
  int B, P, max_blocks, max_new, num_pages;
  const int32_t *prefix_len, *new_len;
  int32_t *n_blocks, *block_table, *free_list, *free_count;
  long long *slot_map;
  int32_t *dev_status;
};

// last index b with cum[b] <= x, for cum[0] = 0 <= ... <= cum[B], x < cum[B]
__device__ __forceinline__ int find_request(const int *cum, int B, int x) {
  int lo = 0, hi = B;  // cum[lo] <= x < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// inclusive sum over the block's threads; `sums` holds 32 entries
__device__ __forceinline__ int block_scan(int v, int *sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sums[w] = v;
  __syncthreads();
  int s = sums[lane];  // kMapThreads / 32 = 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  const int before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
  return v + (w > 0 ? before : 0);
}

__global__ void __launch_bounds__(kMapThreads) k_block_map(MapArgs a) {
  extern __shared__ int map_sm[];
  __shared__ int sums[32];
  int *cum_back = map_sm;                 // [B + 1] pages returned before request b
  int *cum_take = cum_back + a.B + 1;     // [B + 1] pages taken before request b
  int *s_need = cum_take + a.B + 1;       // [B] pages after this call
  int *s_have = s_need + a.B;             // [B] pages before, -1: the request is left alone
  int *s_new = s_have + a.B;              // [B] slots to write
  int *s_len = s_new + a.B;               // [B] tokens before them
  pdl_wait();     // the previous kernel in the stream has completed
  pdl_trigger();  // only now may the next kernel launch
  const int t = threadIdx.x, rank = blockIdx.x, blocks = gridDim.x;
  int bad = 0;
  int F = a.free_count[0];
  if (F < 0 || F > a.num_pages) {
    bad = ET_DEV_BAD_INDEX;
    F = F < 0 ? 0 : a.num_pages;
  }
  // ---- what each request returns and misses, and their sums ----
  int back0 = 0, miss0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += kMapThreads) {
    const int b = b0 + t;
    int back = 0, miss = 0;
    if (b < a.B) {
      const int len = a.prefix_len[b], add = a.new_len[b], have = a.n_blocks[b];
      int need = 0;
      bool ok = len >= 0;
      if (ok) {
        const long long want = ((long long)len + add + a.P - 1) / a.P;
        ok = add >= 0 && (a.max_new == 0 || add <= a.max_new) && have >= 0 && have <= a.max_blocks &&
             want <= a.max_blocks;
        if (!ok) bad |= ET_DEV_BAD_INDEX;
        else need = (int)want;
      }
      s_need[b] = need;
      s_have[b] = ok ? have : -1;
      s_new[b] = ok ? add : 0;
      s_len[b] = len;
      if (ok) {
        back = have > need ? have - need : 0;
        miss = need > have ? need - have : 0;
      }
    }
    const int ib = block_scan(back, sums) + back0, im = block_scan(miss, sums) + miss0;
    if (b < a.B) {
      cum_back[b + 1] = ib;
      cum_take[b + 1] = im;
    }
    __syncthreads();
    const int last = min(a.B, b0 + kMapThreads);
    back0 = cum_back[last];
    miss0 = cum_take[last];
  }
  if (t == 0) cum_back[0] = cum_take[0] = 0;
  __syncthreads();
  const int R = back0;
  const int top = F + R;  // height of the virtual stack (the host keeps num_pages + B * max_blocks below 2^31)
  // requests up to the first that does not fit are served: the sums only grow
  for (int b = t; b < a.B; b += kMapThreads) {
    const int before = cum_take[b], upto = cum_take[b + 1];
    if (upto > before && upto > top) {  // misses pages and does not fit
      bad |= ET_DEV_NO_PAGES;
      s_need[b] = s_have[b];
      s_new[b] = 0;
    }
  }
  __syncthreads();
  // pages taken: the sum of the last request that fits
  int A = miss0;
  if (A > top) {
    const int b = find_request(cum_take, a.B, top);  // cum_take[b] <= top < cum_take[b + 1]
    A = cum_take[b];
  }
  const int left = top - A;
  cl_sync();  // every block has read the lengths, block counts and the free count
  if (bad && rank == 0) flag_status(a.dev_status, bad);
  // ---- pages ----
  // (unsigned: R, A and the slots of a request lie below 2^31, one round past them does not)
  const uint32_t step = (uint32_t)blocks * kMapThreads, first = (uint32_t)(rank * kMapThreads + t);
  auto give = [&](int turn, int page) {  // the turn-th taken page
    const int b = find_request(cum_take, a.B, turn);
    a.block_table[(long long)b * a.max_blocks + s_have[b] + (turn - cum_take[b])] = page;
  };
  for (uint32_t r0 = first; r0 < (uint32_t)R; r0 += kMapBatch * step) {  // loads of a batch first: each is a trip to L2
    int32_t *cell[kMapBatch];
    int page[kMapBatch];
#pragma unroll
    for (int k = 0; k < kMapBatch; ++k) {
      const uint32_t r = r0 + k * step;
      if (r >= (uint32_t)R) continue;
      const int b = find_request(cum_back, a.B, (int)r);
      cell[k] = a.block_table + (long long)b * a.max_blocks + s_need[b] + ((int)r - cum_back[b]);
      page[k] = *cell[k];
    }
#pragma unroll
    for (int k = 0; k < kMapBatch; ++k) {
      if (r0 + k * step >= (uint32_t)R) continue;
      const int place = F + (int)(r0 + k * step);
      if ((unsigned)page[k] >= (unsigned)a.num_pages) bad = ET_DEV_BAD_INDEX;
      if (place >= left) give(top - 1 - place, page[k]);
      else if (place < a.num_pages) a.free_list[place] = page[k];
      *cell[k] = -1;
    }
  }
  for (uint32_t k0 = first; k0 < (uint32_t)A; k0 += kMapBatch * step) {
    int page[kMapBatch];
#pragma unroll
    for (int k = 0; k < kMapBatch; ++k) {
      const uint32_t turn = k0 + k * step;
      const int place = top - 1 - (int)turn;
      page[k] = turn < (uint32_t)A && place < F ? a.free_list[place] : 0;  // (a returned page: its own thread moves it)
    }
#pragma unroll
    for (int k = 0; k < kMapBatch; ++k) {
      const uint32_t turn = k0 + k * step;
      if (turn >= (uint32_t)A || top - 1 - (int)turn >= F) continue;
      if ((unsigned)page[k] >= (unsigned)a.num_pages) bad = ET_DEV_BAD_INDEX;
      give((int)turn, page[k]);
    }
  }
  for (int b = (int)first; b < a.B; b += (int)step)
    if (s_have[b] >= 0) a.n_blocks[b] = s_need[b];
  if (first == 0) {
    a.free_count[0] = min(left, a.num_pages);
    if (left > a.num_pages) bad = ET_DEV_BAD_INDEX;
  }
  if (bad & ET_DEV_BAD_INDEX) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
  if (a.max_new == 0) return;  // uniform over the cluster
  cl_sync();  // the tables are written
  // ---- slots: a warp per request ----
  const int lane = t & 31, warps = blocks * (kMapThreads / 32);
  for (int b = rank * (kMapThreads / 32) + (t >> 5); b < a.B; b += warps) {
    const int count = s_new[b], len = s_len[b];
    const int32_t *row = a.block_table + (long long)b * a.max_blocks;
#pragma unroll 4
    for (uint32_t i = lane; i < (uint32_t)a.max_new; i += 32) {
      long long slot = -1;
      if (i < (uint32_t)count) {
        const int pos = len + (int)i, blk = pos / a.P;  // need pages cover it: no overflow past max_blocks * P
        const int page = __ldcg(row + blk);
        if ((unsigned)page < (unsigned)a.num_pages) slot = (long long)page * a.P + (pos - blk * a.P);
        else flag_status(a.dev_status, ET_DEV_BAD_INDEX);
      }
      a.slot_map[(long long)b * a.max_new + i] = slot;
    }
  }
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
// A unit of threads has one (page that receives rows, head, K or V, sequence):
// it alone reads and writes that page's codes and scale, so nothing is shared
// and no order matters.  An accepted path brings at most 17 rows to a page:
// a warp is the unit, four to a block (32 sequences, 32 heads: 3.8 us in a
// graph, 6.4 with a block per unit).  A prompt fills whole pages: a block is
// the unit, and neighbouring blocks take the heads of one page.
// Either way the rows stay in registers between the search for the largest
// magnitude and the rounding, every load in flight at once; only a prompt's
// pages of more rows than that (64 of 128 dims) are read twice.  Bound by
// latency (one sequence 2.7 us in a graph).  A prompt is bound by HBM and the
// instructions of the conversion: 2 x 2047 rows of 32 heads 18.9 us in a
// graph, 5.3 TB/s; 26.4 us with magnitudes compared as fp32 and codes packed by shifts (20
// instructions an element, 11 now).  Extra blocks copy the feature rows.
constexpr int kCpThreads = 128;

struct CommitPagedArgs {
  int N, Hkv, P, path_len, max_blocks, max_rows;  // max_rows: rows a sequence may append
  long long num_pages, page_stride;
  uint8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  const int32_t *block_table;
  const void *k_tree, *v_tree;
  const int32_t *accept_len, *path, *prefix_len;
  int32_t *new_prefix_len;
  int chunks_f;  // 16-byte chunks per feature row
  const uint4 *features;
  uint4 *feat_out;
  int32_t *dev_status;
};

// eight elements as they lie in memory, and as fp32
template <bool BF16> struct Raw8 { uint4 v; };
template <> struct Raw8<false> { float4 u, v; };
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> raw8(const void *base, long long elem) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.v = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
    r.u = p[0];
    r.v = p[1];
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw8<BF16> &r, float (&x)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
    x[0] = r.u.x; x[1] = r.u.y; x[2] = r.u.z; x[3] = r.u.w;
    x[4] = r.v.x; x[5] = r.v.y; x[6] = r.v.z; x[7] = r.v.w;
  }
}

// magnitudes order like their bits, NaN and infinities above all: the running
// maximum of eight, one instruction for two bf16 values
template <bool BF16>
__device__ __forceinline__ void see8(const Raw8<BF16> &r, uint32_t &top) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(w[e] & 0x7fff7fffu));
  } else {
    float x[8];
    unpack8<BF16>(r, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  }
}

// U threads per unit: 32 (a path's rows) or kCpThreads (a prompt's)
template <bool BF16, int FMT, int D, int U>
__global__ void __launch_bounds__(kCpThreads) k_commit_paged(CommitPagedArgs a) {
  constexpr int CH = D / 8;               // 8-element chunks per row
  constexpr int RP = U / CH;              // rows per pass
  constexpr int UN = kCpThreads / U;      // units per block
  constexpr int KEEP = U == 32 ? (kMaxDepth + 1 + RP - 1) / RP : 8;  // passes whose rows stay in registers
  __shared__ float red[32];
  pdl_wait();     // the previous kernel in the stream has completed
  pdl_trigger();  // only now may the next kernel launch
  // a prompt's neighbouring blocks take the heads of one page, whose rows lie side by side
  const int tp = a.path ? blockIdx.x : blockIdx.x / (2 * a.Hkv), bu = a.path ? blockIdx.y : blockIdx.x - tp * (2 * a.Hkv);
  const int b = blockIdx.z, t = threadIdx.x % U;
  const int unit = bu * UN + threadIdx.x / U, unit_blocks = (2 * a.Hkv + UN - 1) / UN;
  const int alen = a.accept_len[b], base = a.prefix_len[b];
  const bool alen_ok = alen >= -1 && alen < a.max_rows;
  const int rows = (alen_ok && base >= 0) ? alen + 1 : 0;  // rows appended
  if (tp == 0 && unit == 0 && t == 0) {
    if (alen_ok) a.new_prefix_len[b] = base < 0 ? base : (int)min((long long)base + rows, 0x7fffffffll);
    else flag_status(a.dev_status, ET_DEV_BAD_INDEX);
  }
  if ((int)blockIdx.y >= unit_blocks) {  // ---- a feature row, by the whole block ----
    if (tp > 0) return;
    const int i = blockIdx.y - unit_blocks;
    const int row = i < rows ? a.path[(long long)b * a.path_len + i] : -1;
    const bool ok = row >= 0 && row < a.N;
    if (i < rows && !ok) return;  // flagged by the page's units; the row is skipped
    uint4 *dst = a.feat_out + ((long long)b * a.path_len + i) * a.chunks_f;
    const uint4 *src = a.features + ((long long)b * a.N + (ok ? row : 0)) * a.chunks_f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.chunks_f; c += kCpThreads) dst[c] = ok ? src[c] : make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  // ---- one page of one head ----
  const int g = unit >> 1;
  const bool isV = unit & 1;
  const long long blk = base / a.P + tp;  // meaningless unless rows > 0
  const long long start = blk * a.P;      // first token of the page
  const long long end = (long long)base + rows;
  if (unit >= 2 * a.Hkv || rows == 0 || start >= end) return;  // the same in the whole unit
  const int lo = start < base ? base - (int)start : 0;          // first row received
  const int hi = end - start < a.P ? (int)(end - start) : a.P;  // one past the last
  const long long page = blk < a.max_blocks ? a.block_table[(long long)b * a.max_blocks + blk] : -1;
  const int c = t % CH, r0 = t / CH;
  const int skip = (int)(start - base);  // path index of the page's row 0 (may be negative)
  const long long first = ((long long)b * a.N * a.Hkv + g) * D + c * 8;
  const int pitch = a.Hkv * D;
  auto source = [&](int r) -> long long {  // element index of the row that page row r receives, -1: none
    const int i = skip + r;
    const int row = U == 32 ? a.path[(long long)b * a.path_len + i] : i;
    return (unsigned)row < (unsigned)a.N ? first + (long long)row * pitch : -1;
  };
  const void *tree = isV ? a.v_tree : a.k_tree;
  Raw8<BF16> held[KEEP];
  bool have[KEEP];
  int bad = 0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int r = lo + r0 + k * RP;
    have[k] = false;
    if (r < hi) {
      const long long src = source(r);
      if (src < 0) bad |= ET_DEV_BAD_INDEX;
      else {
        have[k] = true;
        held[k] = raw8<BF16>(tree, src);
      }
    }
  }
  if (page < 0 || page >= a.num_pages) {
    if (t == 0) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
    return;
  }
  uint8_t *codes = (isV ? a.v_pages : a.k_pages) + page * a.page_stride + (long long)g * a.P * D;
  float *scale_at = (isV ? a.v_scale : a.k_scale) + page * a.Hkv + g;
  const float was = lo > 0 ? *scale_at : 0.f;
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < KEEP; ++k)
    if (have[k]) see8<BF16>(held[k], top);
#pragma unroll 1
  for (int r = lo + r0 + KEEP * RP; r < hi; r += RP) {  // (a prompt's large pages)
    const long long src = source(r);
    if (src < 0) bad |= ET_DEV_BAD_INDEX;
    else see8<BF16>(raw8<BF16>(tree, src), top);
  }
  if (BF16) top = max(top & 0xffff0000u, top << 16);
  if (top >= 0x7f800000u) {  // once more, without what is not finite
    bad |= ET_DEV_NONFINITE;
    top = 0u;
#pragma unroll 1
    for (int r = lo + r0; r < hi; r += RP) {
      const long long src = source(r);
      if (src < 0) continue;
      float x[8];
      unpack8<BF16>(raw8<BF16>(tree, src), x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(x[e]) <= FLT_MAX) top = max(top, __float_as_uint(fabsf(x[e])));
    }
  }
  float amax = __uint_as_float(top);
  if (U == 32) amax = warp_max(amax);
  else amax = block_max<kCpThreads>(amax, red);
  const float need = page_scale<FMT>(amax);
  const bool was_ok = was > 0.f && was <= FLT_MAX;
  if (lo > 0 && !was_ok) bad |= ET_DEV_NONFINITE;
  const float now = lo > 0 && was_ok ? fmaxf(was, need) : need;
  auto put = [&](int r, const Raw8<BF16> &v, auto scaled) {
    float x[8];
    unpack8<BF16>(v, x);
    *reinterpret_cast<uint2 *>(codes + (long long)r * D + c * 8) =
        make_uint2(f32x4_to_f8x4<FMT>(scaled(x[0]), scaled(x[1]), scaled(x[2]), scaled(x[3])),
                   f32x4_to_f8x4<FMT>(scaled(x[4]), scaled(x[5]), scaled(x[6]), scaled(x[7])));
  };
  if ((__float_as_uint(now) & 0x007fffffu) == 0u) {
    const float inv = 1.f / now;  // exact
    auto scaled = [&](float x) { return x * inv; };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (have[k]) put(lo + r0 + k * RP, held[k], scaled);
#pragma unroll 1
    for (int r = lo + r0 + KEEP * RP; r < hi; r += RP) {
      const long long src = source(r);
      if (src >= 0) put(r, raw8<BF16>(tree, src), scaled);
    }
  } else {  // a page whose scale is of another origin
#pragma unroll 1
    for (int r = lo + r0; r < hi; r += RP) {
      const long long src = source(r);
      if (src >= 0) put(r, raw8<BF16>(tree, src), [&](float x) { return __fdiv_rn(x, now); });
    }
  }
  if (lo > 0 && was_ok && now > was) {  // the rows before, on the grown scale
    const float ratio = __fdiv_rn(was, now);
    for (int r = r0; r < lo; r += RP) {
      uint2 *at = reinterpret_cast<uint2 *>(codes + (long long)r * D + c * 8);
      uint2 v = *at;
      float x[4];
      f8x4_to_f32<FMT>(v.x, x);
      v.x = f32x4_to_f8x4<FMT>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
      f8x4_to_f32<FMT>(v.y, x);
      v.y = f32x4_to_f8x4<FMT>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
      *at = v;
    }
  }
  if (t == 0) *scale_at = now;
  if (bad) flag_status(a.dev_status, bad);
}

template <bool BF16, int FMT>
et_status launch_commit(const CommitPagedArgs &a, int d, int touch, int feature_rows, int B, cudaStream_t st) {
  if (a.path) {  // a warp per unit
    const dim3 grid(touch, (2 * a.Hkv + kCpThreads / 32 - 1) / (kCpThreads / 32) + feature_rows, B);
    if (d == 64) return et_launch(k_commit_paged<BF16, FMT, 64, 32>, grid, dim3(kCpThreads), 0, st, 0, a);
    return et_launch(k_commit_paged<BF16, FMT, 128, 32>, grid, dim3(kCpThreads), 0, st, 0, a);
  }
  const dim3 grid(touch * 2 * a.Hkv, 1, B);
  if (d == 64) return et_launch(k_commit_paged<BF16, FMT, 64, kCpThreads>, grid, dim3(kCpThreads), 0, st, 0, a);
  return et_launch(k_commit_paged<BF16, FMT, 128, kCpThreads>, grid, dim3(kCpThreads), 0, st, 0, a);
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" et_status et_block_map(const et_block_map_shape *s, const int32_t *prefix_len, const int32_t *new_len,
                                  int32_t *n_blocks, int32_t *block_table, int32_t *free_list, int32_t *free_count,
                                  int64_t *slot_map, int32_t *dev_status, et_stream_t stream) {
  ET_RETURN_IF(!s, ET_ERR_INVALID_ARG);
  ET_RETURN_IF(s->B < 1 || s->page_size < 1 || s->max_blocks < 1 || s->max_new < 0 || s->num_pages < 1 ||
                   s->num_pages >= (1ll << 31),
               ET_ERR_INVALID_ARG);
  // positions and stack heights stay below 2^31
  ET_RETURN_IF(s->B > kMapMaxB || (long long)s->B * s->max_blocks + s->num_pages >= (1ll << 31) ||
                   (long long)s->max_blocks * s->page_size >= (1ll << 31),
               ET_ERR_UNSUPPORTED);
  ET_RETURN_IF(!prefix_len || !new_len || !n_blocks || !block_table || !free_list || !free_count, ET_ERR_INVALID_ARG);
  ET_RETURN_IF((s->max_new > 0) != (slot_map != nullptr), ET_ERR_INVALID_ARG);
  MapArgs a;
  a.B = s->B; a.P = s->page_size; a.max_blocks = s->max_blocks; a.max_new = s->max_new;
  a.num_pages = (int)s->num_pages;
  a.prefix_len = prefix_len; a.new_len = new_len;
  a.n_blocks = n_blocks; a.block_table = block_table; a.free_list = free_list; a.free_count = free_count;
  a.slot_map = reinterpret_cast<long long *>(slot_map);
  a.dev_status = dev_status;
  const int smem = (6 * s->B + 2) * (int)sizeof(int);
  const int largest = (6 * kMapMaxB + 2) * (int)sizeof(int);  // the attribute is set once, for every B
  ET_RETURN_IF(et_smem_attr((const void *)k_block_map, largest) != cudaSuccess, ET_ERR_CUDA);
  return et_launch(k_block_map, dim3(kMapCluster), dim3(kMapThreads), smem, (cudaStream_t)stream, kMapCluster, a);
}

extern "C" et_status et_kv_commit_paged(const et_paged_commit_shape *s, const et_paged_cache *cache,
                                        const int32_t *block_table, const void *k_tree, const void *v_tree,
                                        const int32_t *accept_len, const int32_t *path, const int32_t *prefix_len,
                                        int32_t *new_prefix_len, const void *features, void *feat_out,
                                        int32_t *dev_status, et_stream_t stream) {
  ET_RETURN_IF(!s, ET_ERR_INVALID_ARG);
  const et_status cs = paged_cache_status(cache);
  ET_RETURN_IF(cs != ET_OK, cs);
  ET_RETURN_IF(s->dtype != ET_BF16 && s->dtype != ET_F32, ET_ERR_INVALID_ARG);
  const int es = s->dtype == ET_BF16 ? 2 : 4;
  ET_RETURN_IF(s->B < 1 || s->B > 65535 || s->N < 1 || s->path_len < 0 || s->path_len > kMaxDepth + 1 ||
                   s->max_blocks < 1 || s->feat_dim < 0,
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF((path != nullptr) != (s->path_len > 0) || (!path && s->feat_dim > 0), ET_ERR_INVALID_ARG);
  ET_RETURN_IF(((long long)s->feat_dim * es) % 16 != 0, ET_ERR_UNSUPPORTED);
  ET_RETURN_IF(2 * cache->Hkv + s->path_len > 65535 || (long long)s->max_blocks * cache->page_size >= (1ll << 31),
               ET_ERR_UNSUPPORTED);
  ET_RETURN_IF(!block_table || !k_tree || !v_tree || !accept_len || !prefix_len || !new_prefix_len,
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(new_prefix_len == prefix_len, ET_ERR_INVALID_ARG);  // blocks of a sequence read prefix_len
  ET_RETURN_IF(s->feat_dim > 0 && (!features || !feat_out), ET_ERR_INVALID_ARG);
  ET_RETURN_IF(!et_aligned(k_tree, 16) || !et_aligned(v_tree, 16) || (features && !et_aligned(features, 16)) ||
                   (feat_out && !et_aligned(feat_out, 16)),
               ET_ERR_INVALID_ARG);
  CommitPagedArgs a;
  a.N = s->N; a.Hkv = cache->Hkv; a.P = cache->page_size; a.path_len = s->path_len; a.max_blocks = s->max_blocks;
  a.max_rows = path ? s->path_len : s->N;
  a.num_pages = cache->num_pages; a.page_stride = cache->page_stride;
  a.k_pages = static_cast<uint8_t *>(cache->k_pages); a.v_pages = static_cast<uint8_t *>(cache->v_pages);
  a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
  a.block_table = block_table; a.k_tree = k_tree; a.v_tree = v_tree;
  a.accept_len = accept_len; a.path = path; a.prefix_len = prefix_len; a.new_prefix_len = new_prefix_len;
  a.chunks_f = (int)((long long)s->feat_dim * es / 16);
  a.features = s->feat_dim > 0 ? static_cast<const uint4 *>(features) : nullptr;
  a.feat_out = s->feat_dim > 0 ? static_cast<uint4 *>(feat_out) : nullptr;
  a.dev_status = dev_status;
  const int touch = (int)(((long long)a.max_rows + 2ll * a.P - 2) / a.P);  // pages max_rows rows can lie in
  ET_RETURN_IF((long long)touch * 2 * cache->Hkv >= (1ll << 31), ET_ERR_UNSUPPORTED);
  const int feature_rows = s->feat_dim > 0 ? s->path_len : 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (s->dtype == ET_BF16)
    return cache->format == ET_KV_E4M3 ? launch_commit<true, ET_KV_E4M3>(a, cache->d, touch, feature_rows, s->B, st)
                                       : launch_commit<true, ET_KV_E5M2>(a, cache->d, touch, feature_rows, s->B, st);
  return cache->format == ET_KV_E4M3 ? launch_commit<false, ET_KV_E4M3>(a, cache->d, touch, feature_rows, s->B, st)
                                     : launch_commit<false, ET_KV_E5M2>(a, cache->d, touch, feature_rows, s->B, st);
}
