// Tree-masked attention over a paged 8-bit KV cache (EAGLE-2 article,
// attention-mask paragraph: every flattened draft row attends the prefix and
// its own ancestors; EAGLE blog section 1.1: one target pass verifies the
// draft).  N = 1 is plain decoding.
//
// A cached value is code * scale with one scale per (page, head).  The K
// scale multiplies a page's scores.  The V scale is carried in the exponent:
// with t_j = s_j + log2(vs_j) (scores in log2 units) and m >= max t_j,
//   out = (sum 2^(t_j - m) code_j) / (sum 2^(t_j - m) / vs_j),
// so the weights meet the raw codes, no weight overflows whatever the scales
// (the running maximum is taken over t), and the two sums hold the plain
// softmax's numerator and denominator.
#include <cuda_bf16.h>

#include "et_paged.cuh"

namespace et {
namespace {

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

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

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
__device__ __forceinline__ float clamp_v_scale(float s) {
  return fminf(fmaxf(s, 1.f / (1ll << kScaleExp)), (float)(1ll << kScaleExp));  // NaN -> the smallest
}
__device__ __forceinline__ bool tree_keeps(const PagedAttnArgs &a, int b, int i, int tt) {
  if (!a.mask) return tt <= i;
  return (a.mask[((long long)b * a.N + i) * a.W + (tt >> 6)] >> (tt & 63)) & 1ull;
}

// ---------------------------------------------------------------------------
// CUDA cores: one block per (row, head, sequence), fp32 throughout
// ---------------------------------------------------------------------------
// Each warp takes every fourth group of 32 keys: a lane scores one key (its
// whole row, 16 bytes a load), the group's maximum and sum are warp
// reductions, then the lanes turn to the head's dims and add the 32 weighted
// V rows, whose loads do not depend on one another.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(128) k_paged_attn_row(PagedAttnArgs a) {
  constexpr int PL = D / 32;  // dims per lane
  __shared__ float qs[D];
  __shared__ float wm[4], wl[4];
  __shared__ float wacc[4][D];
  pdl_wait();     // the previous kernel in the stream has completed
  pdl_trigger();  // only now may the next kernel launch
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int g = h / a.G, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int bad = 0;
  const int L = paged_prefix(a, b, bad);
  if (L < 0) return;
  const long long orow = ((long long)b * a.N + i) * a.Hq + h;
  for (int c = t; c < D; c += 128) qs[c] = to_f32(static_cast<const T *>(a.q)[orow * D + c]);
  __syncthreads();
  const T *KT = static_cast<const T *>(a.kt), *VT = static_cast<const T *>(a.vt);
  float m = -INFINITY, l = 0.f, acc[PL];
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = 0.f;
  const int nP = (L + 31) / 32, nT = (a.N + 31) / 32;
  for (int grp = warp; grp < nP + nT; grp += 4) {
    const bool cached = grp < nP;
    const int j = cached ? grp * 32 + lane : (grp - nP) * 32 + lane;
    bool ok = cached ? j < L : (j < a.N && tree_keeps(a, b, i, j));
    long long at = 0;  // byte offset of the key's codes, or element offset of its tree row
    float ks = 1.f, vs = 1.f;
    if (ok && cached) {
      const int blk = j / a.P;
      const long long page = a.block_table[(long long)b * a.max_blocks + blk];
      if (page < 0 || page >= a.num_pages) {
        ok = false;
        bad = 1;
      } else {
        at = page * a.page_stride + ((long long)g * a.P + (j - blk * a.P)) * D;
        ks = a.k_scale[page * a.Hkv + g];
        vs = clamp_v_scale(a.v_scale[page * a.Hkv + g]);
      }
    } else if (ok) {
      at = (((long long)b * a.N + j) * a.Hkv + g) * D;
    }
    float s = 0.f;
    if (ok && cached) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a.k_pages + at + 16 * c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[4];
          f8x4_to_f32<FMT>(w[e], x);
#pragma unroll
          for (int u = 0; u < 4; ++u) s = fmaf(qs[16 * c + 4 * e + u], x[u], s);
        }
      }
      s *= ks;
    } else if (ok) {
#pragma unroll 8
      for (int c = 0; c < D; ++c) s = fmaf(qs[c], to_f32(KT[at + c]), s);
    }
    s = ok ? s * a.scale_log2 : -INFINITY;
    const unsigned int keep = __ballot_sync(0xffffffffu, ok);
    if (keep == 0u) continue;  // no key for this row in this group
    float mn = fmaxf(m, warp_max(s));
    if (mn == -INFINITY) mn = 0.f;  // only NaN or -inf scores so far: the weights below become NaN or 0
    const float corr = exp2f(m - mn), p = ok ? exp2f(s - mn) : 0.f;
    l = l * corr + warp_sum(p);
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] *= corr;
    m = mn;
    const float pv = p * vs;
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      const float w = __shfl_sync(0xffffffffu, pv, k);
      const long long row = __shfl_sync(0xffffffffu, at, k);
      if (!((keep >> k) & 1u)) continue;
      float x[PL];
      if (cached) {
        if (PL == 4) {
          float y[4];
          f8x4_to_f32<FMT>(*reinterpret_cast<const uint32_t *>(a.v_pages + row + 4 * lane), y);
#pragma unroll
          for (int c = 0; c < PL; ++c) x[c] = y[c];
        } else {
          const uint32_t hv = f8x2_to_f16x2<FMT>(*reinterpret_cast<const uint16_t *>(a.v_pages + row + 2 * lane));
          const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hv));
          x[0] = y.x;
          x[1] = y.y;
        }
      } else {
#pragma unroll
        for (int c = 0; c < PL; ++c) x[c] = to_f32(VT[row + PL * lane + c]);
      }
#pragma unroll
      for (int c = 0; c < PL; ++c) acc[c] = fmaf(w, x[c], acc[c]);
    }
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < PL; ++c) wacc[warp][PL * lane + c] = acc[c];
  __syncthreads();
  float M = wm[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) M = fmaxf(M, wm[w]);
  float Ls = 0.f, wts[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    wts[w] = wm[w] == -INFINITY ? 0.f : exp2f(wm[w] - M);
    Ls += wl[w] * wts[w];
  }
  for (int c = t; c < D; c += 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += wacc[w][c] * wts[w];
    static_cast<T *>(a.out)[orow * D + c] = from_f32<T>(Ls == 0.f ? 0.f : v / Ls);
  }
  if (t == 0 && a.lse)
    a.lse[((long long)b * a.Hq + h) * a.N + i] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * 0.69314718055994531f;
  if (bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
}

template <typename T, int FMT>
et_status launch_row(const PagedAttnArgs &a, int d, cudaStream_t st) {
  const dim3 grid(a.N, a.Hq, a.B);
  if (d == 64) return et_launch(k_paged_attn_row<T, FMT, 64>, grid, dim3(128), 0, st, 0, a);
  return et_launch(k_paged_attn_row<T, FMT, 128>, grid, dim3(128), 0, st, 0, a);
}

struct PagedPlan {
  int S;      // blocks a sequence's keys are split over
  size_t ws;  // workspace bytes
};

et_status make_plan(const et_paged_attn_shape *s, const et_paged_cache *c, PagedPlan *p) {
  if (!s) return ET_ERR_INVALID_ARG;
  const et_status cs = paged_cache_status(c);
  if (cs != ET_OK) return cs;
  if (s->B < 1 || s->N < 1 || s->N > kMaxN || s->Hq < 1 || s->Hq % c->Hkv || s->max_blocks < 1 || s->max_prefix < 0 ||
      s->num_splits < 0 || !(s->scale > 0.f) || (s->dtype != ET_BF16 && s->dtype != ET_F32))
    return ET_ERR_INVALID_ARG;
  if (s->B > 65535 || s->Hq > 65535 || (long long)s->max_blocks * c->page_size >= (1ll << 31)) return ET_ERR_UNSUPPORTED;
  p->S = 1;
  p->ws = 0;
  return ET_OK;
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" size_t et_tree_attention_paged_workspace_size(const et_paged_attn_shape *shape,
                                                         const et_paged_cache *cache) {
  PagedPlan p;
  return make_plan(shape, cache, &p) == ET_OK ? p.ws : 0;
}

extern "C" int32_t et_tree_attention_paged_splits(const et_paged_attn_shape *shape, const et_paged_cache *cache) {
  PagedPlan p;
  return make_plan(shape, cache, &p) == ET_OK ? p.S : -1;
}

extern "C" et_status et_tree_attention_paged(const et_paged_attn_shape *shape, const et_paged_cache *cache,
                                             const int32_t *block_table, const int32_t *prefix_len, const void *q,
                                             const void *k_tree, const void *v_tree, const uint64_t *mask, void *out,
                                             float *lse, int32_t *dev_status, void *ws, size_t ws_bytes,
                                             et_stream_t stream) {
  PagedPlan plan;
  const et_status ps = make_plan(shape, cache, &plan);
  ET_RETURN_IF(ps != ET_OK, ps);
  ET_RETURN_IF(!block_table || !prefix_len || !q || !k_tree || !v_tree || !out, ET_ERR_INVALID_ARG);
  ET_RETURN_IF(!et_aligned(q, 16) || !et_aligned(k_tree, 16) || !et_aligned(v_tree, 16) || !et_aligned(out, 16) ||
                   !et_aligned(mask, 8),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(plan.ws > 0 && (!ws || ws_bytes < plan.ws || !et_aligned(ws, 256)), ET_ERR_WORKSPACE);
  PagedAttnArgs a;
  a.B = shape->B; a.N = shape->N; a.Hq = shape->Hq; a.Hkv = cache->Hkv; a.G = shape->Hq / cache->Hkv;
  a.P = cache->page_size; a.max_blocks = shape->max_blocks; a.W = (shape->N + 63) / 64;
  a.max_prefix = shape->max_prefix;
  a.scale_log2 = shape->scale * 1.4426950408889634f;
  a.num_pages = cache->num_pages; a.page_stride = cache->page_stride;
  a.k_pages = static_cast<const uint8_t *>(cache->k_pages); a.v_pages = static_cast<const uint8_t *>(cache->v_pages);
  a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
  a.block_table = block_table; a.prefix_len = prefix_len;
  a.q = q; a.kt = k_tree; a.vt = v_tree;
  a.mask = reinterpret_cast<const unsigned long long *>(mask);
  a.out = out; a.lse = lse; a.dev_status = dev_status;
  cudaStream_t st = (cudaStream_t)stream;
  const bool e4m3 = cache->format == ET_KV_E4M3;
  if (shape->dtype == ET_F32)
    return e4m3 ? launch_row<float, ET_KV_E4M3>(a, cache->d, st) : launch_row<float, ET_KV_E5M2>(a, cache->d, st);
  return e4m3 ? launch_row<__nv_bfloat16, ET_KV_E4M3>(a, cache->d, st)
              : launch_row<__nv_bfloat16, ET_KV_E5M2>(a, cache->d, st);
}
