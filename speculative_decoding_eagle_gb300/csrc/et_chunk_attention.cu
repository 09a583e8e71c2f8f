// Attention of new rows over a paged 8-bit prefix and over themselves (EAGLE
// blog 1.1: the target's own forward over a prompt, before the first draft):
// the entry point, and the kernel on fp32 units that takes fp32 inputs.
//
// k_chunk_rows: one block per 32 (token, head) rows of a KV head; online
// softmax over tiles of 32 keys in fp32.  Scores: a thread has two rows and
// two keys of the tile; output: two rows and D / 16 dims.  Bound by shared
// memory reads and the fp32 units, in small calls by latency (17.5 us: two
// sequences of up to 40 rows after 128 cached, 4 heads of 64); fp32 inputs are
// for checks and small models.
#include "et_chunk_attn.cuh"

namespace et {
namespace {

constexpr int kCrThreads = 256, kCrRows = 32, kCrKeys = 32;
// Tiles whose weights and outputs are summed up by themselves before they join the row's: one sum over all keys loses every
// key whose part of it is below 2^-25 (2^18 keys 2^-26 below one: the output off by 0.4%).  Over n keys a value goes through
// 512 sums and n / 512
constexpr int kCrGroup = 16;

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int D, int FMT>
__global__ void __launch_bounds__(kCrThreads) k_chunk_rows(const ChunkArgs c) {
  const PagedAttnArgs &a = c.a;
  constexpr int LD = D + 4;  // rows end four words further each: conflict-free reads of a column of rows
  extern __shared__ __align__(16) float s_rows[];
  float *Q = s_rows, *K = Q + kCrRows * LD, *V = K + kCrKeys * LD, *O = V + kCrKeys * D, *P = O + kCrRows * D;  // P [rows][33]
  const int t = threadIdx.x, ty = t >> 4, tx = t & 15;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, g = blockIdx.y;
  int bad = 0, first, n;
  const int L = paged_prefix(a, b, bad);
  chunk_rows(c, b, first, n, bad);
  int behind = 0;  // some sequence before starts behind this one's first row: a thread looks at a few
#pragma unroll 8
  for (int k = t; k < b; k += kCrThreads) behind |= chunk_start(c, c.row_start[k]) > first;
  if (__syncthreads_or(behind)) n = 0;
  if (bad && t == 0 && blockIdx.x == 0) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
  const long long R0 = (long long)blockIdx.x * kCrRows;  // row of the KV head: token * G + head of the group
  if (L < 0 || R0 >= (long long)n * a.G) return;
  const int real = (int)min((long long)kCrRows, (long long)n * a.G - R0);
  const int last_token = (int)((R0 + real - 1) / a.G);
  for (int x = t; x < kCrRows * (D / 4); x += kCrThreads) {
    const int r = x / (D / 4), e = x % (D / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < real) {
      const long long i = (R0 + r) / a.G;
      const int h = g * a.G + (int)(R0 + r - i * a.G);
      v = load4(static_cast<const float *>(a.q) + (first + i) * c.qs + (long long)h * D + e);
    }
    *reinterpret_cast<float4 *>(Q + r * LD + e) = v;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4 o[2][D / 64];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < D / 64; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M[2] = {-INFINITY, -INFINITY}, A[2] = {0.f, 0.f};  // the same of the groups of tiles before
  float4 *sums[2] = {reinterpret_cast<float4 *>(O + ty * D) + tx, reinterpret_cast<float4 *>(O + (ty + 16) * D) + tx};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < D / 64; ++j) sums[i][16 * j] = make_float4(0.f, 0.f, 0.f, 0.f);
  // own keys that a row may see: 0 .. its token
  const int tok[2] = {(int)((R0 + ty) / a.G), (int)((R0 + ty + 16) / a.G)};
  const int prefix_tiles = (int)(((long long)L + kCrKeys - 1) / kCrKeys), own_tiles = last_token / kCrKeys + 1;
  int page_bad = 0;
  // a tile's rows, four dims of a row a cell: the next tile's are on their way while this one's scores are found
  constexpr int CELLS = kCrKeys * (D / 4) / kCrThreads;
  float4 next_k[CELLS], next_v[CELLS];
  auto fetch = [&](int j) {
    const bool mine = j >= prefix_tiles;
    const int key0 = (mine ? j - prefix_tiles : j) * kCrKeys;
#pragma unroll
    for (int z = 0; z < CELLS; ++z) {
      const int x = t + z * kCrThreads, r = x / (D / 4), e = x % (D / 4) * 4, key = key0 + r;
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      if (mine) {
        if (key <= last_token) {
          const long long row = first + key;
          kv = load4(static_cast<const float *>(a.kt) + row * c.ks + (long long)g * D + e);
          vv = load4(static_cast<const float *>(a.vt) + row * c.vs + (long long)g * D + e);
        }
      } else if (key < L) {
        const int blk = key / a.P, page = a.block_table[(long long)b * a.max_blocks + blk];
        if (page >= 0 && page < a.num_pages) {
          const long long at = (long long)page * a.page_stride + ((long long)g * a.P + (key - blk * a.P)) * D + e;
          const float ks = a.k_scale[(long long)page * a.Hkv + g], vs = clamp_v_scale(a.v_scale[(long long)page * a.Hkv + g]);
          float f[4];
          f8x4_to_f32<FMT>(*reinterpret_cast<const uint32_t *>(a.k_pages + at), f);
          kv = make_float4(f[0] * ks, f[1] * ks, f[2] * ks, f[3] * ks);
          f8x4_to_f32<FMT>(*reinterpret_cast<const uint32_t *>(a.v_pages + at), f);
          vv = make_float4(f[0] * vs, f[1] * vs, f[2] * vs, f[3] * vs);
        } else {
          page_bad = 1;
          kv.x = __uint_as_float(0x7fc00001u);  // marks a key that is not there
        }
      }
      next_k[z] = kv;
      next_v[z] = vv;
    }
  };
  fetch(0);
  for (int j = 0; j < prefix_tiles + own_tiles; ++j) {
    const bool mine = j >= prefix_tiles;
    const int key0 = (mine ? j - prefix_tiles : j) * kCrKeys;
    __syncthreads();
#pragma unroll
    for (int z = 0; z < CELLS; ++z) {
      const int x = t + z * kCrThreads, r = x / (D / 4), e = x % (D / 4) * 4;
      *reinterpret_cast<float4 *>(K + r * LD + e) = next_k[z];
      *reinterpret_cast<float4 *>(V + r * D + e) = next_v[z];
    }
    __syncthreads();
    if (j + 1 < prefix_tiles + own_tiles) fetch(j + 1);
    // ---- scores of rows ty, ty + 16 and keys tx, tx + 16 ----
    float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 8
    for (int e = 0; e < D; e += 4) {
      const float4 q0 = *reinterpret_cast<const float4 *>(Q + ty * LD + e);
      const float4 q1 = *reinterpret_cast<const float4 *>(Q + (ty + 16) * LD + e);
      const float4 k0 = *reinterpret_cast<const float4 *>(K + tx * LD + e);
      const float4 k1 = *reinterpret_cast<const float4 *>(K + (tx + 16) * LD + e);
      s[0][0] = fmaf(q0.x, k0.x, fmaf(q0.y, k0.y, fmaf(q0.z, k0.z, fmaf(q0.w, k0.w, s[0][0]))));
      s[0][1] = fmaf(q0.x, k1.x, fmaf(q0.y, k1.y, fmaf(q0.z, k1.z, fmaf(q0.w, k1.w, s[0][1]))));
      s[1][0] = fmaf(q1.x, k0.x, fmaf(q1.y, k0.y, fmaf(q1.z, k0.z, fmaf(q1.w, k0.w, s[1][0]))));
      s[1][1] = fmaf(q1.x, k1.x, fmaf(q1.y, k1.y, fmaf(q1.z, k1.z, fmaf(q1.w, k1.w, s[1][1]))));
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int key = key0 + tx + 16 * kk;
      const bool gone = !mine && (key >= L || __float_as_uint(K[(tx + 16 * kk) * LD]) == 0x7fc00001u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i][kk] *= a.scale_log2;
        if (gone || (mine && key > tok[i])) s[i][kk] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = fmaxf(s[i][0], s[i][1]);
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float now = fmaxf(m[i], top), ref = now == -INFINITY ? 0.f : now;
      const float old = exp2f(m[i] - ref);
      const float p0 = exp2f(s[i][0] - ref), p1 = exp2f(s[i][1] - ref);
      float sum = p0 + p1;
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = fmaf(l[i], old, sum);
      m[i] = now;
#pragma unroll
      for (int jj = 0; jj < D / 64; ++jj) {
        o[i][jj].x *= old; o[i][jj].y *= old; o[i][jj].z *= old; o[i][jj].w *= old;
      }
      P[(ty + 16 * i) * 33 + tx] = p0;
      P[(ty + 16 * i) * 33 + tx + 16] = p1;
    }
    __syncwarp();  // a row's 32 weights come from its own half warp
    // ---- output: rows ty, ty + 16, dims 4 tx + 64 jj ----
#pragma unroll 8
    for (int kk = 0; kk < kCrKeys; ++kk) {
      const float p0 = P[ty * 33 + kk], p1 = P[(ty + 16) * 33 + kk];
      const int key = key0 + kk;
      // a key that a row does not see stays out of it, whatever its value is
      const bool see0 = !mine || key <= tok[0], see1 = !mine || key <= tok[1];
#pragma unroll
      for (int jj = 0; jj < D / 64; ++jj) {
        const float4 v = *reinterpret_cast<const float4 *>(V + kk * D + 4 * tx + 64 * jj);
        if (see0) {
          o[0][jj].x = fmaf(p0, v.x, o[0][jj].x); o[0][jj].y = fmaf(p0, v.y, o[0][jj].y);
          o[0][jj].z = fmaf(p0, v.z, o[0][jj].z); o[0][jj].w = fmaf(p0, v.w, o[0][jj].w);
        }
        if (see1) {
          o[1][jj].x = fmaf(p1, v.x, o[1][jj].x); o[1][jj].y = fmaf(p1, v.y, o[1][jj].y);
          o[1][jj].z = fmaf(p1, v.z, o[1][jj].z); o[1][jj].w = fmaf(p1, v.w, o[1][jj].w);
        }
      }
    }
    if (j % kCrGroup == kCrGroup - 1 || j + 1 == prefix_tiles + own_tiles) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float by = exp2f(M[i] - (m[i] == -INFINITY ? 0.f : m[i]));
        A[i] = fmaf(A[i], by, l[i]);
        M[i] = m[i];
        l[i] = 0.f;
#pragma unroll
        for (int jj = 0; jj < D / 64; ++jj) {
          float4 v = sums[i][16 * jj];
          v.x = fmaf(v.x, by, o[i][jj].x); v.y = fmaf(v.y, by, o[i][jj].y);
          v.z = fmaf(v.z, by, o[i][jj].z); v.w = fmaf(v.w, by, o[i][jj].w);
          sums[i][16 * jj] = v;
          o[i][jj] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
  }
  if (page_bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = ty + 16 * i;
    if (r >= real) continue;
    const int h = g * a.G + (int)(R0 + r - (long long)tok[i] * a.G);
    const long long row = ((long long)first + tok[i]) * a.Hq + h;
    const float inv = A[i] == 0.f ? 0.f : 1.f / A[i];
#pragma unroll
    for (int jj = 0; jj < D / 64; ++jj) {
      float4 v = sums[i][16 * jj];
      v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
      *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * D + 4 * tx + 64 * jj) = v;
    }
    if (a.lse && tx == 0) a.lse[row] = A[i] == 0.f ? -INFINITY : (M[i] + log2f(A[i])) * 0.69314718055994531f;
  }
}

template <int D, int FMT>
et_status launch_rows(const ChunkArgs &c, cudaStream_t st) {
  constexpr int LD = D + 4;
  constexpr int bytes = (kCrRows * LD + kCrKeys * LD + kCrKeys * D + kCrRows * D + kCrRows * 33) * 4;
  if (et_smem_attr((const void *)k_chunk_rows<D, FMT>, bytes) != cudaSuccess) return ET_ERR_CUDA;
  const long long tiles = ((long long)c.a.N * c.a.G + kCrRows - 1) / kCrRows;
  return et_launch(k_chunk_rows<D, FMT>, dim3((unsigned)tiles, c.a.Hkv, c.a.B), dim3(kCrThreads), bytes, st, 0, c);
}
et_status launch_rows(const ChunkArgs &c, int d, int format, cudaStream_t st) {
  if (d == 64)
    return format == ET_KV_E4M3 ? launch_rows<64, ET_KV_E4M3>(c, st) : launch_rows<64, ET_KV_E5M2>(c, st);
  return format == ET_KV_E4M3 ? launch_rows<128, ET_KV_E4M3>(c, st) : launch_rows<128, ET_KV_E5M2>(c, st);
}

struct ChunkPlan {
  ChunkTcPlan tc;
  size_t ws;
};

constexpr int kChunkCounters = 16384;  // in one place of every workspace, so that calls of other shapes can share it

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 152;
  cudaGetLastError();
  return n;
}

et_status make_plan(const et_chunk_attn_shape *s, const et_paged_cache *c, ChunkPlan *p) {
  if (!s) return ET_ERR_INVALID_ARG;
  const et_status cs = paged_cache_status(c);
  if (cs != ET_OK) return cs;
  if (s->B < 1 || s->rows < 1 || s->max_rows < 1 || s->Hq < 1 || s->Hq % c->Hkv ||
      s->max_blocks < 1 || s->max_prefix < 0 || s->num_splits < 0 || !(s->scale > 0.f) || !(s->scale <= FLT_MAX) ||
      (s->dtype != ET_BF16 && s->dtype != ET_F32))
    return ET_ERR_INVALID_ARG;
  const int es = s->dtype == ET_BF16 ? 2 : 4;
  const long long sizes[3] = {s->Hq, c->Hkv, c->Hkv}, strides[3] = {s->q_stride, s->k_stride, s->v_stride};
  for (int i = 0; i < 3; ++i)
    if (strides[i] < sizes[i] * c->d || strides[i] * es % 16 || strides[i] >= (1ll << 38)) return ET_ERR_INVALID_ARG;
  if (s->B > 65535 || s->Hq > 65535 || (long long)s->max_blocks * c->page_size >= (1ll << 31) ||
      (long long)s->rows * (s->Hq / c->Hkv) >= (1ll << 31))
    return ET_ERR_UNSUPPORTED;
  p->tc.S = 1;
  p->tc.shift = 8;
  p->tc.tiles = p->tc.whole = 0;
  p->tc.ml_off = p->tc.o_off = p->ws = 0;
  if (s->dtype == ET_F32) return ET_OK;
  const long long room = (long long)s->max_blocks * c->page_size;
  const int most = s->max_rows < s->rows ? s->max_rows : s->rows;
  const long long Tp = ((s->max_prefix < room ? s->max_prefix : room) + 127) / 128, T = Tp + (most + 127) / 128;
  const long long G = s->Hq / c->Hkv, rows = (long long)s->rows * G, seqs = s->B < s->rows ? s->B : s->rows;
  // every sequence's rows end in a unit of their own, if they have any
  auto units_of = [&](int shift) { return ((rows + seqs * ((1 << shift) - 1)) >> shift) * c->Hkv; };
  if (units_of(8) >= (1ll << 24)) return ET_ERR_UNSUPPORTED;
  int shift = 8;
  long long S = s->num_splits, whole = 0;
  if (S <= 0) {
    // One block per SM.  In units of 0.88 us, measured: a tile takes 1.2 where both groups have the same rows (1.0 to 1.4, by
    // how many SMs are at it) and 1.9 for 256 rows, a block's start and end 14, a merge through the workspace 1, 0.04 a row
    // and 1 a part.  So parts pay
    //   where blocks are few and tiles many: 64 rows, 32 heads, in 1 / 2 / 3 / 4 parts: 4096 keys 39.7 / 29.2 / 26.9 / 25.5 us,
    //   but 1024 keys 18.3 / 18.4 / 18.9 / 18.6;
    //   where a last round of whole units would leave SMs idle: 512 units of 65 to 80 tiles, the last 56 in two parts 469 us,
    //   whole 516 (that round has the units with the fewest keys, little more than the prefix; of more than 32 sequences it may
    //   have others, and the price is low).
    // Units of 128 rows pay where those of 256 leave half of the SMs idle: 512 rows, 32 heads, 4096 keys 45.5 us,
    // against 53.5 in parts and 70.6 whole
    const long long sms = sm_count(), least = Tp + 1 < T ? Tp + 1 : T;
    double best = 0.0;
    for (int u = 8; u >= 7; --u) {
      if (u == 7 && (most * G <= 128 || units_of(7) >= (1ll << 24))) break;  // the same units, or too many
      const long long units = units_of(u), rounds = units / sms, rest = units % sms;
      const double tile = u == 8 && most * G > 128 ? 1.9 : 1.2;
      const double merge = 1 + 0.04 * (double)(most * G < (1 << u) ? most * G : 1 << u);
      auto block = [&](long long tiles, long long parts) {
        return 14 + tile * (double)((tiles + parts - 1) / parts) + (parts > 1 ? merge + (double)parts : 0.0);
      };
      const double plain = (double)((units + sms - 1) / sms) * block(T, 1);
      double cost = plain;
      long long parts = 1, first = 0;
      for (long long k = 2; k <= 64 && k <= T; ++k) {
        const double all = (double)((units * k + sms - 1) / sms) * block(T, k);
        if (all < cost && all < 0.95 * plain) {
          cost = all;
          parts = k;
          first = 0;
        }
        if (!rounds || !rest) continue;
        const double last = plain - block(least, 1) + (double)((rest * k + sms - 1) / sms) * block(least, k);
        if (last < cost && last < 0.95 * plain) {
          cost = last;
          parts = k;
          first = rounds * sms;
        }
      }
      if (u == 8 || cost < 0.95 * best) {
        best = cost;
        shift = u;
        S = parts;
        whole = first;
      }
    }
  }
  const long long units = units_of(shift);
  if (S > T) S = T;
  if (S > 64) S = 64;
  if (S < 1 || units - whole > kChunkCounters) S = 1;
  p->tc.S = (int)S;
  p->tc.shift = shift;
  p->tc.tiles = (int)(units / c->Hkv);
  p->tc.whole = S > 1 ? (int)whole : 0;
  if (S > 1) {
    const size_t slots = (size_t)(units - whole) * S << shift;
    p->tc.ml_off = kChunkCounters * sizeof(unsigned int);
    p->tc.o_off = p->tc.ml_off + slots * sizeof(float2);
    p->ws = p->tc.o_off + slots * c->d * sizeof(float);
  }
  return ET_OK;
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" size_t et_chunk_attention_paged_workspace_size(const et_chunk_attn_shape *shape, const et_paged_cache *cache) {
  ChunkPlan p;
  return make_plan(shape, cache, &p) == ET_OK ? p.ws : 0;
}

extern "C" int32_t et_chunk_attention_paged_splits(const et_chunk_attn_shape *shape, const et_paged_cache *cache) {
  ChunkPlan p;
  return make_plan(shape, cache, &p) == ET_OK ? p.tc.S : -1;
}

extern "C" et_status et_chunk_attention_paged(const et_chunk_attn_shape *shape, const et_paged_cache *cache,
                                              const int32_t *block_table, const int32_t *prefix_len,
                                              const int32_t *row_start, const void *q, const void *k_new,
                                              const void *v_new, void *out, float *lse, int32_t *dev_status, void *ws,
                                              size_t ws_bytes, et_stream_t stream) {
  ChunkPlan plan;
  const et_status ps = make_plan(shape, cache, &plan);
  ET_RETURN_IF(ps != ET_OK, ps);
  ET_RETURN_IF(!block_table || !prefix_len || !row_start || !q || !k_new || !v_new || !out, ET_ERR_INVALID_ARG);
  ET_RETURN_IF(!et_aligned(q, 16) || !et_aligned(k_new, 16) || !et_aligned(v_new, 16) || !et_aligned(out, 16) ||
                   !et_aligned(block_table, 4) || !et_aligned(prefix_len, 4) || !et_aligned(row_start, 4) ||
                   !et_aligned(lse, 4),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(plan.ws > 0 && (!ws || ws_bytes < plan.ws || !et_aligned(ws, 256)), ET_ERR_WORKSPACE);
  ChunkArgs c = {};
  PagedAttnArgs &a = c.a;
  a.B = shape->B; a.N = shape->max_rows < shape->rows ? shape->max_rows : shape->rows; a.Hq = shape->Hq; a.Hkv = cache->Hkv; a.G = shape->Hq / cache->Hkv;
  a.P = cache->page_size; a.max_blocks = shape->max_blocks; a.max_prefix = shape->max_prefix;
  a.scale_log2 = shape->scale * 1.4426950408889634f;
  a.num_pages = cache->num_pages; a.page_stride = cache->page_stride;
  a.k_pages = static_cast<const uint8_t *>(cache->k_pages); a.v_pages = static_cast<const uint8_t *>(cache->v_pages);
  a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
  a.block_table = block_table; a.prefix_len = prefix_len;
  a.q = q; a.kt = k_new; a.vt = v_new; a.out = out; a.lse = lse; a.dev_status = dev_status;
  c.rows = shape->rows; c.qs = shape->q_stride; c.ks = shape->k_stride; c.vs = shape->v_stride;
  c.row_start = row_start;
  cudaStream_t st = (cudaStream_t)stream;
  if (shape->dtype == ET_BF16) return chunk_tc_launch(cache, c, plan.tc, ws, st);
  return launch_rows(c, cache->d, cache->format, st);
}
