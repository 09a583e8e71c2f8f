// The next token of each row from truncated logits (temperature, top-k, top-p,
// min-p and one given uniform), and the truncated logits themselves, under
// which the acceptance walk is lossless for the truncated distribution (EAGLE
// blog 1.2: lossless in non-greedy decoding).
//
// One thread-block cluster per row; every block keeps its slice of the row in
// shared memory, so that the logits are read from HBM once whatever is asked
// for.  Two questions are put to the row, both "where does a cumulative count
// or mass pass a border": in the order of the logits (top-k by count, top-p by
// mass) and in the order of ids (the draw).
//   Order of logits: a histogram over equal steps of the logit finds the step
// with the border, then histograms over the keys (order-preserving integer
// images of the logits) inside it, until one key value is left; equal keys are
// told apart by id.  Counts and masses are integers, so blocks and atomics may
// come in any order.
//   Order of ids: masses per block, per warp, per 32 tokens.
// Masses are sums of weights 2^44 exp((z - max) / T) rounded to integers.  The
// exponential is evaluated in pairs of fp32 numbers (error-free sums and
// products after T. J. Dekker, Numer. Math. 18, 1971; reduction to 2^(k/64) and
// a Taylor polynomial) to about 2^-40: with plain fp32 exponentials a row of
// 10^5 tokens would give another token than 64-bit arithmetic in one draw of
// some hundred.
#include "et_common.cuh"

namespace et {
namespace {

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaBins = 1024;
constexpr int kSaLimbs = 3;          // a mass of 45 bits in three sums of 15 bits
constexpr int kSaMaxCluster = 8;
constexpr int kSaMaxSlice = 32768;   // tokens per block: 8 * 32768 = the largest vocabulary
constexpr int kSaFrac = 44;

struct SampleArgs {
  int B, V, slice, cluster;
  long long row_stride, out_stride;
  int vec4;  // rows 16-byte aligned
  const float *logits, *temperature, *top_p, *min_p, *uniforms;
  const int32_t *top_k;
  int32_t *token, *dev_status;
  float *logprob, *truncated;
};

// what a block's peers read of it
struct SampleShared {
  float zmax, zmin;                      // of the block's slice (zmin: of what is above -inf)
  unsigned int first;                    // lowest id of the block's largest
  int odd;
  unsigned int key_lo, key_hi;           // of the slice's members of the current bin
  unsigned long long mass;               // of the slice's kept tokens
  unsigned int ties;
  unsigned long long warp_mass[kSaWarps];
  unsigned int hist[2][kSaLimbs][kSaBins];  // alternating: a pass clears the other one
};

// order-preserving image of a logit: larger logit, larger key; -0 as +0
__device__ __forceinline__ unsigned int order_key(float z) {
  const unsigned int u = __float_as_uint(z == 0.f ? 0.f : z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned int cl_ld_u32(uint32_t addr) { return (unsigned int)cl_ld_s32(addr); }
__device__ __forceinline__ unsigned long long cl_ld_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 2^44 * exp((z - zm) / T), rounded; ch + cl = log2(e) / T
struct Weigher {
  float zm, ch, cl;
  const float2 *table;  // [64] 2^(j / 64) in two fp32 numbers
  __device__ __forceinline__ unsigned long long operator()(float z) const {
    const float s = z - zm, p = s * ch;
    if (!(p > -46.f)) return 0ull;
    const float back = s - z;                                  // z - zm = s + err exactly
    const float err = (z - (s - back)) - (zm + back);
    float e = fmaf(s, ch, -p);
    e = fmaf(err, ch, fmaf(s, cl, e));                         // the exponent is p + e
    const float k = rintf(p * 64.f), r = fmaf(k, -0.015625f, p);
    const float yh = r + e, yl = e - (yh - r);
    // u = y ln 2
    const float L1 = 0.693147182464599609375f, L2 = -1.904654299957767e-9f;
    const float uh = yh * L1, ul = fmaf(yl, L1, fmaf(yh, L2, fmaf(yh, L1, -uh)));
    const float q = fmaf(uh * uh, fmaf(uh, fmaf(uh, 0.041666667f, 0.16666667f), 0.5f), ul);  // exp(u) - 1 - uh
    const int ki = (int)k;
    const float2 t = table[ki & 63];
    const float a = t.x * uh, al = fmaf(t.x, uh, -a);
    const float wh = t.x + a, wl = (a - (wh - t.x)) + (fmaf(t.x, q, al) + fmaf(t.y, uh, t.y));
    const long long w = ((long long)__float2int_rn(wh * 16777216.f) << (kSaFrac - 24)) + __float2int_rn(wl * 17592186044416.f);
    const int n = -(ki >> 6);  // 0..46
    return (unsigned long long)(n ? (w + (1ll << (n - 1))) >> n : w);
  }
};

// the three limbs of a mass into a bin; high limbs are rarely there
__device__ __forceinline__ void add_mass(unsigned int (*h)[kSaBins], int bin, unsigned long long w) {
  const unsigned int l0 = (unsigned int)w & 0x7fffu, l1 = (unsigned int)(w >> 15) & 0x7fffu, l2 = (unsigned int)(w >> 30);
  if (l0) atomicAdd(&h[0][bin], l0);
  if (l1) atomicAdd(&h[1][bin], l1);
  if (l2) atomicAdd(&h[2][bin], l2);
}

// what is kept: keys above tau, and of those equal to it ids up to cut
struct Kept {
  unsigned int tau;
  int cut;
  __device__ __forceinline__ bool operator()(unsigned int key, int id) const { return key > tau || (key == tau && id <= cut); }
};

struct Row {
  SampleShared *sh;
  const float *z;   // the slice
  int base, n;      // first id, tokens of the slice
  int rank, C;      // of the cluster
  int buf;          // histogram of the next pass
};

// Warp w of the block has tokens [w * span, ...) of the slice, in steps of 32.
__device__ __forceinline__ int warp_span(int slice) { return ((slice + kSaWarps - 1) / kSaWarps + 31) & ~31; }

// The id of the token at which the cumulative weight, in ascending id, passes
// `target` (target < the cluster's total, else -1).  w(key, id, z) weighs.  Every thread
// of the cluster calls it and gets the id.
template <typename W>
__device__ int locate(const Row &row, int slice, unsigned long long *s_red, int *s_id, W weigh, unsigned long long target,
                      unsigned long long *total, bool fraction, float uniform) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, span = warp_span(slice);
  const int i0 = warp * span, i1 = min(i0 + span, row.n);
  unsigned long long mine = 0ull;
  for (int i = i0 + lane; i < i1; i += 32) mine += weigh(row.z[i], row.base + i);
  mine = warp_sum_u64(mine);
  if (lane == 0) row.sh->warp_mass[warp] = mine;
  __syncthreads();
  if (t == 0) {
    unsigned long long sum = 0ull;
    for (int k = 0; k < kSaWarps; ++k) sum += row.sh->warp_mass[k];
    row.sh->mass = sum;
    *s_id = -1;
  }
  cl_sync();
  unsigned long long before = 0ull, all = 0ull;
  for (int k = 0; k < row.C; ++k) {
    const unsigned long long m = cl_ld_u64(cl_map(&row.sh->mass, (uint32_t)k));
    if (k < row.rank) before += m;
    all += m;
  }
  if (total) *total = all;
  if (fraction) target = (unsigned long long)((double)uniform * (double)all);
  // this warp's tokens begin behind `before`
  for (int k = 0; k < warp; ++k) before += row.sh->warp_mass[k];
  if (before <= target && target < before + mine) {  // one warp of the cluster
    for (int i = i0; i < i1; i += 32) {
      const unsigned long long w = i + lane < i1 ? weigh(row.z[i + lane], row.base + i + lane) : 0ull;
      unsigned long long incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned int hit = __ballot_sync(0xffffffffu, before + incl > target);
      if (hit) {
        const int id = row.base + i + __ffs(hit) - 1;
        for (int k = lane; k < row.C; k += 32)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cl_map(s_id, (uint32_t)k)), "r"(id) : "memory");
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  cl_sync();
  const int id = *s_id;
  __syncthreads();
  return id;
}

// Where the cumulative weight in the order of the logits passes `target`: the
// kept set that ends with that token.  MASS: weights are masses of the tokens
// in `in`, and target a share of their sum; else counts.
template <bool MASS>
__device__ Kept border(Row &row, const SampleArgs &a, const Kept &in, const Weigher &weigh, float zm, float step,
                       unsigned long long count, float share, unsigned long long *s_red, int *s_id) {
  SampleShared *sh = row.sh;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  unsigned long long target = count;  // the border lies in the first bin whose cumulative weight reaches it
  unsigned long long above = 0ull;    // weight of the bins above
  unsigned int lo = 0u, hi = 0xffffffffu;
  int shift = -1;                     // -1: bins are steps of the logit below the maximum; else (key - lo) >> shift from above
  bool first = true;
  for (int round = 0; round < 8; ++round) {  // 1 + at most 4 rounds: a round leaves 2^22 of 2^32 keys, 2^12, 2^2, one
    unsigned int (*h)[kSaBins] = sh->hist[row.buf];
    auto bin_of = [&](unsigned int key, float z) -> int {
      if (shift < 0) return min(kSaBins - 1, (int)((zm - z) * step));
      return (int)((hi - key) >> shift);
    };
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = row.z[i];
      const unsigned int key = order_key(z);
      if (z == -INFINITY || key < lo || key > hi || !in(key, row.base + i)) continue;
      if (MASS) add_mass(h, bin_of(key, z), weigh(z));
      else atomicAdd(&h[0][bin_of(key, z)], 1u);
    }
    cl_sync();
    // every block adds the cluster's histograms up: thread t has bins 2 t and 2 t + 1
    unsigned long long w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      w[e] = 0ull;
      for (int k = 0; k < row.C; ++k) {
#pragma unroll
        for (int l = 0; l < (MASS ? kSaLimbs : 1); ++l)
          w[e] += (unsigned long long)cl_ld_u32(cl_map(&h[l][2 * t + e], (uint32_t)k)) << (15 * l);
      }
    }
    unsigned long long incl = w[0] + w[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_red[warp] = incl;
    if (t == 0) *s_id = -1;
    // the other histogram is free: its readers have passed this pass's first barrier
    for (int x = t; x < kSaLimbs * kSaBins; x += kSaThreads) (&sh->hist[row.buf ^ 1][0][0])[x] = 0u;
    __syncthreads();
    unsigned long long before = above, all = above;
    for (int k = 0; k < kSaWarps; ++k) {
      if (k < warp) before += s_red[k];
      all += s_red[k];
    }
    if (MASS && first) {  // tokens before which less than the share of the mass lies: ceil(share * mass), one at least
      target = (unsigned long long)ceil((double)share * (double)all);
      if (target < 1ull) target = 1ull;
    }
    first = false;
    before += incl - w[0] - w[1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < target && target <= before + w[e]) {
        s_id[0] = 2 * t + e;
        s_red[kSaWarps] = before;
      }
      before += w[e];
    }
    if (t == 0) {
      sh->key_lo = 0xffffffffu;
      sh->key_hi = 0u;
    }
    __syncthreads();
    const int bin = *s_id;
    above = s_red[kSaWarps];
    if (bin < 0) {  // more was asked for than there is: everything stays
      cl_sync();
      row.buf ^= 1;
      return in;
    }
    // the bin's keys
    unsigned int kl = 0xffffffffu, kh = 0u;
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = row.z[i];
      const unsigned int key = order_key(z);
      if (z == -INFINITY || key < lo || key > hi || !in(key, row.base + i) || bin_of(key, z) != bin) continue;
      kl = min(kl, key);
      kh = max(kh, key);
    }
    kl = __reduce_min_sync(0xffffffffu, kl);
    kh = __reduce_max_sync(0xffffffffu, kh);
    if (lane == 0 && kl <= kh) {
      atomicMin(&sh->key_lo, kl);
      atomicMax(&sh->key_hi, kh);
    }
    cl_sync();
    lo = 0xffffffffu;
    hi = 0u;
    for (int k = 0; k < row.C; ++k) {
      lo = min(lo, cl_ld_u32(cl_map(&sh->key_lo, (uint32_t)k)));
      hi = max(hi, cl_ld_u32(cl_map(&sh->key_hi, (uint32_t)k)));
    }
    row.buf ^= 1;
    if (lo >= hi) break;
    shift = max(0, 22 - __clz(hi - lo));  // at most 1024 bins of 2^shift keys
  }
  // one key value: the first of its tokens, in ascending id, up to the border
  Kept out;
  out.tau = lo;
  out.cut = 0x7fffffff;
  const unsigned long long each = MASS ? weigh(__uint_as_float((lo & 0x80000000u) ? (lo & 0x7fffffffu) : ~lo)) : 1ull;
  const unsigned long long nth = each ? (target - above + each - 1) / each : 1ull;  // how many of them
  const int id = locate(row, a.slice, s_red, s_id, [&](float z, int i) -> unsigned long long {
    const unsigned int key = order_key(z);
    return key == lo && in(key, i) ? 1ull : 0ull;
  }, nth - 1, nullptr, false, 0.f);
  if (id >= 0) out.cut = id;
  return out;
}

__global__ void __launch_bounds__(kSaThreads) k_sample(const SampleArgs a) {
  extern __shared__ __align__(16) float s_z[];
  __shared__ SampleShared sh;
  __shared__ float2 s_table[64];
  __shared__ unsigned long long s_red[kSaWarps + 1];
  __shared__ int s_id;
  __shared__ float s_f[32];
  __shared__ unsigned int s_u[kSaWarps];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  Row row;
  row.sh = &sh;
  row.z = s_z;
  row.C = a.cluster;
  row.rank = a.cluster > 1 ? (int)cl_rank() : 0;
  row.base = row.rank * a.slice;
  row.n = max(0, min(a.slice, a.V - row.base));
  row.buf = 0;
  const int b = blockIdx.x / a.cluster;
  if (t < 64) {
    const double x = exp2((double)t / 64);
    const float h = (float)x;
    s_table[t] = make_float2(h, (float)(x - (double)h));
  }
  for (int x = t; x < kSaLimbs * kSaBins; x += kSaThreads) (&sh.hist[0][0][0])[x] = 0u;
  pdl_wait();
  pdl_trigger();
  // ---- the slice into shared memory; its extremes ----
  const float *zr = a.logits + (long long)b * a.row_stride + row.base;
  float zmax = -INFINITY, zmin = INFINITY;
  int odd = 0;
  auto take = [&](float z) -> float {
    z = sanitize_logit(z, odd);
    zmax = fmaxf(zmax, z);
    if (z > -INFINITY) zmin = fminf(zmin, z);
    return z;
  };
  if (a.vec4) {  // the slice is a multiple of 4: only the row's end is ragged
    const int n4 = row.n >> 2;
    for (int i = t; i < n4; i += kSaThreads) {
      float4 v = __ldcs(reinterpret_cast<const float4 *>(zr) + i);
      v.x = take(v.x); v.y = take(v.y); v.z = take(v.z); v.w = take(v.w);
      reinterpret_cast<float4 *>(s_z)[i] = v;
    }
    for (int i = 4 * n4 + t; i < row.n; i += kSaThreads) s_z[i] = take(zr[i]);
  } else {
    for (int i = t; i < row.n; i += kSaThreads) s_z[i] = take(zr[i]);
  }
  zmax = block_max<kSaThreads>(zmax, s_f);
  zmin = -block_max<kSaThreads>(-zmin, s_f);
  odd = __syncthreads_or(odd);
  unsigned int first = 0xffffffffu;  // lowest id of the largest logit
  for (int i = t; i < row.n; i += kSaThreads)
    if (s_z[i] == zmax) first = min(first, (unsigned int)(row.base + i));
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0) s_u[warp] = first;
  __syncthreads();
  if (t == 0) {
    for (int k = 0; k < kSaWarps; ++k) first = min(first, s_u[k]);
    sh.zmax = zmax;
    sh.zmin = zmin;
    sh.first = first;
    sh.odd = odd;
  }
  cl_sync();
  float zm = -INFINITY, zl = INFINITY;
  unsigned int top = 0xffffffffu;
  for (int k = 0; k < a.cluster; ++k) {
    const float m = cl_ld_f32(cl_map(&sh.zmax, (uint32_t)k));
    const unsigned int f = cl_ld_u32(cl_map(&sh.first, (uint32_t)k));
    if (m > zm) { zm = m; top = f; }  // blocks hold ascending ids: the first one wins a tie
    zl = fminf(zl, cl_ld_f32(cl_map(&sh.zmin, (uint32_t)k)));
  }
  if (odd && t == 0) flag_status(a.dev_status, ET_DEV_NONFINITE);

  float T = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  float u = a.uniforms[b];
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  const bool none = zm == -INFINITY, greedy = !(T > 0.f) || k == 1 || p <= 0.f;
  Kept kept;
  kept.tau = 0u;
  kept.cut = -1;  // every key above zero: -inf is above it, and left out where it matters
  int token = -1;
  float logprob = -INFINITY;
  if (none) {
    if (t == 0 && row.rank == 0) flag_status(a.dev_status, ET_DEV_NONFINITE);
    kept.tau = 0xffffffffu;
  } else if (greedy) {
    token = (int)top;
    logprob = 0.f;
    kept.tau = order_key(zm);
    kept.cut = token;
  } else {
    T = fminf(fmaxf(T, 1e-30f), 1e30f);
    const double c = 1.4426950408889634074 / (double)T;
    Weigher weigh;
    weigh.zm = zm;
    weigh.ch = (float)c;
    weigh.cl = (float)(c - (double)weigh.ch);
    weigh.table = s_table;
    // steps of the logit: the row's own range, but no more than what has mass
    const float range = fminf(zm - zl, fmaxf(32.f * T, 32.f));
    const float step = range > 0.f ? (float)(kSaBins - 1) / range : 0.f;
    if (k > 0 && k < a.V) kept = border<false>(row, a, kept, weigh, zm, step, (unsigned long long)k, 0.f, s_red, &s_id);
    if (p < 1.f) kept = border<true>(row, a, kept, weigh, zm, step, 0ull, p, s_red, &s_id);
    if (mp > 0.f) {
      // the smallest logit with (z - max) / T >= log(min_p)
      const double depth = (double)T * log((double)mp);
      float zf = (float)((double)zm + depth);
      if ((double)zf - (double)zm < depth) zf = nextafterf(zf, INFINITY);
      const unsigned int key = order_key(fminf(zf, zm));
      if (mp > 1.f || zf > zm) {  // the largest token alone
        kept.tau = order_key(zm);
        kept.cut = (int)top;
      } else if (key > kept.tau) {
        kept.tau = key;
        kept.cut = 0x7fffffff;
      }
    }
    unsigned long long total = 0ull;
    token = locate(row, a.slice, s_red, &s_id, [&](float z, int i) -> unsigned long long {
      return kept(order_key(z), i) ? weigh(z) : 0ull;
    }, 0ull, &total, true, u);
    if (t == 0 && row.rank == 0 && a.logprob && token >= 0) {
      const float z = a.logits[(long long)b * a.row_stride + token];
      int ignore = 0;
      const double depth = ((double)sanitize_logit(z, ignore) - (double)zm) / (double)T;
      logprob = (float)(depth - log((double)total / (double)(1ll << kSaFrac)));
    }
  }
  if (a.truncated) {
    float *out = a.truncated + (long long)b * a.out_stride + row.base;
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = s_z[i];
      out[i] = kept(order_key(z), row.base + i) ? z : -INFINITY;
    }
  }
  if (t == 0 && row.rank == 0) {
    a.token[b] = token;
    if (a.logprob) a.logprob[b] = logprob;
  }
  cl_sync();  // no block leaves while another reads its memory
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" et_status et_sample(const et_sample_shape *s, const float *logits, const float *temperature,
                               const int32_t *top_k, const float *top_p, const float *min_p, const float *uniforms,
                               int32_t *token, float *logprob, float *truncated, int32_t *dev_status,
                               et_stream_t stream) {
  ET_RETURN_IF(!s || !logits || !uniforms || !token, ET_ERR_INVALID_ARG);
  ET_RETURN_IF(s->B < 1 || s->V < 1 || s->row_stride < s->V || (truncated && s->out_stride < s->V), ET_ERR_INVALID_ARG);
  ET_RETURN_IF(s->V > kMaxV || s->B > (1 << 24), ET_ERR_UNSUPPORTED);
  ET_RETURN_IF(!et_aligned(logits, 4) || !et_aligned(temperature, 4) || !et_aligned(top_k, 4) ||
                   !et_aligned(top_p, 4) || !et_aligned(min_p, 4) || !et_aligned(uniforms, 4) || !et_aligned(token, 4) ||
                   !et_aligned(logprob, 4) || !et_aligned(truncated, 4),
               ET_ERR_INVALID_ARG);
  SampleArgs a = {};
  a.B = s->B; a.V = s->V; a.row_stride = s->row_stride; a.out_stride = s->out_stride;
  a.vec4 = et_aligned(logits, 16) && s->row_stride % 4 == 0;
  a.logits = logits; a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.uniforms = uniforms; a.token = token; a.logprob = logprob; a.truncated = truncated; a.dev_status = dev_status;
  int C = kSaMaxCluster;
  while (C > 1 && s->V <= 4096 * (C / 2)) C /= 2;
  a.cluster = C;
  a.slice = ((s->V + C - 1) / C + 3) & ~3;
  const size_t smem = (size_t)a.slice * sizeof(float);
  if (et_smem_attr((const void *)k_sample, kSaMaxSlice * (int)sizeof(float)) != cudaSuccess) return ET_ERR_CUDA;
  return et_launch(k_sample, dim3((unsigned)(s->B * (long long)C)), dim3(kSaThreads), smem, (cudaStream_t)stream, C, a);
}
