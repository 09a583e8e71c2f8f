// The next token of each row from truncated logits (temperature, top-k, top-p,
// min-p and one given uniform), and the truncated logits themselves, under
// which the acceptance walk is lossless for the truncated distribution (EAGLE
// blog 1.2: lossless in non-greedy decoding).
//
// One thread-block cluster per row (of one block where there are rows enough);
// every block keeps its slice of the row in shared memory, so that the logits
// are read from HBM once whatever is asked for.  Two questions are put to the
// row, both "where does a cumulative count or mass pass a border": in the
// order of the logits (top-k by count, top-p by mass) and in the order of ids
// (the draw).
//   Order of logits: a histogram over equal steps of the logit finds the step
// with the border.  If it and the steps above hold few tokens, as they do for
// all but flat rows, one block sorts these and answers everything.  Else, if
// that step alone holds few, one block sorts it and finds the border.  Else
// histograms over the keys (order-preserving integer images of the logits)
// inside the step follow, until one key value is left; equal keys are told
// apart by id.  Counts and masses are integers, so blocks and atomics may come
// in any order.
//   Order of ids: masses per block, per warp, per 32 tokens.
// Masses are sums of weights 2^44 exp((z - max) / T) rounded to integers.  The
// exponential is evaluated in pairs of fp32 numbers (error-free sums and
// products after T. J. Dekker, Numer. Math. 18, 1971; reduction to 2^(k/64) and
// a Taylor polynomial) to 2^-36.8, 2^-39 in the mean square (its fp32 steps
// against long doubles, 16 million logits): with plain fp32 exponentials a row of
// 10^5 tokens would give another token than 64-bit arithmetic in one draw of
// some hundred.
// Measured: nothing comes near the memory's rate.  One row of 32000: 16 us, the
// latency of a dozen steps that follow on one another (load, extremes,
// histogram, crossing, list, sort by weight, sort by id, draw), each gone
// through once.  244 rows of 32000, top-p and truncated logits: 79 us.  128 rows
// of 100003: 110 to 129 us by the draw of rows; two blocks of an SM issue in 37%
// of the cycles, and most of a warp's waiting is at barriers (8.4 of 20 warps
// per issue), where the steps follow on one another.
#include "et_common.cuh"

namespace et {
namespace {

constexpr int kSaThreads = 512;      // two blocks per SM: one's barriers under the other's arithmetic
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaBins = 512;
constexpr int kSaLimbs = 3;          // a mass of 45 bits in three sums of 15 bits; a count is the first alone
constexpr int kSaMaxCluster = 8;
constexpr int kSaMaxSlice = 32768;   // tokens per block: 8 * 32768 = the largest vocabulary
constexpr int kSaSlice = 20000;      // tokens per block that two blocks of an SM can hold
constexpr int kSaFrac = 44;
constexpr int kSaList = 1024;        // tokens that one block sorts, two per thread

struct SampleArgs {
  int B, V, slice, cluster;
  long long row_stride, out_stride;
  int vec4;  // rows 16-byte aligned
  const float *logits, *temperature, *top_p, *min_p, *uniforms;
  const int32_t *top_k;
  int32_t *token, *dev_status;
  float *logprob, *truncated;
};

// where a cumulative weight passes a border
struct Crossing {
  int bin;                               // -1: nowhere
  unsigned long long above;              // weight of the bins above
};
// what a block's peers read and write of it
struct SampleShared {
  float zmax, zmin;                      // of the block's slice (zmin: of what is above -inf)
  unsigned int first;                    // lowest id of the block's largest
  int odd;
  unsigned int key_lo, key_hi;           // of the slice's members of the current bin
  unsigned long long mass;               // of the slice's kept tokens, or of the block's share of the bins
  Crossing crossing;
  unsigned int listed[3];                // tokens for each list that may be made (block 0)
  unsigned int kept_tau;
  int kept_cut;
  unsigned long long warp_mass[kSaWarps];
  unsigned int hist[2][kSaLimbs][kSaBins];  // alternating: a pass clears the other one
  unsigned long long list[kSaList], weight[kSaList];
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
// all blocks of the row
__device__ __forceinline__ void row_sync(int C) {
  if (C > 1) cl_sync();
  else __syncthreads();
}
__device__ __forceinline__ float key_value(unsigned int key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
// floor or ceil of f * m, exactly: f in [0, 1), m < 2^62 (fp64 arithmetic takes a sixtieth of fp32's rate)
__device__ __forceinline__ unsigned long long fraction_of(float f, unsigned long long m, bool up) {
  const unsigned int bits = __float_as_uint(f);
  const int e = max((int)(bits >> 23), 1), s = 150 - e;  // f = q 2^-s, s >= 24
  const unsigned long long q = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
  unsigned long long lo = q * m, hi = __umul64hi(q, m);
  if (s >= 128) return up && q && m ? 1ull : 0ull;       // less than 2^86 / 2^128
  const unsigned long long rest = s >= 64 ? lo | (hi & ((1ull << (s - 64)) - 1ull)) : lo & ((1ull << s) - 1ull);
  const unsigned long long whole = s >= 64 ? (hi >> (s - 64)) : (hi << (64 - s)) | (lo >> s);
  return whole + (up && rest ? 1ull : 0ull);
}
__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 2^(j / 64) in two fp32 numbers, by repeated products in fp64 (off by 2^-47 at most)
struct PowerTable {
  float hi[64], lo[64];
  constexpr PowerTable() : hi(), lo() {
    double x = 1.0;
    for (int j = 0; j < 64; ++j) {
      hi[j] = (float)x;
      lo[j] = (float)(x - (double)hi[j]);
      x *= 1.01088928605170046002;  // 2^(1 / 64)
    }
  }
};
__constant__ constexpr PowerTable kPowers{};

// 2^44 * exp((z - zm) / T), rounded; ch + cl = log2(e) / T
struct Weigher {
  float zm, ch, cl;
  const float2 *table;  // [64] 2^(j / 64) in two fp32 numbers
  __device__ __forceinline__ unsigned long long operator()(float z) const {
    const float s = z - zm, back = s - z;                      // z - zm = s + err exactly
    const float p = s * ch;
    if (!(p > -46.f)) return 0ull;                             // -inf, too
    const float err = (z - (s - back)) - (zm + back);
    const float e = fmaf(err, ch, fmaf(s, cl, fmaf(s, ch, -p)));  // the exponent of 2 is p + e
    // k = round(64 p): the sum's last bits hold it (1.5 2^23)
    const float kk = fmaf(p, 64.f, 12582912.f);
    const float r = fmaf(kk - 12582912.f, -0.015625f, p);
    const float yh = r + e, yl = e - (yh - r);
    // u = y ln 2
    const float L1 = 0.693147182464599609375f, L2 = -1.904654299957767e-9f;
    const float uh = yh * L1, ul = fmaf(yl, L1, fmaf(yh, L2, fmaf(yh, L1, -uh)));
    const float q = fmaf(uh * uh, fmaf(uh, fmaf(uh, 0.041666667f, 0.16666667f), 0.5f), ul);  // exp(u) - 1 - uh
    const int ki = __float_as_int(kk) - 0x4b400000;
    const float2 t = table[ki & 63];
    const float a = t.x * uh, al = fmaf(t.x, uh, -a);
    const float wh = t.x + a, wl = (a - (wh - t.x)) + (fmaf(t.x, q, al) + fmaf(t.y, uh, t.y));
    // wh, between 1/2 and 2, in units of 2^-24 from its bits; wl, below 2^-15, in units of 2^-37
    const int d = __float_as_int(wh) - 0x3f800000, ih = 0x1000000 + (d < 0 ? d : 2 * d);
    const int il = __float_as_int(fmaf(wl, 137438953472.f, 12582912.f)) - 0x4b400000;
    const long long w = ((long long)ih << (kSaFrac - 24)) + ((long long)il << (kSaFrac - 37));
    const int n = -(ki >> 6);  // 0..46
    return (unsigned long long)(n ? (w + (1ll << (n - 1))) >> n : w);
  }
};

// a token's mass into a bin, in three limbs of which the high ones are rarely there
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

// A mass of every block of the row: their sum, and the sum of the blocks before this one.  Lane k reads block k's, so that
// the reads of other blocks' memory run at once.
__device__ __forceinline__ unsigned long long peers_mass(const Row &row, unsigned long long &before) {
  const int lane = threadIdx.x & 31;
  unsigned long long m = 0ull;
  if (lane < row.C) m = row.C > 1 ? cl_ld_u64(cl_map(&row.sh->mass, (uint32_t)lane)) : row.sh->mass;
  before = warp_sum_u64(lane < row.rank ? m : 0ull);
  return warp_sum_u64(m);
}

// Warp w of the block has tokens [w * span, ...) of the slice, in steps of 32.
__device__ __forceinline__ int warp_span(int slice) { return ((slice + kSaWarps - 1) / kSaWarps + 31) & ~31; }

// The id of the token at which the cumulative weight, in ascending id, passes
// `target` (target < the cluster's total, else -1).  weigh(z, id) is a token's weight.  Every thread of the cluster
// calls it and gets the id.
template <typename W>
__device__ int locate(const Row &row, int slice, int *s_id, W weigh, unsigned long long target,
                      unsigned long long *total, bool fraction, float uniform) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, span = warp_span(slice);
  const int i0 = warp * span, i1 = min(i0 + span, row.n);
  unsigned long long mine = 0ull;
#pragma unroll 2
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
  row_sync(row.C);
  unsigned long long before;
  const unsigned long long all = peers_mass(row, before);
  if (total) *total = all;
  if (fraction) target = fraction_of(uniform, all, false);
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
  row_sync(row.C);
  const int id = *s_id;
  __syncthreads();
  return id;
}

// inclusive sums over the block's threads in order, of a mass and (if asked for) a count; red holds twice kSaWarps
template <bool COUNT>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned int n, unsigned long long *red,
                                                         unsigned long long &all, unsigned int &incl_n, unsigned int &all_n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int *red_n = reinterpret_cast<unsigned int *>(red + kSaWarps);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    const unsigned int yn = COUNT ? __shfl_up_sync(0xffffffffu, n, o) : 0u;
    if (lane >= o) {
      v += y;
      n += yn;
    }
  }
  if (lane == 31) {
    red[warp] = v;
    if (COUNT) red_n[warp] = n;
  }
  __syncthreads();
  unsigned long long mine = lane < kSaWarps ? red[lane] : 0ull;
  unsigned int mine_n = COUNT && lane < kSaWarps ? red_n[lane] : 0u;
#pragma unroll
  for (int o = 1; o < kSaWarps; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, mine, o);
    const unsigned int yn = COUNT ? __shfl_up_sync(0xffffffffu, mine_n, o) : 0u;
    if (lane >= o) {
      mine += y;
      mine_n += yn;
    }
  }
  all = __shfl_sync(0xffffffffu, mine, kSaWarps - 1);
  const unsigned long long before = __shfl_sync(0xffffffffu, mine, (warp + 31) & 31);
  if (COUNT) {
    all_n = __shfl_sync(0xffffffffu, mine_n, kSaWarps - 1);
    const unsigned int before_n = __shfl_sync(0xffffffffu, mine_n, (warp + 31) & 31);
    incl_n = n + (warp ? before_n : 0u);
  }
  __syncthreads();
  return v + (warp ? before : 0ull);
}
__device__ __forceinline__ unsigned long long block_scan_u64(unsigned long long v, unsigned long long *red, unsigned long long &all) {
  unsigned int n, all_n;
  return block_scan<false>(v, 0u, red, all, n, all_n);
}

// The cluster's histogram `h`, its bins in order, and where the cumulative weight reaches `target` (share >= 0: that share
// of the sum, rounded up, one at least).  Block r adds up its share of the bins over the blocks.
template <bool MASS>
__device__ Crossing cross(const Row &row, unsigned int (*h)[kSaBins], unsigned long long above, float share,
                          unsigned long long *target, unsigned long long *s_red) {
  SampleShared *sh = row.sh;
  const int t = threadIdx.x, C = row.C, per = kSaBins / C;
  row_sync(C);  // every block's histogram is whole
  unsigned long long w = 0ull;
  static_assert(kSaBins <= kSaThreads, "a thread per bin and block");
  if (t < kSaBins) {  // bin t / C of the share, as block t % C has it
    const int bin = row.rank * per + t / C;
    const uint32_t k = (uint32_t)(t % C);
    unsigned int l[kSaLimbs];
#pragma unroll
    for (int x = 0; x < kSaLimbs; ++x) l[x] = !MASS && x ? 0u : C > 1 ? cl_ld_u32(cl_map(&h[x][bin], k)) : h[x][bin];
    w = (unsigned long long)l[0] + ((unsigned long long)l[1] << 15) + ((unsigned long long)l[2] << 30);
  }
  // the sum over a bin's C threads comes out of a running sum over all of them
  unsigned long long all;
  const unsigned long long incl = block_scan_u64(w, s_red, all);
  if (t == 0) {
    sh->mass = all;
    sh->crossing.bin = -1;
  }
  row_sync(C);
  unsigned long long before;
  const unsigned long long sum = peers_mass(row, before);
  before += above;
  if (MASS && share >= 0.f) {
    *target = fraction_of(share, sum, true);
    if (*target < 1ull) *target = 1ull;
  }
  // the last of a bin's threads knows the weight up to its end; the bin before, up to its beginning
  unsigned long long begin = __shfl_up_sync(0xffffffffu, incl, C);
  if ((t & 31) == 31) s_red[t >> 5] = incl;
  __syncthreads();
  if ((t & 31) < C) begin = t < 32 ? 0ull : s_red[(t >> 5) - 1];  // the bin before is the previous warp's last
  if (t < kSaBins && t % C == C - 1) {
    const unsigned long long from = before + begin, to = before + incl;
    if (from < *target && *target <= to) {
      Crossing c;
      c.bin = row.rank * per + t / C;
      c.above = from;
      for (int k = 0; k < C; ++k) {
        const uint32_t at = cl_map(&sh->crossing, (uint32_t)k);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at + 8u), "l"(c.above) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(c.bin) : "memory");
      }
    }
  }
  row_sync(C);
  return sh->crossing;
}

// steps of the logit below the maximum
__device__ __forceinline__ int step_of(float z, float zm, float step) { return min(kSaBins - 1, (int)((zm - z) * step)); }

// v[e] of thread t, number t + e * kSaThreads of n, ascending: a bitonic network; beyond n everything is ~0
__device__ void block_sort(unsigned long long (&v)[2], int n, unsigned long long *buf) {
  const int t = threadIdx.x;
  const int count = n > kSaThreads ? 2 : 1;
  for (int k = 2; k < 2 * n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (j == kSaThreads) {
        if (v[1] < v[0]) {
          const unsigned long long x = v[0];
          v[0] = v[1];
          v[1] = x;
        }
        continue;
      }
      if (j >= 32) {
        __syncthreads();
        for (int e = 0; e < count; ++e) buf[t + e * kSaThreads] = v[e];
        __syncthreads();
      } else if (k <= 32 && (t & ~31) >= n) {
        continue;  // whole warps
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (e >= count) break;
        const int i = t + e * kSaThreads;
        const unsigned long long o = j >= 32 ? buf[i ^ j] : __shfl_xor_sync(0xffffffffu, v[e], j);
        const bool low = ((i & j) == 0) == ((i & k) == 0);  // this place takes the smaller one
        v[e] = low == (o < v[e]) ? o : v[e];
      }
    }
}

// The tokens that `in` holds of, from every block of the row into block 0's list, which has room for kSaList of them; how many
// there are comes back.  `count` is zero before, and not used again.
template <typename In>
__device__ unsigned int gather(const Row &row, unsigned int *count, In in) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i0 = 0; i0 < row.n; i0 += kSaThreads) {
    const int i = i0 + threadIdx.x;
    const float z = i < row.n ? row.z[i] : -INFINITY;
    const bool here = z > -INFINITY && in(z, row.base + i);
    const unsigned int m = __ballot_sync(0xffffffffu, here);
    if (!m) continue;
    unsigned int at = 0u;
    if (lane == 0)
      asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(cl_map(count, 0u)), "r"((unsigned int)__popc(m)) : "memory");
    at = __shfl_sync(0xffffffffu, at, 0) + (unsigned int)__popc(m & ((1u << lane) - 1u));
    if (here && at < kSaList)
      cl_st_u64(cl_map(&row.sh->list[0], 0u) + 8u * at, ((unsigned long long)~order_key(z) << 32) | (unsigned int)(row.base + i));
  }
  row_sync(row.C);
  return row.C > 1 ? cl_ld_u32(cl_map(count, 0u)) : *count;
}

// Where the cumulative weight in the order of the logits passes the border: the kept set that ends with that token.  The
// first histogram's crossing is `c`.  MASS: weights are masses of the tokens in `in`; else counts.
template <bool MASS>
__device__ Kept border(Row &row, const SampleArgs &a, const Kept &in, const Weigher &weigh, float zm, float step, Crossing c,
                       unsigned long long target, unsigned int *count, unsigned long long *s_red, int *s_id) {
  SampleShared *sh = row.sh;
  const int t = threadIdx.x, lane = t & 31;
  if (c.bin < 0) return in;  // more was asked for than there is: everything stays
  // ---- the step's tokens, if they are few: block 0 sorts them ----
  if (gather(row, count, [&](float z, int id) { return step_of(z, zm, step) == c.bin && in(order_key(z), id); }) <= kSaList) {
    if (row.rank == 0) {
      const int n = (int)*count, places = n > kSaThreads ? 2 : 1;
      unsigned long long mine[2], sum = c.above;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = t + e * kSaThreads;
        mine[e] = i < n ? sh->list[i] : ~0ull;
      }
      block_sort(mine, n, sh->weight);
      for (int e = 0; e < places; ++e) {
        const unsigned int key = ~(unsigned int)(mine[e] >> 32);
        const unsigned long long w = t + e * kSaThreads >= n ? 0ull : MASS ? weigh(key_value(key)) : 1ull;
        unsigned long long all;
        const unsigned long long incl = sum + block_scan_u64(w, s_red, all);
        if (incl - w < target && target <= incl) {  // one token
          sh->kept_tau = key;
          sh->kept_cut = (int)(unsigned int)mine[e];
        }
        sum += all;
      }
    }
    row_sync(row.C);
    Kept out;
    out.tau = row.C > 1 ? cl_ld_u32(cl_map(&sh->kept_tau, 0u)) : sh->kept_tau;
    out.cut = row.C > 1 ? cl_ld_s32(cl_map(&sh->kept_cut, 0u)) : sh->kept_cut;
    return out;
  }
  unsigned int lo = 0u, hi = 0xffffffffu;
  int shift = -1;  // -1: bins are steps of the logit below the maximum; else (hi - key) >> shift
  for (int round = 0; round < 8; ++round) {  // 1 + at most 4 rounds: a round leaves 2^23 of 2^32 keys, 2^14, 2^5, one
    auto bin_of = [&](unsigned int key, float z) -> int { return shift < 0 ? step_of(z, zm, step) : (int)((hi - key) >> shift); };
    if (t == 0) {
      sh->key_lo = 0xffffffffu;
      sh->key_hi = 0u;
    }
    __syncthreads();
    unsigned int kl = 0xffffffffu, kh = 0u;  // the bin's keys
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = row.z[i];
      const unsigned int key = order_key(z);
      if (z == -INFINITY || key < lo || key > hi || !in(key, row.base + i) || bin_of(key, z) != c.bin) continue;
      kl = min(kl, key);
      kh = max(kh, key);
    }
    kl = __reduce_min_sync(0xffffffffu, kl);
    kh = __reduce_max_sync(0xffffffffu, kh);
    if (lane == 0 && kl <= kh) {
      atomicMin(&sh->key_lo, kl);
      atomicMax(&sh->key_hi, kh);
    }
    row_sync(row.C);
    lo = 0xffffffffu;
    hi = 0u;
    if (lane < row.C) {
      lo = row.C > 1 ? cl_ld_u32(cl_map(&sh->key_lo, (uint32_t)lane)) : sh->key_lo;
      hi = row.C > 1 ? cl_ld_u32(cl_map(&sh->key_hi, (uint32_t)lane)) : sh->key_hi;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lo >= hi) break;
    shift = max(0, 23 - __clz(hi - lo));  // at most 512 bins of 2^shift keys
    // the other histogram has been clear since the last pass; this pass clears the one before
    row.buf ^= 1;
    unsigned int (*h)[kSaBins] = sh->hist[row.buf];
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = row.z[i];
      const unsigned int key = order_key(z);
      if (z == -INFINITY || key < lo || key > hi || !in(key, row.base + i)) continue;
      if (MASS) add_mass(h, bin_of(key, z), weigh(z));
      else atomicAdd(&h[0][bin_of(key, z)], 1u);
    }
    for (int x = t; x < kSaLimbs * kSaBins; x += kSaThreads) (&sh->hist[row.buf ^ 1][0][0])[x] = 0u;
    c = cross<MASS>(row, h, c.above, -1.f, &target, s_red);
  }
  // one key value: the first of its tokens, in ascending id, up to the border
  Kept out;
  out.tau = lo;
  out.cut = 0x7fffffff;
  const unsigned long long each = MASS ? weigh(key_value(lo)) : 1ull;
  const unsigned long long nth = each ? (target - c.above + each - 1) / each : 1ull;  // how many of them
  const int id = locate(row, a.slice, s_id, [&](float z, int i) -> unsigned long long {
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
  __shared__ unsigned long long s_red[2 * kSaWarps];
  __shared__ int s_id;
  __shared__ float s_f[2 * kSaWarps], s_row[3];
  __shared__ int s_odd[kSaWarps];
  const int t = threadIdx.x, lane = t & 31;
  Row row;
  row.sh = &sh;
  row.z = s_z;
  row.C = a.cluster;
  row.rank = a.cluster > 1 ? (int)cl_rank() : 0;
  row.base = row.rank * a.slice;
  row.n = max(0, min(a.slice, a.V - row.base));
  row.buf = 0;
  const int b = blockIdx.x / a.cluster;
  if (t < 64) s_table[t] = make_float2(kPowers.hi[t], kPowers.lo[t]);
  for (int x = t; x < 2 * kSaLimbs * kSaBins; x += kSaThreads) (&sh.hist[0][0][0])[x] = 0u;
  if (t < 3) sh.listed[t] = 0u;
  pdl_wait();
  pdl_trigger();
  // ---- the slice into shared memory; its extremes ----
  const float *zr = a.logits + (long long)b * a.row_stride + row.base;
  float T = a.temperature ? a.temperature[b] : 1.f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
  float u = a.uniforms[b];
  T = T > 0.f ? fminf(fmaxf(T, 1e-30f), 1e30f) : 0.f;
  double depth = 0.0;  // of min-p
  if (t == 0 && T > 0.f) {  // what takes fp64 arithmetic, by one thread and while the logits come
    const double c = 1.4426950408889634074 / (double)T;
    s_row[0] = (float)c;
    s_row[1] = (float)(c - (double)(float)c);
    if (mp > 0.f) depth = (double)T * log((double)mp);
  }
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
#pragma unroll 4
    for (int i = t; i < n4; i += kSaThreads) {
      float4 v = __ldcs(reinterpret_cast<const float4 *>(zr) + i);
      v.x = take(v.x); v.y = take(v.y); v.z = take(v.z); v.w = take(v.w);
      reinterpret_cast<float4 *>(s_z)[i] = v;
    }
    for (int i = 4 * n4 + t; i < row.n; i += kSaThreads) s_z[i] = take(zr[i]);
  } else {
#pragma unroll 8
    for (int i = t; i < row.n; i += kSaThreads) s_z[i] = take(zr[i]);
  }
  zmax = warp_max(zmax);
  zmin = -warp_max(-zmin);
  const float warp_top = zmax;
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) {
    s_f[t >> 5] = zmax;
    s_f[kSaWarps + (t >> 5)] = zmin;
    s_odd[t >> 5] = odd;
  }
  __syncthreads();
  zmax = warp_max(lane < kSaWarps ? s_f[lane] : -INFINITY);
  zmin = -warp_max(lane < kSaWarps ? -s_f[kSaWarps + lane] : -INFINITY);
  odd = __any_sync(0xffffffffu, lane < kSaWarps && s_odd[lane]);
  if (t == 0) {
    sh.zmax = zmax;
    sh.zmin = zmin;
    sh.first = 0xffffffffu;
    sh.odd = odd;
  }
  __syncthreads();
  // the lowest id of the largest logit: a warp that has it looks for it
  if (warp_top == zmax) {
    const int stride = a.vec4 ? 4 : 1;  // what a thread has read
    unsigned int found = 0xffffffffu;
    for (int i = stride * t; i < row.n; i += stride * kSaThreads)
      for (int e = 0; e < stride && i + e < row.n; ++e)
        if (s_z[i + e] == zmax) found = min(found, (unsigned int)(row.base + i + e));
    if (a.vec4)  // the row's ragged end was read one by one
      for (int i = (row.n & ~3) + t; i < row.n; i += kSaThreads)
        if (s_z[i] == zmax) found = min(found, (unsigned int)(row.base + i));
    found = __reduce_min_sync(0xffffffffu, found);
    if (lane == 0) atomicMin(&sh.first, found);
  }
  row_sync(row.C);
  float zm = -INFINITY, zl = INFINITY;
  unsigned int top = 0xffffffffu;
  if (lane < row.C) {
    zm = row.C > 1 ? cl_ld_f32(cl_map(&sh.zmax, (uint32_t)lane)) : sh.zmax;
    zl = row.C > 1 ? cl_ld_f32(cl_map(&sh.zmin, (uint32_t)lane)) : sh.zmin;
    top = row.C > 1 ? cl_ld_u32(cl_map(&sh.first, (uint32_t)lane)) : sh.first;
  }
  const float mine_max = zm;
  zm = warp_max(zm);
  zl = -warp_max(-zl);
  top = __reduce_min_sync(0xffffffffu, mine_max == zm ? top : 0xffffffffu);  // the lowest id of the largest
  if (odd && t == 0) flag_status(a.dev_status, ET_DEV_NONFINITE);

  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  const bool none = zm == -INFINITY, greedy = !(T > 0.f) || k == 1 || p <= 0.f;
  Kept kept;
  kept.tau = 0u;
  kept.cut = -1;  // every key above zero: -inf is above it, and left out where it matters
  int token = -1;
  bool listed_one = false;  // block 0 has answered everything from the list
  float logprob = -INFINITY;
  if (t == 0 && !none && !greedy) {
    unsigned int key_min = 0u;  // min-p: keys from this one on
    if (mp > 0.f) {
      // the smallest logit with (z - max) / T >= log(min_p)
      float zf = (float)((double)zm + depth);
      if ((double)zf - (double)zm < depth) zf = nextafterf(zf, INFINITY);
      key_min = mp > 1.f || zf > zm ? 0xffffffffu : order_key(zf);
    }
    s_row[2] = __uint_as_float(key_min);
  }
  __syncthreads();
  auto log_share = [&](float z, unsigned long long total) -> float {
    return (float)(((double)z - (double)zm) / (double)T - log((double)total / (double)(1ll << kSaFrac)));
  };
  if (none) {
    if (t == 0 && row.rank == 0) flag_status(a.dev_status, ET_DEV_NONFINITE);
    kept.tau = 0xffffffffu;
  } else if (greedy) {
    token = (int)top;
    logprob = 0.f;
    kept.tau = order_key(zm);
    kept.cut = token;
  } else {
    Weigher weigh;
    weigh.zm = zm;
    weigh.ch = s_row[0];
    weigh.cl = s_row[1];
    weigh.table = s_table;
    const unsigned int key_min = __float_as_uint(s_row[2]);
    const bool by_count = k > 0 && k < a.V, by_mass = p < 1.f;
    if (by_count || by_mass) {
      // steps of the logit: the row's own range, but no more than what has mass
      const float range = fminf(zm - zl, fmaxf(32.f * T, 32.f));
      const float step = range > 0.f ? (float)(kSaBins - 1) / range : 0.f;
      unsigned int (*h)[kSaBins] = sh.hist[0];
      unsigned long long target = by_count ? (unsigned long long)k : 0ull;
      Crossing x;
      if (by_count) {
#pragma unroll 4
        for (int i = t; i < row.n; i += kSaThreads) {
          const float z = s_z[i];
          if (z > -INFINITY) atomicAdd(&h[0][step_of(z, zm, step)], 1u);
        }
        x = cross<false>(row, h, 0ull, -1.f, &target, s_red);
      } else {
#pragma unroll 2
        for (int i = t; i < row.n; i += kSaThreads) {
          const float z = s_z[i];
          if (z > -INFINITY) add_mass(h, step_of(z, zm, step), weigh(z));
        }
        x = cross<true>(row, h, 0ull, p, &target, s_red);
      }
      unsigned int listed = ~0u;
      if (x.bin >= 0) {
        // ---- the tokens up to the border's step go to block 0, if they are few ----
        listed = gather(row, &sh.listed[0], [&](float z, int) { return step_of(z, zm, step) <= x.bin; });
      }
      if (listed <= kSaList) {
        // ---- one block sorts them and answers everything ----
        if (row.rank == 0) {
          const int n = (int)listed, places = n > kSaThreads ? 2 : 1;
          unsigned long long mine[2], w[2], incl[2], sum = 0ull;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = t + e * kSaThreads;
            mine[e] = i < n ? sh.list[i] : ~0ull;
          }
          block_sort(mine, n, sh.weight);
          for (int e = 0; e < places; ++e) {
            const int i = t + e * kSaThreads;
            w[e] = i < n && !(by_count && i >= k) ? weigh(key_value(~(unsigned int)(mine[e] >> 32))) : 0ull;
            unsigned long long all;
            incl[e] = sum + block_scan_u64(w[e], s_red, all);
            sum += all;
          }
          if (by_mass && by_count) {
            target = fraction_of(p, sum, true);
            if (target < 1ull) target = 1ull;
          }
          int m = 0;  // how many stay: every rule keeps a leading part
          for (int e = 0; e < places; ++e) {
            const int i = t + e * kSaThreads;
            const unsigned int key = ~(unsigned int)(mine[e] >> 32);
            m += __syncthreads_count(i < n && !(by_count && i >= k) && (!by_mass || incl[e] - w[e] < target) && (key >= key_min || i == 0));
          }
          // the draw: the kept tokens in the order of ids
          for (int e = 0; e < places; ++e) {
            const int i = t + e * kSaThreads;
            if (i == m - 1) {
              sh.kept_tau = ~(unsigned int)(mine[e] >> 32);
              sh.kept_cut = (int)(unsigned int)mine[e];
            }
            sh.weight[i] = w[e];
            mine[e] = i < m ? (mine[e] << 32) | (unsigned int)i : ~0ull;
          }
          if (a.truncated && row.C > 1) cl_arrive();  // the other blocks know what is kept while this one draws
          block_sort(mine, m, sh.list);
          __syncthreads();
          unsigned long long all = 0ull;
          for (int e = 0; e < places; ++e) {
            const int i = t + e * kSaThreads;
            w[e] = i < m ? sh.weight[(unsigned int)mine[e]] : 0ull;
            unsigned long long part;
            incl[e] = all + block_scan_u64(w[e], s_red, part);
            all += part;
          }
          const unsigned long long aim = fraction_of(u, all, false);
          for (int e = 0; e < places; ++e)
            if (t + e * kSaThreads < m && incl[e] - w[e] <= aim && aim < incl[e]) {  // one token
              token = (int)(mine[e] >> 32);
              a.token[b] = token;
              int ignore = 0;
              if (a.logprob) a.logprob[b] = log_share(sanitize_logit(a.logits[(long long)b * a.row_stride + token], ignore), all);
            }
          __syncwarp();
          if (!a.truncated) {
            if (row.C > 1) cl_sync();  // no block leaves while another reads its memory
            return;
          }
          if (row.C > 1) cl_wait();
          kept.tau = sh.kept_tau;
          kept.cut = sh.kept_cut;
        } else {
          if (!a.truncated) {  // this block's memory is not read any more, and it has read block 0's
            cl_arrive();
            return;
          }
          cl_sync();
          kept.tau = cl_ld_u32(cl_map(&sh.kept_tau, 0u));
          kept.cut = cl_ld_s32(cl_map(&sh.kept_cut, 0u));
        }
        listed_one = true;
      } else if (by_count) {
        kept = border<false>(row, a, kept, weigh, zm, step, x, target, &sh.listed[1], s_red, &s_id);
        if (by_mass) {
          row.buf ^= 1;
          h = sh.hist[row.buf];
          row_sync(row.C);  // the histogram that is used next has been cleared, or never used
          for (int i = t; i < kSaLimbs * kSaBins; i += kSaThreads) (&sh.hist[row.buf ^ 1][0][0])[i] = 0u;
          for (int i = t; i < row.n; i += kSaThreads) {
            const float z = s_z[i];
            if (z > -INFINITY && kept(order_key(z), row.base + i)) add_mass(h, step_of(z, zm, step), weigh(z));
          }
          x = cross<true>(row, h, 0ull, p, &target, s_red);
          kept = border<true>(row, a, kept, weigh, zm, step, x, target, &sh.listed[2], s_red, &s_id);
        }
      } else {
        kept = border<true>(row, a, kept, weigh, zm, step, x, target, &sh.listed[1], s_red, &s_id);
      }
    }
    if (!listed_one) {
      if (key_min > order_key(zm)) {  // the largest token alone
        kept.tau = order_key(zm);
        kept.cut = (int)top;
      } else if (key_min > kept.tau) {
        kept.tau = key_min;
        kept.cut = 0x7fffffff;
      }
      unsigned long long total = 0ull;
      token = locate(row, a.slice, &s_id, [&](float z, int i) -> unsigned long long {
        return kept(order_key(z), i) ? weigh(z) : 0ull;
      }, 0ull, &total, true, u);
      if (t == 0 && row.rank == 0) {
        a.token[b] = token;
        int ignore = 0;
        if (a.logprob && token >= 0)
          a.logprob[b] = log_share(sanitize_logit(a.logits[(long long)b * a.row_stride + token], ignore), total);
      }
    }
  }
  if ((none || greedy) && t == 0 && row.rank == 0) {
    a.token[b] = token;
    if (a.logprob) a.logprob[b] = logprob;
  }
  if (a.truncated) {
    float *out = a.truncated + (long long)b * a.out_stride + row.base;
#pragma unroll 4
    for (int i = t; i < row.n; i += kSaThreads) {
      const float z = s_z[i];
      out[i] = kept(order_key(z), row.base + i) ? z : -INFINITY;
    }
  }
  __syncwarp();
  if (row.C > 1) {
    if (listed_one && row.rank > 0) cl_arrive();
    else cl_sync();
  }
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
  // blocks of a row: slices of at most kSaSlice tokens, so that two blocks fit an SM, or less while every block of the call has
  // an SM to itself
  int C = 1, dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 152;
  cudaGetLastError();
  while (C < kSaMaxCluster && (s->V + C - 1) / C > kSaSlice) C *= 2;
  while (C < kSaMaxCluster && 2ll * C * s->B <= sms && s->V > 2048 * C) C *= 2;
  a.cluster = C;
  a.slice = ((s->V + C - 1) / C + 3) & ~3;
  const size_t smem = (size_t)a.slice * sizeof(float);
  if (et_smem_attr((const void *)k_sample, kSaMaxSlice * (int)sizeof(float)) != cudaSuccess) return ET_ERR_CUDA;
  return et_launch(k_sample, dim3((unsigned)(s->B * (long long)C)), dim3(kSaThreads), smem, (cudaStream_t)stream, C, a);
}
