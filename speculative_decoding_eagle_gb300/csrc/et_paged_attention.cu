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
//
// A tree row, whose V is not quantised, gets a scale of the same kind: vt, the
// power of two that a page of this V alone would have.  t then bounds p |v|
// for both kinds of key, whatever the size of V, and no key's weight falls out
// of fp16's range because another kind's V is held in another unit.  (One
// scale for the whole tree would let a row that others do not attend, padding
// for one, decide about them.)  Its weight is 2^(t - m) / vt (bf16, whose range
// has room for it), so that V meets it as it is.
#include <cuda_bf16.h>

#include "et_paged_attn.cuh"

namespace et {
namespace {

// ---------------------------------------------------------------------------
// fp32: CUDA cores, one block per (row, head, sequence)
// ---------------------------------------------------------------------------
// Each warp takes every eighth group of 32 keys: a lane scores one key (its
// whole row, 16 bytes a load), the group's maximum and sum are warp
// reductions, then the lanes turn to the head's dims and add the 32 weighted
// V rows, whose loads do not depend on one another.  For small models and
// checks: it reads a sequence's codes once per row and head out of L2.  Bound
// by latency (17 rows, 4 heads of 64 dims, 128 tokens: 5.1 us in a graph).
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) k_paged_attn_row(PagedAttnArgs a) {
  constexpr int PL = D / 32;  // dims per lane
  __shared__ float qs[D];
  __shared__ float wm[kRowWarps], wl[kRowWarps];
  __shared__ float wacc[kRowWarps][D];
  pdl_wait();     // the previous kernel in the stream has completed
  pdl_trigger();  // only now may the next kernel launch
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int g = h / a.G, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int bad = 0;
  const int L = paged_prefix(a, b, bad);
  if (L < 0) return;
  const long long orow = ((long long)b * a.N + i) * a.Hq + h;
  for (int c = t; c < D; c += kRowThreads) qs[c] = static_cast<const float *>(a.q)[orow * D + c];
  __syncthreads();
  const float *KT = static_cast<const float *>(a.kt), *VT = static_cast<const float *>(a.vt);
  float m = -INFINITY, l = 0.f, acc[PL];
#pragma unroll
  for (int c = 0; c < PL; ++c) acc[c] = 0.f;
  const int nP = tiles_of(L, 32), nT = (a.N + 31) / 32;
  for (int grp = warp; grp < nP + nT; grp += kRowWarps) {
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
#pragma unroll
      for (int c = 0; c < D / 4; ++c) {
        const float4 v = *reinterpret_cast<const float4 *>(KT + at + 4 * c);
        s = fmaf(qs[4 * c], v.x, s);
        s = fmaf(qs[4 * c + 1], v.y, s);
        s = fmaf(qs[4 * c + 2], v.z, s);
        s = fmaf(qs[4 * c + 3], v.w, s);
      }
    }
    s = ok ? s * a.scale_log2 : -INFINITY;
    const unsigned int keep = __ballot_sync(0xffffffffu, ok);
    if (keep == 0u) continue;  // no key for this row in this group
    const float was = m;
    m = fmaxf(m, warp_max(s));
    const float ref = m == -INFINITY ? 0.f : m;  // only NaN or -inf scores so far: the weights below become NaN or 0
    const float corr = exp2f(was - ref), p = ok ? exp2f(s - ref) : 0.f;
    l = l * corr + warp_sum(p);
#pragma unroll
    for (int c = 0; c < PL; ++c) acc[c] *= corr;
    const float pv = p * vs;
#pragma unroll 1
    for (int k0 = 0; k0 < 32; k0 += 16) {
      uint32_t code[16];
      float xt[16][PL];
#pragma unroll
      for (int k = 0; k < 16; ++k) {  // sixteen rows' loads in flight
        const long long row = __shfl_sync(0xffffffffu, at, k0 + k);
        const bool on = (keep >> (k0 + k)) & 1u;
        code[k] = 0u;
#pragma unroll
        for (int c = 0; c < PL; ++c) xt[k][c] = 0.f;
        if (on && cached) {
          if (PL == 4) code[k] = *reinterpret_cast<const uint32_t *>(a.v_pages + row + 4 * lane);
          else code[k] = *reinterpret_cast<const uint16_t *>(a.v_pages + row + 2 * lane);
        } else if (on) {
#pragma unroll
          for (int c = 0; c < PL; c += 2) {
            const float2 y = *reinterpret_cast<const float2 *>(VT + row + PL * lane + c);
            xt[k][c] = y.x;
            xt[k][c + 1] = y.y;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float w = __shfl_sync(0xffffffffu, pv, k0 + k);
        if (!((keep >> (k0 + k)) & 1u)) continue;
        if (cached) {
          float y[4];
          f8x4_to_f32<FMT>(code[k], y);
#pragma unroll
          for (int c = 0; c < PL; ++c) xt[k][c] = y[c];
        }
#pragma unroll
        for (int c = 0; c < PL; ++c) acc[c] = fmaf(w, xt[k][c], acc[c]);
      }
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
  for (int w = 1; w < kRowWarps; ++w) M = fmaxf(M, wm[w]);
  float Ls = 0.f, wts[kRowWarps];
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    wts[w] = wm[w] == -INFINITY ? 0.f : exp2f(wm[w] - M);
    Ls += wl[w] * wts[w];
  }
  for (int c = t; c < D; c += kRowThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) v += wacc[w][c] * wts[w];
    static_cast<float *>(a.out)[orow * D + c] = Ls == 0.f ? 0.f : v / Ls;
  }
  if (t == 0 && a.lse)
    a.lse[((long long)b * a.Hq + h) * a.N + i] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * 0.69314718055994531f;
  if (bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
}

template <int FMT>
et_status launch_row(const PagedAttnArgs &a, int d, cudaStream_t st) {
  const dim3 grid(a.N, a.Hq, a.B);
  if (d == 64) return et_launch(k_paged_attn_row<FMT, 64>, grid, dim3(kRowThreads), 0, st, 0, a);
  return et_launch(k_paged_attn_row<FMT, 128>, grid, dim3(kRowThreads), 0, st, 0, a);
}

// ---------------------------------------------------------------------------
// bf16: tensor cores (mma.sync), cached codes as operands
// ---------------------------------------------------------------------------
// Codes become fp16 exactly, so both products are fp16 m16n8k16 into fp32
// sums.  q is lifted by a power of two per row to [2^14, 2^15) before it is
// rounded to fp16: nothing above 2^-38 of its row's largest element is lost.
// Weights stay below 2^15 and lose only what lies 2^-28 below the largest.
// (8-bit mma.sync is no way out here: on this part it runs as two fp16
// products and conversions; 479 TFLOP/s against 573 for fp16 in a loop with
// changing operands.)
//
// A block of four warps owns R = 16 * WR * MT query rows (token, head in
// group) of one KV head and a chunk of the prefix.  WR warps share the rows,
// KG = 4 / WR groups of them take alternate tiles of 32 keys.  Each group has
// its own ring of tiles, brought by TMA (one box of 32 rows, two of 16 where
// a page is not a multiple of 32) into the 128- or 64-byte swizzle, in which
// every operand load is conflict-free.  Page ids and scales are fetched 32
// units of 16 keys at a time, one per lane, a batch ahead.
// d = 128 runs 16 rows a block (more go to the tcgen05 kernel), d = 64 also 32
// (MT = 2) and 64 (WR = 2).  16 rows: three blocks of 64 KB of tiles an SM.
//
// Bound by HBM once blocks are long: 64 sequences of 4096 tokens, 32 heads,
// one row each: 320 us, 6.7 TB/s.  A block takes about 10 us beside its stream (its
// lengths, page table and first tiles one after the other; its groups' rows
// and the sequence's chunks merged): 16 sequences of 512..16384 tokens, 8 KV
// heads of 8 query heads: 57.4 us in a graph, 5.1 TB/s; one of 1023, 32 heads: 8.7 us in a
// graph, 1.0 TB/s.
constexpr int kPaThreads = 128;
constexpr int kPaWarps = 4;
constexpr int kPaTile = 32;  // keys per tile
constexpr int kPaLeast = 8;  // tiles in a chunk, at least
// arrival counters in every workspace, at its start: the same place whatever the shape, so that calls of different
// shapes can use one workspace one after the other
constexpr int kPaCounters = 1 << 16;

template <int D, int WR, int MT>
struct PaShape {
  static constexpr int KG = kPaWarps / WR;
  static constexpr int R = 16 * WR * MT;
  static constexpr int kBlocks = MT == 1 ? 3 : 2;           // resident blocks per SM
  static constexpr int kStages = WR == 2 ? 4 : 2;           // 64 KB of tiles a block
  static constexpr int kTileBytes = kPaTile * D;            // K or V
  static constexpr int kRing = KG * kStages * 2 * kTileBytes;
  static constexpr int kOffQ = kRing;                       // lifted fp16, fragment order
  static constexpr int kOffQ16 = kOffQ + R * D * 2;         // bf16, fragment order
  static constexpr int kOffRow = kOffQ16 + R * D * 2;       // row factors
  static constexpr int kOffBar = kOffRow + R * 4;
  static constexpr int kBytes = kOffBar + KG * kStages * 8 + 1024;  // + slack for 1024-byte alignment
  static_assert(KG * R * D * 4 + (KG + 1) * R * 8 <= kOffRow, "the groups' rows are merged in the space of the ring and q");
  static_assert((kPaMaxSplits + 1) * R * 8 <= kOffRow, "the chunks' pairs, too");
  static_assert(kBlocks * (kBytes + 1024 + 64 + kMaxN * 4) <= 228 * 1024, "the blocks of an SM");
};

template <bool BF16>
__device__ __forceinline__ void mma_16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// 16-byte chunk c of row r of a merged fp32 row set: rotated so that the four
// lanes of a quad and two neighbouring rows hit different banks
template <int D>
__device__ __forceinline__ int merge_chunk(int r, int c) {
  return (c & ~7) | ((c + (c >> 3) + (D == 128 ? 4 : 2) * r) & 7);
}

// Weights of NT n-tiles of scores (16 keys = two n-tiles share a scale): x =
// score * f + lv relative to the row's reference mr, which moves only when a
// weight would pass 2^15 (then it becomes the row maximum - 3 and what was
// summed is rescaled).  keep: bit (8 * n-tile + key) per row, all ones when
// `masked` is false.  On return p holds the weights as packed pairs.  The
// tree's rows (BF16) have a V scale each, 2 * n-tile + (column & 1), and their
// weights are divided by it.
template <int NT, int MT, int NTO, bool BF16>
__device__ __forceinline__ void paged_softmax(const float (&s)[MT][NT][4], const float (&rf)[2 * MT],
                                              const float (&ks)[NT / 2], const float (&lv)[BF16 ? 2 * NT : NT / 2],
                                              const float (&iv)[BF16 ? 2 * NT : NT / 2], bool masked,
                                              const uint32_t (&keep)[2 * MT], float (&mr)[2 * MT], float (&l)[2 * MT], float (&o)[MT][NTO][4],
                                              uint32_t (&p)[MT][NT][2]) {
  const int t2 = 2 * (threadIdx.x & 3);
  float x[MT][NT][4];
  auto weigh = [&]() {
    float top = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int u = 0; u < NT / 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = rf[2 * mt + h] * ks[u];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int nt = 2 * u + (e >> 1), i = 2 * h + (e & 1);
            const float c = lv[BF16 ? 2 * nt + (e & 1) : u] - mr[2 * mt + h];
            float v = fmaf(s[mt][nt][i], f, c);
            if (masked && !((keep[2 * mt + h] >> (8 * nt + t2 + (e & 1))) & 1u)) v = -INFINITY;
            x[mt][nt][i] = v;
            top = fmaxf(top, v);
          }
        }
    return top;
  };
  if (__any_sync(0xffffffffu, weigh() > kPaTop + kPaSlack)) {
    // a weight too large (or the first key of a row): the maxima of the rows, from the scores themselves
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
      const int mt = r >> 1, h = r & 1;
      float top = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!masked || ((keep[r] >> (8 * nt + t2 + e)) & 1u))
            top = fmaxf(top, fmaf(s[mt][nt][2 * h + e], rf[r] * ks[nt / 2], lv[BF16 ? 2 * nt + e : nt / 2]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float now = fmaxf(mr[r], top - kPaTop), corr = ex2_fast(mr[r] - now);
      mr[r] = now;
      l[r] *= corr;
#pragma unroll
      for (int nt = 0; nt < NTO; ++nt) {
        o[mt][nt][2 * h] *= corr;
        o[mt][nt][2 * h + 1] *= corr;
      }
    }
    weigh();
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int u = 0; u < NT / 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w0 = ex2_fast(x[mt][2 * u][2 * h]), w1 = ex2_fast(x[mt][2 * u][2 * h + 1]);
        float w2 = ex2_fast(x[mt][2 * u + 1][2 * h]), w3 = ex2_fast(x[mt][2 * u + 1][2 * h + 1]);
        if (BF16) {
          w0 *= iv[4 * u]; w1 *= iv[4 * u + 1]; w2 *= iv[4 * u + 2]; w3 *= iv[4 * u + 3];
          l[2 * mt + h] += (w0 + w1) + (w2 + w3);
        } else {
          l[2 * mt + h] = fmaf((w0 + w1) + (w2 + w3), iv[u], l[2 * mt + h]);
        }
        p[mt][2 * u][h] = BF16 ? pack_bf16x2(w0, w1) : pack_f16x2(w0, w1);
        p[mt][2 * u + 1][h] = BF16 ? pack_bf16x2(w2, w3) : pack_f16x2(w2, w3);
      }
}

// A batch of up to 32 sequences shared among `blocks` blocks per tile of rows, all chunks of one length: the shortest,
// to a 31st of its range, that needs no more blocks.  Every warp works it out for itself, a sequence a lane.
struct Share { int b, chunk, chunks, per; };  // b < 0: nothing for block c
__device__ __forceinline__ Share share_batch(const PagedAttnArgs &a, int lane, int blocks, int c) {
  int ignore = 0;
  const int L = lane < a.B ? paged_prefix(a, lane, ignore) : -1, T = L < 0 ? 0 : tiles_of(L, kPaTile);
  const int present = __popc(__ballot_sync(0xffffffffu, L >= 0));
  const int longest = __reduce_max_sync(0xffffffffu, T);
  const float total = (float)__reduce_add_sync(0xffffffffu, (unsigned)T);  // < 2^31: 32 sequences of 2^26 tiles at most
  // sum of ceil(T / per) <= total / per + present, so the upper end needs no more than `blocks`
  const int lo = max(max(kPaLeast, (longest + kPaMaxSplits - 1) / kPaMaxSplits), (int)(total / (float)blocks));
  const int hi = max(lo, (int)(total * 1.000001f / (float)(blocks - present)) + 1), step = (hi - lo + 30) / 31;
  const int mine = lo + lane * step;
  // ceil(T / per): at most kPaMaxSplits, so the quotient in fp32 is off by one at most
  auto pieces = [&](int tiles, int per) -> int {
    const int x = tiles + per - 1;
    int q = (int)((float)x * (1.f / (float)per));
    const int r = x - q * per;
    q += (r >= per ? 1 : 0) - (r < 0 ? 1 : 0);
    return max(q, 1);
  };
  int need = 0;
#pragma unroll 4
  for (int k = 0; k < a.B; ++k) {
    const int Lk = __shfl_sync(0xffffffffu, L, k), Tk = __shfl_sync(0xffffffffu, T, k);
    need += Lk < 0 ? 0 : pieces(Tk, mine);
  }
  const uint32_t fits = __ballot_sync(0xffffffffu, need <= blocks);
  Share s;
  s.per = __shfl_sync(0xffffffffu, mine, fits ? __ffs(fits) - 1 : 31);
  const int own = L < 0 ? 0 : pieces(T, s.per);
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int before = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += before;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, upto > c);
  s.b = past ? __ffs(past) - 1 : -1;
  const int at = max(s.b, 0);
  s.chunks = __shfl_sync(0xffffffffu, own, at);
  s.chunk = c - __shfl_sync(0xffffffffu, upto - own, at);
  return s;
}

template <int D, int FMT, int WR, int MT>
__global__ void __launch_bounds__(kPaThreads, (PaShape<D, WR, MT>::kBlocks))
    k_paged_attn_mma(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ PagedSplitArgs ma) {
  using Sh = PaShape<D, WR, MT>;
  constexpr int KG = Sh::KG, R = Sh::R, ST = Sh::kStages, TB = Sh::kTileBytes;
  constexpr int K16 = D / 16, NTO = D / 8;
  const PagedAttnArgs &a = ma.a;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_abort, s_last;
  __shared__ int s_red[kPaWarps];
  __shared__ float s_tree_lv[kMaxN];  // log2 of the tree rows' V scales
  unsigned char *sm = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = saddr(sm);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g8 = lane >> 2, tq = lane & 3;
  const int wr = warp % WR, kg = warp / WR;
  auto bar = [&](int stage) -> uint32_t { return sb + Sh::kOffBar + 8u * (uint32_t)(kg * ST + stage); };

  // ---- set-up that touches no global memory ----
  static_assert(kPaThreads >= kMaxN, "an entry a thread");
  if (t < kMaxN) s_tree_lv[t] = 0.f;  // (entries past the tree's rows are read, for keys that are masked)
  if (t == 0) {
    s_abort = 0;
    for (int i = 0; i < KG * ST; ++i) mbar_init(sb + Sh::kOffBar + 8u * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  pdl_wait();     // the previous kernel in the stream has completed
  pdl_trigger();  // only now may the next kernel launch
  const int g = blockIdx.y / ma.row_tiles, rt = blockIdx.y - g * ma.row_tiles;
  // chunks are as long in every sequence: the length that shares the batch among the grid's blocks, or the longest
  // sequence's share
  int b = blockIdx.z, chunk = blockIdx.x, per, chunks, bad = 0;
  long long slot0 = ((long long)b * ma.tiles_y + blockIdx.y) * ma.S;  // of the sequence's first chunk, in the workspace
  if (ma.flat) {
    const Share share = share_batch(a, lane, gridDim.x, blockIdx.x);
    if (share.b < 0) return;
    b = share.b;
    chunk = share.chunk;
    per = share.per;
    chunks = share.chunks;
    slot0 = (long long)blockIdx.y * gridDim.x + blockIdx.x - chunk;
  }
  const int L = paged_prefix(a, b, bad);
  if (!ma.flat) {
    int longest = L;
    if (a.B > 1) {
      int other = 0;
      if (a.B <= kPaThreads) {
        int ignore = 0;
        if (t < a.B) other = paged_prefix(a, t, ignore);
      } else {
        other = min((long long)a.max_prefix, (long long)a.max_blocks * a.P);
      }
      other = __reduce_max_sync(0xffffffffu, other);
      if (lane == 0) s_red[warp] = other;
      __syncthreads();
      longest = max(max(s_red[0], s_red[1]), max(s_red[2], s_red[3]));
    }
    if (L < 0) return;
    per = max((tiles_of(longest, kPaTile) + ma.S - 1) / ma.S, 1);
    chunks = max(1, (tiles_of(L, kPaTile) + per - 1) / per);
    if (chunk >= chunks) return;
  }
  __syncthreads();  // the barriers are initialised
  const int T = tiles_of(L, kPaTile);
  const int t0 = chunk * per, t1 = min(T, t0 + per);
  const int first = t0 + kg;  // this group's i-th tile: first + KG * i
  const int n = t1 > first ? (t1 - first + KG - 1) / KG : 0;

  // ---- units of 16 keys, two per tile: lane l holds unit l of a batch of 16 tiles ----
  int page = -1, slot = 0, page_n = -1, slot_n = 0;
  float ksc = 0.f, vsc = 1.f, ksc_n = 0.f, vsc_n = 1.f;
  auto fetch_page = [&](int batch, int &pg, int &sl) {
    const int i = 16 * batch + (lane >> 1);
    const long long key = (long long)(first + (long long)KG * i) * kPaTile + 16 * (lane & 1);
    pg = sl = -1;
    if (i < n && key < L) {
      const int blk = page_index(ma, (int)key);
      sl = (int)key - blk * a.P;
      pg = a.block_table[(long long)b * a.max_blocks + blk];
    }
  };
  auto check_page = [&](int &pg, int sl) {  // apart from the load, which it would wait for
    if (pg >= 0 && pg < a.num_pages) return;
    if (sl >= 0) bad = 1;
    pg = -1;
  };
  auto fetch_scale = [&](int pg, float &ks, float &vs) {
    ks = 0.f;
    vs = 1.f;
    if (pg >= 0) {
      ks = a.k_scale[(long long)pg * a.Hkv + g];
      vs = clamp_v_scale(a.v_scale[(long long)pg * a.Hkv + g]);
    }
  };
  // the group's i-th tile into its stage (the whole warp wr == 0 calls it); pg, sl: the batch that holds it
  auto issue = [&](int i, int pg, int sl) {
    const int u = 2 * (i & 15);
    const int p0 = __shfl_sync(0xffffffffu, pg, u), p1 = __shfl_sync(0xffffffffu, pg, u + 1);
    const int s0 = __shfl_sync(0xffffffffu, sl, u), s1 = __shfl_sync(0xffffffffu, sl, u + 1);
    if (lane != 0) return;
    const int stage = i % ST;
    const uint32_t kd = sb + (uint32_t)((kg * ST + stage) * 2 * TB), vd = kd + TB, fb = bar(stage);
    if (ma.box == kPaTile) {  // both units in one page
      if (p0 >= 0) {
        mbar_expect_tx(fb, 2 * TB);
        tma_4d(kd, &tm_k, 0, s0, g, p0, fb);
        tma_4d(vd, &tm_v, 0, s0, g, p0, fb);
      } else {
        mbar_arrive(fb);
      }
    } else {
      const int boxes = (p0 >= 0 ? 1 : 0) + (p1 >= 0 ? 1 : 0);
      if (boxes == 0) {
        mbar_arrive(fb);
      } else {
        mbar_expect_tx(fb, (uint32_t)(boxes * TB));
        if (p0 >= 0) {
          tma_4d(kd, &tm_k, 0, s0, g, p0, fb);
          tma_4d(vd, &tm_v, 0, s0, g, p0, fb);
        }
        if (p1 >= 0) {
          tma_4d(kd + TB / 2, &tm_k, 0, s1, g, p1, fb);
          tma_4d(vd + TB / 2, &tm_v, 0, s1, g, p1, fb);
        }
      }
    }
  };
  fetch_page(0, page, slot);
  check_page(page, slot);
  if (wr == 0)
    for (int i = 0; i < n && i < ST; ++i) issue(i, page, slot);

  // ---- q into fragment order: D / 8 lanes per row, eight dims a lane ----
  float *row_f = reinterpret_cast<float *>(sm + Sh::kOffRow);
  {
    constexpr int LR = D / 8, RW = 32 / LR;       // lanes per row, rows a warp takes at once
    constexpr int QR = R / (kPaWarps * RW);       // rounds
    const int lr = lane % LR, sub = lane / LR;
    // the tree's V once over, for its rows' scales (its products read it again, out of L1)
    const int r_tree = warp * RW + sub;
    auto tree_cell = [&](int r) {
      return r < a.N && chunk == 0 ? *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.vt) +
                                                                      (((long long)b * a.N + r) * a.Hkv + g) * D + 8 * lr)
                                   : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 tree_v = tree_cell(r_tree);
    uint4 raw[QR];
#pragma unroll
    for (int k = 0; k < QR; ++k) {
      const int r = (warp + kPaWarps * k) * RW + sub, Rg = rt * R + r, i = row_token(ma, Rg);
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i < a.N)
        raw[k] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                  (((long long)b * a.N + i) * a.Hq + g * a.G + (Rg - i * a.G)) * D +
                                                  8 * lr);
    }
    fetch_scale(page, ksc, vsc);  // in flight while q is staged
    for (int r = r_tree; r - sub < a.N && chunk == 0; r += kPaWarps * RW) {  // whole warps
      const uint32_t w[4] = {tree_v.x, tree_v.y, tree_v.z, tree_v.w};
      tree_v = tree_cell(r + kPaWarps * RW);
      uint32_t top = 0u;  // largest finite magnitudes of the low and of the high halves
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7fffu, hi = w[e] & 0x7fff0000u;
        top = __vmaxu2(top, (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f800000u ? hi : 0u));
      }
      top = max(top << 16, top & 0xffff0000u);
#pragma unroll
      for (int x = 1; x < LR; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      if (lr == 0) s_tree_lv[r] = (float)page_exponent<FMT>(__uint_as_float(top));
    }
#pragma unroll
    for (int k = 0; k < QR; ++k) {
      const int r = (warp + kPaWarps * k) * RW + sub, mt = r >> 4, up = (r >> 3) & 1, r8 = r & 7;
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      uint32_t top = 0u;  // the row's largest magnitude, as the bits of a bf16 value: they order like the values
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
      for (int x = 1; x < LR; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      const bool odd = top >= 0x7f80u;  // NaN or infinity
      // 2^e2 lifts the largest magnitude into [2^14, 2^15); e2 may leave fp32's exponents, half of it cannot
      const int e2 = top == 0u || odd ? 0 : 141 - max((int)(top >> 7), 1);
      const int ea = e2 >> 1, eb = e2 - ea;
      const float lift_a = __uint_as_float((uint32_t)(127 + ea) << 23), lift_b = __uint_as_float((uint32_t)(127 + eb) << 23);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // thread (g, t) of a k-step holds dims (D / 4) t + 4 ks + {0, 1} and + {2, 3} of rows g and g + 8
        const int d = 8 * lr + 4 * half, tt = d / (D / 4), ks = (d % (D / 4)) / 4;
        const uint32_t at = (uint32_t)((((mt * K16 + ks) * 32) + 4 * r8 + tt) * 16 + up * 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t v = w[2 * half + e];
          *reinterpret_cast<uint32_t *>(sm + Sh::kOffQ + at + 8 * e) =
              pack_f16x2(__uint_as_float(v << 16) * lift_a * lift_b, __uint_as_float(v & 0xffff0000u) * lift_a * lift_b);
          if (chunk == 0) *reinterpret_cast<uint32_t *>(sm + Sh::kOffQ16 + at + 8 * e) = v;  // for the tree's rows
        }
      }
      // what a score of lifted q and codes stands for, in log2 units; a row that is not finite scores NaN
      if (lr == 0)
        row_f[r] = odd ? __uint_as_float(0x7fc00000u)
                       : a.scale_log2 * __uint_as_float((uint32_t)(127 - ea) << 23) * __uint_as_float((uint32_t)(127 - eb) << 23);
    }
  }
  __syncthreads();

  float rf[2 * MT], mr[2 * MT], l[2 * MT];
  int tok[2 * MT];
#pragma unroll
  for (int r = 0; r < 2 * MT; ++r) {
    const int row = wr * 16 * MT + 16 * (r >> 1) + 8 * (r & 1) + g8;
    rf[r] = row_f[row];
    tok[r] = row_token(ma, rt * R + row);  // >= N: no such row
    mr[r] = -3e38f;
    l[r] = 0.f;
  }
  float o[MT][NTO][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NTO; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;

  // ---- the tree's own rows, 16 keys at a time, while the first tiles arrive ----
  if (chunk == 0) {
    const __nv_bfloat16 *KT = static_cast<const __nv_bfloat16 *>(a.kt), *VT = static_cast<const __nv_bfloat16 *>(a.vt);
    for (int tc = kg; 16 * tc < a.N; tc += KG) {
      uint32_t keep[2 * MT];
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) {
        const int i = tok[r];
        uint32_t w = 0u;
        if (i < a.N) {
          if (a.mask) w = (uint32_t)(a.mask[((long long)b * a.N + i) * a.W + (tc >> 2)] >> (16 * (tc & 3))) & 0xffffu;
          else w = i >= 16 * tc + 15 ? 0xffffu : (i < 16 * tc ? 0u : (2u << (i - 16 * tc)) - 1u);
        }
        if (16 * tc + 16 > a.N) w &= (1u << (a.N - 16 * tc)) - 1u;
        keep[r] = w;
      }
      uint32_t kw[2][D / 8];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int key = 16 * tc + 8 * nt + g8;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (key < a.N)
            v = *reinterpret_cast<const uint4 *>(KT + (((long long)b * a.N + key) * a.Hkv + g) * D + (D / 4) * tq + 8 * c);
          kw[nt][4 * c] = v.x; kw[nt][4 * c + 1] = v.y; kw[nt][4 * c + 2] = v.z; kw[nt][4 * c + 3] = v.w;
        }
      }
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < K16; ++ks)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 q = lds128(sb + Sh::kOffQ16 + (uint32_t)((((wr * MT + mt) * K16 + ks) * 32 + lane) * 16));
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma_16<true>(s[mt][nt], q.x, q.y, q.z, q.w, kw[nt][2 * ks], kw[nt][2 * ks + 1]);
        }
      float fs[2 * MT];
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) fs[r] = rf[r] == rf[r] ? a.scale_log2 : rf[r];  // NaN: q is not finite
      const float one[1] = {1.f};
      float lvt[4], ivt[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lvt[k] = s_tree_lv[16 * tc + 2 * tq + 8 * (k >> 1) + (k & 1)];
        ivt[k] = power_of_two(-(int)lvt[k]);
      }
      uint32_t p[MT][2][2];
      paged_softmax<2, MT, NTO, true>(s, fs, one, lvt, ivt, true, keep, mr, l, o, p);
      bool odd = false;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {  // 8 of the thread's dims at a time
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 16 * tc + 2 * tq + (k & 1) + 8 * (k >> 1);
          v[k] = make_uint4(0u, 0u, 0u, 0u);
          if (key < a.N)
            v[k] = *reinterpret_cast<const uint4 *>(VT + (((long long)b * a.N + key) * a.Hkv + g) * D + (D / 8) * g8 + 8 * c);
        }
        uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                            {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
        // NaN and infinities would reach rows that do not attend their key (0 * inf): they are added by hand below
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((w[k][e] & 0x7f80u) == 0x7f80u) { w[k][e] &= 0xffff0000u; odd = true; }
            if ((w[k][e] & 0x7f800000u) == 0x7f800000u) { w[k][e] &= 0xffffu; odd = true; }
          }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(w[0][e >> 1], w[1][e >> 1], sel), b1 = __byte_perm(w[2][e >> 1], w[3][e >> 1], sel);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            mma_16<true>(o[mt][8 * c + e], p[mt][0][0], p[mt][0][1], p[mt][1][0], p[mt][1][1], b0, b1);
        }
      }
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
        for (int k = 0; k < 16 && 16 * tc + k < a.N; ++k) {
          const __nv_bfloat16 *vr = VT + (((long long)b * a.N + 16 * tc + k) * a.Hkv + g) * D + (D / 4) * tq;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int nt = 0; nt < NTO; ++nt) {
              const float x = __bfloat162float(vr[(D / 8) * half + nt]);
              if (fabsf(x) <= FLT_MAX) continue;
#pragma unroll
              for (int r = 0; r < 2 * MT; ++r)
                if ((keep[r] >> k) & 1u) o[r >> 1][nt][2 * (r & 1) + half] += x;
            }
        }
      }
    }
  }

  // ---- the cached keys ----
  bool dead = false;  // a wait gave up: go on without waiting, computing or fetching, in step with the partner warp
  int issued = n < ST ? n : ST;
  for (int i = 0; i < n; ++i) {
    if ((i & 15) == 0) {
      if (i > 0) {
        page = page_n; slot = slot_n; ksc = ksc_n; vsc = vsc_n;
      }
      fetch_page((i >> 4) + 1, page_n, slot_n);
    } else if ((i & 15) == 1) {
      check_page(page_n, slot_n);
      fetch_scale(page_n, ksc_n, vsc_n);
    }
    const int stage = i % ST;
    if (!dead && !mbar_try(bar(stage), (uint32_t)(i / ST) & 1u))
      dead = !mbar_wait(bar(stage), (uint32_t)(i / ST) & 1u, &s_abort, ma.wait_cycles);
    dead = __any_sync(0xffffffffu, dead);
    if (!dead) {
      const int u = 2 * (i & 15), key0 = (first + KG * i) * kPaTile;
      float ks[2], vs[2], lv[2], iv[2];
      bool there[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ks[h] = __shfl_sync(0xffffffffu, ksc, u + h);
        vs[h] = __shfl_sync(0xffffffffu, vsc, u + h);
        there[h] = __shfl_sync(0xffffffffu, page, u + h) >= 0;
        lv[h] = __log2f(vs[h]);
        iv[h] = __frcp_rn(vs[h]);
      }
      const bool whole = there[0] && there[1] && L - key0 >= kPaTile;
      uint32_t valid = 0xffffffffu;  // bit k: key key0 + k is there
      if (!whole) {
        valid = L - key0 >= kPaTile ? 0xffffffffu : (1u << (L - key0)) - 1u;
        if (!there[0]) valid &= 0xffff0000u;
        if (!there[1]) valid &= 0x0000ffffu;
      }
      const uint32_t kb = sb + (uint32_t)((kg * ST + stage) * 2 * TB), vb = kb + TB;
      // S = q K^T: a thread's 32 (16) bytes of a key row are one word a k-step
      float s[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
      uint4 kw[4][D / 64];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const uint32_t row = kb + (uint32_t)((8 * nt + g8) * D);
        if (D == 128) {
          kw[nt][0] = lds128(row + (uint32_t)(((2 * tq) ^ g8) << 4));
          kw[nt][D / 64 - 1] = lds128(row + (uint32_t)(((2 * tq + 1) ^ g8) << 4));
        } else {
          kw[nt][0] = lds128(row + (uint32_t)((tq ^ ((g8 >> 1) & 3)) << 4));
        }
      }
#pragma unroll
      for (int k = 0; k < K16; ++k) {
        uint32_t b0[4], b1[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint4 x = kw[nt][k >> 2];
          f8x4_to_f16<FMT>((k & 3) == 0 ? x.x : (k & 3) == 1 ? x.y : (k & 3) == 2 ? x.z : x.w, b0[nt], b1[nt]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 q = lds128(sb + Sh::kOffQ + (uint32_t)((((wr * MT + mt) * K16 + k) * 32 + lane) * 16));
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) mma_16<false>(s[mt][nt], q.x, q.y, q.z, q.w, b0[nt], b1[nt]);
        }
      }
      uint32_t keep[2 * MT];
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) keep[r] = valid;
      uint32_t p[MT][4][2];
      if (whole) paged_softmax<4, MT, NTO, false>(s, rf, ks, lv, iv, false, keep, mr, l, o, p);
      else paged_softmax<4, MT, NTO, false>(s, rf, ks, lv, iv, true, keep, mr, l, o, p);
      // O += P V: the bytes of two keys at one dim become a pair of fp16
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t w[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 16 * j + 2 * tq + (k & 1) + 8 * (k >> 1);
          const uint32_t row = vb + (uint32_t)(key * D);
          if (D == 128) {
            const uint4 v = lds128(row + (uint32_t)((g8 ^ (key & 7)) << 4));
            w[k][0] = v.x; w[k][1] = v.y; w[k][D / 32 - 2] = v.z; w[k][D / 32 - 1] = v.w;
          } else {
            const uint2 v = lds64(row + (uint32_t)((((g8 >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (g8 & 1)));
            w[k][0] = v.x; w[k][1] = v.y;
          }
          if (!whole && !((valid >> key) & 1u)) {  // whatever the page holds there must not meet a zero weight
#pragma unroll
            for (int c = 0; c < D / 32; ++c) w[k][c] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t b0[4], b1[4];
          f8x4_to_f16<FMT>(__byte_perm(w[0][c], w[1][c], 0x5140), b0[0], b0[1]);
          f8x4_to_f16<FMT>(__byte_perm(w[0][c], w[1][c], 0x7362), b0[2], b0[3]);
          f8x4_to_f16<FMT>(__byte_perm(w[2][c], w[3][c], 0x5140), b1[0], b1[1]);
          f8x4_to_f16<FMT>(__byte_perm(w[2][c], w[3][c], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma_16<false>(o[mt][4 * c + e], p[mt][2 * j][0], p[mt][2 * j][1], p[mt][2 * j + 1][0],
                            p[mt][2 * j + 1][1], b0[e], b1[e]);
        }
      }
    }
    // the stage is free once both warps of the group have read it
    if (WR == 2) asm volatile("bar.sync %0, 64;" ::"r"(1 + kg) : "memory");
    else __syncwarp();
    if (wr == 0 && !dead && i + ST < n) {
      const bool later = ((i + ST) >> 4) != (i >> 4);
      issue(i + ST, later ? page_n : page, later ? slot_n : slot);
      issued = i + ST + 1;
    }
  }
  if (dead && wr == 0 && lane == 0)  // copies still in flight land before the block reuses or leaves its memory
    for (int i = issued > ST ? issued - ST : 0; i < issued; ++i) mbar_drain(bar(i % ST), (uint32_t)(i / ST) & 1u);
  if (bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
  __syncthreads();
  const bool aborted = *(volatile int *)&s_abort != 0;
  if (aborted && t == 0) flag_status(a.dev_status, ET_DEV_TIMEOUT);

  // ---- the groups' rows, merged through shared memory ----
  float4 *rows = reinterpret_cast<float4 *>(sm);                       // [KG][R][D / 4]
  float2 *ml = reinterpret_cast<float2 *>(sm + KG * R * D * 4);        // [KG][R]
#pragma unroll
  for (int r = 0; r < 2 * MT; ++r) {
    const int mt = r >> 1, h = r & 1, row = wr * 16 * MT + 16 * mt + 8 * h + g8;
    float sum = l[r];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (tq == 0) ml[kg * R + row] = make_float2(mr[r], sum);
#pragma unroll
    for (int half = 0; half < 2; ++half)  // column 2 tq + half of n-tile nt is dim (D / 8) (2 tq + half) + nt
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        rows[(kg * R + row) * (D / 4) + merge_chunk<D>(row, (D / 16) * tq + (D / 32) * half + c)] =
            make_float4(o[mt][4 * c][2 * h + half], o[mt][4 * c + 1][2 * h + half], o[mt][4 * c + 2][2 * h + half],
                        o[mt][4 * c + 3][2 * h + half]);
  }
  __syncthreads();
  const int real = min(R, a.N * a.G - rt * R);  // rows that exist are a prefix of the tile
  const long long tile_id = (long long)b * ma.tiles_y + blockIdx.y;
  const bool cluster = ma.cnt == nullptr;
  auto write_row = [&](int r, int c, const float4 &v, float M, float sum) {
    const int Rg = rt * R + r, i = row_token(ma, Rg), h = g * a.G + (Rg - i * a.G);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2 w;
    w.x = pack_bf16x2(v.x * inv, v.y * inv);
    w.y = pack_bf16x2(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + (((long long)b * a.N + i) * a.Hq + h) * D + 4 * c) = w;
    if (c == 0 && a.lse)
      a.lse[((long long)b * a.Hq + h) * a.N + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
  };
  for (int x = t; x < real * (D / 4); x += kPaThreads) {
    const int r = x / (D / 4), c = x - r * (D / 4);
    float M = ml[r].x;
#pragma unroll
    for (int k = 1; k < KG; ++k) M = fmaxf(M, ml[k * R + r].x);
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const float2 e = ml[k * R + r];
      const float w = ex2_fast(e.x - M);
      const float4 y = rows[(k * R + r) * (D / 4) + merge_chunk<D>(r, c)];
      sum = fmaf(e.y, w, sum);
      v.x = fmaf(y.x, w, v.x); v.y = fmaf(y.y, w, v.y); v.z = fmaf(y.z, w, v.z); v.w = fmaf(y.w, w, v.w);
    }
    if (chunks == 1) {
      write_row(r, c, v, M, sum);
    } else if (cluster) {  // for the cluster to read: a cell where only this thread read one
      rows[r * (D / 4) + merge_chunk<D>(r, c)] = v;
      if (c == 0) ml[KG * R + r] = make_float2(M, sum);
    } else {
      const long long at = (slot0 + chunk) * R + r;
      ma.part_o[at * (D / 4) + c] = v;
      if (c == 0) ma.part_ml[at] = make_float2(M, sum);
    }
  }
  if (chunks == 1) return;
  if (cluster) {
    // ---- the chunks' rows, each merged by one of the cluster's blocks ----
    // (blocks without keys have left: the barrier counts the others)
    __syncwarp();
    cl_sync();
    for (int x = t; x < (real - chunk + chunks - 1) / chunks * (D / 4); x += kPaThreads) {
      const int r = chunk + x / (D / 4) * chunks, c = x % (D / 4);
      float4 y[kPaMaxCluster];
      float2 e[kPaMaxCluster];
#pragma unroll
      for (int k = 0; k < kPaMaxCluster; ++k) {  // every load in flight before any arithmetic
        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        e[k] = make_float2(-3e38f, 0.f);
        if (k < chunks) {
          y[k] = cl_ld_f32x4(cl_map(&rows[r * (D / 4) + merge_chunk<D>(r, c)], (uint32_t)k));
          const uint32_t at = cl_map(&ml[KG * R + r], (uint32_t)k);
          e[k] = make_float2(cl_ld_f32(at), cl_ld_f32(at + 4u));
        }
      }
      float M = e[0].x, sum = 0.f;
#pragma unroll
      for (int k = 1; k < kPaMaxCluster; ++k) M = fmaxf(M, e[k].x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPaMaxCluster; ++k) {
        const float w = ex2_fast(e[k].x - M);
        sum = fmaf(e[k].y, w, sum);
        v.x = fmaf(y[k].x, w, v.x); v.y = fmaf(y[k].y, w, v.y); v.z = fmaf(y[k].z, w, v.z); v.w = fmaf(y[k].w, w, v.w);
      }
      write_row(r, c, v, M, sum);
    }
    __syncwarp();
    cl_sync();  // no block leaves while another reads its rows
    return;
  }
  // ---- the chunks' rows, merged by the last block to arrive ----
  if (!arrive_last(ma.cnt + tile_id, (unsigned)chunks, &s_last)) return;
  merge_chunks<D, R, kPaThreads>(ma, slot0, chunks, real, sm, write_row);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <int D, int FMT, int WR, int MT>
et_status launch_mma(const CUtensorMap &mk, const CUtensorMap &mv, const PagedSplitArgs &ma, cudaStream_t st) {
  using Sh = PaShape<D, WR, MT>;
  if (et_smem_attr((const void *)k_paged_attn_mma<D, FMT, WR, MT>, Sh::kBytes) != cudaSuccess) return ET_ERR_CUDA;
  const dim3 grid = ma.flat ? dim3(ma.flat, ma.tiles_y) : dim3(ma.S, ma.tiles_y, ma.a.B);
  return et_launch(k_paged_attn_mma<D, FMT, WR, MT>, grid, dim3(kPaThreads), Sh::kBytes, st,
                   ma.cnt || ma.S == 1 ? 0 : ma.S, mk, mv, ma);
}
template <int D, int FMT>
et_status launch_mma_rows(int R, const CUtensorMap &mk, const CUtensorMap &mv, const PagedSplitArgs &ma, cudaStream_t st) {
  if constexpr (D == 64) {  // with d = 128 more rows go to the tcgen05 kernel
    if (R == 32) return launch_mma<D, FMT, 1, 2>(mk, mv, ma, st);
    if (R == 64) return launch_mma<D, FMT, 2, 2>(mk, mv, ma, st);
  }
  return launch_mma<D, FMT, 1, 1>(mk, mv, ma, st);
}

struct PagedPlan {
  int S;      // blocks a sequence's keys are split over (with flat: at most)
  int flat;   // blocks per tile of rows that share the batch, 0: S of each sequence
  int R;      // query rows per block
  int row_tiles;
  bool tc;    // tcgen05 kernel (bf16, d = 128, more than 16 rows per KV head), else mma.sync
  size_t ws;  // workspace bytes: counters, (maximum, sum) pairs, partial rows
  size_t ml_off, o_off;
};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    n = 152;
  cudaGetLastError();
  return n;
}

long long least(long long a, long long b) { return a < b ? a : b; }

// Chunks of the tcgen05 kernel, one block per SM.  A block costs about ten of its 128-key tiles before its first and
// after its last (measured: 11 against 1.0 us), a merge about three in a cluster and eight through the workspace.  One
// sequence: whole waves of equal blocks.  Several, of any length up to T: the work of half the bound over all SMs, and
// half of the longest block at the end.
int tc_splits(long long tiles, int T, int B) {
  constexpr double kBlock = 10;
  const int sms = sm_count();
  int best = 1;
  double least = 1e30;
  for (int S = 1; S <= kPaMaxSplits && S <= T; ++S) {
    const bool cluster = S > 1 && S <= kPaMaxCluster;
    const long long together = cluster ? paged_tc_clusters(S, sms) : sms, units = cluster ? tiles : tiles * S;
    const double chunk = (T + S - 1) / S, merge = cluster ? 3 : S > 1 ? 8 : 0;
    const double cost = B == 1 ? (double)((units + together - 1) / together) * (kBlock + chunk + merge)
                               : (double)tiles * (S * (kBlock + merge) + 0.5 * T) / sms + 0.5 * (kBlock + chunk + merge);
    if (cost < least) {
      least = cost;
      best = S;
    }
  }
  return best;
}

et_status make_plan(const et_paged_attn_shape *s, const et_paged_cache *c, PagedPlan *p) {
  if (!s) return ET_ERR_INVALID_ARG;
  const et_status cs = paged_cache_status(c);
  if (cs != ET_OK) return cs;
  if (s->B < 1 || s->N < 1 || s->N > kMaxN || s->Hq < 1 || s->Hq % c->Hkv || s->max_blocks < 1 || s->max_prefix < 0 ||
      s->num_splits < 0 || !(s->scale > 0.f) || (s->dtype != ET_BF16 && s->dtype != ET_F32))
    return ET_ERR_INVALID_ARG;
  if (s->B > 65535 || s->Hq > 65535 || (long long)s->max_blocks * c->page_size >= (1ll << 31)) return ET_ERR_UNSUPPORTED;
  p->S = 1;
  p->ws = p->ml_off = p->o_off = 0;
  p->R = p->row_tiles = 1;
  p->tc = false;
  p->flat = 0;
  if (s->dtype == ET_F32) return ET_OK;
  const long long rows = (long long)s->N * (s->Hq / c->Hkv);
  // mma.sync and tcgen05 from a graph, 16 rows and 24 (two of mma.sync's row tiles): 16 sequences of 8880 tokens, 8 KV
  // heads: 57.3 and 87.4 us, 99.6 and 88.3; one of 8192: 16.9 and 17.8, 20.0 and 18.1; 8 of 4096, 32 KV heads: 24 rows
  // 96.4 and 80.5.  One of 1024, 32 KV heads, is the exception: 24 rows 11.6 and 12.9, 32 rows 11.8 and 13.1
  p->tc = c->d == 128 && rows > 16;
  p->R = rows <= 16 ? 16 : rows <= 32 && !p->tc ? 32 : 64;
  p->row_tiles = (int)((rows + p->R - 1) / p->R);
  const long long tiles = (long long)s->B * c->Hkv * p->row_tiles;
  if ((long long)c->Hkv * p->row_tiles > 65535) return ET_ERR_UNSUPPORTED;
  const long long room = (long long)s->max_blocks * c->page_size;
  const int tile = p->tc ? kPtKeys : kPaTile;
  const int T = (int)(((s->max_prefix < room ? s->max_prefix : room) + tile - 1) / tile);
  int S = s->num_splits;
  if (S <= 0) {
    if (p->tc) {
      S = tc_splits(tiles, T, s->B);
    } else if (s->B == 1) {
      // one block per SM, of eight 32-key tiles at least (8 KV heads, prefix 16384: 20.7 us in 19 chunks, 21.9 in 38)
      S = (int)least(sm_count() / tiles, T / 8);
    } else {
      // Where one wave of blocks gives every sequence three chunks, the lengths themselves share it out (8 KV heads,
      // 16 sequences: of 512..16384 tokens 59.4 us, 65.1 in 16 chunks each; of 8880 each 59.4, 58.2 in 3 chunks each,
      // 73.2 in 16).  Short ones (4 of 1024: 16.0 us against 14.4) and larger batches take chunks of the longest's
      // share: a wave of eight tiles at least, or many waves of long chunks (32 KV heads: 16 sequences of up to 8192
      // 110.7 us in 4 chunks, 113.3 in one; 32 of up to 2048 61 in one, 71 in two, 107 shared out by length).
      const long long slots = (p->R <= 16 ? 3ll : 2ll) * sm_count() / (tiles / s->B);  // blocks per tile of rows at once
      const long long wave = least(3ll * sm_count() / tiles, T / 8), waves = least(14ll * sm_count() / tiles, T / 64);
      S = (int)(waves >= 2 * wave ? waves : wave);
      if (s->B <= 32 && slots >= 3 * s->B && T >= 8 * kPaLeast) {
        p->flat = (int)slots;
        S = (int)least(slots - s->B + 1, T / kPaLeast);
      }
    }
  }
  if (S > T) S = T;
  if (S > kPaMaxSplits) S = kPaMaxSplits;
  if (S < 1) S = 1;
  // one sequence's blocks merge as a cluster where they can (32 KV heads, prefix 1023, side by side: 8.4 us in a graph,
  // 10.0 through the workspace); a batch's blocks of few rows do not, its short sequences leave clusters half empty (32
  // KV heads, 16 sequences of up to 8192: 131 us, 110 through the workspace).  Of the tcgen05 kernel's blocks an SM holds
  // one, so few wait (32 KV heads, 2 sequences of up to 16384: 68.3 us, 71.2 through the workspace)
  const bool cluster = S > 1 && S <= kPaMaxCluster && (p->tc || s->B == 1);
  if (tiles > kPaCounters && !cluster) S = 1;  // far more blocks than SMs as it is
  if (S == 1) p->flat = 0;
  p->S = S;
  if (S > 1 && !cluster) {
    const size_t parts = p->flat ? (size_t)(tiles / s->B) * p->flat : (size_t)tiles * S;
    const size_t cnt = kPaCounters * sizeof(unsigned int);
    const size_t ml = (parts * p->R * sizeof(float2) + 255) & ~(size_t)255;
    p->ml_off = cnt;
    p->o_off = cnt + ml;
    p->ws = cnt + ml + parts * p->R * c->d * sizeof(float);
  }
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
    return e4m3 ? launch_row<ET_KV_E4M3>(a, cache->d, st) : launch_row<ET_KV_E5M2>(a, cache->d, st);
  if (!encode_fn()) return ET_ERR_CUDA;
  PagedSplitArgs ma;
  ma.a = a;
  ma.S = plan.S;
  ma.flat = plan.flat;
  ma.row_tiles = plan.row_tiles;
  ma.tiles_y = cache->Hkv * plan.row_tiles;
  ma.box = cache->page_size % kPaTile == 0 ? kPaTile : 16;
  unsigned char *wsb = static_cast<unsigned char *>(ws);
  ma.cnt = plan.ws > 0 ? reinterpret_cast<unsigned int *>(wsb) : nullptr;
  ma.part_ml = plan.ws > 0 ? reinterpret_cast<float2 *>(wsb + plan.ml_off) : nullptr;
  ma.part_o = plan.ws > 0 ? reinterpret_cast<float4 *>(wsb + plan.o_off) : nullptr;
  const uint32_t units = (uint32_t)cache->page_size / 16;
  ma.page_magic = units == 1 ? 0u : (uint32_t)(((1ull << 32) + units - 1) / units);
  ma.group_shift = 0;
  while ((2ll << ma.group_shift) < a.G) ++ma.group_shift;
  ma.group_magic = a.G == 1 ? 0u : (uint32_t)(((1ull << (32 + ma.group_shift)) + a.G - 1) / a.G);
  ma.wait_cycles = et_wait_limit_cycles();
  if (plan.tc) return paged_tc_launch(cache, ma, st);
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, cache->k_pages, cache, ma.box) || !make_page_map(&mv, cache->v_pages, cache, ma.box))
    return ET_ERR_INVALID_ARG;
  if (cache->d == 64)
    return e4m3 ? launch_mma_rows<64, ET_KV_E4M3>(plan.R, mk, mv, ma, st)
                : launch_mma_rows<64, ET_KV_E5M2>(plan.R, mk, mv, ma, st);
  return e4m3 ? launch_mma_rows<128, ET_KV_E4M3>(plan.R, mk, mv, ma, st)
              : launch_mma_rows<128, ET_KV_E5M2>(plan.R, mk, mv, ma, st);
}
