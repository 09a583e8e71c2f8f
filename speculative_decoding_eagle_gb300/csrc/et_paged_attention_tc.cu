// Paged 8-bit attention on the 5th-generation tensor cores (tcgen05): the many
// rows of a draft tree (EAGLE-2 article, attention-mask paragraph) against a
// cache whose codes go to the tensor cores as they lie in the page.  D = 128.
//
// Everything is transposed: keys are the rows of the products, query rows
// their columns.
//   S^T [128 keys x 64 rows] = K8 . Q8^T   (kind::f8f6f4; K's codes by TMA, q
//        lifted by a power of two per row and split into two e4m3 terms, two
//        products into one sum)
//   O^T [128 dims x 64 rows] += V16^T . P^T (kind::f16; V's codes as fp16)
// A tree of up to 64 rows per KV head (every MHA tree) then fills the 128
// lanes of tensor memory with keys instead of padding them with rows that do
// not exist; the softmax runs one key per thread, and a tile of a page's
// codes needs no conversion before the scores.
//
// One block per SM, nineteen warps:
//   warps 0-7, 8-15  two softmax groups on alternate tiles, each with its own
//               weights, running maximum and O in TMEM: independent online
//               softmaxes, joined at the end.  A thread has one key and half
//               of the rows.  The group also turns its tile's V codes into
//               fp16, before its scores arrive
//   warp 16     TMA: a 128-key tile of K and of V, into rings of 2 (the 32 KB
//               of a third stage hold a third V16 buffer: 327 us against 334
//               for the 16 sequences below).  It also publishes the tile's scales,
//               so that no softmax thread looks a page up (331 against 305 us)
//   warp 17     owns 512 columns of TMEM, issues the score products
//   warp 18     issues the P.V products.  A thread that issues waits for its
//               products to be taken (measured: 71 cycles an fp16 product of
//               up to 128 columns, 47 an 8-bit one of 64), so one warp for
//               both spent more time polling between them than computing
// A weight's reference moves only when some weight would pass 2^15 (one vote
// of the group in place of a maximum over the lanes); the slow path finds the
// maxima, and rescales the group's sums and O.  The tree's own rows are one
// more tile in bf16, staged by all warps before the roles part.
// Up to eight chunks of a sequence form a cluster and merge through its shared
// memory (7B heads, prefix 1024, side by side when it was chosen: 16.0 us, 18.9
// through the workspace; 14.3 now); more go through the workspace, and the last
// block merges them.
//
// Measured: 32 heads, N = 61, 16 sequences of 512..16384 tokens: 304 us, 3.9
// TB/s of codes and 466 TFLOP/s, 1.7 times what the bytes take.  A tile costs
// 1.1 us with every SM at work (0.73 for its bytes).  What bounds it is the
// softmax warps' chain of instructions and of waits (issue slots 66% taken in
// the busiest SM, half of its ALU's cycles, tensor pipe 24%, shared memory 0.5
// wavefronts a cycle); a block spends about 10 us before its first and after its last
// tile, which is most of the time of one short sequence.  Every mbarrier wait is bounded: a block that gives up
// sets ET_DEV_TIMEOUT, drains what it issued and leaves.
#include <atomic>
#include <type_traits>

#include "et_paged_attn.cuh"

namespace et {
namespace {

constexpr int kPtThreads = 608;
constexpr int kPtGroup = 256;   // threads of a softmax group
constexpr int kPtQ = kPtRows / 2;  // rows per softmax thread
constexpr int kPtD = 128;
constexpr int kPtStages = 2;
constexpr int kPtVBuf = 3;  // V16 buffers: one more than groups, so that a conversion waits for no product of its group
constexpr int kPtTmaWarp = 16, kPtScoreWarp = 17, kPtPvWarp = 18;
constexpr uint32_t kPtTile8 = kPtKeys * kPtD;            // 16 KB: K8 or V8
constexpr uint32_t kPtTile16 = 2 * kPtTile8;             // 32 KB: V16, two halves of 64 dims
constexpr uint32_t kPtHalf16 = kPtKeys * 128;            // 16 KB
constexpr uint32_t kPtP = kPtKeys * kPtRows * 2;         // 16 KB
constexpr uint32_t kPtOffQ = 0;                          // Q8: 64 rows hi, 64 rows lo, 128 bytes each
constexpr uint32_t kPtOffK = kPtOffQ + 2 * kPtRows * kPtD;
constexpr uint32_t kPtOffV = kPtOffK + kPtStages * kPtTile8;
constexpr uint32_t kPtOffVH = kPtOffV + kPtStages * kPtTile8;
constexpr uint32_t kPtOffP = kPtOffVH + kPtVBuf * kPtTile16;
constexpr uint32_t kPtOffBar = kPtOffP + 2 * kPtP;
constexpr uint32_t kPtOffFC = kPtOffBar + 256;           // [2 groups][32 pairs of rows] factors, -references
constexpr uint32_t kPtOffRed = kPtOffFC + 2 * kPtRows * 8;     // [2][4 warps][64]
constexpr uint32_t kPtOffAdj = kPtOffRed + 2 * 4 * kPtRows * 4;  // [2][32 pairs] reference changes, factors
constexpr uint32_t kPtOffMask = kPtOffAdj + 2 * kPtRows * 8;   // [64] two mask words
constexpr uint32_t kPtOffML = kPtOffMask + kPtRows * 16;       // [2][64] (reference, sum)
constexpr uint32_t kPtBytes = kPtOffML + 2 * kPtRows * 8 + 1024;  // + slack for 1024-byte alignment
static_assert(kPtBytes <= 227 * 1024 - 256, "one block per SM");
// before the first products the tree's rows use the weights' and V16's space
constexpr uint32_t kPtOffTreeK = kPtOffP;                    // K tree, bf16, two halves of 128 rows
constexpr uint32_t kPtOffTreeV = kPtOffVH;                   // V tree, bf16, as V16 buffer 0
constexpr uint32_t kPtOffTreeQ = kPtOffVH + kPtTile16;       // q, bf16, two halves of 64 rows
// TMEM columns
constexpr uint32_t kPtColS = 0, kPtColO = 192, kPtTmemCols = 512;  // three score buffers, two O

enum { T_KFULL = 0, T_KEMPTY = 2, T_VFULL = 4, T_VEMPTY = 6, T_SFULL = 8, T_SFREE = 11, T_PFULL = 14, T_PVDONE = 16,
       T_VHFREE = 18, T_TREE = 21, T_DRAIN = 22 /* two */, T_COUNT = 24 };

// instruction descriptors: fp32 sums (bits 4-5 = 1), A type in bits 7-9, B
// type in 10-12, A / B stored MN-major in bits 15 / 16, N >> 3, M >> 4
constexpr uint32_t pt_idesc(int a_type, int b_type, bool a_mn, bool b_mn, int M, int N) {
  return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)b_type << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void pt_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// pairs of fp32 values: one instruction for two
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t &a, uint64_t &b) {
  asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
__device__ __forceinline__ void pt_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void pt_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void pt_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
__device__ __forceinline__ void lds_f4(uint32_t addr, float &x, float &y, float &z) {
  asm volatile("{\n .reg .f32 w;\n ld.shared.v4.f32 {%0, %1, %2, w}, [%3];\n}\n" : "=f"(x), "=f"(y), "=f"(z) : "r"(addr) : "memory");
}
// read anew each time: what is needed rarely is not kept in registers
__device__ __forceinline__ int thread_now() {
  int t;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
  return t;
}
// OR of a condition over a softmax group's threads, and a barrier
__device__ __forceinline__ bool group_any(int group, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(1 + group), "r"(p ? 1u : 0u)
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 256;" ::"r"(1 + group) : "memory");
}
// mbar_wait without a call: the warps that wait hold most of their registers live
__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, volatile int *abort, long long limit) {
  if (mbar_try(bar, parity)) return true;
  const long long start = clock64();
  auto parked = [&]() -> bool {  // parked by the hardware up to 2 us at a time: a spinning warp takes issue slots
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0u;
  };
#pragma unroll 1
  while (!parked()) {
    if (*abort) return false;
    if (clock64() - start > limit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// tables of two values per row, by pairs of rows: x of both, then y of both
__device__ __forceinline__ int px(int row) { return 4 * (row >> 1) + (row & 1); }
__device__ __forceinline__ int py(int row) { return px(row) + 2; }
// chunk c (16 bytes) of row r in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// maximum over the warp's lanes; NaN is passed over
__device__ __forceinline__ float warp_max_f32(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

template <int FMT>
__global__ void __launch_bounds__(kPtThreads, 1)
    k_paged_attn_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ PagedSplitArgs ma) {
  const PagedAttnArgs &a = ma.a;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_abort, s_last, s_odd;
  __shared__ int s_red[kPtThreads / 32];
  __shared__ uint32_t s_tmem, s_units[kPtStages];
  __shared__ float s_tree_lv[kPtKeys];  // log2 of the tree rows' V scales
  __shared__ float4 s_scale[kPtStages][kPtKeys / 16];  // a unit's K scale, log2 of its V scale, the inverse of that
  unsigned char *sm = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = saddr(sm);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  auto bar = [&](int i) -> uint32_t { return sb + kPtOffBar + 8u * (uint32_t)i; };

  // ---- set-up that touches no global memory ----
  if (t == 0) {
    s_abort = 0;
    s_odd = 0;
    for (int i = 0; i < T_COUNT; ++i) {
      int count = 1;
      if (i >= T_VFULL && i < T_VEMPTY) count = 2;  // the copies, the scales
      if ((i >= T_VEMPTY && i < T_SFULL) || (i >= T_SFREE && i < T_PVDONE)) count = kPtGroup / 32;  // a group's warps
      mbar_init(bar(i), (uint32_t)count);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  pdl_wait();  // the previous kernel in the stream has completed
  const int b = blockIdx.z, g = blockIdx.y / ma.row_tiles, rt = blockIdx.y - g * ma.row_tiles, chunk = blockIdx.x;
  int bad = 0;
  const int L = paged_prefix(a, b, bad);
  int longest = L;  // chunks are as long in every sequence: the longest sequence's share
  if (a.B > 1) {
    int other = 0;
    if (a.B <= kPtThreads) {
      int ignore = 0;
      if (t < a.B) other = paged_prefix(a, t, ignore);
    } else {
      other = (int)min((long long)a.max_prefix, (long long)a.max_blocks * a.P);
    }
    other = __reduce_max_sync(0xffffffffu, other);
    if (lane == 0) s_red[warp] = other;
    __syncthreads();
    longest = s_red[0];
    for (int w = 1; w < kPtThreads / 32; ++w) longest = max(longest, s_red[w]);
  }
  if (L < 0) return;
  const int T = tiles_of(L, kPtKeys), Tl = tiles_of(longest, kPtKeys);
  const int per = max((Tl + ma.S - 1) / ma.S, 1);
  const int chunks = max(1, (T + per - 1) / per);
  if (chunk >= chunks) return;
  const int t0 = chunk * per, n = min(T, t0 + per) - t0;  // prefix tiles t0 .. t0 + n - 1
  const int tree = chunk == 0 ? 1 : 0;                    // item 0 is the tree's tile
  const int items = n + tree;
  if (warp == kPtScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&s_tmem)), "r"(kPtTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();  // barriers initialised (and the longest prefix read by all)
  pdl_trigger();    // after the TMEM allocation: a waiting dependent block must not hold what this block needs

  // ---- TMA: tile j of this block into ring stage j % stages ----
  // lane: unit (lane & 7) of tile 4 * (j / 4) + (lane >> 3), 16 keys a unit; the next four tiles' (_n) in flight ahead
  int page = -1, slot = 0, page_n = -1, slot_n = 0;
  float ks = 0.f, vs = 1.f, ks_n = 0.f, vs_n = 1.f;
  auto unit_key = [&](int j0) -> long long {
    const int j = j0 + (lane >> 3);
    const long long key = (long long)(t0 + j) * kPtKeys + 16 * (lane & 7);
    return j < n && key < L ? key : -1;
  };
  auto fetch_pages = [&](int j0, int &pg, int &sl) {
    const int key = (int)unit_key(j0);
    pg = -1;
    if (key >= 0) {
      const int blk = page_index(ma, key);
      sl = key - blk * a.P;
      pg = a.block_table[(long long)b * a.max_blocks + blk];
    }
  };
  auto fetch_scales = [&](int j0, int &pg, float &k, float &v) {
    if (pg < 0 || pg >= a.num_pages) {
      if (unit_key(j0) >= 0) bad = 1;
      pg = -1;
    }
    k = 0.f;
    v = 1.f;
    if (pg >= 0) {
      k = a.k_scale[(long long)pg * a.Hkv + g];
      v = a.v_scale[(long long)pg * a.Hkv + g];
    }
  };
  auto issue = [&](int j) {
    const int stage = j % kPtStages, src = 8 * (j & 3), per_box = ma.box / 16;
    const int pg = __shfl_sync(0xffffffffu, page, src + (lane & 7)), sl = __shfl_sync(0xffffffffu, slot, src + (lane & 7));
    const uint32_t there = __ballot_sync(0xffffffffu, lane < 8 && pg >= 0);
    const uint32_t mine = __ballot_sync(0xffffffffu, lane < 8 && lane % per_box == 0 && pg >= 0);
    const uint32_t bytes = (uint32_t)__popc(mine) * (uint32_t)ma.box * kPtD;
    if (lane == 0) {
      s_units[stage] = there;
      if (bytes) {
        mbar_expect_tx(bar(T_KFULL + stage), bytes);
        mbar_expect_tx(bar(T_VFULL + stage), bytes);
      } else {
        mbar_arrive(bar(T_KFULL + stage));
        mbar_arrive(bar(T_VFULL + stage));
      }
    }
    __syncwarp();
    if ((mine >> lane) & 1u) {
      const uint32_t off = (uint32_t)(stage * kPtTile8 + lane * 16 * kPtD);
      tma_4d(sb + kPtOffK + off, &tm_k, 0, sl, g, pg, bar(T_KFULL + stage));
      tma_4d(sb + kPtOffV + off, &tm_v, 0, sl, g, pg, bar(T_VFULL + stage));
    }
  };
  auto publish = [&](int j) {  // the tile's scales, and the arrival that goes with them
    const int stage = j % kPtStages, src = 8 * (j & 3) + (lane & 7);
    const float k = __shfl_sync(0xffffffffu, ks, src), v = clamp_v_scale(__shfl_sync(0xffffffffu, vs, src));
    if (lane < 8) s_scale[stage][lane] = make_float4(k, __log2f(v), __fdividef(1.f, v), 0.f);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(T_VFULL + stage));
  };
  if (warp == kPtTmaWarp) {
    fetch_pages(0, page, slot);
    fetch_scales(0, page, ks, vs);
    for (int j = 0; j < n && j < kPtStages; ++j) issue(j);
  }

  // ---- q and, in the block that takes it, the tree's rows: every load in flight first ----
  constexpr int kQRounds = (kPtRows * 16 + kPtThreads - 1) / kPtThreads, kTreeRounds = 2;
  const __nv_bfloat16 *KT = static_cast<const __nv_bfloat16 *>(a.kt), *VT = static_cast<const __nv_bfloat16 *>(a.vt);
  const int tree_cells = tree ? ((a.N + 15) & ~15) * 16 : 0;  // 16-byte cells, rows in whole k-steps of 16 keys
  auto tree_cell = [&](int x, uint4 &k, uint4 &v) {
    const int r = x >> 4;
    k = v = make_uint4(0u, 0u, 0u, 0u);
    if (x < tree_cells && r < a.N) {
      const long long at = (((long long)b * a.N + r) * a.Hkv + g) * kPtD + 8 * (x & 15);
      k = *reinterpret_cast<const uint4 *>(KT + at);
      v = *reinterpret_cast<const uint4 *>(VT + at);
    }
  };
  float *fc = reinterpret_cast<float *>(sm + kPtOffFC);  // group w at 2 * kPtRows * w
  bool odd_v = false;
  auto store_cell = [&](int x, const uint4 &k, const uint4 &v) {  // whole warps: 16 lanes have a row
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0u;  // largest finite magnitudes of the low and of the high halves
    // NaN and infinities would reach rows that do not attend their key (0 * inf): they are added at the end
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; odd_v = true; }
      if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0xffffu; odd_v = true; }
      top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    }
    top = max(top << 16, top & 0xffff0000u);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o, 16));
    if ((x & 15) == 0) s_tree_lv[x >> 4] = (float)page_exponent<FMT>(__uint_as_float(top));
    const uint32_t at = (uint32_t)(((x & 15) >> 3) * kPtHalf16) + sw128(x >> 4, x & 7);
    sts128(sb + kPtOffTreeK + at, k.x, k.y, k.z, k.w);
    sts128(sb + kPtOffTreeV + at, w[0], w[1], w[2], w[3]);
  };
  {
    const int lr = t & 15;
    uint4 raw[kQRounds], tk[kTreeRounds], tv[kTreeRounds];
#pragma unroll
    for (int k = 0; k < kQRounds; ++k) {
      const int r = (t >> 4) + k * (kPtThreads / 16), Rg = rt * kPtRows + r, i = row_token(ma, Rg);
      raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < kPtRows && i < a.N)
        raw[k] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                  (((long long)b * a.N + i) * a.Hq + g * a.G + (Rg - i * a.G)) * kPtD + 8 * lr);
    }
    if (tree) {
#pragma unroll
      for (int k = 0; k < kTreeRounds; ++k) tree_cell(t + k * kPtThreads, tk[k], tv[k]);
    }
    // two e4m3 terms, K-major; 16 lanes a row, eight dims a lane
#pragma unroll
    for (int k = 0; k < kQRounds; ++k) {
      const int r = (t >> 4) + k * (kPtThreads / 16);
      if (r >= kPtRows) break;  // whole warps
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      uint32_t top = 0u;  // the row's largest magnitude, as the bits of a bf16 value: they order like the values
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x, 16));
      const bool odd = top >= 0x7f80u;  // NaN or infinity
      // 2^e2 lifts the largest magnitude into (224, 448], 448 = 1.75 * 2^8; half of e2 stays within fp32's exponents
      const int e2 = top == 0u || odd ? 0 : 135 - max((int)(top >> 7), 1) - ((top & 0x7fu) > 0x60u ? 1 : 0);
      const int ea = e2 >> 1, eb = e2 - ea;
      const float lift_a = __uint_as_float((uint32_t)(127 + ea) << 23), lift_b = __uint_as_float((uint32_t)(127 + eb) << 23);
      uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y0 = __uint_as_float(w[e] << 16) * lift_a * lift_b, y1 = __uint_as_float(w[e] & 0xffff0000u) * lift_a * lift_b;
        const uint32_t h2 = f32x2_to_f8x2<ET_KV_E4M3>(y0, y1);
        const uint32_t hf = f8x2_to_f16x2<ET_KV_E4M3>((uint16_t)h2);
        const float2 hv = __half22float2(*reinterpret_cast<const __half2 *>(&hf));
        hi[e >> 1] |= h2 << (16 * (e & 1));
        lo[e >> 1] |= f32x2_to_f8x2<ET_KV_E4M3>(y0 - hv.x, y1 - hv.y) << (16 * (e & 1));
      }
      unsigned char *dst = sm + kPtOffQ + sw128(r, lr >> 1) + 8 * (lr & 1);
      *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2 *>(dst + kPtRows * kPtD) = make_uint2(lo[0], lo[1]);
      if (tree) sts128(sb + kPtOffTreeQ + (uint32_t)((lr >> 3) * kPtRows * 128) + sw128(r, lr & 7), w[0], w[1], w[2], w[3]);
      if (lr == 0) {
        // what a score of lifted q and codes stands for, in log2 units; a row that is not finite scores NaN
        const float f = odd ? __uint_as_float(0x7fc00000u)
                            : a.scale_log2 * __uint_as_float((uint32_t)(127 - ea) << 23) * __uint_as_float((uint32_t)(127 - eb) << 23);
        fc[2 * kPtRows + px(r)] = f;
        fc[px(r)] = tree && !odd ? a.scale_log2 : f;  // group 0 takes the tree's tile first: q as it is
        fc[py(r)] = fc[2 * kPtRows + py(r)] = 0.f;
      }
    }
    if (tree) {
#pragma unroll
      for (int k = 0; k < kTreeRounds; ++k)
        if (t + k * kPtThreads < tree_cells) store_cell(t + k * kPtThreads, tk[k], tv[k]);
    }
  }
  if (tree) {
#pragma unroll 1
    for (int x = t + kTreeRounds * kPtThreads; x < tree_cells; x += kPtThreads) {
      uint4 k, v;
      tree_cell(x, k, v);
      store_cell(x, k, v);
    }
    if (odd_v) s_odd = 1;
    if (t < kPtRows) {
      const int i = row_token(ma, rt * kPtRows + t);
      unsigned long long m0 = 0ull, m1 = 0ull;
      if (i < a.N) {
        if (a.mask) {
          m0 = a.mask[((long long)b * a.N + i) * a.W];
          if (a.W > 1) m1 = a.mask[((long long)b * a.N + i) * a.W + 1];
        } else {
          m0 = i >= 63 ? ~0ull : (2ull << i) - 1ull;
          m1 = i < 64 ? 0ull : (i >= 127 ? ~0ull : (2ull << (i - 64)) - 1ull);
        }
      }
      unsigned long long *m = reinterpret_cast<unsigned long long *>(sm + kPtOffMask) + 2 * t;
      m[0] = m0;
      m[1] = m1;
    }
  }
  fence_async_smem();  // q and the tree's rows are read by the tensor cores
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const long long limit = ma.wait_cycles;

  if (warp == kPtTmaWarp) {
    // ---------------- TMA ----------------
    bool ok = true;
    int issued = n < kPtStages ? n : kPtStages;
    fetch_pages(4, page_n, slot_n);
    for (int j = 0; j < issued; ++j) publish(j);
    for (int j = kPtStages; j < n; ++j) {
      if ((j & 3) == 2) fetch_scales(j + 2, page_n, ks_n, vs_n);
      if ((j & 3) == 0) {
        page = page_n; slot = slot_n; ks = ks_n; vs = vs_n;
        fetch_pages(j + 4, page_n, slot_n);
      }
      const int stage = j % kPtStages;
      const uint32_t phase = (uint32_t)(j / kPtStages - 1) & 1u;
      ok = pt_wait(bar(T_KEMPTY + stage), phase, &s_abort, limit) && pt_wait(bar(T_VEMPTY + stage), phase, &s_abort, limit);
      if (!__all_sync(0xffffffffu, ok)) break;
      issue(j);
      publish(j);
      issued = j + 1;
    }
    if (lane == 0)  // no copy may be in flight when the block leaves
      for (int j = issued > kPtStages ? issued - kPtStages : 0; j < issued; ++j) {
        mbar_drain(bar(T_KFULL + j % kPtStages), (uint32_t)(j / kPtStages) & 1u);
        mbar_drain(bar(T_VFULL + j % kPtStages), (uint32_t)(j / kPtStages) & 1u);
      }
    if (bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
  } else if (warp == kPtScoreWarp) {
    // ---------------- score products, three items ahead of the weights at most ----------------
    if (lane == 0) {
      constexpr uint32_t iS = pt_idesc(FMT == ET_KV_E4M3 ? 0 : 1, 0, false, false, 128, 64);
      constexpr uint32_t iSt = pt_idesc(1, 1, false, false, 128, 64);
      for (int i = 0; i < items; ++i) {
        const int buf = i % 3;
        const uint32_t d = tmem + kPtColS + 64u * (uint32_t)buf;
        if (i >= 3 && !pt_wait(bar(T_SFREE + buf), (uint32_t)(i / 3 - 1) & 1u, &s_abort, limit)) break;
        if (tree && i == 0) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma(d, sw128_desc(sb + kPtOffTreeK + (kk >> 2) * kPtHalf16 + (kk & 3) * 32, 16, 1024),
                   sw128_desc(sb + kPtOffTreeQ + (kk >> 2) * (kPtRows * 128) + (kk & 3) * 32, 16, 1024), iSt, kk > 0);
          tc_commit(bar(T_TREE));
        } else {
          const int j = i - tree, stage = j % kPtStages;
          if (!pt_wait(bar(T_KFULL + stage), (uint32_t)(j / kPtStages) & 1u, &s_abort, limit)) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // the two terms of q one after the other
            pt_mma_f8(d, sw128_desc(sb + kPtOffK + stage * kPtTile8 + (kk & 3) * 32, 16, 1024),
                      sw128_desc(sb + kPtOffQ + (kk >> 2) * (kPtRows * kPtD) + (kk & 3) * 32, 16, 1024), iS, kk > 0);
          if (j + kPtStages < n) tc_commit(bar(T_KEMPTY + stage));
        }
        tc_commit(bar(T_SFULL + buf));
      }
      // every product this thread issued has finished before TMEM is freed
      tc_commit(bar(T_DRAIN));
      mbar_drain(bar(T_DRAIN), 0);
    }
  } else if (warp == kPtPvWarp) {
    // ---------------- P.V products ----------------
    if (lane == 0) {
      constexpr uint32_t iO = pt_idesc(0, 0, true, true, 128, 64), iOt = pt_idesc(1, 1, true, true, 128, 64);
      for (int i = 0; i < items; ++i) {
        const int w = i & 1;
        if (!pt_wait(bar(T_PFULL + w), (uint32_t)(i >> 1) & 1u, &s_abort, limit)) break;
        tc_fence_after();
        const bool is_tree = tree && i == 0;
        const int steps = is_tree ? (a.N + 15) >> 4 : kPtKeys / 16;
        for (int kk = 0; kk < steps; ++kk)
          tc_mma(tmem + kPtColO + 64u * (uint32_t)w,
                 sw128_desc(sb + kPtOffVH + (i % kPtVBuf) * kPtTile16 + kk * 2048, kPtHalf16, 1024),
                 sw128_desc(sb + kPtOffP + w * kPtP + kk * 2048, kPtHalf16, 1024), is_tree ? iOt : iO, (i >= 2 || kk > 0) ? 1u : 0u);
        tc_commit(bar(T_VHFREE + i % kPtVBuf));
        tc_commit(bar(T_PVDONE + w));
      }
      tc_commit(bar(T_DRAIN + 1));
      mbar_drain(bar(T_DRAIN + 1), 0);
    }
  } else {
    // ---------------- softmax: group w, one key and half of the rows per thread ----------------
    const int w = warp >> 3, quarter = warp & 3, col = (warp >> 2) & 1, tid = 32 * quarter + lane;
    const int gt = t & (kPtGroup - 1), r0 = kPtQ * col;  // thread of the group; first of its rows
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)r0;
    const uint32_t fcb = sb + kPtOffFC + (uint32_t)((2 * kPtRows * w + 2 * r0) * 4), prow = sb + kPtOffP + (uint32_t)(w * kPtP);
    uint64_t l2[kPtQ / 2];
#pragma unroll
    for (int q = 0; q < kPtQ / 2; ++q) l2[q] = 0ull;
    bool dead = false;
    bool fresh = true;       // some row has no reference yet (the same in the whole group)
    bool mine_fresh = true;  // threads 0..63 of the group: row gt has none
    // one item; the tree's tile (group 0's first) is compiled apart, which keeps its choices out of the others
    auto item = [&](int i, auto is_tree_) {
      constexpr bool is_tree = decltype(is_tree_)::value;
      const int buf = i % 3;  // of the scores and of V16
      static_assert(kPtVBuf == 3, "as many as score buffers");
      bool there = is_tree && tid < a.N;
      float ks = 1.f, lv = 0.f, iv = 1.f;
      if (is_tree) {
        lv = there ? s_tree_lv[tid] : 0.f;
        iv = power_of_two(-(int)lv);
      }
      // V16 buffer 1 held q of the tree's scores; else the buffer is free once the other group's product has run
      if (!is_tree && !dead) {
        if (i >= kPtVBuf) dead = !pt_wait(bar(T_VHFREE + buf), (uint32_t)(i / 3 - 1) & 1u, &s_abort, limit);
        else if (tree && i == 1) dead = !pt_wait(bar(T_TREE), 0, &s_abort, limit);
      }
      if (!is_tree) {
        // V's codes -> fp16: 16 codes of a row a thread, read as two chunks of eight.  The row's place in its group of
        // eight is the thread's own, so addresses advance by whole groups.  Dims 16 c .. + 15 become two 16-byte chunks
        // of half c / 4; which one a lane takes first alternates between the halves, which keeps the stores free of
        // bank conflicts, and between rows, which keeps the reads free of them
        const int j = i - tree, stage = j % kPtStages;
        if (!dead) dead = !pt_wait(bar(T_VFULL + stage), (uint32_t)(j / kPtStages) & 1u, &s_abort, limit);
        const uint32_t units = *(volatile uint32_t *)&s_units[stage];
        const int lim = L - (t0 + j) * kPtKeys;  // rows past it hold no key of this sequence
        lds_f4(saddr(&s_scale[stage][tid >> 4]), ks, lv, iv);
        there = tid < lim && ((units >> (tid >> 4)) & 1u);
        const int c = gt & 7, r7 = (gt >> 3) & 7, r64 = gt >> 6, c0 = 2 * (c & 3);
        const int swap = (c >> 2) ^ (r7 & 1);
        const uint32_t from = sb + kPtOffV + stage * kPtTile8 + 1024u * (uint32_t)r64 + sw128(r7, c);
        const uint32_t half = sb + kPtOffVH + (uint32_t)buf * kPtTile16 + (uint32_t)((c >> 2) * kPtHalf16) + 1024u * (uint32_t)r64;
        const uint32_t from0 = from + 8u * (uint32_t)swap, from1 = from + 8u - 8u * (uint32_t)swap;
        const uint32_t to0 = half + sw128(r7, c0 + swap), to1 = half + sw128(r7, c0 + 1 - swap);
        const bool whole = lim >= kPtKeys && units == 0xffu;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[k].x), "=r"(v[k].y) : "r"(from0 + 4096u * k));
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[k].z), "=r"(v[k].w) : "r"(from1 + 4096u * k));
        }
        if (!whole) {  // whatever lies in rows without a key must not meet a zero weight
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = r7 + 8 * (r64 + 4 * k);
            if (r >= lim || !((units >> (r >> 4)) & 1u)) v[k] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h[8];
          f8x4_to_f16<FMT>(v[k].x, h[0], h[1]);
          f8x4_to_f16<FMT>(v[k].y, h[2], h[3]);
          f8x4_to_f16<FMT>(v[k].z, h[4], h[5]);
          f8x4_to_f16<FMT>(v[k].w, h[6], h[7]);
          sts128(to0 + 4096u * k, h[0], h[1], h[2], h[3]);
          sts128(to1 + 4096u * k, h[4], h[5], h[6], h[7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T_VEMPTY + stage));
      }
      uint32_t keep = there ? 0xffffffffu : 0u;  // bit q: row r0 + q attends this thread's key
      if (is_tree && there) {
        keep = 0u;
#pragma unroll 4
        for (int q = 0; q < kPtQ; ++q) {
          const unsigned long long m =
              *(reinterpret_cast<const unsigned long long *>(sm + kPtOffMask) + 2 * (r0 + q) + (tid >> 6));
          keep |= (uint32_t)((m >> (tid & 63)) & 1ull) << q;
        }
      }
      const bool masked = __any_sync(0xffffffffu, keep != 0xffffffffu);
      if (!dead) dead = !pt_wait(bar(T_SFULL + buf), (uint32_t)(i / 3) & 1u, &s_abort, limit);
      // this group's weights (and O) are free once its last product has run, long before now
      if (!dead && i >= 2) dead = !pt_wait(bar(T_PVDONE + w), (uint32_t)((i >> 1) - 1) & 1u, &s_abort, limit);
      dead = __any_sync(0xffffffffu, dead);
      tc_fence_after();
      float x[kPtQ];
      const uint64_t ks2 = pair(ks, ks), lv2 = pair(lv, lv), iv2 = pair(iv, iv);
#pragma unroll
      for (int part = 0; part < kPtQ / 8; ++part) {
        uint32_t sc[8];
        pt_ld8(lanes + kPtColS + 64u * (uint32_t)buf + 8u * part, sc);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          uint64_t f, c;  // two rows' factors and -references
          lds_pairs(fcb + 8u * (uint32_t)(8 * part + e), f, c);
          uint64_t y = pair(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
          y = fma2(is_tree ? y : mul2(y, ks2), f, add2(lv2, c));
          unpair(y, x[8 * part + e], x[8 * part + e + 1]);
        }
      }
      tc_fence_before();  // the scores sit in registers: their buffer is free
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T_SFREE + buf));
      if (masked) {  // whatever was scored there
#pragma unroll
        for (int q = 0; q < kPtQ; ++q) x[q] = (keep >> q) & 1u ? x[q] : -INFINITY;
        __syncwarp();
      }
      float top = x[0];
#pragma unroll
      for (int q = 1; q + 1 < kPtQ; q += 2) top = fmaxf(top, fmaxf(x[q], x[q + 1]));
      top = fmaxf(top, x[kPtQ - 1]);
      if (group_any(w, fresh || top > kPaTop + kPaSlack)) {
        // the rows' maxima over the tile: a warp's 32 keys, then the four quarters
        const int now_t = thread_now(), sw = now_t / kPtGroup, sgt = now_t % kPtGroup, sl = now_t & 31;
        const int sr0 = kPtQ * ((now_t >> 7) & 1);
        const uint32_t redb = sb + kPtOffRed + (uint32_t)(sw * 4 * kPtRows * 4);
        const uint32_t adjb = sb + kPtOffAdj + (uint32_t)(sw * 2 * kPtRows * 4);
        float highest = -INFINITY;
#pragma unroll
        for (int q = 0; q < kPtQ; ++q) {
          const float m = warp_max_f32(x[q]);
          if (sl == q) highest = m;
        }
        sts32(redb + (uint32_t)((((now_t >> 5) & 3) * kPtRows + sr0 + sl) * 4), highest);
        group_sync(sw);
        bool still = false;
        if (sgt < kPtRows) {
          const uint32_t at = redb + 4u * (uint32_t)sgt, refb = sb + kPtOffFC + (uint32_t)((2 * kPtRows * sw + py(sgt)) * 4);
          const float m = fmaxf(fmaxf(lds32(at), lds32(at + 4 * kPtRows)), fmaxf(lds32(at + 8 * kPtRows), lds32(at + 12 * kPtRows)));
          const float was = -lds32(refb);  // the reference; 0 while the row is fresh
          float now = was;
          if (m > -INFINITY) now = mine_fresh ? m - kPaTop : fmaxf(was, m + was - kPaTop);
          const float corr = mine_fresh ? 0.f : ex2_fast(was - now);
          mine_fresh = mine_fresh && !(m > -INFINITY);
          still = mine_fresh;
          sts32(refb, -now);
          sts32(adjb + 4u * (uint32_t)px(sgt), was - now);
          sts32(adjb + 4u * (uint32_t)py(sgt), corr);
        }
        fresh = group_any(sw, still);
#pragma unroll
        for (int q = 0; q < kPtQ; q += 2) {
          uint64_t d, f;
          lds_pairs(adjb + 8u * (uint32_t)(sr0 + q), d, f);
          unpair(add2(pair(x[q], x[q + 1]), d), x[q], x[q + 1]);
          l2[q / 2] = mul2(l2[q / 2], f);
        }
        if (i >= 2) {  // O holds the sums of this group's earlier tiles
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < kPtQ / 8; ++part) {
            uint32_t o[8];
            const uint32_t at = lanes + kPtColO + 64u * (uint32_t)sw + 8u * part;
            pt_ld8(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * lds32(adjb + 4u * (uint32_t)py(sr0 + 8 * part + e)));
            pt_st8(at, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        group_sync(sw);  // the changes are read before they may change again
      }
#pragma unroll
      for (int c = 0; c < kPtQ / 8; ++c) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = 8 * c + 2 * e;
          const float w0 = ex2_fast(x[q]), w1 = ex2_fast(x[q + 1]);
          l2[q / 2] = fma2(pair(w0, w1), iv2, l2[q / 2]);
          p[e] = is_tree ? pack_bf16x2(w0 * iv, w1 * iv) : pack_f16x2(w0, w1);
        }
        sts128(prow + sw128(tid, 4 * col + c), p[0], p[1], p[2], p[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T_PFULL + w));
      if (is_tree) {  // cached tiles from here on: the rows' own factors
        group_sync(w);
        if (gt < kPtRows) fc[px(gt)] = fc[2 * kPtRows + px(gt)];
        group_sync(w);
      }
    };
    int i0 = w;
    if (tree && w == 0) {
      item(0, std::true_type{});
      i0 = 2;
    }
#pragma unroll 1
    for (int i = i0; i < items; i += 2) item(i, std::false_type{});
    // the group's sums: a warp's 32 rows over its 32 keys; after the step of offset o a lane holds the rows whose
    // index agrees with it in the bits done, in the end row r0 + lane
    float l[kPtQ];
#pragma unroll
    for (int q = 0; q < kPtQ; q += 2) unpair(l2[q / 2], l[q], l[q + 1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int q = 0; q < o; ++q) {
        const float kept = up ? l[q + o] : l[q], send = up ? l[q] : l[q + o];
        l[q] = kept + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    float *red = reinterpret_cast<float *>(sm + kPtOffRed) + w * 4 * kPtRows;
    const float *ref = fc + 2 * kPtRows * w;
    red[quarter * kPtRows + r0 + lane] = l[0];
    group_sync(w);
    const int mine = items > w ? (items - w + 1) / 2 : 0;  // this group's items
    if (gt < kPtRows)
      reinterpret_cast<float2 *>(sm + kPtOffML)[w * kPtRows + gt] =
          make_float2(mine && !mine_fresh ? -ref[py(gt)] : -3e38f,
                      (red[gt] + red[kPtRows + gt]) + (red[2 * kPtRows + gt] + red[3 * kPtRows + gt]));
    if (mine && !dead) dead = !pt_wait(bar(T_PVDONE + w), (uint32_t)(mine - 1) & 1u, &s_abort, limit);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool aborted = *(volatile int *)&s_abort != 0;
  if (aborted && t == 0) flag_status(a.dev_status, ET_DEV_TIMEOUT);

  // ---- the two groups' O, joined; thread = dim ----
  const int real = min(kPtRows, a.N * a.G - rt * kPtRows);  // rows that exist are a prefix of the tile
  const long long tile_id = (long long)b * ma.tiles_y + blockIdx.y;
  auto place = [&](int r) -> long long {  // element index of row r in out
    const int Rg = rt * kPtRows + r, i = row_token(ma, Rg);
    return (((long long)b * a.N + i) * a.Hq + g * a.G + (Rg - i * a.G)) * kPtD;
  };
  auto write_lse = [&](int r, float M, float sum) {
    const int Rg = rt * kPtRows + r, i = row_token(ma, Rg), h = g * a.G + (Rg - i * a.G);
    if (a.lse) a.lse[((long long)b * a.Hq + h) * a.N + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
  };
  // a chunk's rows go to the workspace or, for its cluster to read, to shared memory where the rings and the tables of
  // factors were
  const bool cluster = ma.cnt == nullptr;
  const long long part = cluster ? 0 : (tile_id * ma.S + chunk) * kPtRows;
  float2 *part_ml = cluster ? reinterpret_cast<float2 *>(sm + kPtOffFC) : ma.part_ml;
  float *part_o = cluster ? reinterpret_cast<float *>(sm + kPtOffK) : reinterpret_cast<float *>(ma.part_o);
  // factors of the two groups' sums and the row's place, per row (short loops: cold code runs at the speed of its fetch)
  float2 *mix = reinterpret_cast<float2 *>(sm + kPtOffAdj);
  long long *to = reinterpret_cast<long long *>(sm + kPtOffRed);
  if (t < real) {
    const float2 *ml = reinterpret_cast<const float2 *>(sm + kPtOffML);
    const float2 x = ml[t], y = ml[kPtRows + t];
    const float M = fmaxf(x.x, y.x), wx = ex2_fast(x.x - M), wy = ex2_fast(y.x - M), sum = fmaf(x.y, wx, y.y * wy);
    if (chunks == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      mix[t] = make_float2(wx * inv, wy * inv);
      to[t] = place(t);
      write_lse(t, M, sum);
    } else {
      mix[t] = make_float2(wx, wy);
      to[t] = (part + t) * kPtD;
      part_ml[part + t] = make_float2(M, sum);
    }
  }
  __syncthreads();
  if (warp < kPtTmaWarp) {
    const int quarter = warp & 3, d = 32 * quarter + lane, q0 = 16 * (warp >> 2);  // 16 rows a warp
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16) + kPtColO;
    const bool odd = tree && s_odd, two = items > 1;  // a group without items left its columns unwritten
    if (q0 < real) {
      uint32_t o0[16], o1[16];
      pt_ld16(lanes + (uint32_t)q0, o0);
      pt_ld16(lanes + 64u + (uint32_t)q0, o1);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 f = mix[q0 + e];
        o0[e] = __float_as_uint(__uint_as_float(o0[e]) * f.x + (two ? __uint_as_float(o1[e]) * f.y : 0.f));
      }
      if (odd) {
#pragma unroll 1
        for (int k = 0; k < a.N; ++k) {
          const float z = __bfloat162float(
              static_cast<const __nv_bfloat16 *>(a.vt)[(((long long)b * a.N + k) * a.Hkv + g) * kPtD + d]);
          if (fabsf(z) <= FLT_MAX) continue;
          const unsigned long long *m = reinterpret_cast<const unsigned long long *>(sm + kPtOffMask) + (k >> 6);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((m[2 * (q0 + e)] >> (k & 63)) & 1ull) o0[e] = __float_as_uint(__uint_as_float(o0[e]) + z);
        }
      }
      if (chunks == 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (q0 + e < real)
            static_cast<__nv_bfloat16 *>(a.out)[to[q0 + e] + d] = __float2bfloat16_rn(__uint_as_float(o0[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (q0 + e < real) part_o[to[q0 + e] + d] = __uint_as_float(o0[e]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == kPtScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPtTmemCols) : "memory");
  if (chunks == 1) return;
  auto write4 = [&](int r, int c, const float4 &v, float M, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint2 u;
    u.x = pack_bf16x2(v.x * inv, v.y * inv);
    u.y = pack_bf16x2(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + place(r) + 4 * c) = u;
    if (c == 0) write_lse(r, M, sum);
  };
  if (cluster) {
    // ---- the chunks' rows, each merged by a warp of one of the cluster's blocks ----
    // (blocks without keys have left: the barrier counts the others)
    __syncwarp();
    cl_sync();
#pragma unroll 1
    for (int r = chunk + warp * chunks; r < real; r += kPtThreads / 32 * chunks) {
      float4 v[kPaMaxCluster];
#pragma unroll
      for (int k = 0; k < kPaMaxCluster; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < chunks) v[k] = cl_ld_f32x4(cl_map(part_o, (uint32_t)k) + (uint32_t)((r * kPtD + 4 * lane) * 4));
      }
      float m = -3e38f, l = 0.f;
      if (lane < chunks) {
        const uint32_t at = cl_map(part_ml, (uint32_t)lane) + 8u * (uint32_t)r;
        m = cl_ld_f32(at);
        l = cl_ld_f32(at + 4u);
      }
      const float M = warp_max_f32(m), f = ex2_fast(m - M);
      float sum = l * f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum = __shfl_sync(0xffffffffu, sum, 0);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPaMaxCluster; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k);
        if (k < chunks) {
          y.x = fmaf(v[k].x, fk, y.x); y.y = fmaf(v[k].y, fk, y.y);
          y.z = fmaf(v[k].z, fk, y.z); y.w = fmaf(v[k].w, fk, y.w);
        }
      }
      write4(r, lane, y, M, sum);
    }
    __syncwarp();
    cl_sync();  // no block leaves while another reads its rows
    return;
  }
  // ---- more chunks than a cluster has blocks: merged by the last block to arrive ----
  if (!arrive_last(ma.cnt + tile_id, (unsigned)chunks, &s_last)) return;
  merge_chunks<kPtD, kPtRows, kPtThreads>(ma, tile_id * ma.S, chunks, real, sm, write4);
}

}  // namespace

bool make_page_map(CUtensorMap *m, const void *base, const et_paged_cache *c, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c->d, (cuuint64_t)c->page_size, (cuuint64_t)c->Hkv, (cuuint64_t)c->num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c->d, (cuuint64_t)c->d * c->page_size, (cuuint64_t)c->page_stride};
  const cuuint32_t boxes[4] = {(cuuint32_t)c->d, (cuuint32_t)box, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, boxes, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     c->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

et_status paged_tc_launch(const et_paged_cache *cache, const PagedSplitArgs &args, cudaStream_t stream) {
  PagedSplitArgs ma = args;
  ma.box = cache->page_size % 128 == 0 ? 128 : cache->page_size % 64 == 0 ? 64 : cache->page_size % 32 == 0 ? 32 : 16;
  CUtensorMap mk, mv;
  if (!make_page_map(&mk, cache->k_pages, cache, ma.box) || !make_page_map(&mv, cache->v_pages, cache, ma.box))
    return ET_ERR_INVALID_ARG;
  const dim3 grid(ma.S, ma.tiles_y, ma.a.B);
  const int cluster = ma.cnt || ma.S == 1 ? 0 : ma.S;
  auto *kernel = cache->format == ET_KV_E4M3 ? k_paged_attn_tc<ET_KV_E4M3> : k_paged_attn_tc<ET_KV_E5M2>;
  if (et_smem_attr((const void *)kernel, (int)kPtBytes) != cudaSuccess) return ET_ERR_CUDA;
  return et_launch(kernel, grid, dim3(kPtThreads), kPtBytes, stream, cluster, mk, mv, ma);
}

int paged_tc_clusters(int S, int sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kPaMaxCluster + 1];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  if (dev >= 0 && dev < kDevices && (n = known[dev][S].load(std::memory_order_relaxed)) > 0) return n;
  auto *kernel = k_paged_attn_tc<ET_KV_E4M3>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)S;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)S);
  cfg.blockDim = dim3(kPtThreads);
  cfg.dynamicSmemBytes = kPtBytes;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (dev < 0 || et_smem_attr((const void *)kernel, (int)kPtBytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return sms / S > 0 ? sms / S : 1;
  }
  if (dev < kDevices) known[dev][S].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace et
