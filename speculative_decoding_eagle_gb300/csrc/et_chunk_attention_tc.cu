// Chunk attention on the 5th-generation tensor cores (tcgen05): many new rows
// of a sequence over its paged 8-bit prefix and over themselves, bf16 inputs,
// D = 64 or 128 (EAGLE blog 1.1: the target's forward over a prompt).
//
// One block per SM and a unit of 256 (token, head) rows of a KV head, two
// tiles of 128 rows, a row to a TMEM lane (units of 128 rows where they would
// leave half of the SMs idle); keys in tiles of 128:
//   S [128 rows x 128 keys] = Q8 . K8^T  (kind::f8f6f4: K's codes by TMA as they
//        lie in the page; q lifted by a power of two per row and split into
//        two e4m3 terms, two products into one sum), or Q . K^T in bf16 for
//        the new rows' own keys;
//   O [128 rows x D] += P . V  (kind::f16, P from TMEM where S was): V's codes
//        as fp16, or the new rows' V in bf16.
// Sixteen warps:
//   warps 0-3, 4-7  a softmax group each, one row per thread: the row's 128
//              scores go through registers once, no exchange between threads.
//              More than 128 rows: each group has its own 128, over the same
//              tiles.  Fewer (decoded tokens, short pieces): both have the
//              same rows and alternate tiles, joined at the end, so that one
//              group's products run under the other's softmax either way
//   warps 8-11 turn V's codes into fp16, stage q, and clear what no row of
//              the block may see from the new rows' V
//   warps 12, 15  TMA for K (with the scales) and for V;  warp 13 issues the score products, warp 14 those of P.V
// The prefix comes first.  A weight's reference moves only when some weight
// would pass 2^15; a row is a thread's own, so nothing but the warp has to
// agree.  A cached key's weight carries its page's V scale and is rounded to
// fp16; the new keys' weights are rounded to bf16, whose range does not depend
// on how large their V is against the cache's.
// Few rows, or a last round of blocks that would not fill the SMs: a unit's
// tiles are split over several blocks, which leave their rows in the
// workspace; the last one to arrive merges them.
// Bounds, measured: 2048 rows after 8192 cached, 64 / 8 heads, 470 us = 1316
// TFLOP/s (68% of the measured bf16 rate); a tile of 256 x 128 takes about 3000
// cycles of which the tensor cores work 2048: the rest is the softmax warps'
// chain (scores out of tensor memory, exponentials, weights back) against the
// two groups' turns.  16 sequences, mostly one row each, 182 us = 3.4 TB/s of
// codes: about 1900 cycles a tile where its bytes take 1400.  Beside its
// tiles a block costs 11000 cycles to the first scores (rows, pages, q and the
// first keys one after the other) and 9000 behind the last, which is most of a
// call over a short prefix.
// Every mbarrier wait is bounded: a block that gives up sets ET_DEV_TIMEOUT,
// drains what it issued and leaves.
#include "et_chunk_attn.cuh"
#include "et_paged_tc.cuh"

#include <type_traits>

namespace et {
namespace {

constexpr int kCtThreads = 512;
constexpr int kCtKeys = 128;                          // keys per tile
constexpr int kCtTmaWarp = 12, kCtScoreWarp = 13, kCtPvWarp = 14, kCtTmaVWarp = 15;
constexpr int kCtStages8 = 4, kCtStages16 = 2;        // K ring: stages of codes, or of bf16 rows, in one space
constexpr int kCtOrdered = 32;                        // sequences up to which a batch goes out by length
constexpr int kCtSlots = 8;                           // tiles whose scales are kept
constexpr uint32_t kCtColS = 0, kCtColO = 256, kCtTmemCols = 512;  // S / P of the two groups, O of the two groups

template <int D>
struct CtShape {
  static constexpr uint32_t tile8 = kCtKeys * D;          // codes of a tile of keys, or one term of 128 q rows
  static constexpr uint32_t tile16 = 2 * tile8;           // bf16 / fp16 rows of a tile
  static constexpr uint32_t half16 = kCtKeys * 128;       // 64 dims of it
  static constexpr uint32_t off_q = 0;                    // two groups: two e4m3 terms, later bf16
  static constexpr uint32_t off_k = 2 * tile16;
  static constexpr uint32_t off_v8 = off_k + kCtStages16 * tile16;
  static constexpr uint32_t off_v16 = off_v8 + 2 * tile8;
  static constexpr uint32_t off_bar = off_v16 + 2 * tile16;
  static constexpr uint32_t bytes = off_bar + 512 + 1024;  // + slack for 1024-byte alignment
};
static_assert(CtShape<128>::bytes <= 227 * 1024 - 1536, "one block per SM, static shared memory besides");

enum {
  C_KFULL = 0,                        // four stages of codes
  C_KEMPTY = C_KFULL + kCtStages8,
  C_K2FULL = C_KEMPTY + kCtStages8,   // two stages of bf16 keys
  C_K2EMPTY = C_K2FULL + kCtStages16,
  C_VFULL = C_K2EMPTY + kCtStages16,  // V's codes, two stages or four
  C_VEMPTY = C_VFULL + 4,
  C_VTMA = C_VEMPTY + 4,              // bf16 V has landed
  C_VHFULL = C_VTMA + 2,              // V as the products take it
  C_VHFREE = C_VHFULL + 2,
  C_SFULL = C_VHFREE + 2,             // per group from here on
  C_PFULL = C_SFULL + 2,
  C_PHALF = C_PFULL + 2,
  C_PVDONE = C_PHALF + 2,
  C_QFREE = C_PVDONE + 2,             // the prefix's score products have run: q and the K ring are free
  C_QFULL = C_QFREE + 1,              // q in bf16
  C_SCALES = C_QFULL + 1,             // eight slots: a tile's scales are there
  C_QRAW = C_SCALES + kCtSlots,       // q has landed as it is
  C_DRAIN = C_QRAW + 1,               // two
  C_COUNT = C_DRAIN + 2
};
static_assert(C_COUNT * 8 <= 512, "barriers");

// descriptor of 8-bit rows of D bytes: 128-byte or 64-byte swizzle (mode 2 or 4), eight rows to a group
template <int D>
__device__ __forceinline__ uint64_t desc8(uint32_t start) {
  const uint64_t mode = D == 128 ? 2ull : 4ull;
  return (uint64_t)((start >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(8 * D >> 4) << 32) | (1ull << 46) | (mode << 61);
}
// chunk c (16 bytes) of row r among rows of D bytes
template <int D>
__device__ __forceinline__ uint32_t at8(int r, int c) {
  return D == 128 ? sw128(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
// mbar_drain without a call: registers are split unevenly over the warps, which a call's fixed set does not allow
__device__ __forceinline__ void ct_drain(uint32_t bar, uint32_t parity) {
  const long long start = clock64();
#pragma unroll 1
  while (!mbar_try(bar, parity) && clock64() - start < kTcWaitCycles) {
  }
}
// all warps at the end of their roles: registers are handed back before any warp asks for its share again (a warp that took
// them back while a softmax warp still waits for them would leave it waiting)
__device__ __forceinline__ void roles_end() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kCtThreads) : "memory"); }
template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// One lane of a converged warp.  Products are issued from control flow that the whole warp shares, under this predicate:
// their descriptors then stay in uniform registers (a product of 128 x 128 x 16 every 64 cycles; 130 to 160 from a loop that
// one lane alone runs)
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0u;
}
// Products and commits by the one lane whose `lead` is set, without a branch: the operands stay in uniform registers
__device__ __forceinline__ void ct_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void ct_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void ct_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void ct_commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(lead)
      : "memory");
}
// two values -> two codes, round to nearest even, saturating, NaN kept
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
  return r;
}
struct ChunkTcArgs {
  ChunkArgs c;
  int S;                 // parts of a unit's tiles at most
  int shift;             // a unit: 1 << shift (token, head) rows of a KV head, 128 or 256
  int tiles;             // units per KV head in the grid
  int whole;             // the first units, each a block
  int q_tma;             // q by TMA: the heads of a group divide a tile's 128 rows
  int box;               // rows per TMA box of a page
  unsigned int *cnt;     // arrival counters (null with S = 1)
  float2 *part_ml;
  float4 *part_o;
  uint32_t page_magic, group_magic, group_shift;
  long long wait_cycles;
};
__device__ __forceinline__ int ct_page_index(const ChunkTcArgs &a, int token) {
  const uint32_t u = (uint32_t)token >> 4;
  return (int)(a.page_magic ? __umulhi(u, a.page_magic) : u);
}
__device__ __forceinline__ int ct_token(const ChunkTcArgs &a, int row) {
  return (int)(a.group_magic ? __umulhi((uint32_t)row, a.group_magic) >> a.group_shift : (uint32_t)row);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kCtThreads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
               const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ ChunkTcArgs ca) {
  using Sh = CtShape<D>;
  const PagedAttnArgs &a = ca.c.a;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_abort, s_last, s_odd, s_seq, s_tile, s_longest, s_first, s_rows, s_prefix;
  __shared__ int s_red[kCtThreads / 32], s_len[kCtThreads / 32];
  __shared__ int2 s_seqs[kCtOrdered];
  __shared__ uint32_t s_tmem, s_units[kCtSlots];
  __shared__ __align__(16) float4 s_scale[kCtSlots][kCtKeys / 16];  // a unit's K scale, log2 of its V scale, the inverse of that
  unsigned char *sm = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = saddr(sm);
  const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
  auto bar = [&](int i) -> uint32_t { return sb + Sh::off_bar + 8u * (uint32_t)i; };

  // ---- set-up that touches no global memory ----
  if (t < C_COUNT) {
    const bool warps = (t >= C_VEMPTY && t < C_VTMA) || (t >= C_VHFULL && t < C_VHFREE) || (t >= C_PFULL && t < C_PVDONE) || (t == C_QFULL && !ca.q_tma);
    mbar_init(bar(t), warps ? 4u : 1u);  // the warps of a group, or one
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (t == C_COUNT) {
    s_abort = 0;
    s_odd = 0;
    s_seq = -1;
    s_longest = 0;
  } else if (warp == 3 && lane < 5) {
    prefetch_tmap(lane == 0 ? &tm_k : lane == 1 ? &tm_v : lane == 2 ? &tm_kn : lane == 3 ? &tm_vn : &tm_q);
  }
  __syncthreads();
  pdl_wait();  // the previous kernel in the stream has completed

  // ---- which rows: unit `index` of a KV head's units, in the sequences' order ----
  const int behind = (int)blockIdx.x - ca.whole;  // a block of the units in parts
  const int cut = behind < 0 ? 0 : behind / ca.S, part = behind < 0 ? 0 : behind - cut * ca.S;
  const int unit = behind < 0 ? (int)blockIdx.x : ca.whole + cut;
  const int index = unit / a.Hkv, g = unit - index * a.Hkv;
  int bad = 0;
  {
    // Sequences of the most keys go out first (ties: lower index), as far as one round of threads ranks them: a block that
    // starts last should not be the longest.  Larger batches keep their order
    int done = 0;  // tiles of the sequences before this round's
    int wrong = 0, top = -1;  // a row_start so far was; the largest start so far, once one was
    for (int b0 = 0; b0 < a.B; b0 += kCtThreads) {
      const int b = b0 + t;
      int mine = 0, keys = 0, first = 0, n = 0, L = -1, odd = 0;
      if (b < a.B) {
        int ignore = 0;
        L = paged_prefix(a, b, ignore);
        chunk_rows(ca.c, b, first, n, odd);
        if ((ignore | odd) && blockIdx.x == 0) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
      }
      // Some start is wrong: a sequence whose first row lies before an earlier one is left out (chunk_start).  Up to kCtOrdered
      // sequences lie in one warp
      if (a.B <= kCtOrdered ? __any_sync(0xffffffffu, odd) : __syncthreads_or(odd | wrong)) {
        if (!wrong && b0 > 0) top = ca.c.row_start[b0];  // they ascended up to here
        wrong = 1;
        int high = b < a.B ? chunk_start(ca.c, first) : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, high, o);
          if (lane >= o) high = max(high, y);
        }
        if (a.B > kCtOrdered) {
          if (lane == 31) s_red[warp] = high;
          __syncthreads();
          for (int w = 0; w < warp; ++w) high = max(high, s_red[w]);
          high = max(high, top);
          for (int w = 0; w < kCtThreads / 32; ++w) top = max(top, s_red[w]);
          __syncthreads();
        }
        if (first < high) n = 0;
      }
      if (L >= 0 && n > 0) {
        mine = (int)(((long long)n * a.G + (1 << ca.shift) - 1) >> ca.shift);
        keys = tiles_of(L, kCtKeys) + tiles_of(n, kCtKeys);
      }
      const int longest_here = __reduce_max_sync(0xffffffffu, keys);
      if (lane == 0) s_len[warp] = longest_here;
      int before = done;
      if (a.B <= kCtOrdered) {
        if (t < kCtOrdered) s_seqs[t] = make_int2(keys, mine);
        __syncthreads();
        if (b < a.B)
          for (int c = 0; c < a.B; ++c) {
            const int2 o = s_seqs[c];
            if (o.x > keys || (o.x == keys && c < b)) before += o.y;
          }
      } else {
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) s_red[warp] = incl;
        __syncthreads();
        int all = done;
        for (int w = 0; w < kCtThreads / 32; ++w) {
          if (w < warp) before += s_red[w];
          all += s_red[w];
        }
        before += incl - mine;
        done = all;
      }
      if (before <= index && index < before + mine) {
        s_seq = b;
        s_tile = index - before;
        s_first = first;
        s_rows = n;
        s_prefix = L;
      }
      if (t == 0)
        for (int w = 0; w < kCtThreads / 32; ++w) s_longest = max(s_longest, s_len[w]);
      __syncthreads();
    }
  }
  auto uni = [](int x) -> int { return __shfl_sync(0xffffffffu, x, 0); };  // the same in every lane, and known to be so
  const int b = uni(s_seq);
  if (b < 0) return;  // fewer tiles than the grid has places for
  const int first = uni(s_first), nrows = uni(s_rows), L = uni(s_prefix);
  // the last tiles have the most keys: they go out first
  const long long all_rows = (long long)nrows * a.G;
  const int row_tiles = (int)((all_rows + (1 << ca.shift) - 1) >> ca.shift);
  const int R0 = (row_tiles - 1 - uni(s_tile)) << ca.shift;             // first row of the KV head's (token, head) rows
  const int real = (int)min(1ll << ca.shift, all_rows - R0);
  const bool shared_rows = uni(real <= 128) != 0;                            // both groups have the same rows
  const int tok_first = ct_token(ca, R0), tok_last = ct_token(ca, R0 + real - 1);
  const int Tp = tiles_of(L, kCtKeys), To = tok_last / kCtKeys + 1, T = Tp + To;
  int parts = 1, per = T;
  if (behind >= 0 && ca.S > 1) {  // shorter sequences have fewer parts
    const int most = max((s_longest + ca.S - 1) / ca.S, 1);
    per = tiles_of(T, (T + most - 1) / most);
    parts = tiles_of(T, per);
  }
  if (part >= parts) return;
  const int t0 = part * per, t1 = min(T, t0 + per);
  const int n8 = uni(max(0, min(t1, Tp) - t0));                         // tiles of the prefix
  const int o0 = uni(max(t0 - Tp, 0)), n16 = uni(max(0, t1 - Tp - o0));      // tiles of the new rows: o0 .. o0 + n16 - 1
  const int n = n8 + n16;
  // tiles that group 0 needs: its last row sees fewer of the new rows
  const int To0 = shared_rows ? To : ct_token(ca, R0 + 127) / kCtKeys + 1;
  const int n_first = uni(shared_rows ? n : n8 + max(0, min(n16, To0 - o0)));
  if (warp == kCtScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&s_tmem)), "r"(kCtTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // users of tile i: group 0 and 1, or i & 1
  auto uses = [&](int w, int i) -> bool { return shared_rows ? (i & 1) == w : (w == 1 || i < n_first); };

  // ---- TMA: the prefix's tiles, K four ahead of its products, V two ahead of its conversion; four where the groups share
  // their rows, in the room of the second group's q (each byte is then used once, and what is in flight bounds the rate) ----
  const int v_stages = shared_rows ? 4 : 2;
  auto v8_at = [&](int stage) -> uint32_t {
    return sb + (stage < 2 ? Sh::off_v8 + (uint32_t)stage * Sh::tile8 : Sh::off_q + Sh::tile16 + (uint32_t)(stage - 2) * Sh::tile8);
  };
  // lane: unit (lane & 7) of tile 4 * (j / 4) + (lane >> 3), 16 keys a unit; pages and scales of the four tiles that come
  // next (n) are in flight ahead
  int pg = -1, sl = 0, pg_n = -1, sl_n = 0;
  float ks = 0.f, vs = 1.f, ks_n = 0.f, vs_n = 1.f;
  auto unit_key = [&](int j0) -> long long {
    const int j = j0 + (lane >> 3);
    const long long key = (long long)(t0 + j) * kCtKeys + 16 * (lane & 7);
    return j < n8 && key < L ? key : -1;
  };
  auto fetch_pages = [&](int j0, int &page, int &slot) {
    const int key = (int)unit_key(j0);
    page = -1;
    if (key >= 0) {
      const int blk = ct_page_index(ca, key);
      slot = key - blk * a.P;
      page = a.block_table[(long long)b * a.max_blocks + blk];
    }
  };
  auto fetch_scales = [&](int j0, int &page, float &k, float &v, bool scales) {
    if (page < 0 || page >= a.num_pages) {
      if (unit_key(j0) >= 0) bad = 1;
      page = -1;
    }
    k = 0.f;
    v = 1.f;
    if (scales && page >= 0) {
      k = a.k_scale[(long long)page * a.Hkv + g];
      v = a.v_scale[(long long)page * a.Hkv + g];
    }
  };
  const int per_box = ca.box / 16;
  // the boxes of tile j into a stage
  auto load8 = [&](int j, const CUtensorMap *map, uint32_t dst, uint32_t full) {
    const int src = 8 * (j & 3) + (lane & 7);
    const int page = __shfl_sync(0xffffffffu, pg, src), slot = __shfl_sync(0xffffffffu, sl, src);
    const uint32_t mine = __ballot_sync(0xffffffffu, lane < 8 && lane % per_box == 0 && page >= 0);
    const uint32_t bytes = (uint32_t)__popc(mine) * (uint32_t)ca.box * D;
    if (lane == 0) {
      if (bytes) mbar_expect_tx(full, bytes);
      else mbar_arrive(full);
    }
    __syncwarp();
    if ((mine >> lane) & 1u) tma_4d(dst + (uint32_t)(lane * 16 * D), map, 0, slot, g, page, full);
  };
  auto load_k8 = [&](int j) {
    // the scales' slot was last read for tile j - 8, whose softmax is past: tile j - 4's scores have run
    const int src = 8 * (j & 3) + (lane & 7), sk = j % kCtStages8;
    const int page = __shfl_sync(0xffffffffu, pg, src);
    const float k = __shfl_sync(0xffffffffu, ks, src), v = clamp_v_scale(__shfl_sync(0xffffffffu, vs, src));
    const uint32_t there = __ballot_sync(0xffffffffu, lane < 8 && page >= 0);
    if (lane < 8) s_scale[j % kCtSlots][lane] = make_float4(k, __log2f(v), __fdividef(1.f, v), 0.f);
    if (lane == 0) s_units[j % kCtSlots] = there;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C_SCALES + j % kCtSlots));
    load8(j, &tm_k, sb + Sh::off_k + (uint32_t)sk * Sh::tile8, bar(C_KFULL + sk));
  };
  auto load_v8 = [&](int j) {
    const int sv = j & (v_stages - 1);
    load8(j, &tm_v, v8_at(sv), bar(C_VFULL + sv));
  };
  // pages of the next tiles, as tile j comes up
  auto turn_pages = [&](int j, bool scales) {
    if ((j & 3) == 0) {
      if (j > 0) {
        pg = pg_n; sl = sl_n; ks = ks_n; vs = vs_n;
      }
      fetch_pages(j + 4, pg_n, sl_n);
    }
    if ((j & 3) == 2) fetch_scales(j + 2, pg_n, ks_n, vs_n, scales);
  };
  auto load16 = [&](int j, bool is_v) {  // one lane; tile j of the new rows
    const int sv = is_v ? (n8 + j) & 1 : j & 1, row = first + (o0 + j) * kCtKeys;
    const uint32_t full = bar((is_v ? C_VTMA : C_K2FULL) + sv), dst = sb + (is_v ? Sh::off_v16 : Sh::off_k) + (uint32_t)sv * Sh::tile16;
    mbar_expect_tx(full, Sh::tile16);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) tma_3d(dst + (uint32_t)x * Sh::half16, is_v ? &tm_vn : &tm_kn, 64 * x, g, row, full);
  };

  // ---- q: D / 8 lanes a row; two e4m3 terms for the prefix, else bf16 at once ----
  const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(a.q);
  auto q_row = [&](int r) -> const __nv_bfloat16 * {  // row r of the block; null past the last
    if (r >= real) return nullptr;
    const int R = R0 + r, i = ct_token(ca, R), h = g * a.G + (R - i * a.G);
    return Q + (long long)(first + i) * ca.c.qs + (long long)h * D;
  };
  constexpr int kLanes = D / 8;  // of a row, eight dims each
  const int qrows = shared_rows ? 128 : 256;
  const long long limit = ca.wait_cycles;
  auto load_q = [&](uint32_t dst, uint32_t full) {  // one lane
    const int token = first + ct_token(ca, R0), tiles = qrows >> 7;
    mbar_expect_tx(full, (uint32_t)tiles * Sh::tile16);
    for (int w = 0; w < tiles; ++w)
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        tma_4d(dst + (uint32_t)w * Sh::tile16 + (uint32_t)x * Sh::half16, &tm_q, 64 * x, 0, g, token + w * (128 / a.G), full);
  };
  // q lands as it is, in two halves of 64 dims a tile and in its place for bf16 products, or where V's fp16 tiles will be
  const uint32_t raw_q = sb + (n8 > 0 ? Sh::off_v16 : Sh::off_q);
  if (warp == kCtTmaWarp || warp == kCtTmaVWarp) {  // the first tiles
    const bool is_v = warp == kCtTmaVWarp;
    if (!is_v && ca.q_tma && lane == 0) load_q(raw_q, bar(C_QRAW));
    __syncwarp();
    if (n8 > 0) {
      fetch_pages(0, pg, sl);
      fetch_scales(0, pg, ks, vs, !is_v);
      for (int j = 0; j < n8 && j < (is_v ? 2 : kCtStages8); ++j) {
        turn_pages(j, !is_v);
        if (is_v) load_v8(j);
        else load_k8(j);
      }
    } else if (lane == 0) {
      for (int j = 0; j < n16 && j < 2; ++j) load16(j, is_v);
    }
  } else if (!ca.q_tma && warp < kCtTmaWarp) {
#pragma unroll 4
    for (int x = t; x < qrows * kLanes; x += kCtTmaWarp * 32) {
      const int r = x / kLanes, c = x % kLanes;
      const uint32_t dst = raw_q + (uint32_t)(r >> 7) * Sh::tile16 + (uint32_t)(c >> 3) * Sh::half16 + sw128(r & 127, c & 7);
      const __nv_bfloat16 *src = q_row(r);
      if (src) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + 8 * c) : "memory");
      else sts128(dst, 0u, 0u, 0u, 0u);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  if (!ca.q_tma) __syncthreads();
  float f8 = 0.f, f16 = a.scale_log2;  // what a score of lifted q and codes, or of bf16 values, stands for in log2 units
  const uint32_t my_q = raw_q + (shared_rows ? 0u : (uint32_t)(warp >> 2) * Sh::tile16);  // a softmax warp's tile
  auto piece = [&](int c, uint32_t (&x)[4]) {  // eight dims of a softmax thread's row
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(my_q + (uint32_t)(c >> 3) * Sh::half16 + sw128(t & 127, c & 7))
                 : "memory");
  };
  auto row_exponent = [&]() -> int {
    // the row's largest magnitude, as the bits of a bf16 value (they order like the values)
    if (ca.q_tma) pt_wait(bar(C_QRAW), 0, &s_abort, limit);
    uint32_t top = 0u;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      uint32_t x[4];
      piece(c, x);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu), __vmaxu2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu)));
    }
    top = max(top & 0xffffu, top >> 16);
    const bool odd = top >= 0x7f80u;  // NaN or infinity: the row scores NaN
    // 2^e2 lifts the largest magnitude into (224, 448], 448 = 1.75 * 2^8 (or, of rows below 2^-118, as far as fp32 goes)
    const int e2 = top == 0u || odd ? 0 : min(126, 135 - max((int)(top >> 7), 1) - ((top & 0x7fu) > 0x60u ? 1 : 0));
    f8 = a.scale_log2 * power_of_two(-e2);
    if (odd) f8 = f16 = __uint_as_float(0x7fc00000u);
    return e2;
  };
  if (warp < 8 && n8 > 0) {
    // (fp16 holds the lifted bf16 values, and their distance to the first term, as they are down to 2^-14, and with an error of
    // 2^-25 below; the second term's last bit is 2^-9.)  Groups that share their rows take half of the dims each
    const float lift = power_of_two(row_exponent());
    const int r = t & 127;
    const uint32_t dst = sb + Sh::off_q + (shared_rows ? 0u : (uint32_t)(warp >> 2) * Sh::tile16);
    const int c0 = shared_rows && warp >= 4 ? D / 32 : 0, c1 = shared_rows && warp < 4 ? D / 32 : D / 16;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
        piece(2 * c + h, x);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t h2[2], l2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const __half2 y = __floats2half2_rn(__uint_as_float(x[2 * e + k] << 16) * lift, __uint_as_float(x[2 * e + k] & 0xffff0000u) * lift);
            h2[k] = f16x2_to_e4m3x2(y);
            const uint32_t hf = f8x2_to_f16x2<ET_KV_E4M3>((uint16_t)h2[k]);
            l2[k] = f16x2_to_e4m3x2(__hsub2(y, *reinterpret_cast<const __half2 *>(&hf)));
          }
          hi[2 * h + e] = h2[0] | h2[1] << 16;
          lo[2 * h + e] = l2[0] | l2[1] << 16;
        }
      }
      sts128(dst + at8<D>(r, c), hi[0], hi[1], hi[2], hi[3]);
      sts128(dst + Sh::tile8 + at8<D>(r, c), lo[0], lo[1], lo[2], lo[3]);
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // after the TMEM allocation: a waiting dependent block must not hold what this block needs
  const uint32_t tmem = (uint32_t)uni((int)s_tmem);
  const uint32_t lead = elect_lane() ? 1u : 0u;
  float l = 0.f, ref = 0.f;   // a softmax thread's row: sum of weights, reference
  bool fresh = true;          // no key seen yet
  int items = 0;              // tiles this group has taken

  // a softmax thread holds a row's 128 scores: it gets registers of the other warps (512 x 128 = 256 x 48 + 256 x 208; at 64 and 192 it spills)
  if (warp >= kCtTmaWarp) {
  regs_down<48>();
  if (warp == kCtTmaWarp) {
    // ---------------- TMA: K ----------------
    bool ok = true;
    int issued = min(n8, kCtStages8), issued16 = n8 == 0 ? min(n16, 2) : 0;
    for (int j = issued; j < n8; ++j) {
      turn_pages(j, true);
      ok = pt_wait(bar(C_KEMPTY + j % kCtStages8), (uint32_t)(j / kCtStages8 - 1) & 1u, &s_abort, limit);
      if (!__all_sync(0xffffffffu, ok)) break;
      load_k8(j);
      issued = j + 1;
    }
    if (bad) flag_status(a.dev_status, ET_DEV_BAD_INDEX);
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
      bool q_again = false;
      if (n8 > 0 && n16 > 0) {
        ok = ok && pt_wait(bar(C_QFREE), 0, &s_abort, limit);
        if (ok && ca.q_tma) {  // q as it is, for the new rows' keys
          load_q(sb + Sh::off_q, bar(C_QFULL));
          q_again = true;
        }
      }
      for (int j = issued16; ok && j < n16; ++j) {
        if (j >= 2 && !pt_wait(bar(C_K2EMPTY + (j & 1)), (uint32_t)((j >> 1) - 1) & 1u, &s_abort, limit)) break;
        load16(j, false);
        issued16 = j + 1;
      }
      // no copy may be in flight when the block leaves
      if (ca.q_tma) ct_drain(bar(C_QRAW), 0);
      if (q_again) ct_drain(bar(C_QFULL), 0);
      for (int j = max(0, issued - kCtStages8); j < issued; ++j)
        ct_drain(bar(C_KFULL + j % kCtStages8), (uint32_t)(j / kCtStages8) & 1u);
      for (int j = max(0, issued16 - 2); j < issued16; ++j) ct_drain(bar(C_K2FULL + (j & 1)), (uint32_t)(j >> 1) & 1u);
    }
  } else if (warp == kCtTmaVWarp) {
    // ---------------- TMA: V ----------------
    bool ok = true;
    int issued = min(n8, 2), issued16 = n8 == 0 ? min(n16, 2) : 0;
    for (int j = issued; j < n8; ++j) {
      turn_pages(j, false);
      if (j >= v_stages)
        ok = pt_wait(bar(C_VEMPTY + (j & (v_stages - 1))), (uint32_t)(j / v_stages - 1) & 1u, &s_abort, limit);
      if (!__all_sync(0xffffffffu, ok)) break;
      load_v8(j);
      issued = j + 1;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
      // The buffers' phases have not been followed so far.  With the prefix's scores done, the product of tile n8 - 3 has run:
      // from there on a buffer is at the phase before the one that is waited for, and a parity tells them apart
      if (n8 > 0 && n16 > 0) ok = ok && pt_wait(bar(C_QFREE), 0, &s_abort, limit);
      for (int j = issued16; ok && j < n16; ++j) {
        const int i = n8 + j;
        if (i >= 2 && !pt_wait(bar(C_VHFREE + (i & 1)), (uint32_t)((i >> 1) - 1) & 1u, &s_abort, limit)) break;
        load16(j, true);
        issued16 = j + 1;
      }
      for (int j = max(0, issued - v_stages); j < issued; ++j)
        ct_drain(bar(C_VFULL + (j & (v_stages - 1))), (uint32_t)(j / v_stages) & 1u);
      // bf16 tiles of V: the k-th of a buffer is its k-th arrival
      for (int j = max(0, issued16 - 2); j < issued16; ++j) {
        const int sv = (n8 + j) & 1, first_j = (n8 & 1) == sv ? 0 : 1;
        ct_drain(bar(C_VTMA + sv), (uint32_t)((j - first_j) >> 1) & 1u);
      }
    }
  } else if (warp == kCtScoreWarp) {
    // ---------------- score products ----------------
    {
      constexpr uint32_t i8 = pt_idesc(0, FMT == ET_KV_E4M3 ? 0 : 1, false, false, 128, kCtKeys);
      constexpr uint32_t i16 = pt_idesc(1, 1, false, false, 128, kCtKeys);
      int k[2] = {0, 0};
      bool ok = !ca.q_tma || pt_wait(bar(C_QRAW), 0, &s_abort, limit);
      ok = __all_sync(0xffffffffu, ok);
      for (int i = 0; ok && i < n; ++i) {
        const int j = i - n8, sk = i < n8 ? i % kCtStages8 : j & 1;
        if (i < n8) {
          ok = pt_wait(bar(C_KFULL + sk), (uint32_t)(i / kCtStages8) & 1u, &s_abort, limit);
        } else {
          if (j == 0 && n8 > 0) ok = pt_wait(bar(C_QFULL), 0, &s_abort, limit);
          ok = ok && pt_wait(bar(C_K2FULL + sk), (uint32_t)(j >> 1) & 1u, &s_abort, limit);
        }
        ok = __all_sync(0xffffffffu, ok);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || !uses(w, i)) continue;
          // S lies where P of the group's last tile was: that product has run
          if (k[w] > 0) ok = pt_wait(bar(C_PVDONE + w), (uint32_t)(k[w] - 1) & 1u, &s_abort, limit);
          // the groups run half a turn apart, so that one's products find the tensor cores free
          else if (w == 1 && k[0] > 0 && !shared_rows) ok = pt_wait(bar(C_PHALF), 0, &s_abort, limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          tc_fence_after();
          const uint32_t q = sb + Sh::off_q + (shared_rows ? 0u : (uint32_t)w * Sh::tile16), d = tmem + kCtColS + 128u * (uint32_t)w;
          if (i < n8) {
            const uint64_t qd = desc8<D>(q), kd = desc8<D>(sb + Sh::off_k + (uint32_t)sk * Sh::tile8);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)  // the two terms of q one after the other
              ct_mma_f8(d, qd + (((kk / (D / 32)) * Sh::tile8 + (kk % (D / 32)) * 32) >> 4), kd + ((kk % (D / 32)) * 32 >> 4), i8, kk > 0, lead);
          } else {
            const uint64_t qd = sw128_desc(q, 16, 1024), kd = sw128_desc(sb + Sh::off_k + (uint32_t)sk * Sh::tile16, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              ct_mma(d, qd + (((kk >> 2) * Sh::half16 + (kk & 3) * 32) >> 4), kd + (((kk >> 2) * Sh::half16 + (kk & 3) * 32) >> 4), i16, kk > 0, lead);
          }
          ct_commit(bar(C_SFULL + w), lead);
          ++k[w];
        }
        if (!ok) break;
        {
          if (i < n8 && i + kCtStages8 < n8) ct_commit(bar(C_KEMPTY + sk), lead);
          if (i >= n8 && j + 2 < n16) ct_commit(bar(C_K2EMPTY + sk), lead);
          if (i == n8 - 1 && n16 > 0) ct_commit(bar(C_QFREE), lead);
        }
      }
      // every product this thread issued has finished before TMEM is freed
      ct_commit(bar(C_DRAIN), lead);
      ct_drain(bar(C_DRAIN), 0);
    }
  } else if (warp == kCtPvWarp) {
    // ---------------- P.V products ----------------
    {
      constexpr uint32_t i8 = pt_idesc(0, 0, false, true, 128, D), i16 = pt_idesc(1, 1, false, true, 128, D);
      int k[2] = {0, 0};
      bool ok = true;
      for (int i = 0; ok && i < n; ++i) {
        ok = pt_wait(bar(C_VHFULL + (i & 1)), (uint32_t)(i >> 1) & 1u, &s_abort, limit);
        ok = __all_sync(0xffffffffu, ok);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || !uses(w, i)) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && pt_wait(bar((h ? C_PFULL : C_PHALF) + w), (uint32_t)k[w] & 1u, &s_abort, limit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            {
              const uint64_t vd = sw128_desc(sb + Sh::off_v16 + (uint32_t)(i & 1) * Sh::tile16, Sh::half16, 1024);
              const uint32_t o = tmem + kCtColO + 128u * (uint32_t)w, p = tmem + kCtColS + 128u * (uint32_t)w;
              const uint32_t id = i < n8 ? i8 : i16;
#pragma unroll
              for (int kk = 4 * h; kk < 4 * h + 4; ++kk) ct_mma_ts(o, p + 8u * kk, vd + (kk * 2048 >> 4), id, (k[w] > 0 || kk > 0) ? 1u : 0u, lead);
              if (h) ct_commit(bar(C_PVDONE + w), lead);
            }
          }
          if (!ok) continue;
          ++k[w];
        }
        if (!ok) break;
        ct_commit(bar(C_VHFREE + (i & 1)), lead);
      }
      ct_commit(bar(C_DRAIN + 1), lead);
      ct_drain(bar(C_DRAIN + 1), 0);
    }
  }
  __syncwarp();
  roles_end();
  regs_up<128>();
  } else if (warp >= 8) {
    regs_down<48>();
    // ---------------- V as the products take it ----------------
    const int gt = t & 127;
    bool ok = true;
    for (int i = 0; i < n8; ++i) {
      const int sv = i & 1, s8 = i & (v_stages - 1);
      ok = ok && pt_wait(bar(C_VFULL + s8), (uint32_t)(i / v_stages) & 1u, &s_abort, limit);
      // the K warp says which units there are
      if (ok) ok = pt_wait(bar(C_SCALES + i % kCtSlots), (uint32_t)(i / kCtSlots) & 1u, &s_abort, limit);
      if (ok && i >= 2) ok = pt_wait(bar(C_VHFREE + sv), (uint32_t)((i >> 1) - 1) & 1u, &s_abort, limit);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      const uint32_t units = *(volatile uint32_t *)&s_units[i % kCtSlots];
      const int lim = L - (t0 + i) * kCtKeys;  // rows past it hold no key of this sequence
      const bool whole = lim >= kCtKeys && units == 0xffu;
      // 16 codes of a row a thread, read as two chunks of eight.  Which one it takes first alternates between the 64-dim
      // halves, which keeps the stores free of bank conflicts, and between rows, which keeps the reads free of them
      constexpr int C = D / 16, RP = 128 / C, ROUNDS = kCtKeys / RP;  // 16-code chunks of a row; rows the threads take at once
      const int c = gt % C, r0 = gt / C, c0 = 2 * (c & 3), s = (c >> 2) ^ (r0 & 1);
      const uint32_t from = v8_at(s8) + at8<D>(r0, c), to = sb + Sh::off_v16 + (uint32_t)sv * Sh::tile16 + (uint32_t)(c >> 2) * Sh::half16;
      const uint32_t from0 = from + 8u * (uint32_t)s, from1 = from + 8u - 8u * (uint32_t)s;
      const uint32_t to0 = to + sw128(r0, c0 + s), to1 = to + sw128(r0, c0 + 1 - s);
      static_assert(RP % 8 == 0, "a row's place in its group of eight is the thread's own");
#pragma unroll 2
      for (int k = 0; k < ROUNDS; ++k) {
        const uint32_t in = (uint32_t)(k * RP * D), out = (uint32_t)(k * RP * 128);
        uint4 v;
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(from0 + in));
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.z), "=r"(v.w) : "r"(from1 + in));
        if (!whole) {
          const int r = r0 + RP * k;
          if (r >= lim || !((units >> (r >> 4)) & 1u)) v = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t h[8];
        f8x4_to_f16<FMT>(v.x, h[0], h[1]);
        f8x4_to_f16<FMT>(v.y, h[2], h[3]);
        f8x4_to_f16<FMT>(v.z, h[4], h[5]);
        f8x4_to_f16<FMT>(v.w, h[6], h[7]);
        sts128(to0 + out, h[0], h[1], h[2], h[3]);
        sts128(to1 + out, h[4], h[5], h[6], h[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C_VEMPTY + s8));
        mbar_arrive(bar(C_VHFULL + sv));
      }
    }
    if (n16 > 0) {
      if (ok && n8 > 0 && !ca.q_tma) {  // q as it is, once the prefix's score products have run
        ok = __all_sync(0xffffffffu, pt_wait(bar(C_QFREE), 0, &s_abort, limit));
        if (ok) {
#pragma unroll 4
          for (int x = gt; x < qrows * kLanes; x += 128) {
            const int qr = x / kLanes, c = x % kLanes;
            const uint32_t dst = sb + Sh::off_q + (uint32_t)(qr >> 7) * Sh::tile16 + (uint32_t)(c >> 3) * Sh::half16 + sw128(qr & 127, c & 7);
            const __nv_bfloat16 *src = q_row(qr);
            if (src) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + 8 * c) : "memory");
            else sts128(dst, 0u, 0u, 0u, 0u);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C_QFULL));
        }
      }
      bool odd = false;
      for (int j = 0; ok && j < n16; ++j) {
        const int i = n8 + j, sv = i & 1, first_j = (n8 & 1) == sv ? 0 : 1;
        ok = __all_sync(0xffffffffu, pt_wait(bar(C_VTMA + sv), (uint32_t)((j - first_j) >> 1) & 1u, &s_abort, limit));
        if (!ok) break;
        const int key0 = (o0 + j) * kCtKeys;
        if (key0 + kCtKeys - 1 > tok_first) {
          // some row does not see some key here: 0 * NaN must not reach it.  What is not finite is taken out and added
          // to the rows that see it at the end; rows past the block's last token are nobody's
          for (int x = gt; x < kCtKeys * (D / 8); x += 128) {
            const int r = x / (D / 8), c = x % (D / 8);
            const uint32_t at = sb + Sh::off_v16 + (uint32_t)sv * Sh::tile16 + (uint32_t)(c >> 3) * Sh::half16 + sw128(r, c & 7);
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
            bool change = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; change = true; }
              if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0xffffu; change = true; }
            }
            if (change) sts128(at, w[0], w[1], w[2], w[3]);
            odd = odd || (change && key0 + r <= tok_last);
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C_VHFULL + sv));
      }
      if (odd) s_odd = 1;
    }
    __syncwarp();
    roles_end();
    regs_up<128>();
  } else {
    regs_up<208>();
    // ---------------- softmax: group w, a row per thread ----------------
    const int w = warp >> 2, r = t & 127, Rr = shared_rows ? r : 128 * w + r;
    const int tok = Rr < real ? ct_token(ca, R0 + Rr) : -1;  // rows that do not exist see nothing
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sc = lanes + kCtColS + 128u * (uint32_t)w, oc = lanes + kCtColO + 128u * (uint32_t)w;
    if (n8 == 0) row_exponent();  // under the first product
    bool dead = false;
    // the weights of one tile from its scores; `own`: the new rows' keys
    auto tile = [&](int i, auto own_, auto masked_) {
      constexpr bool own = decltype(own_)::value, masked = decltype(masked_)::value;
      const int slot = i % kCtSlots;
      // a unit's factor, offset and inverse V scale, before the scores are there
      float fu[kCtKeys / 16], cu[kCtKeys / 16], iu[kCtKeys / 16];
      if (!own) {
#pragma unroll
        for (int u = 0; u < kCtKeys / 16; ++u) {
          float ks, lv;
          lds_f4(saddr(&s_scale[slot][u]), ks, lv, iu[u]);
          fu[u] = f8 * ks;
          cu[u] = lv - ref;
        }
      }
      int lim = 0;
      uint32_t units = 0xffu;
      if (masked) {
        if (own) {
          lim = tok - (o0 + i - n8) * kCtKeys + 1;
        } else {
          units = *(volatile uint32_t *)&s_units[slot];
          lim = tok < 0 ? 0 : L - (t0 + i) * kCtKeys;
        }
      }
      dead = dead || !pt_wait(bar(C_SFULL + w), (uint32_t)items & 1u, &s_abort, limit);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) return;
      tc_fence_after();
      uint32_t raw[kCtKeys / 32][32];
#pragma unroll
      for (int p = 0; p < kCtKeys / 32; ++p) tmem_ld32(sc + 32u * p, raw[p]);
      tmem_wait_ld();
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains: one would wait for itself
#pragma unroll
      for (int u = 0; u < kCtKeys / 16; ++u) {
        const float f = own ? f16 : fu[u], c = own ? -ref : cu[u];
        const uint64_t f2 = pair(f, f), c2 = pair(c, c);
        int limu = masked ? lim - 16 * u : 16;
        if (masked && !own && !((units >> u) & 1u)) limu = 0;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          uint32_t *x = &raw[u >> 1][16 * (u & 1) + e];
          float x0, x1;
          unpair(fma2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, c2), x0, x1);
          if (masked) {
            x0 = e < limu ? x0 : -INFINITY;
            x1 = e + 1 < limu ? x1 : -INFINITY;
          }
          tops[(e >> 1) & 3] = fmaxf(tops[(e >> 1) & 3], fmaxf(x0, x1));
          x[0] = __float_as_uint(x0);
          x[1] = __float_as_uint(x1);
        }
      }
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      const bool move = top > kPaTop + kPaSlack || (fresh && top > -INFINITY);
      if (__any_sync(0xffffffffu, move)) {
        const float now = move ? top + ref - kPaTop : ref, by = move ? ref - now : 0.f;
        const float corr = fresh ? 0.f : ex2_fast(by);
        if (move) {
          l *= corr;
          ref = now;
        }
#pragma unroll
        for (int p = 0; p < kCtKeys / 32; ++p)
#pragma unroll
          for (int e = 0; e < 32; ++e) raw[p][e] = __float_as_uint(__uint_as_float(raw[p][e]) + by);
        if (items > 0) {  // O holds the sums of this group's earlier tiles
          const float by_o = move ? corr : 1.f;
#pragma unroll 1
          for (int p = 0; p < D / 8; ++p) {
            uint32_t o[8];
            pt_ld8(oc + 8u * p, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by_o);
            pt_st8(oc + 8u * p, o);
          }
        }
        if (move) fresh = false;
      }
      uint64_t l2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int p = 0; p < kCtKeys / 32; ++p) {
        uint32_t pk[16];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint64_t iv2 = own ? 0ull : pair(iu[2 * p + u], iu[2 * p + u]);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float w0 = ex2_fast(__uint_as_float(raw[p][16 * u + e])), w1 = ex2_fast(__uint_as_float(raw[p][16 * u + e + 1]));
            l2[(e >> 1) & 3] = own ? add2(pair(w0, w1), l2[(e >> 1) & 3]) : fma2(pair(w0, w1), iv2, l2[(e >> 1) & 3]);
            pk[8 * u + (e >> 1)] = own ? pack_bf16x2(w0, w1) : pack_f16x2(w0, w1);
          }
        }
        tmem_st16(sc + 16u * p, pk);
        if (p == 1) {  // the first 64 keys' weights: their product may begin
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C_PHALF + w));
        }
      }
      float s0, s1;
      unpair(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])), s0, s1);
      l += s0 + s1;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C_PFULL + w));
      ++items;
    };
    // A warp without a row that exists (few rows) leaves its lanes of P as they are, which is its own rows' matter, and the
    // issue slots to the others
    const bool idle = uni((Rr & ~31) >= real) != 0;
    for (int i = 0; idle && i < n; ++i) {
      if (!uses(w, i)) continue;
      dead = __any_sync(0xffffffffu, !pt_wait(bar(C_SFULL + w), (uint32_t)items & 1u, &s_abort, limit));
      if (dead) break;
      if (lane == 0) {
        mbar_arrive(bar(C_PHALF + w));
        mbar_arrive(bar(C_PFULL + w));
      }
      ++items;
    }
    for (int i = idle ? n : 0; i < n; ++i) {
      if (!uses(w, i)) continue;
      if (i < n8) dead = dead || !pt_wait(bar(C_SCALES + i % kCtSlots), (uint32_t)(i / kCtSlots) & 1u, &s_abort, limit);
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      if (i < n8) {
        const bool whole = L - (t0 + i) * kCtKeys >= kCtKeys && *(volatile uint32_t *)&s_units[i % kCtSlots] == 0xffu;
        if (whole) tile(i, std::false_type{}, std::false_type{});
        else tile(i, std::false_type{}, std::true_type{});
      } else {
        const bool whole = (o0 + i - n8) * kCtKeys + kCtKeys - 1 <= ct_token(ca, R0 + (shared_rows ? 0 : 128 * w));
        if (whole) tile(i, std::true_type{}, std::false_type{});
        else tile(i, std::true_type{}, std::true_type{});
      }
    }
    if (items && !dead) pt_wait(bar(C_PVDONE + w), (uint32_t)(items - 1) & 1u, &s_abort, limit);
    __syncwarp();
    regs_down<128>();
    roles_end();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*(volatile int *)&s_abort != 0 && t == 0) flag_status(a.dev_status, ET_DEV_TIMEOUT);

  // ---- the rows: one group's, or the two groups' halves of the keys joined ----
  float *xo = reinterpret_cast<float *>(sm + Sh::off_q);     // [D][128]: of each dim what the group gives that does not join it
  float2 *xm = reinterpret_cast<float2 *>(sm + Sh::off_v8);  // [2][128]
  // the rows as they go out: behind the other group's, or (fp32 rows of both groups) from the start
  const uint32_t stage = sb + (parts > 1 && !shared_rows ? Sh::off_q : Sh::off_k);
  const long long slot0 = (((long long)cut * ca.S + part) << ca.shift);
  const int w = warp >> 2, r = t & 127, Rr = shared_rows ? r : 128 * w + r;
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kCtColO + 128u * (uint32_t)w;
  if (shared_rows && warp < 8) {  // a group joins half of the dims and gives the other half away
    xm[128 * w + r] = make_float2(fresh ? -3e38f : ref, l);
    float *give = xo + (1 - w) * (D / 2) * 128 + r;
#pragma unroll 1
    for (int p = 0; p < D / 64; ++p) {
      uint32_t o[32];
      if (items > 0) {
        tmem_ld32(lanes + (uint32_t)((1 - w) * (D / 2) + 32 * p), o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) give[(32 * p + e) * 128] = items > 0 ? __uint_as_float(o[e]) : 0.f;
    }
  }
  __syncthreads();
  if (warp < 8) {
    float M = fresh ? -3e38f : ref, mine = 1.f, other = 0.f;
    if (shared_rows) {
      const float2 y = xm[128 * (1 - w) + r];
      const float both = fmaxf(M, y.x);
      mine = ex2_fast(M - both);
      other = ex2_fast(y.x - both);
      l = fmaf(l, mine, y.y * other);
      M = both;
    }
    const bool mine_any = items > 0;
    const int R = R0 + Rr, i = ct_token(ca, R), h = g * a.G + (R - i * a.G);
    const long long row = (long long)(first + i) * a.Hq + h;
    const bool odd = s_odd != 0;
    if (parts == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      mine *= inv;
      other *= inv;
      if (Rr < real && a.lse && (w == 0 || !shared_rows)) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
    } else if (Rr < real && (w == 0 || !shared_rows)) {
      ca.part_ml[slot0 + Rr] = make_float2(M, l);
    }
#pragma unroll 1
    for (int p = shared_rows ? w * (D / 64) : 0; p < (shared_rows ? (w + 1) * (D / 64) : D / 32); ++p) {
      uint32_t o[32];
      tmem_ld32(lanes + 32u * p, o);
      tmem_wait_ld();
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = mine_any ? __uint_as_float(o[e]) * mine : 0.f;
      if (shared_rows) {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = fmaf(xo[(32 * p + e) * 128 + r], other, x[e]);
      }
      if (odd && Rr < real) {
        // values that are not finite, taken out of the tiles that not every row sees whole
        const int from = max(tok_first / kCtKeys, o0) * kCtKeys, to = min(i, (o0 + n16) * kCtKeys - 1);
#pragma unroll 1
        for (int key = from; key <= to; ++key) {
          const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.vt) + (long long)(first + key) * ca.c.vs + (long long)g * D + 32 * p;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float z = __bfloat162float(v[e]);
            if (!(fabsf(z) <= FLT_MAX)) x[e] += z;
          }
        }
      }
      // through shared memory, where rows are written one by one: a row's 16-byte pieces trade places by the row's number
      if (parts == 1) {
        const uint32_t dst = stage + (uint32_t)(Rr * D * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sts128(dst + (uint32_t)(((4 * p + e) ^ (Rr & 7)) << 4), pack_bf16x2(x[8 * e], x[8 * e + 1]), pack_bf16x2(x[8 * e + 2], x[8 * e + 3]),
                 pack_bf16x2(x[8 * e + 4], x[8 * e + 5]), pack_bf16x2(x[8 * e + 6], x[8 * e + 7]));
      } else {
        const uint32_t dst = stage + (uint32_t)(Rr * D * 4);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sts128(dst + (uint32_t)(((8 * p + e) ^ (Rr & 7)) << 4), __float_as_uint(x[4 * e]), __float_as_uint(x[4 * e + 1]),
                 __float_as_uint(x[4 * e + 2]), __float_as_uint(x[4 * e + 3]));
      }
    }
  }
  __syncthreads();
  {
    const int per_row = parts == 1 ? D / 8 : D / 4;  // 16-byte pieces
#pragma unroll 4
    for (int x = t; x < real * per_row; x += kCtThreads) {
      const int rr = x / per_row, c = x - rr * per_row;
      const uint4 v = *reinterpret_cast<const uint4 *>(sm + (stage - sb) + (uint32_t)(16 * (rr * per_row + (c ^ (rr & 7)))));
      if (parts == 1) {
        const int R = R0 + rr, i = ct_token(ca, R), h = g * a.G + (R - i * a.G);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + ((long long)(first + i) * a.Hq + h) * D + 8 * c) = v;
      } else {
        reinterpret_cast<uint4 *>(ca.part_o)[(slot0 + rr) * (D / 4) + c] = v;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kCtScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCtTmemCols) : "memory");
  if (parts == 1) return;
  // ---- the parts' rows, merged by the last block to arrive ----
  if (!arrive_last(ca.cnt + cut, (unsigned)parts, &s_last)) return;
  const long long base = (long long)cut * ca.S << ca.shift;
  float *share = reinterpret_cast<float *>(sm);  // [parts][256]: what a part's row counts for
  if (t < real) {
    float M = -3e38f, sum = 0.f;
    for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(&ca.part_ml[base + (k << ca.shift) + t]).x);
    for (int k = 0; k < parts; ++k) {
      const float2 e = __ldcg(&ca.part_ml[base + (k << ca.shift) + t]);
      const float f = ex2_fast(e.x - M);
      sum = fmaf(e.y, f, sum);
      share[k * 256 + t] = f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int k = 0; k < parts; ++k) share[k * 256 + t] *= inv;
    const int R = R0 + t, i = ct_token(ca, R);
    if (a.lse)
      a.lse[(long long)(first + i) * a.Hq + g * a.G + (R - i * a.G)] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
  }
  __syncthreads();
  // four pieces a thread, two parts at a time: eight loads under way
  const int pieces = real * (D / 4);
#pragma unroll 1
  for (int x0 = t; x0 < pieces; x0 += 4 * kCtThreads) {
    float4 v[4] = {};
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
      const float4 *from = ca.part_o + (base + (k << ca.shift)) * (D / 4);
      float4 y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __ldcg(&from[min(x0 + e * kCtThreads, pieces - 1)]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = share[k * 256 + min(x0 + e * kCtThreads, pieces - 1) / (D / 4)];
        v[e].x = fmaf(y[e].x, f, v[e].x); v[e].y = fmaf(y[e].y, f, v[e].y);
        v[e].z = fmaf(y[e].z, f, v[e].z); v[e].w = fmaf(y[e].w, f, v[e].w);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = x0 + e * kCtThreads, rr = x / (D / 4), c = x % (D / 4);
      if (x >= pieces) break;
      const int R = R0 + rr, i = ct_token(ca, R), h = g * a.G + (R - i * a.G);
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + ((long long)(first + i) * a.Hq + h) * D + 4 * c) =
          make_uint2(pack_bf16x2(v[e].x, v[e].y), pack_bf16x2(v[e].z, v[e].w));
    }
  }
}

// new keys or values: [rows][Hkv][D], rows `stride` elements apart; a box is 128 rows of 64 dims of one head
bool make_new_map(CUtensorMap *m, const void *base, const ChunkArgs &c, int d, long long stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)c.a.Hkv, (cuuint64_t)c.rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t boxes[3] = {64, 1, kCtKeys};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, boxes, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q: [rows][Hkv][G][D]; a box is the rows of 128 / G tokens of one KV head, 64 dims
bool make_q_map(CUtensorMap *m, const ChunkArgs &c, int d) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)c.a.G, (cuuint64_t)c.a.Hkv, (cuuint64_t)c.rows};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)c.a.G * d * 2, (cuuint64_t)c.qs * 2};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)c.a.G, 1, (cuuint32_t)(128 / c.a.G)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(c.a.q), dims, strides, boxes, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT>
et_status launch_tc(const CUtensorMap (&m)[5], const ChunkTcArgs &ca, cudaStream_t st) {
  if (et_smem_attr((const void *)k_chunk_tc<D, FMT>, (int)CtShape<D>::bytes) != cudaSuccess) return ET_ERR_CUDA;
  const long long blocks = ca.whole + ((long long)ca.tiles * ca.c.a.Hkv - ca.whole) * ca.S;
  return et_launch(k_chunk_tc<D, FMT>, dim3((unsigned)blocks), dim3(kCtThreads), CtShape<D>::bytes, st, 0, m[0], m[1], m[2],
                   m[3], m[4], ca);
}

}  // namespace

et_status chunk_tc_launch(const et_paged_cache *cache, const ChunkArgs &c, const ChunkTcPlan &p, void *ws, cudaStream_t st) {
  if (!encode_fn()) return ET_ERR_CUDA;
  ChunkTcArgs ca;
  ca.c = c;
  ca.S = p.S;
  ca.shift = p.shift;
  ca.tiles = p.tiles;
  ca.whole = p.whole;
  const int P = cache->page_size;
  ca.box = P % 128 == 0 ? 128 : P % 64 == 0 ? 64 : P % 32 == 0 ? 32 : 16;
  unsigned char *wsb = static_cast<unsigned char *>(ws);
  ca.cnt = p.S > 1 ? reinterpret_cast<unsigned int *>(wsb) : nullptr;
  ca.part_ml = p.S > 1 ? reinterpret_cast<float2 *>(wsb + p.ml_off) : nullptr;
  ca.part_o = p.S > 1 ? reinterpret_cast<float4 *>(wsb + p.o_off) : nullptr;
  const uint32_t units = (uint32_t)P / 16, G = (uint32_t)c.a.G;
  ca.page_magic = units == 1 ? 0u : (uint32_t)(((1ull << 32) + units - 1) / units);
  ca.group_shift = 0;
  while ((2ull << ca.group_shift) < G) ++ca.group_shift;
  ca.group_magic = G == 1 ? 0u : (uint32_t)(((1ull << (32 + ca.group_shift)) + G - 1) / G);
  ca.wait_cycles = et_wait_limit_cycles();
  CUtensorMap m[5];
  ca.q_tma = G <= 128 && 128 % G == 0;
  if (!make_page_map(&m[0], cache->k_pages, cache, ca.box) || !make_page_map(&m[1], cache->v_pages, cache, ca.box) ||
      !make_new_map(&m[2], c.a.kt, c, cache->d, c.ks) || !make_new_map(&m[3], c.a.vt, c, cache->d, c.vs) || (ca.q_tma && !make_q_map(&m[4], c, cache->d)))
    return ET_ERR_INVALID_ARG;
  if (!ca.q_tma) m[4] = m[2];  // not read
  const bool e4m3 = cache->format == ET_KV_E4M3;
  if (cache->d == 64) return e4m3 ? launch_tc<64, ET_KV_E4M3>(m, ca, st) : launch_tc<64, ET_KV_E5M2>(m, ca, st);
  return e4m3 ? launch_tc<128, ET_KV_E4M3>(m, ca, st) : launch_tc<128, ET_KV_E5M2>(m, ca, st);
}

}  // namespace et
