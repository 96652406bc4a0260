// Attention over the paged cache for many rows per request (prompts, chunks of
// prompts, mixed steps), on the 5th-generation tensor cores.
//
// A CTA takes tiles of 128 rows ((token, query head of the group) pairs) of one
// key/value head: two tiles that share the cache blocks (bf16 activations), or
// one (fp32, whose query takes three times the shared memory).  The cache comes in
// blocks of BT tokens: 128, or 64 (fp32: the weights' three parts lie over their
// scores, and two score regions and O have to fit the 512 columns of TMEM).  Per block and tile
//   S = Q K^T        tcgen05.mma, both operands in shared memory, S in TMEM
//   P = exp2(S - m)  one thread per row reads S, writes P over it (in bf16 parts)
//   O += P V         tcgen05.mma, P from TMEM, V^T straight from V's rows (MN-major)
// Roles: 4 warps per tile for the rows (fp32: 16 warps, four threads per row), 1
// thread issues MMAs, 3 to 7 warps load.  While one tile's rows are worked on, the
// tensor cores run the other tile's products (fp32: the next block's scores).
// A row's maximum moves only when it grows by more than 2^8, so that O is
// seldom rescaled; the weights are then at most 2^8, far inside bf16 and fp32.
//
// fp32 activations: query and weights as three bf16 parts each (24 bits), their
// products added in the accumulator; every block's O leaves the accumulator,
// which truncates, and is added in registers with rounding.
//
// bf16 activations: the query is exact, a weight has two bf16 parts (16 bits).  With
// one, the rounding of the weights is as large as the output's own (four windowed
// prompts, error against 64 bits: 2.1e-3 instead of 1.6e-3, at 219 us instead of 248),
// and a row's precision would depend on how many rows its request has.
//
// A 4-bit cache is widened by the loading warps to bf16 integers q (exact); the
// token's scale multiplies its score or its weight.
//
// The work line (paged_sched.cuh) is divided evenly among the CTAs whatever the
// lengths are; units that fall on two CTAs are joined by attn_join_kernel.
//
// Measured (32 query and 8 key/value heads of 128):
//   bf16, four prompts with a window: 239 us, 368 TFLOP/s of the seen pairs; two without
//     a window: 192 us, 650 TFLOP/s.  The windowed ones have fewer blocks per CTA (45
//     against 51) but more that are partial (11.6 against 2.1: copied by the threads, one
//     slot at a time) and more units (5 against 2.5: the next unit's scores wait for all
//     values of the last).  With one part per weight a block of 2 x 128 rows x 128 tokens
//     took 2.2 us, by timestamps: a tile's rows work 1.1 us, in which they read the scores
//     from TMEM twice, a chunk at a time, and 1.1 pass from its weights to its next
//     scores, while the rows of the other tile work; the 16 MMAs between are 0.5 us by
//     themselves.  The second part costs 14 us of MMAs and 20 of the rows (192 us).
//   fp32 over 4 bits, two prompts: 470 us, 264 TFLOP/s, three times that in MMAs: each is
//     done for three parts.  A block of 64 tokens takes 1.9 us, all of it on the MMA
//     thread; its 36 MMAs run in 1.05 alone, the scores' at the rate at which shared
//     memory gives the query.
//   fp32 over bf16: 443 us.
// fp32 rows over 4 bits took 700 us with two threads per row, whose queries the loaders brought in
// between two units and whose MMA thread walked the work line itself.
#include <cfloat>
#include <cuda.h>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"
#include "paged_sched.cuh"
#include "tc.cuh"

namespace dualar {

// Limit of every wait inside the kernel.  A constant: read from the arguments it costs
// fp32 rows over 4 bits 3% (two prompts: 488 us instead of 474).
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLazyMax = 8.f;                     // a row's maximum may lag by this (log2)

template <int HD, int BITS, bool F32>
struct Pro {
  static constexpr int NT = F32 ? 1 : 2;             // tiles of 128 rows
  static constexpr int NP = F32 ? 3 : 1;             // bf16 parts of a query element
  static constexpr int PP = F32 ? 3 : 2;             // and of a weight
  static constexpr int BT = F32 ? 64 : 128;          // tokens per block
  static constexpr int TILE = 128 * NT;
  static constexpr int SUBS = HD / 64;               // 128-byte wide sub-tiles of an operand row
  static constexpr int QTILE = SUBS * 128 * 128;     // bytes of one part of one tile's query
  static constexpr int QBYTES = NT * NP * QTILE;
  static constexpr int SLOT = SUBS * BT * 128;       // bytes of a block's keys or values
  static constexpr int STG = 2048;                   // per row warp: 64 bytes of each of its rows, for the output
  static constexpr int H = F32 ? 4 : 1;              // threads per row: shares of a block's tokens and of the dims
  static constexpr int ROWS = NT * H * 128;          // threads of the rows
  // loading threads: 4-bit codes take 7 warps to widen beside two tiles (16 in all, 128
  // registers); fp32 rows leave room for 3 (20 in all, 96 registers; with 7 there are
  // 80, the rows spill, and 461 us become 640); bf16 blocks come by TMA, and 4 warps
  // copy the ones that need zeros (one warp: 173 us instead of 154)
  static constexpr int LOAD = F32 ? 96 : BITS == 4 ? 224 : 128;
  static constexpr int ROOM = 214 * 1024 - QBYTES - ROWS / 32 * STG;
  static constexpr int NSLOT = ROOM / SLOT > 8 ? 8 : ROOM / SLOT;
  static constexpr int THREADS = ROWS + 32 + LOAD;
  static constexpr int PCOLS = BT / 2;               // TMEM columns of one part of the weights
  static constexpr int SCOLS = PP * PCOLS > BT ? PP * PCOLS : BT;   // of a tile's scores, or weights over them
  // Column of part q of the weights of 16 tokens from 16 k.  bf16 rows read their scores
  // in chunks of 32 columns (32 tokens) and put both parts of those weights over each;
  // fp32 rows hold theirs by then, and the parts lie one after the other.
  static constexpr int weight_col(int q, int k) { return F32 ? q * PCOLS + k * 8 : (k >> 1) * 32 + q * 16 + (k & 1) * 8; }
  static constexpr int RB = F32 ? 2 : 1;             // score regions of a tile
  static constexpr int TCOLS = RB * SCOLS + HD;      // of a tile
  static constexpr uint32_t ALLOC = NT * TCOLS <= 256 ? 256 : 512;
  static constexpr int SMEM = QBYTES + NSLOT * SLOT + ROWS / 32 * STG + 1024;
  static constexpr int PART = TILE * (HD + 2);       // floats of a partial result
};

// Blocks whose scales are kept.  A slot ring of NSLOT <= 8 lets the loaders run at
// most NSLOT / 2 + 1 blocks ahead of the rows, so a block's entry is free again
// when they come back to it.
constexpr int kMeta = 8;
// the block is its unit's last here; the next block begins a unit
constexpr int kLast = 1, kNextFresh = 2;

// B operand whose rows are K (tokens) and whose 64-element wide sub-tiles lie
// `sub` bytes apart (128-byte swizzle): MN-major.
DEVI uint64_t smem_desc_mn_sw128(uint32_t addr, uint32_t sub) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(sub >> 4) << 16;        // next 64 elements of N
  d |= static_cast<uint64_t>(1024u >> 4) << 32;      // next 8 rows of K
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
DEVI uint64_t smem_desc_k_sw128(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// D[tmem] (+)= A[tmem] B[smem]
DEVI void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
DEVI void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
DEVI void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
DEVI void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 columns, valid behind tmem_wait_ld
DEVI void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  uint32_t (&lo)[16] = *reinterpret_cast<uint32_t (*)[16]>(&r[0]);
  uint32_t (&hi)[16] = *reinterpret_cast<uint32_t (*)[16]>(&r[16]);
  tmem_ld16_async(taddr, lo);
  tmem_ld16_async(taddr + 16, hi);
}
DEVI void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
DEVI void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
DEVI void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 8 codes as 8 bf16 integers q.
DEVI uint4 widen_codes(uint32_t w) {
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {     // codes j and j + 4
    const uint32_t m = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;                       // 128 + u
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r[j]) : "r"(m), "r"(0x43084308u));               // - 136
  }
  return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410), __byte_perm(r[0], r[1], 0x7632),
                    __byte_perm(r[2], r[3], 0x7632));
}

// A tile's rows as (token of the request, query head of the group) without a
// division each: exact for row < 256, group <= 32.
struct RowMap {
  int t0, rem, mul, group;
  DEVI RowMap(int r0, int group_) : t0(r0 / group_), rem(r0 % group_), mul((65536 + group_ - 1) / group_), group(group_) {}
  // (token, head) of row `row` of the tile
  DEVI int2 at(int row) const {
    const int x = rem + row, t = (x * mul) >> 16;
    return make_int2(t0 + t, x - t * group);
  }
};

template <int HD, int BITS, bool F32>
__global__ void __launch_bounds__(Pro<HD, BITS, F32>::THREADS, 1) 
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tkv, const __grid_constant__ CUtensorMap tq, const AttnArgs a,
                       const int use_tma) {
  using D = Pro<HD, BITS, F32>;
  constexpr int NT = D::NT, NP = D::NP, PP = D::PP, BT = D::BT, TILE = D::TILE, NSLOT = D::NSLOT, LT = D::LOAD, RB = D::RB, H = D::H;
  constexpr bool Q4 = BITS == 4;
  using Walk = AttnWalk<TILE, BT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ ShareScratch<D::THREADS> sc;
  __shared__ uint64_t full[NSLOT], empty[NSLOT], qfull, qempty, sfull[NT * RB], pready[NT], odone[NT], drained, bready[kMeta], rowx, suml;
  __shared__ uint32_t tmem_slot;
  __shared__ int gave_up;                              // a wait ran out
  __shared__ float row_max[2][H][H > 1 ? 128 : 1], row_sum[H][H > 1 ? 128 : 1];   // the shares' maxima (two blocks) and sums
  // what the rows need of a block beside its products; block b's is at b % kMeta
  __shared__ int page_ok[kMeta];                       // per 64 tokens: the page is in range
  __shared__ int steps[kMeta];                         // for the MMA thread: kLast, kNextFresh
  __shared__ __align__(16) float scales[Q4 ? kMeta : 1][2][BT];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_a = smem_addr(smem), ring_a = q_a + D::QBYTES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.n_head / a.kv.n_kv_head;
  constexpr int MMA_WARP = D::ROWS / 32, LOAD0 = D::ROWS + 32;

  if (tid == 0) {
    gave_up = a.no_waiting;
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&full[s], LT);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&qfull, F32 ? D::ROWS : LT);
    for (int i = 0; i < kMeta; ++i) mbar_init(&bready[i], LT);
    mbar_init(&qempty, 1);
    for (int t = 0; t < NT; ++t) {
      for (int r = 0; r < RB; ++r) mbar_init(&sfull[t * RB + r], 1);
      mbar_init(&pready[t], 128 * H);
      mbar_init(&odone[t], 1);
    }
    mbar_init(&drained, 1);
    mbar_init(&rowx, 128 * H);
    mbar_init(&suml, 128 * H);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch();
  find_share<TILE, BT, D::THREADS>(a, group, 1, sc);
  const AttnShare sh = sc.share;
  int* heads = reinterpret_cast<int*>(a.ws) + blockIdx.x * kHeadInts;
  float* parts = a.ws + gridDim.x * kHeadInts;
  if (tid == 0) heads[0] = heads[kHeadLost] = 0;
  if (sh.w0 >= sh.w1) return;   // the whole CTA
  // Every wait of the roles has a limit; behind one that ran out no other waits any
  // more.  What the CTA leaves behind is then not the call's result: the join, told by
  // its header, makes all rows NaN.
  auto reached = [&](uint64_t* bar, int phase) {
    if (mbar_try_wait(bar, phase & 1)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, phase & 1))
      if (*const_cast<volatile int*>(&gave_up) || global_timer_ns() - t0 > kWaitNs) {
        raise_error(a.err, DEV_ERR_MBAR_TIMEOUT);
        gave_up = 1;
        return false;
      }
    return true;
  };
  if (warp == MMA_WARP) {
    tmem_alloc(&tmem_slot, D::ALLOC);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_slot;
  const int n_blocks = static_cast<int>(sh.w1 - sh.w0);   // blocks of this CTA, over all its units

  Walk wk;
  wk.seek(a, group, sh, sh.w0);

  // queries: 8 consecutive dims of a row at a time
  constexpr int PR = HD / 8;
  auto q_place = [&](int row, int c8) {
    return q_a + (row >> 7) * (NP * D::QTILE) + (c8 >> 3) * (128 * 128) + (row & 127) * 128 + (((c8 & 7) ^ (row & 7)) << 4);
  };
  auto q_source = [&](const RowMap& rows, int row, int c8) {
    const int2 th = rows.at(row);
    return static_cast<int64_t>(wk.u.q0 + th.x) * a.ldq + static_cast<int64_t>(wk.head * group + th.y) * HD + c8 * 8;
  };

  if (tid >= LOAD0) {
    // ---- loaders: queries of a unit (bf16 ones), then keys and values of its blocks
    const int t = tid - LOAD0;
    // A block as the loaders see it; a 4-bit one with this thread's codes and scales.
    constexpr int PC4 = HD / 32;                       // 16-byte pieces (32 codes) per token
    constexpr int RN = Q4 ? (BT * PC4 + LT - 1) / LT : 1, SN = Q4 ? (BT + LT - 1) / LT : 1;
    struct Look {
      int pos, hi, lo, sink, head, okm, page0, page1;
      uint4 raw[2][RN];
      uint16_t scale[2][SN];
    };
    Look cur;
    // its entries of the page table, read a block ahead (need: which pages some row needs)
    int page[BT / 64], need = 0;
    auto peek = [&]() {
      need = 0;
#pragma unroll
      for (int h = 0; h < BT / 64; ++h) {
        const int pg = wk.pos / kPageTokens + h;
        const bool any = pg * kPageTokens < wk.u.hi && (pg * kPageTokens + kPageTokens > wk.u.lo || pg * kPageTokens < wk.u.sink);
        need |= static_cast<int>(any) << h;
        page[h] = any && pg < a.width ? table_of(a, wk.seq)[pg] : -1;
      }
    };
    peek();
    auto look = [&](Look& k) {
      k.pos = wk.pos;
      k.hi = wk.u.hi;
      k.lo = wk.u.lo;
      k.sink = wk.u.sink;
      k.head = wk.head;
      k.okm = 0;
      k.page1 = 0;
#pragma unroll
      for (int h = 0; h < BT / 64; ++h) {
        const bool ok = page[h] >= 0 && page[h] < a.kv.n_pages;
        if (((need >> h) & 1) && !ok && t == 0) raise_error(a.err, DEV_ERR_BAD_PAGE);
        k.okm |= static_cast<int>(ok) << h;
        (h ? k.page1 : k.page0) = ok ? page[h] : 0;
      }
      if constexpr (Q4) {
        // (a page out of range: page 0, whose codes are finite, with scales of 0)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const unsigned char* b0 = kv_block(a.kv, k.page0, kv, k.head);
          const unsigned char* b1 = kv_block(a.kv, k.page1, kv, k.head);
#pragma unroll
          for (int i = 0; i < RN; ++i) {
            const int id = i * LT + t, tok = id / PC4;
            k.raw[kv][i] = make_uint4(0, 0, 0, 0);
            if (id < BT * PC4)
              k.raw[kv][i] = *reinterpret_cast<const uint4*>((BT > 64 && tok >= 64 ? b1 : b0) + (tok & 63) * (HD / 2) + id % PC4 * 16);
          }
#pragma unroll
          for (int i = 0; i < SN; ++i) {
            const int tok = i * LT + t;
            k.scale[kv][i] = 0;
            if (tok < BT)
              k.scale[kv][i] = *reinterpret_cast<const uint16_t*>((BT > 64 && tok >= 64 ? b1 : b0) + 64 * (HD / 2) + (tok & 63) * 2);
          }
        }
      }
    };
    int unit_n = 0;            // units begun
    int issued = 0;            // slots filled, or being filled
    bool fresh = true;
    auto publish = [&](int slot) {
      fence_async_smem();
      mbar_arrive(&full[slot]);
    };
#pragma unroll 1
    for (int b = 0; b < n_blocks; ++b) {
      if (!F32 && fresh) {
        fresh = false;
        if (unit_n > 0 && !reached(&qempty, unit_n - 1)) break;
        ++unit_n;
        const RowMap rows(wk.u.r0, group);
        if (use_tma & 2) {
          // 128 / group tokens of the group's heads are a tile's rows in order
          if (t == 0) {
            mbar_arrive_expect_tx(&qfull, static_cast<uint32_t>(D::QBYTES));
#pragma unroll
            for (int tile = 0; tile < NT; ++tile)
#pragma unroll
              for (int sub = 0; sub < HD / 64; ++sub)
                tma_load_3d(q_a + tile * D::QTILE + sub * (128 * 128), &tq, sub * 64, wk.head * group,
                            wk.u.q0 + rows.t0 + tile * (128 / group), &qfull);
          } else {
            mbar_arrive(&qfull);
          }
        } else {
          // as they are: all copies in flight at once
#pragma unroll 4
          for (int id = t; id < TILE * PR; id += LT) {
            const int row = id / PR, c8 = id % PR;
            const bool live = row < wk.u.nr;
            cp16_or_zero(q_place(row, c8), static_cast<const uint16_t*>(a.q) + (live ? q_source(rows, row, c8) : 0), live);
          }
          cp_async_commit();
          cp_wait<0>();
          fence_async_smem();
          mbar_arrive(&qfull);
        }
      }
      look(cur);
      const Look& k = cur;
      const int okm = k.okm;
      auto take = [&](int tok) {   // some row sees the token
        const int j = k.pos + tok;
        return ((okm >> (tok >> 6)) & 1) && j < k.hi && (j >= k.lo || j < k.sink);
      };
      // every token of the block is seen by some row: copied by the TMA
      const bool whole = !Q4 && (use_tma & 1) && okm == (1 << (BT / 64)) - 1 && k.pos + BT <= k.hi &&
                         (k.pos >= k.lo || k.pos + BT <= k.sink);
      bool next_fresh = false;
      if (b + 1 < n_blocks) {
        const long long was = wk.start;
        wk.next_chunk(a, group);
        next_fresh = wk.start != was;
        peek();
        if constexpr (F32) {
          // the next unit's queries into L2: their reading stands between two units
          if (next_fresh) {
            constexpr int LINES = HD / 32;
            const RowMap rows(wk.u.r0, group);
            for (int id = t; id < min(wk.u.nr, TILE) * LINES; id += LT)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const float*>(a.q) + q_source(rows, id / LINES, id % LINES * 4)));
          }
        }
      }
      // (published with the keys; an entry is free again like page_ok's)
      if (t == 0) steps[b % kMeta] = (next_fresh || b + 1 == n_blocks ? kLast : 0) | (next_fresh ? kNextFresh : 0);
      bool dead = false;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int n = 2 * b + kv, slot = n % NSLOT;
        if (n >= NSLOT && !reached(&empty[slot], n / NSLOT - 1)) {
          dead = true;
          break;
        }
        const uint32_t dst = ring_a + slot * D::SLOT;
        if constexpr (!Q4) {
          if (whole) {
            if (t == 0) {
              mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(D::SLOT));
#pragma unroll
              for (int h = 0; h < BT / 64; ++h)
#pragma unroll
                for (int sub = 0; sub < HD / 64; ++sub)
                  tma_load_4d(dst + sub * (BT * 128) + h * (64 * 128), &tkv, sub * 64, 0, kv * a.kv.n_kv_head + k.head,
                              h ? k.page1 : k.page0, &full[slot]);
            } else {
              mbar_arrive(&full[slot]);
            }
          } else {
            // tokens that no row sees are filled with zeros
            constexpr int PC = HD / 8;        // 16-byte pieces per token
#pragma unroll 4
            for (int id = t; id < BT * PC; id += LT) {
              const int tok = id / PC, c = id % PC;
              cp16_or_zero(dst + (c >> 3) * (BT * 128) + tok * 128 + (((c & 7) ^ (tok & 7)) << 4),
                    kv_block(a.kv, BT > 64 && tok >= 64 ? k.page1 : k.page0, kv, k.head) + (tok & 63) * (HD * 2) + c * 16, take(tok));
            }
            cp_async_commit();
            cp_wait<0>();
            publish(slot);
          }
        } else {
#pragma unroll
          for (int i = 0; i < SN; ++i) {
            const int tok = i * LT + t;
            if (tok < BT) scales[b % kMeta][kv][tok] = take(tok) ? bf16bits_to_f32(kv ? k.scale[1][i] : k.scale[0][i]) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < RN; ++i) {
            const int id = i * LT + t, tok = id / PC4, c = id % PC4;
            const uint4 raw = kv ? k.raw[1][i] : k.raw[0][i];
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            const uint32_t at0 = dst + (c >> 1) * (BT * 128) + tok * 128 + ((((c & 1) * 4) ^ (tok & 7)) << 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 v = widen_codes(w[e]);
              const uint32_t at = at0 ^ (e << 4);
              if (id < BT * PC4)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            }
          }
          publish(slot);
        }
        ++issued;
      }
      if (dead) break;
      if (t == 0) page_ok[b % kMeta] = okm;
      mbar_arrive(&bready[b % kMeta]);
      fresh = next_fresh;
    }
    // every copy issued here has landed before the CTA may exit (where other loaders
    // gave up, a barrier stays open: one limit is enough for all copies)
    if (t == 0) {
      bool landed = F32 || unit_n == 0 || mbar_wait(&qfull, (unit_n - 1) & 1, a.err, kWaitNs);
      for (int n = issued > NSLOT ? issued - NSLOT : 0; n < issued && landed; ++n)
        landed = mbar_wait(&full[n % NSLOT], (n / NSLOT) & 1, a.err, kWaitNs);
    }
  } else if (warp == MMA_WARP) {
    if (lane == 0) {
      // ---- MMA issuer
      constexpr uint32_t id_s = idesc_bf16_f32(128, BT);
      constexpr uint32_t id_o = idesc_bf16_f32(128, HD) | (1u << 16);   // B is MN-major
      int units = 0;
      bool dead = false;
      auto scores = [&](int t, int b) {      // S of tile t, block b
        const uint32_t td = tm + t * D::TCOLS + (b % RB) * D::SCOLS;
        // (descriptors move by their address field: 16-byte units)
        const uint64_t kd = smem_desc_k_sw128(ring_a + (2 * b % NSLOT) * D::SLOT);
        const uint64_t qd = smem_desc_k_sw128(q_a + t * (NP * D::QTILE));
        // small parts first: the accumulator truncates at its size
#pragma unroll
        for (int p = NP - 1; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t ko = (k >> 2) * (BT * 128) + (k & 3) * 32, qo = p * D::QTILE + (k >> 2) * (128 * 128) + (k & 3) * 32;
            tc_mma_bf16(td, qd + (qo >> 4), kd + (ko >> 4), id_s, p < NP - 1 || k > 0);
          }
        tc_commit(&sfull[t * RB + b % RB]);
      };
      auto values = [&](int t, int b, bool first) {   // O of tile t, block b
        const uint32_t td = tm + t * D::TCOLS + (b % RB) * D::SCOLS, to = tm + t * D::TCOLS + RB * D::SCOLS;
        const uint64_t vd = smem_desc_mn_sw128(ring_a + ((2 * b + 1) % NSLOT) * D::SLOT, BT * 128);
#pragma unroll
        for (int p = PP - 1; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < BT / 16; ++k)
            tc_mma_ts(to, td + D::weight_col(p, k), vd + ((k * 2048) >> 4), id_o,
                      p < PP - 1 || k > 0 || (!first && !F32));
      };
      auto wait = [&](uint64_t* bar, int phase) {
        if (dead) return;
        if (!reached(bar, phase)) dead = true;
        tc_fence_after();
      };
      bool fresh = true;                      // the block begins its unit
      int step = 0, next = 0;                 // what the loaders say of the block, of the next
      for (int b = 0; b < n_blocks && !dead; ++b) {
        // S of block 0; later blocks' S were issued behind the O of the one before
        if (b == 0) {
          wait(&qfull, units);
          ++units;
          wait(&full[0], 0);
          if (dead) break;
          step = steps[0];
          for (int t = 0; t < NT; ++t) scores(t, 0);
          tc_commit(&empty[0]);
          if (step & kLast) tc_commit(&qempty);   // the unit's last S: its queries may go
        }
        const bool more = b + 1 < n_blocks, turn = step & kNextFresh;
        auto next_scores = [&](int t) {
          if (t == 0) {
            if (turn) {
              wait(&qfull, units);
              ++units;
            }
            wait(&full[(2 * b + 2) % NSLOT], (2 * b + 2) / NSLOT);
          }
          if (dead) return;
          next = steps[(b + 1) % kMeta];
          scores(t, b + 1);
          if (t == NT - 1) {
            tc_commit(&empty[(2 * b + 2) % NSLOT]);
            if (next & kLast) tc_commit(&qempty);
          }
        };
        // with two score regions the next block's S goes before this one's O
        // (but for a new unit's, which waits for its queries)
        const bool ahead = RB == 2 && more && !turn;
        if (ahead) next_scores(0);
        wait(&full[(2 * b + 1) % NSLOT], (2 * b + 1) / NSLOT);
        for (int t = 0; t < NT && !dead; ++t) {
          wait(&pready[t], b);
          if (dead) break;
          values(t, b, fresh);
          tc_commit(&odone[t]);
          if (t == NT - 1) tc_commit(&empty[(2 * b + 1) % NSLOT]);
          if (more && !ahead && !turn) next_scores(t);
        }
        if (more && turn)
          for (int t = 0; t < NT && !dead; ++t) next_scores(t);
        fresh = turn;
        step = next;
      }
      // every MMA issued has completed before the CTA gives its memory back
      tc_commit(&drained);
      mbar_wait(&drained, 0, a.err, kWaitNs);
    }
  } else {
    // ---- rows: thread = row of its tile (fp32: four threads, a share each)
    // (all lanes of a warp go on or stop together: its tensor-memory instructions take
    // them all)
    auto ready = [&](uint64_t* bar, int phase) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
      const uint64_t t0 = global_timer_ns();
      while (!__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1)))
        if (__any_sync(0xffffffffu, *const_cast<volatile int*>(&gave_up) || global_timer_ns() - t0 > kWaitNs)) {
          raise_error(a.err, DEV_ERR_MBAR_TIMEOUT);
          gave_up = 1;
          return false;
        }
      return true;
    };
    const int tile = H > 1 ? 0 : warp >> 2, share = H > 1 ? warp >> 2 : 0, row = tid & 127;
    constexpr int HDH = HD / H;              // dims of a thread
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts0 = tm + tile * D::TCOLS + lanes, to = ts0 + RB * D::SCOLS;
    const float sc2 = a.scale * 1.4426950408889634f;
    float m = -FLT_MAX, l = 0.f;
    float o[F32 ? HDH : 1];                  // fp32 activations: the running output
    int units = 0;                           // units ended
    int p = 0;
    bool fresh = true, live = false, first = true;   // first: no block of the unit yet
    int pmin = 0, pmax = 0;
    bool begins = wk.start >= sh.w0;         // the unit's first block is this CTA's
#pragma unroll 1
    for (int b = 0; b < n_blocks; ++b) {
      if (fresh) {
        fresh = false;
        if constexpr (F32) {
          // the unit's queries in parts: four loads in flight per thread
          if (!first && !ready(&qempty, units - 1)) break;
          constexpr int QB = TILE * PR / D::ROWS < 4 ? TILE * PR / D::ROWS : 4;
          static_assert(TILE * PR % (D::ROWS * QB) == 0, "whole rounds");
          const RowMap rows(wk.u.r0, group);
#pragma unroll 1
          for (int id0 = tid; id0 < TILE * PR; id0 += D::ROWS * QB) {
            float x[QB][8];
#pragma unroll
            for (int k = 0; k < QB; ++k) {
              const int id = id0 + k * D::ROWS, qr = id / PR;
#pragma unroll
              for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
              if (qr < wk.u.nr) {
                const float* src = static_cast<const float*>(a.q) + q_source(rows, qr, id % PR);
                const float4 v0 = *reinterpret_cast<const float4*>(src), v1 = *reinterpret_cast<const float4*>(src + 4);
                x[k][0] = v0.x;
                x[k][1] = v0.y;
                x[k][2] = v0.z;
                x[k][3] = v0.w;
                x[k][4] = v1.x;
                x[k][5] = v1.y;
                x[k][6] = v1.z;
                x[k][7] = v1.w;
              }
            }
#pragma unroll
            for (int k = 0; k < QB; ++k) {
              const int id = id0 + k * D::ROWS;
              const uint32_t at = q_place(id / PR, id % PR);
#pragma unroll
              for (int q = 0; q < NP; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  w[e] = pack_bf16(x[k][2 * e], x[k][2 * e + 1]);
                  x[k][2 * e] -= bf16lo(w[e]);
                  x[k][2 * e + 1] -= bf16hi(w[e]);
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + q * D::QTILE), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                             "r"(w[3])
                             : "memory");
              }
            }
          }
          fence_async_smem();
          mbar_arrive(&qfull);
        }
        first = true;
        const int r = wk.u.r0 + tile * 128 + row;
        live = tile * 128 + row < wk.u.nr;
        const long long top = 0x7ffffff0ll;
        p = live ? static_cast<int>(max(-1ll, min(wk.u.pbase + r / group, top))) : -1;
        const int r1 = wk.u.r0 + min(wk.u.nr, tile * 128 + 128) - 1, ra = wk.u.r0 + tile * 128;
        pmin = static_cast<int>(max(-1ll, min(wk.u.pbase + ra / group, top)));
        pmax = static_cast<int>(max(-1ll, min(wk.u.pbase + max(ra, r1) / group, top)));
        m = -FLT_MAX;
        l = 0.f;
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < HDH; ++i) o[i] = 0.f;
        }
      }
      const int pos = wk.pos, meta = b % kMeta;
      const uint32_t ts = ts0 + (b % RB) * D::SCOLS;
      if (!ready(&sfull[tile * RB + b % RB], b / RB)) break;
      if (!ready(&bready[meta], b / kMeta)) break;
      tc_fence_after();
      const int okm = page_ok[meta];
      bool see_all = okm == (1 << (BT / 64)) - 1 && pos + BT <= pmin + 1 && pos + BT <= wk.u.hi;
      if (a.window > 0) see_all = see_all && (pos > pmax - a.window || pos + BT <= a.sinks);
      // tokens of the block that this row sees: [lo_l, hi_l] and [0, sink_l)
      const int hi_l = min(p, wk.u.hi - 1) - pos;
      const int lo_l = a.window > 0 ? (p < a.window ? 0 : p - a.window + 1 - pos) : 0;
      const int sink_l = a.window > 0 ? a.sinks - pos : 0;
      auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
      auto seen = [&](int t0) {   // of 32 tokens from t0, one bit each
        const uint32_t v = below(hi_l + 1 - t0) & (~below(lo_l - t0) | below(sink_l - t0));
        return (okm >> (t0 >> 6)) & 1 ? v : 0u;
      };
      // Scores of a chunk of CW tokens, without the softmax's constant (4 bits: with the
      // keys' scales); -inf where the row sees nothing.
      constexpr int CW = F32 ? BT / H : 32, CH = BT / H / CW;
      static_assert(!F32 || (CW == 16 && CH == 1), "fp32: one chunk of 16 tokens per thread");
      auto load_scores = [&](int ch, float (&x)[CW]) {
        uint32_t v[CW];
#pragma unroll
        for (int i = 0; i < CW; i += 16) tmem_ld16_async(ts + ch * CW + i, *reinterpret_cast<uint32_t (*)[16]>(&v[i]));
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < CW; ++i) x[i] = __uint_as_float(v[i]);
        if constexpr (Q4) {
#pragma unroll
          for (int i = 0; i < CW; i += 4) {
            const float4 k = *reinterpret_cast<const float4*>(&scales[meta][0][ch * CW + i]);
            x[i] *= k.x;
            x[i + 1] *= k.y;
            x[i + 2] *= k.z;
            x[i + 3] *= k.w;
          }
        }
        if (!see_all) {
          const uint32_t bits = seen(ch * CW);
#pragma unroll
          for (int i = 0; i < CW; ++i) x[i] = bits & (1u << i) ? x[i] : -INFINITY;
        }
      };
      // maximum (fp32 activations keep the scores; bf16 ones read them again)
      float x[CW];
      float mx = -FLT_MAX;
#pragma unroll 1
      for (int ch = share * CH; ch < (share + 1) * CH; ++ch) {
        load_scores(ch, x);
        float m4[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
        for (int i = 0; i < CW; ++i) m4[i & 3] = fmaxf(m4[i & 3], x[i]);
        mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
      }
      if constexpr (H > 1) {
        // the other shares' (also: all have read their scores, which the weights overwrite)
        row_max[b & 1][share][row] = mx;
        tc_fence_before();
        mbar_arrive(&rowx);
        if (!ready(&rowx, b)) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < H; ++h) mx = fmaxf(mx, row_max[b & 1][h][row]);
      }
      mx = mx > -FLT_MAX ? mx * sc2 : -FLT_MAX;
      const bool grow = mx > m + kLazyMax || m == -FLT_MAX;
      const float mn = grow ? fmaxf(mx, m) : m;
      const float f = exp2_fast(m - mn);
      if constexpr (!F32) {
        if (__any_sync(0xffffffffu, grow && l > 0.f)) {
#pragma unroll 1
          for (int ch = 0; ch < HD / 32; ++ch) {
            uint32_t v[32];
            tmem_ld32(to + ch * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st16(to + ch * 32, *reinterpret_cast<uint32_t (*)[16]>(&v[0]));
            tmem_st16(to + ch * 32 + 16, *reinterpret_cast<uint32_t (*)[16]>(&v[16]));
          }
          tmem_wait_st();
        }
      }
      m = mn;
      float lb = 0.f;
      // weights
#pragma unroll 1
      for (int ch = share * CH; ch < (share + 1) * CH; ++ch) {
        if constexpr (!F32) load_scores(ch, x);
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          x[i] = exp2_fast(fmaf(x[i], sc2, -m));
          l4[i & 3] += x[i];
        }
        lb += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        if constexpr (Q4) {
#pragma unroll
          for (int i = 0; i < CW; i += 4) {
            const float4 k = *reinterpret_cast<const float4*>(&scales[meta][1][ch * CW + i]);
            x[i] *= k.x;
            x[i + 1] *= k.y;
            x[i + 2] *= k.z;
            x[i + 3] *= k.w;
          }
        }
#pragma unroll
        for (int q = 0; q < PP; ++q) {
          uint32_t w[CW / 2];
#pragma unroll
          for (int i = 0; i < CW / 2; ++i) {
            w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            if (q + 1 < PP) {
              x[2 * i] -= bf16lo(w[i]);
              x[2 * i + 1] -= bf16hi(w[i]);
            }
          }
          if constexpr (CW == 32) tmem_st16(ts + D::weight_col(q, 2 * ch), w);
          else tmem_st8(ts + D::weight_col(q, ch), w);
        }
      }
      l = fmaf(l, f, lb);
      tmem_wait_st();
      // fp32: block b's output, added to the running one
      auto take_output = [&](int b, float scale) {
        if (!ready(&odone[tile], b)) return false;
        tc_fence_after();
#pragma unroll
        for (int ch = 0; ch < HDH / 16; ++ch) {
          uint32_t v[16];
          tmem_ld16_async(to + share * HDH + ch * 16, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float& y = o[F32 ? ch * 16 + i : 0];
            y = (y + __uint_as_float(v[i])) * scale;
          }
        }
        return true;
      };
      if constexpr (F32) {
        if (!first && !take_output(b - 1, f)) break;
      }
      first = false;
      tc_fence_before();
      mbar_arrive(&pready[tile]);
      const bool more = b + 1 < n_blocks;
      const bool unit_end = wk.left == 1;
      const bool last = unit_end || !more;
      if constexpr (F32) {
        if (last) {
          if (!take_output(b, 1.f)) break;
          tc_fence_before();
        }
      } else if (last) {
        if (!ready(&odone[tile], b)) break;
        tc_fence_after();
      }
      if (last) {
        if constexpr (H > 1) {
          row_sum[share][row] = l;
          mbar_arrive(&suml);
          if (!ready(&suml, units)) break;
          l = row_sum[0][row];
#pragma unroll
          for (int h = 1; h < H; ++h) l += row_sum[h][row];
          ++units;
        }
        const bool whole = begins && unit_end;
        const int slot = begins ? 1 : 0;
        const float inv = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
        float* part = parts + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * D::PART;
        const int lr = tile * 128 + row;
        const RowMap rows(wk.u.r0, group);
        // 64 bytes of every row of the warp, from byte `off` of the thread's dims:
        // through shared memory, so that neighbouring lanes write neighbouring bytes
        unsigned char* stg = smem + D::QBYTES + NSLOT * D::SLOT + warp * D::STG;
        auto put = [&](const uint4 (&v)[4], int off) {
#pragma unroll
          for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v[c];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = i * 8 + (lane >> 2), c = lane & 3, tr = tile * 128 + (warp & 3) * 32 + rr;
            const uint4 y = *reinterpret_cast<const uint4*>(stg + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
            if (tr < wk.u.nr) {
              unsigned char* dst;
              if (whole) {
                const int2 th = rows.at(tr);
                dst = static_cast<unsigned char*>(a.out) +
                      (static_cast<int64_t>(wk.u.q0 + th.x) * a.ldo + static_cast<int64_t>(wk.head * group + th.y) * HD +
                       share * HDH) * (F32 ? 4 : 2);
              } else {
                dst = reinterpret_cast<unsigned char*>(part + static_cast<int64_t>(tr) * HD + share * HDH);
              }
              *reinterpret_cast<uint4*>(dst + off + c * 16) = y;
            }
          }
          __syncwarp();
        };
        // fp32 values, 16 at a time
        auto put16 = [&](const float* y, int off) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                              __float_as_uint(y[4 * i + 3]));
          put(v, off);
        };
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < HDH; ++i) o[i] *= inv;
#pragma unroll
          for (int ch = 0; ch < HDH / 16; ++ch) put16(o + ch * 16, ch * 64);
        } else {
#pragma unroll
          for (int ch = 0; ch < HDH / 32; ++ch) {
            float y[32];
            uint32_t v[32];
            tmem_ld32(to + ch * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(v[i]) * inv;
            if (whole) {
              uint4 w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = make_uint4(pack_bf16(y[8 * i], y[8 * i + 1]), pack_bf16(y[8 * i + 2], y[8 * i + 3]),
                                  pack_bf16(y[8 * i + 4], y[8 * i + 5]), pack_bf16(y[8 * i + 6], y[8 * i + 7]));
              put(w, ch * 64);
            } else {
              put16(y, ch * 128);
              put16(y + 16, ch * 128 + 64);
            }
          }
        }
        if (!F32) tc_fence_before();
        if (!whole && share == 0) {
          part[TILE * HD + lr] = m;
          part[TILE * HD + TILE + lr] = l;
          if (begins && tid == 0) {
            const long long e = wk.start + wk.u.n;
            int k = static_cast<int>((e - 1) * sh.n_cta / sh.total);
            while (k + 1 < sh.n_cta && share_start(sh.total, sh.n_cta, k + 1) < e) ++k;
            heads[1] = k - static_cast<int>(blockIdx.x);
            heads[2] = wk.u.q0;
            heads[3] = wk.u.r0;
            heads[4] = wk.u.nr;
            heads[5] = wk.head;
            heads[0] = 1;
          }
        }
      }
      if (more) {
        const long long was = wk.start;
        wk.next_chunk(a, group);
        if (wk.start != was) {
          fresh = true;
          begins = true;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tm, D::ALLOC);
  }
  if (tid == 0) heads[kHeadLost] = gave_up;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A bf16 tensor map with 128-byte swizzle, encoded anew for every call.
static bool encode_map(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box) {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The cache: (dim, token of the page, key or value head, page), boxes of 64 dims x 64 tokens.
static bool kv_tensor_map(CUtensorMap* m, const KvView& kv) {
  if (kv.page_stride >= (1ll << 40)) return false;
  const cuuint64_t hd = static_cast<cuuint64_t>(kv.head_dim);
  const cuuint64_t dims[4] = {hd, kPageTokens, static_cast<cuuint64_t>(2 * kv.n_kv_head), static_cast<cuuint64_t>(kv.n_pages)};
  const cuuint64_t strides[3] = {hd * 2, hd * 2 * kPageTokens, static_cast<cuuint64_t>(kv.page_stride)};
  const cuuint32_t box[4] = {64, kPageTokens, 1, 1};
  return encode_map(m, 4, kv.data, dims, strides, box);
}
// bf16 queries: (dim, head, row), boxes of 64 dims x the group x the tokens that
// make 128 rows; a group that is no divisor of 128 has none.
static bool q_tensor_map(CUtensorMap* m, const AttnArgs& a) {
  const int group = a.n_head / a.kv.n_kv_head;
  if (128 % group || a.ldq >= (1ll << 38)) return false;
  const cuuint64_t hd = static_cast<cuuint64_t>(a.kv.head_dim);
  const cuuint64_t dims[3] = {hd, static_cast<cuuint64_t>(a.n_head), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[2] = {hd * 2, static_cast<cuuint64_t>(a.ldq) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)};
  return encode_map(m, 3, a.q, dims, strides, box);
}

template <int HD, int BITS, bool F32>
static cudaError_t launch_one(const AttnArgs& a, int n_sm, cudaStream_t st) {
  using D = Pro<HD, BITS, F32>;
  // what has no map is copied by the threads
  CUtensorMap tkv{}, tq{};
  const int use_tma = (BITS == 16 && kv_tensor_map(&tkv, a.kv) ? 1 : 0) | (!F32 && q_tensor_map(&tq, a) ? 2 : 0);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_prompt_kernel<HD, BITS, F32>), D::SMEM, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_prompt_kernel<HD, BITS, F32>, dim3(n_sm), dim3(D::THREADS), D::SMEM, st, tkv, tq, a, use_tma);
  if (e != cudaSuccess) return e;
  return launch_attn_join(a, !F32, D::TILE, n_sm, st);
}

int64_t prompt_workspace_floats(bool f32, int head_dim) {
  return static_cast<int64_t>(kAttnSms) * (kHeadInts + 2 * (f32 ? 128 : 256) * (head_dim + 2));
}

cudaError_t launch_attn_prompt(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  if (a.kv.head_dim == 128) {
    if (a.kv.bits == 16) return bf16 ? launch_one<128, 16, false>(a, n_sm, st) : launch_one<128, 16, true>(a, n_sm, st);
    return bf16 ? launch_one<128, 4, false>(a, n_sm, st) : launch_one<128, 4, true>(a, n_sm, st);
  }
  if (a.kv.bits == 16) return bf16 ? launch_one<64, 16, false>(a, n_sm, st) : launch_one<64, 16, true>(a, n_sm, st);
  return bf16 ? launch_one<64, 4, false>(a, n_sm, st) : launch_one<64, 4, true>(a, n_sm, st);
}

}  // namespace dualar
