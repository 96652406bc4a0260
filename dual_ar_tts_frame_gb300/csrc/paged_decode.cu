// Attention over the paged cache for few rows per request (single tokens and
// short drafts).
//
// Memory bound: each cached vector that a tile of rows sees is read once, 4 HD
// (bf16) or HD + 4 (4-bit) bytes per token and head for 4 HD FLOP per row.  So
// the kernel is a stream of chunks: a warp owns a piece of the work line
// (paged_sched.cuh), copies its chunks into a ring of its own with cp.async
// (no barrier between warps; cells that no row sees are zero-filled, never
// read), and keeps the running maximum, sum and output of its rows in
// registers.
//
// Products run as mma.sync m16n8k16 with the cache as the 16-row operand and the
// tile's 8 rows as the 8 columns: scores S^T = K Q^T (16 tokens x 8 rows), then
// O^T = V^T P^T (16 dims x 8 rows), the weights turned from one layout into the
// other by movmatrix.  tcgen05's 64 rows and more would need the whole group's
// cache staged as bf16 in shared memory.  (With the queries as the 16-row operand
// half of every MMA is empty at 8 rows; that took twice the tensor time.)
//
// Precision.  bf16 cache: bf16 parts of the other factor, multiplied one after
// the other into one accumulator: fp32 activations 3 (24 bits of query and
// weight), bf16 activations 1 of the query (exact) and 2 of the weight.
// 4-bit cache: fp16 parts, 2 of the weight (22 bits) and of an fp32 query, 1 of a bf16
// query (exact).  (With 1 part of the weight, 11 bits, bf16 rows take 161 us instead of
// 172 for 64 requests; the error of typical rows is the output's rounding either way,
// that of rows whose values cancel is not.)  The tensor cores' accumulators truncate (measured);
// for fp32 activations and the 4-bit cache a chunk's sums leave them and are
// added to the running output with rounding.
//
// A 4-bit code u = q + 8 is an fp16 number as it stands: the bits 0000..u are the
// subnormal u 2^-24, and one place up (bits 4-7) u 2^-20.  So a word of 8 codes
// becomes four operand registers by four ANDs and one shift, where bf16 integers
// take three shifts, four ORs and four subtractions.  The place is made up for by
// the query (keys) or when an output row is added (values); the 8 is taken off
// in the accumulator's initial value, -8 times the sum of what multiplies the
// codes (the sums' terms are then up to 15 of a token's scale: at most 2^-15 of sum_j
// w_j s_j of error, below the output's rounding of typical rows).  fp32 activations take
// q itself, 1024 + u less 1032, one more instruction per register: with u the larger
// sums cost a truncating accumulator accuracy, and the tensor cores align a subnormal
// operand's product by the exponent that it does not have, which left 18 bits of a query
// beside a code of 1 (one request of 32K, error: 4.4e-6 with u, 6.9e-7 with q as
// subnormals, 1.3e-7).  The token's scale multiplies its score or its weight, never an
// element.  Queries are scaled by a power of two to their row's largest element, weights
// to their chunk's, which keeps them inside fp16's range.  Any order of the head's
// dimensions serves in the first product as long as the query uses it too, and any order
// of output rows in the second; so a lane reads its codes as
// one contiguous vector, and its outputs are contiguous.
//
// Measured (32 query and 8 key/value heads of 128):
//   bf16 cache, 64 requests, window 1024 + 4 first tokens: 54 us, 5.0 TB/s, 74% of a
//     copy's rate; bound by memory, and by the start and the join of a short kernel.
//   4 bits, 64 requests of 2000 to 16384 tokens, bf16 rows: 170 us, 3.7 TB/s, 54%.  59% of
//     issue slots are in use, with four warps per scheduler: a chunk is one dependent
//     chain (scores, maximum, exponentials, the weights' scale, values), and nothing of
//     a warp's next chunk runs beside it.
//   4 bits, one request of 32K: 28 us; 304 CTAs, of which each has 7 chunks per warp:
//     the start (work shares, first loads) and the join are most of it.
#include <cfloat>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"
#include "paged_sched.cuh"

namespace dualar {

constexpr int kDecTile = 8;      // rows per unit

template <int HD, int BITS, bool F32>
struct Dec {
  static constexpr int WARPS = 8;
  // 4 bits: two CTAs per SM (the arithmetic wants 16 warps); bf16: one, whose
  // rings fill the shared memory
  static constexpr int CTAS = BITS == 4 ? 2 : 1;
  static constexpr int CT = BITS == 16 && HD == 128 ? 16 : 32;   // tokens per chunk
  static constexpr int ROWB = BITS == 4 ? HD / 2 : HD * 2;       // bytes per token
  static constexpr int KB = CT * ROWB;
  static constexpr int STAGE = 2 * KB + (BITS == 4 ? 4 * CT : 0);
  static constexpr int PART = kDecTile * (HD + 2);               // floats of a partial result
  static constexpr int ROOM = (225 * 1024 / CTAS - 2304) / WARPS - PART * 4;
  static constexpr int NST = ROOM / STAGE > 4 ? 4 : ROOM / STAGE;   // ring stages: 2 to 4
  static constexpr int RING = NST * STAGE > PART * 4 ? NST * STAGE : (PART * 4 + 127) / 128 * 128;
  static constexpr int SMEM = WARPS * (RING + PART * 4);
  static constexpr int KS = HD / 16;                             // k steps of the first product
  static constexpr int QP = F32 ? (BITS == 4 ? 2 : 3) : 1;       // parts of a query element
  static constexpr int PP = BITS == 4 || !F32 ? 2 : 3;   // parts of a weight
  static constexpr bool OWN = BITS == 4 || F32;                  // a chunk has its own accumulators
};

// A requested chunk, for its use: its position, and of its unit what the rows
// need.  One per ring stage.
struct DecChunk {
  int pos, flags;              // kPageOk, kUnitEnd
  int q0, r0nr, head;          // r0nr: first row (token, head) of the tile * 2 + how many
  int pbase, hi;               // position of the request's first row; positions below hi are seen
  long long end;               // the unit's end on the line
};
constexpr int kPageOk = 1, kUnitEnd = 2, kBegins = 4;

DEVI void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
DEVI void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 16-bit transpose across the warp.
DEVI uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c += A B; fp16 operands (F16) or bf16
template <bool F16>
DEVI void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = A B + {i0, i1, i0, i1} in fp16
DEVI void mma_from(float (&c)[4], float i0, float i1, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                   uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(i0), "f"(i1));
}
DEVI void cp_async16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
DEVI float pow2_biased(int e) { return __uint_as_float(static_cast<uint32_t>(e) << 23); }

// Two values as N parts of 16 bits, largest first; each part rounds what the
// ones before it leave.
template <bool F16, int N>
DEVI void split_parts(float x, float y, uint32_t (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (F16) {
      const __half2 a = __floats2half2_rn(x, y);
      h[i] = *reinterpret_cast<const uint32_t*>(&a);
      if (i + 1 < N) {
        const float2 f = __half22float2(a);
        x -= f.x;
        y -= f.y;
      }
    } else {
      h[i] = pack_bf16(x, y);
      x -= bf16lo(h[i]);
      y -= bf16hi(h[i]);
    }
  }
}

// 8 codes -> fp16 pairs of codes (j, j + 4), j = 0..3: u 2^-24 for even j, u 2^-20
// for odd j; SIGNED: q and 16 q, as normal numbers (exact: 1024 + u less 1032).
template <bool SIGNED>
DEVI void codes_f16(uint32_t w, uint32_t (&r)[4]) {
  constexpr uint32_t one = SIGNED ? 0x64006400u : 0u;
  r[0] = (w & 0x000F000Fu) | one;
  r[1] = (w & 0x00F000F0u) | one;
  const uint32_t v = w >> 8;
  r[2] = (v & 0x000F000Fu) | one;
  r[3] = (v & 0x00F000F0u) | one;
  if constexpr (SIGNED) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r[j]) : "r"(r[j]), "r"(j & 1 ? 0x64806480u : 0x64086408u));
  }
}

// Byte offset of 16-byte piece c of token t inside a chunk: shared-memory banks
// are hit once per access in both products (keys by token, values by token pair).
template <int HD, int BITS>
DEVI uint32_t cell(int t, int c) {
  if constexpr (BITS == 16) {
    return static_cast<uint32_t>(t * HD * 2 + ((c ^ (t & 7)) << 4));
  } else if constexpr (HD == 128) {
    return static_cast<uint32_t>((t >> 1) * 128 + ((t ^ (t >> 1)) & 1) * 64 + ((c ^ (((t >> 2) & 1) << 1)) << 4));
  } else {
    return static_cast<uint32_t>(((t >> 3) * 2 + (t & 1)) * 128 + ((((t >> 1) & 3) ^ ((t & 1) << 1)) << 5) + (c << 4));
  }
}

// Element offset in out of row r (token, head of the group) of a request.
DEVI int64_t out_at(const AttnArgs& a, int group, int hd, int q0, int r, int head) {
  return static_cast<int64_t>(q0 + r / group) * a.ldo + static_cast<int64_t>(head * group + r % group) * hd;
}

// Lane's HD / 32 consecutive dims of an output row.
template <int HD, bool F32>
DEVI void store_row(const AttnArgs& a, int64_t at, const float (&v)[HD / 32], float inv) {
  float y[HD / 32];
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) y[i] = v[i] * inv;
  store_act<!F32, HD / 32>(a.out, at, y);
}

// Joins n <= 32 pieces of one row: piece i's sums, maximum and sum of weights are
// at of(i).  The result is in the lanes' acc (HD / 32 dims each).
template <int HD, int TILE, typename Of>
DEVI void join_row(int n, int r, Of of, float (&acc)[HD / 32], float& m, float& l) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  float pm = -FLT_MAX, pl = 0.f;
  if (lane < n) {
    const float* q = of(lane);
    pm = q[TILE * HD + r];
    pl = q[TILE * HD + TILE + r];
  }
  const float top = fmaxf(m, warp_max(pm));
  const float w = lane < n ? exp2_fast(pm - top) : 0.f;
  const float old = exp2_fast(m - top);
  l = l * old + warp_sum(pl * w);
  m = top;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    float v[E];
    load_act<false, E>(of(i), r * HD + lane * E, v);
    const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(v[e], wi, acc[e]);
  }
}

template <int HD, int BITS, bool F32>
__global__ void __launch_bounds__(Dec<HD, BITS, F32>::WARPS * 32, Dec<HD, BITS, F32>::CTAS)
    attn_decode_kernel(const AttnArgs a) {
  using D = Dec<HD, BITS, F32>;
  constexpr int TILE = kDecTile, CT = D::CT, KS = D::KS, NST = D::NST, W = D::WARPS, QP = D::QP, PP = D::PP;
  constexpr bool Q4 = BITS == 4;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ ShareScratch<W * 32> sc;
  __shared__ AttnWalk<TILE, CT> walks[W];
  __shared__ DecChunk chunks[W][NST];
  __shared__ struct Seg {
    int used, ends, q0, r0nr, head;
  } seg[W][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int group = a.n_head / a.kv.n_kv_head;
  pdl_wait();
  pdl_launch();
  if (tid < W * 2) seg[tid >> 1][tid & 1].used = 0;
  find_share<TILE, CT, W * 32>(a, group, W, sc);
  const AttnShare sh = sc.share;
  int* heads = reinterpret_cast<int*>(a.ws) + blockIdx.x * kHeadInts;
  float* parts = a.ws + gridDim.x * kHeadInts;
  if (tid == 0) heads[0] = 0;
  if (sh.w0 >= sh.w1) return;   // the whole CTA
  unsigned char* ring = smem + warp * D::RING;
  // a warp's piece of a unit that came in from before it, and of one that goes on
  // behind it (in the drained ring)
  auto part_of = [&](int w, int slot) {
    return reinterpret_cast<float*>(slot ? smem + w * D::RING : smem + W * D::RING + w * D::PART * 4);
  };
  const uint32_t ring_a = smem_addr(ring);

  const long long span = sh.w1 - sh.w0;
  const long long a0 = sh.w0 + span * warp / W, a1 = sh.w0 + span * (warp + 1) / W;
  if (a0 < a1) {
    constexpr int PC = D::ROWB / 16;    // 16-byte pieces per token
    constexpr int NP = CT * PC / 32;    // pieces per lane and side
    uint32_t dst[NP];                   // their places in a stage
#pragma unroll
    for (int i = 0; i < NP; ++i) dst[i] = ring_a + cell<HD, BITS>((i * 32 + lane) / PC, (i * 32 + lane) % PC);
    // the next chunk to request; what changes with the unit alone is in shared
    // memory (all lanes hold and write the same)
    AttnWalk<TILE, CT>& walk = walks[warp];
    int pos, left, hi, lo, sink, sink_end, win_from, seq, head;
    auto take_unit = [&](const AttnWalk<TILE, CT>& w) {
      pos = w.pos;
      left = w.left;
      hi = w.u.hi;
      lo = w.u.lo;
      sink = w.u.sink;
      sink_end = w.u.ns * CT;
      win_from = w.u.wf * CT;
      seq = w.seq;
      head = w.head;
      __syncwarp();
      walk = w;
      __syncwarp();
    };
    {
      AttnWalk<TILE, CT> w;
      w.seek(a, group, sh, a0);
      take_unit(w);
    }
    int to_req = static_cast<int>(a1 - a0), to_use = to_req;
    int tab_seq = -1, tab0 = 0, tab = 0;   // 32 table entries, one per lane
    int rstage = 0;                        // stage of the next request
    const int64_t kv_gap = static_cast<int64_t>(a.kv.n_kv_head) * kv_block_bytes(HD, BITS);
    auto request = [&]() {
      if (to_req > 0) {
        const int pg = pos / kPageTokens, t0 = pos % kPageTokens;
        if (tab_seq != seq || static_cast<unsigned>(pg - tab0) >= 32u) {
          tab_seq = seq;
          tab0 = pg;
          tab = pg + lane < a.width ? table_of(a, seq)[pg + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, tab, pg - tab0);
        const bool any = pos < hi;           // (an empty unit has one chunk that no row sees)
        const bool ok = page >= 0 && page < a.kv.n_pages;
        if (any && !ok && lane == 0) raise_error(a.err, DEV_ERR_BAD_PAGE);
        const unsigned char* kb = kv_block(a.kv, ok ? page : 0, 0, head);
        const uint32_t st = static_cast<uint32_t>(rstage) * D::STAGE;
        const unsigned char* src = kb + t0 * D::ROWB + lane * 16;   // pieces lie in order
        if (ok && pos + CT <= hi && (pos >= lo || pos + CT <= sink)) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            cp_async16_at(dst[i] + st, src + i * 512);
            cp_async16_at(dst[i] + st + D::KB, src + kv_gap + i * 512);
          }
        } else {
          // tokens that no row sees are filled with zeros
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int j = pos + (i * 32 + lane) / PC;
            const bool take = ok && j < hi && (j >= lo || j < sink);
            cp16_or_zero(dst[i] + st, src + i * 512, take);
            cp16_or_zero(dst[i] + st + D::KB, src + kv_gap + i * 512, take);
          }
        }
        if constexpr (Q4) {
          constexpr int SP = CT * 2 / 16;   // pieces of one side's scales
          if (lane < 2 * SP)
            cp16_or_zero(ring_a + st + 2 * D::KB + lane * 16,
                         kb + (lane < SP ? 0 : kv_gap) + kPageTokens * HD / 2 + t0 * 2 + (lane % SP) * 16, any && ok);
        }
        if (lane == 0) {
          DecChunk& d = chunks[warp][rstage];
          d.pos = pos;
          d.flags = (ok ? kPageOk : 0) | (left == 1 ? kUnitEnd : 0) | (walk.start >= a0 ? kBegins : 0);
          d.q0 = walk.u.q0;
          d.r0nr = walk.u.r0 * 2 + walk.u.nr;
          d.head = head;
          d.pbase = static_cast<int>(max(-0x40000000ll, min(walk.u.pbase, 0x7fff0000ll)));
          d.hi = hi;
          d.end = walk.start + walk.u.n;
        }
        rstage = rstage + 1 == NST ? 0 : rstage + 1;
        if (--to_req > 0) {
          pos += CT;
          if (pos == sink_end) pos = win_from;   // the sinks are done
          if (--left == 0) {
            AttnWalk<TILE, CT> w = walk;
            w.next_unit(a, group);
            take_unit(w);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) request();

    // this lane's cells of the first 8 tokens: of token g (keys), of 2c and 2c + 1 (values)
    const uint32_t k_at = Q4 ? (HD == 128 ? cell<HD, 4>(g, c) : cell<HD, 4>(g, c >> 1) + (c & 1) * 8) : 0;
    uint32_t v_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      v_at[e] = HD == 128 ? cell<HD, 4>(2 * c + e, g >> 1) + (g & 1) * 8 : cell<HD, 4>(2 * c + e, g >> 2) + (g & 3) * 4;
    const float sc2 = a.scale * 1.4426950408889634f;
    // B operand of the scores: row g, this lane's k pairs.  Accumulators and
    // statistics: rows 2c and 2c + 1.
    uint32_t qf[KS][2][QP];
    float qinit[2] = {0.f, 0.f}, qscale[2] = {sc2, sc2};   // 4 bits: -8 * (the row's sum); what its scaling stands for
    float o[HD / 16][4], m[2], l[2];    // [16 dims][row of the two + 2 * second dim]
    int p[2] = {0, 0};                  // the rows' positions, -1: no row
    int seen_from = 0, seen_to = 0;     // positions that every row sees (beside the sinks)
    bool fresh = true;
    int stage = NST - 1;

#pragma unroll 1
    while (true) {
      stage = stage + 1 == NST ? 0 : stage + 1;
      const DecChunk& ck = chunks[warp][stage];
      if (fresh) {
        fresh = false;
        __syncwarp();
        const int r0 = (ck.r0nr >> 4) * 8, nr = ck.r0nr & 15;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          p[r] = 2 * c + r < nr ? max(-1, ck.pbase + (r0 + 2 * c + r) / group) : -1;
          m[r] = -FLT_MAX;
          l[r] = 0.f;
        }
        const int pmin = max(-1, ck.pbase + r0 / group), pmax = max(-1, ck.pbase + (r0 + nr - 1) / group);
        seen_from = a.window > 0 ? pmax - a.window + 1 : 0;
        seen_to = min(pmin + 1, ck.hi);
#pragma unroll
        for (int t = 0; t < HD / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
        const int r = r0 + g;
        const bool live = g < nr;
        const int64_t at = static_cast<int64_t>(ck.q0 + r / group) * a.ldq + static_cast<int64_t>(ck.head * group + r % group) * HD;
        if constexpr (!Q4) {
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x[2] = {0.f, 0.f};
              if (live) load_act<!F32, 2>(a.q, at + 16 * s + 8 * h + 2 * c, x);
              split_parts<false, QP>(x[0], x[1], qf[s][h]);
            }
        } else {
          // this lane's quarter of the row, scaled to 2^13 .. 2^14 at its largest
          constexpr int N = HD / 4;
          float x[N], top_x = 0.f;
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (live) load_act<!F32, 4>(a.q, at + c * N + i, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[i + e] = v[e];
              top_x = max_nan(top_x, fabsf(v[e]));
            }
          }
          top_x = max_nan(top_x, __shfl_xor_sync(0xffffffffu, top_x, 1));
          top_x = max_nan(top_x, __shfl_xor_sync(0xffffffffu, top_x, 2));
          const bool finite = top_x <= FLT_MAX;
          const int k = finite && top_x > 0.f ? 13 - ilogbf(top_x) : 0;
          // (2^k in two factors: it may lie outside fp32)
          const float u0 = finite ? scalbnf(1.f, k / 2) : 0.f, u1 = scalbnf(1.f, k - k / 2);
          float sum = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // elements j, j + 4 of word s / 2, j = 2 (s % 2) + h; odd j against
              // codes that stand 16 times as high
              const int e0 = 8 * (s >> 1) + 2 * (s & 1) + h;
              const float w = h ? u1 * 0.0625f : u1;
              split_parts<true, QP>(x[e0] * u0 * w, x[e0 + 4] * u0 * w, qf[s][h]);
              float v = 0.f;
#pragma unroll
              for (int i = QP - 1; i >= 0; --i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[s][h][i]));
                v += f.x + f.y;
              }
              sum += h ? 16.f * v : v;
            }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const float qs = finite ? scalbnf(sc2, (F32 ? 0 : 24) - k) : NAN;
#pragma unroll
          for (int r2 = 0; r2 < 2; ++r2) {
            qinit[r2] = F32 ? 0.f : -0x1p-21f * __shfl_sync(0xffffffffu, sum, (2 * c + r2) * 4);
            qscale[r2] = __shfl_sync(0xffffffffu, qs, (2 * c + r2) * 4);
          }
        }
      }
      cp_wait<NST - 2>();
      __syncwarp();
      request();                        // into the stage used last time
      const int at_pos = ck.pos, flags = ck.flags;
      const uint32_t st = ring_a + stage * D::STAGE;
      const unsigned char* sp = ring + stage * D::STAGE;

      // ---- scores x[16 tokens][half of 8][row]: token 16 t + 8 h + g
      constexpr int NT = CT / 16;
      float x[NT][2][2];
      {
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] = Q4 ? qinit[e & 1] : 0.f;
        if constexpr (!Q4) {
          // the small parts first: the accumulator truncates at its size
#pragma unroll
          for (int i = QP - 1; i >= 0; --i)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                uint32_t f[4];   // 16 tokens x 16 dims
                ldsm4(f, st + cell<HD, 16>(t * 16 + (lane & 15), k * 2 + (lane >> 4)));
                mma<false>(s[t], f[0], f[1], f[2], f[3], qf[k][0][i], qf[k][1][i]);
              }
        } else {
          uint32_t wd[NT][2][HD / 32];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (HD == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(sp + k_at + (t * 2 + h) * 512);
                wd[t][h][0] = v.x;
                wd[t][h][1] = v.y;
                wd[t][h][HD / 32 - 2] = v.z;
                wd[t][h][HD / 32 - 1] = v.w;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(sp + k_at + (t * 2 + h) * 256);
                wd[t][h][0] = v.x;
                wd[t][h][1] = v.y;
              }
            }
#pragma unroll
          for (int q = 0; q < HD / 32; ++q)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              uint32_t f0[4], f1[4];
              codes_f16<F32>(wd[t][0][q], f0);
              codes_f16<F32>(wd[t][1][q], f1);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = QP - 1; i >= 0; --i)
                  mma<true>(s[t], f0[2 * h], f1[2 * h], f0[2 * h + 1], f1[2 * h + 1], qf[2 * q + h][0][i], qf[2 * q + h][1][i]);
            }
        }
        const uint16_t* ks = reinterpret_cast<const uint16_t*>(sp + 2 * D::KB);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float k = Q4 ? bf16bits_to_f32(ks[t * 16 + h * 8 + g]) : 1.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) x[t][h][r] = s[t][2 * h + r] * (Q4 ? qscale[r] * k : sc2);
          }
      }
      // ---- mask: all of the chunk is seen by all rows, or per row and token
      const bool ok = flags & kPageOk;  // a page out of range counts as not seen
      const bool see_all = ok && at_pos + CT <= seen_to && (at_pos >= seen_from || at_pos + CT <= a.sinks);
      uint32_t seen = 0;                // one bit per score of this lane
      if (!see_all) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = at_pos + t * 16 + h * 8 + g;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              bool v = ok && j <= p[r] && j < ck.hi;
              if (a.window > 0) v = v && (j > p[r] - a.window || j < a.sinks);
              seen |= static_cast<uint32_t>(v) << (t * 4 + h * 2 + r);
              if (!v) x[t][h][r] = -INFINITY;
            }
          }
      }
      // ---- running maximum and sum
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = m[r];
#pragma unroll
        for (int t = 0; t < NT; ++t) mx[r] = fmaxf(mx[r], fmaxf(x[t][0][r], x[t][1][r]));
      }
#pragma unroll
      for (int b = 4; b < 32; b <<= 1)
#pragma unroll
        for (int r = 0; r < 2; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], b));
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = exp2_fast(m[r] - mx[r]);
          l[r] *= f;
          m[r] = mx[r];
#pragma unroll
          for (int t = 0; t < HD / 16; ++t) {
            o[t][r] *= f;
            o[t][2 + r] *= f;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[t][h][r] = exp2_fast(x[t][h][r] - m[r]);
            l[r] += x[t][h][r];
          }
      // ---- weighted values
      uint32_t pf[NT][2][PP];           // B operand: row g, tokens 16 t + 8 h + 2c, + 1
      if constexpr (!Q4) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            split_parts<false, PP>(x[t][h][0], x[t][h][1], pf[t][h]);
#pragma unroll
            for (int i = 0; i < PP; ++i) pf[t][h][i] = movm(pf[t][h][i]);
          }
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          float own[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t f[4];   // dims 0-7 and 8-15 of 16 x tokens 0-7, then tokens 8-15
            ldsm4_t(f, st + D::KB + cell<HD, 16>(t * 16 + (lane & 7) + ((lane >> 4) << 3), d * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int i = PP - 1; i >= 0; --i) {
              if constexpr (D::OWN) mma<false>(own, f[0], f[1], f[2], f[3], pf[t][0][i], pf[t][1][i]);
              else mma<false>(o[d], f[0], f[1], f[2], f[3], pf[t][0][i], pf[t][1][i]);
            }
          }
          if constexpr (D::OWN) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] += own[e];
          }
        }
      } else {
        const uint16_t* vs = reinterpret_cast<const uint16_t*>(sp + 2 * D::KB) + CT;
        float cm[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float v = bf16bits_to_f32(vs[t * 16 + h * 8 + g]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              x[t][h][r] *= v;
              if (!see_all && !((seen >> (t * 4 + h * 2 + r)) & 1u)) x[t][h][r] = 0.f;   // (a hidden token's scale may be a NaN)
              cm[r] = max_nan(cm[r], x[t][h][r]);
            }
          }
#pragma unroll
        for (int b = 4; b < 32; b <<= 1)
#pragma unroll
          for (int r = 0; r < 2; ++r) cm[r] = max_nan(cm[r], __shfl_xor_sync(0xffffffffu, cm[r], b));
        // weights scaled to 2^13 .. 2^14 at the chunk's largest
        float up[2], f0[2], f1[2];      // f0: their unit, but for a constant power of 2; f1: that of codes 16 times as high
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int ce = max(static_cast<int>(__float_as_uint(cm[r]) >> 23), 30);
          up[r] = pow2_biased(254 + 13 - ce);
          f0[r] = cm[r] <= FLT_MAX ? pow2_biased(F32 ? ce - 13 : ce) : NAN;
          f1[r] = f0[r] * 0.0625f;
        }
        // and 8 times their sum, by a row of codes 8
        float s8[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            split_parts<true, PP>(x[t][h][0] * up[0], x[t][h][1] * up[1], pf[t][h]);
#pragma unroll
            for (int i = 0; i < PP; ++i) pf[t][h][i] = movm(pf[t][h][i]);
          }
#pragma unroll
          for (int i = PP - 1; i >= 0 && !F32; --i)
            mma<true>(s8, 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, pf[t][0][i], pf[t][1][i]);
        }
        // tokens 2c, 2c + 1, 8 + 2c, 8 + 2c + 1 of each 16; HD / 8 dims from (HD / 8) g
        constexpr int VW = HD / 64;
        uint32_t tw[NT][4][VW];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tk = (t * 2 + (e >> 1)) * 8 * D::ROWB;   // 8 tokens on: the cells repeat
            if constexpr (HD == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(sp + D::KB + v_at[e & 1] + tk);
              tw[t][e][0] = v.x;
              tw[t][e][VW - 1] = v.y;
            } else {
              tw[t][e][0] = *reinterpret_cast<const uint32_t*>(sp + D::KB + v_at[e & 1] + tk);
            }
          }
#pragma unroll
        for (int q = 0; q < VW; ++q)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7632u : 0x5410u;   // codes 4 half .. 4 half + 3 of two tokens
            float acc[2][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              uint32_t r0[4], r1[4];
              codes_f16<F32>(__byte_perm(tw[t][0][q], tw[t][1][q], sel), r0);
              codes_f16<F32>(__byte_perm(tw[t][2][q], tw[t][3][q], sel), r1);
#pragma unroll
              for (int j = 0; j < 2; ++j)     // codes j and j + 2
#pragma unroll
                for (int i = PP - 1; i >= 0; --i) {
                  if (t == 0 && i == PP - 1)
                    mma_from(acc[j], j ? -16.f * s8[0] : -s8[0], j ? -16.f * s8[1] : -s8[1], r0[j], r0[j + 2], r1[j], r1[j + 2],
                             pf[t][0][i], pf[t][1][i]);
                  else
                    mma<true>(acc[j], r0[j], r0[j + 2], r1[j], r1[j + 2], pf[t][0][i], pf[t][1][i]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& y = o[q * 4 + half * 2 + j][e];
                y = fmaf(acc[j][e], j ? f1[e & 1] : f0[e & 1], y);
              }
          }
      }
      // ---- end of the unit or of this warp's piece
      const bool unit_end = flags & kUnitEnd;
      --to_use;
      if (unit_end || to_use == 0) {
        fresh = true;
#pragma unroll
        for (int b = 4; b < 32; b <<= 1)
#pragma unroll
          for (int r = 0; r < 2; ++r) l[r] += __shfl_xor_sync(0xffffffffu, l[r], b);
        const bool begins = flags & kBegins;
        const int slot = begins ? 1 : 0;
        float* dst = part_of(warp, slot);
        const int r0 = (ck.r0nr >> 4) * 8, nr = ck.r0nr & 15;
        const bool whole = begins && unit_end;
        if (!whole && begins) {
          cp_wait<0>();
          __syncwarp();
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int lr = 2 * c + r;
          const float inv = l[r] != 0.f ? 1.f / l[r] : 0.f;
          const float unit = Q4 && !F32 ? 0x1p11f : 1.f;   // 2^24 (codes) / 2^13 (weights)
          const int64_t at = out_at(a, group, HD, ck.q0, r0 + lr, ck.head);
          const bool live = lr < nr;
          if constexpr (Q4) {
            // dims (HD / 8) g + 8 q + 4 half + j (+ 2)
#pragma unroll
            for (int q = 0; q < HD / 32; ++q) {   // four dims at a time
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = o[q * 2 + (e & 1)][(e & 2) + r] * unit;
              const int d = (HD / 8) * g + 4 * q;
              if (whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= inv;
                if (live) store_act<!F32, 4>(a.out, at + d, v);
              } else {
                store_act<false, 4>(dst, lr * HD + d, v);
              }
            }
          } else {
#pragma unroll
            for (int t = 0; t < HD / 16; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int d = 16 * t + 8 * h + g;
                const float v = o[t][2 * h + r];
                if (!whole) dst[lr * HD + d] = v;
                else if (live && F32) static_cast<float*>(a.out)[at + d] = v * inv;
                else if (live) static_cast<uint16_t*>(a.out)[at + d] = f32_to_bf16bits(v * inv);
              }
          }
          if (!whole && g == 0) {
            dst[TILE * HD + lr] = m[r];
            dst[TILE * HD + TILE + lr] = l[r];
          }
        }
        if (!whole && lane == 0) {
          seg[warp][slot] = Seg{1, unit_end, ck.q0, ck.r0nr, ck.head};
          if (slot == 1 && ck.end > sh.w1) {
            // goes on behind this CTA: the last CTA whose share begins before its end
            int k = static_cast<int>((ck.end - 1) * sh.n_cta / sh.total);
            while (k + 1 < sh.n_cta && share_start(sh.total, sh.n_cta, k + 1) < ck.end) ++k;
            heads[1] = k - static_cast<int>(blockIdx.x);
          }
        }
        if (to_use == 0) break;
      }
    }
    cp_wait<0>();
  }
  __syncthreads();
  // ---- joining the warps' pieces: the unit that came in from the CTA before
  // (slot 0 of the first warps), and each unit that began in a warp and went on
  // (its slot 1, then slot 0 of the following ones).  A thread per row and four dims.
  const int jr = tid / (HD / 4), jd = (tid % (HD / 4)) * 4;
  bool came_in = true;       // no piece yet: a slot 0 is of the unit that came in
#pragma unroll 1
  for (int w0 = 0; w0 < W; ++w0) {
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
      if (!seg[w0][slot].used) continue;
      if (slot == 0 && !came_in) continue;
      came_in = false;
      const Seg info = seg[w0][slot];
      uint32_t pieces = 1u << w0;
      bool ends = info.ends != 0;
      for (int w = w0 + 1; w < W && !ends; ++w)
        if (seg[w][0].used) {      // (a warp without work has none)
          pieces |= 1u << w;
          ends = seg[w][0].ends != 0;
        }
      const bool whole = slot == 1 && ends;
      const int nr = info.r0nr & 15;
      if (jr < nr) {
        auto of = [&](int w) { return part_of(w, w == w0 ? slot : 0); };
        float top = -FLT_MAX, ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t q = pieces; q; q &= q - 1) top = fmaxf(top, of(__ffs(q) - 1)[TILE * HD + jr]);
        for (uint32_t q = pieces; q; q &= q - 1) {
          const float* part = of(__ffs(q) - 1);
          const float f = exp2_fast(part[TILE * HD + jr] - top);
          float v[4];
          load_act<false, 4>(part, jr * HD + jd, v);
          ll = fmaf(part[TILE * HD + TILE + jr], f, ll);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fmaf(v[e], f, acc[e]);
        }
        if (whole) {
          const float inv = ll != 0.f ? 1.f / ll : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] *= inv;
          store_act<!F32, 4>(a.out, out_at(a, group, HD, info.q0, (info.r0nr >> 4) * 8 + jr, info.head) + jd, acc);
        } else {
          float* out = parts + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * D::PART;
          store_act<false, 4>(out, jr * HD + jd, acc);
          if (jd == 0) {
            out[TILE * HD + jr] = top;
            out[TILE * HD + TILE + jr] = ll;
          }
        }
      }
      if (!whole && slot == 1 && tid == 0) {
        heads[2] = info.q0;
        heads[3] = (info.r0nr >> 4) * 8;
        heads[4] = nr;
        heads[5] = info.head;
        heads[0] = 1;
      }
    }
  }
}

// NaN in all rows of the call: a wait of the attention kernel ran out, and which rows
// are right is not known.
template <int HD, bool F32>
__device__ __noinline__ void rows_are_lost(const AttnArgs& a) {
  const int begin = min(a.rows, max(0, a.row_start[0])), end = min(a.rows, a.row_start[a.n_seq]), width = a.n_head * HD;
  const float nan[2] = {NAN, NAN};
  for (int row = begin + blockIdx.y * gridDim.x + blockIdx.x; row < end; row += gridDim.x * gridDim.y)
    for (int i = threadIdx.x * 2; i < width; i += 512) store_act<!F32, 2>(a.out, static_cast<int64_t>(row) * a.ldo + i, nan);
}

// Joins the units that several CTAs worked on, in CTA order: CTA c's header
// names the unit that began in it, whose pieces are (c, 1), (c + 1, 0), ..  A warp
// per row, 8 rows a CTA.  The weights e^(m_i - m) and sums are fp32, added in piece
// order: a result does not depend on which CTA ended first.  Bound by latency: 6 us
// after a decode step, 15 us after long prompts (up to 40 MB of pieces), most of either
// hidden by the launch's overlap with the attention kernel's end.
template <int HD, bool F32, int TILE>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, int n_cta) {
  constexpr int PART = TILE * (HD + 2), E = HD / 32;
  pdl_wait();
  if constexpr (TILE != kDecTile) {
    bool lost = false;
    for (int c = threadIdx.x; c < n_cta; c += 256) lost |= reinterpret_cast<const int*>(a.ws)[c * kHeadInts + kHeadLost] != 0;
    if (__syncthreads_or(lost)) {
      rows_are_lost<HD, F32>(a);
      return;
    }
  }
  const int4* h4 = reinterpret_cast<const int4*>(a.ws) + blockIdx.x * (kHeadInts / 4);
  const int4 h = h4[0], h2 = h4[1];
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (!h.x || r >= h2.x) return;
  const float* parts = a.ws + n_cta * kHeadInts;
  const int group = a.n_head / a.kv.n_kv_head, n = h.y + 1;
  float acc[E], m = -FLT_MAX, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    auto of = [&](int i) {
      return parts + (static_cast<int64_t>(blockIdx.x + i0 + i) * 2 + (i0 + i == 0 ? 1 : 0)) * PART;
    };
    join_row<HD, TILE>(min(32, n - i0), r, of, acc, m, l);
  }
  store_row<HD, F32>(a, out_at(a, group, HD, h.z, h.w + r, h2.y) + lane * E, acc, l != 0.f ? 1.f / l : 0.f);
}

template <int HD, bool F32, int TILE>
static cudaError_t join_one(const AttnArgs& a, int grid, cudaStream_t st) {
  return launch_pdl(attn_join_kernel<HD, F32, TILE>, dim3(grid, TILE / 8), dim3(256), 0, st, a, grid);
}

cudaError_t launch_attn_join(const AttnArgs& a, bool bf16, int tile, int grid, cudaStream_t st) {
  const bool wide = a.kv.head_dim == 128;
  if (tile == kDecTile) {
    if (bf16) return wide ? join_one<128, false, kDecTile>(a, grid, st) : join_one<64, false, kDecTile>(a, grid, st);
    return wide ? join_one<128, true, kDecTile>(a, grid, st) : join_one<64, true, kDecTile>(a, grid, st);
  }
  if (bf16) return wide ? join_one<128, false, 256>(a, grid, st) : join_one<64, false, 256>(a, grid, st);
  return wide ? join_one<128, true, 128>(a, grid, st) : join_one<64, true, 128>(a, grid, st);
}

template <int HD, int BITS, bool F32>
static cudaError_t launch_one(const AttnArgs& a, int n_sm, cudaStream_t st) {
  using D = Dec<HD, BITS, F32>;
  const int grid = n_sm * D::CTAS;
  static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its shared memory
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_decode_kernel<HD, BITS, F32>), D::SMEM, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_decode_kernel<HD, BITS, F32>, dim3(grid), dim3(D::WARPS * 32), D::SMEM, st, a);
  if (e != cudaSuccess) return e;
  return launch_attn_join(a, !F32, kDecTile, grid, st);
}

int64_t decode_workspace_floats(int bits, int head_dim) {
  const int64_t grid = kAttnSms * (bits == 4 ? 2 : 1), part = kDecTile * (head_dim + 2);
  return grid * (kHeadInts + 2 * part);
}

cudaError_t launch_attn_decode(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  if (a.kv.head_dim == 128) {
    if (a.kv.bits == 16) return bf16 ? launch_one<128, 16, false>(a, n_sm, st) : launch_one<128, 16, true>(a, n_sm, st);
    return bf16 ? launch_one<128, 4, false>(a, n_sm, st) : launch_one<128, 4, true>(a, n_sm, st);
  }
  if (a.kv.bits == 16) return bf16 ? launch_one<64, 16, false>(a, n_sm, st) : launch_one<64, 16, true>(a, n_sm, st);
  return bf16 ? launch_one<64, 4, false>(a, n_sm, st) : launch_one<64, 4, true>(a, n_sm, st);
}

}  // namespace dualar
