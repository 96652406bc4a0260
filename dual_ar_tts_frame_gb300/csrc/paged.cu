// Paged key/value operators: step plans, QK-norm + rotation + append, cache
// read-back, and the choice of an attention kernel.
//
// Formulas and layouts: include/dualar_paged.h.
#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "paged.h"

namespace dualar {

// ============================================================================
// Step plan
// ============================================================================
// A cluster of CTAs.  Each takes the prefix sums of the requests' rows and pages
// (redundantly: a few thousand numbers), counts the free pages of its slice of
// the pool, learns the lower slices' counts through distributed shared memory,
// hands its free pages out, and after a second cluster barrier, which makes the
// table's new cells visible, lays out its share of the rows.  Bound by a chain of
// dependent reads (lengths, pool, table), not by bytes.
// Measured: 16 requests, 2048 pages, one CTA: 10 us.  500 requests of 1 to 401 new
// tokens, 131072 pages, a cluster of 8: 28 us; a call of it took 63 us when the cluster
// came and 96 us with one CTA, through which all 512 KB of page counts went.
constexpr int kPlanThreads = 1024;

// Inclusive prefix sums over the CTA of (v, w); *tv, *tw receive the sums.
// tot: 2 * kPlanThreads / 32 values.
DEVI void block_scan2(long long& v, long long& w, long long* tot, long long* tv, long long* tw) {
  constexpr int NW = kPlanThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v, o), b = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) {
      v += a;
      w += b;
    }
  }
  __syncthreads();
  if (lane == 31) {
    tot[warp] = v;
    tot[NW + warp] = w;
  }
  __syncthreads();
  // every warp scans the warps' totals for itself
  long long a = tot[lane], b = tot[NW + lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += c;
      b += d;
    }
  }
  *tv = __shfl_sync(0xffffffffu, a, 31);
  *tw = __shfl_sync(0xffffffffu, b, 31);
  const long long before_v = __shfl_sync(0xffffffffu, a, (warp + 31) & 31);
  const long long before_w = __shfl_sync(0xffffffffu, b, (warp + 31) & 31);
  if (warp > 0) {
    v += before_v;
    w += before_w;
  }
}

DEVI uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
DEVI void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Value of a shared variable in CTA `rank` of the cluster.
DEVI int cluster_load(const int* p, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return static_cast<int>(v);
}

// Which of pages 4 q .. 4 q + 3 are free.
DEVI uint32_t free_mask(const PlanArgs& a, int q) {
  uint32_t m = 0;
  if (4 * q + 3 < a.n_pages && (reinterpret_cast<uintptr_t>(a.page_refs) & 15u) == 0) {
    const int4 r = *reinterpret_cast<const int4*>(a.page_refs + 4 * q);
    m = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
  } else {
    for (int e = 0; e < 4; ++e)
      if (4 * q + e < a.n_pages) m |= static_cast<uint32_t>(a.page_refs[4 * q + e] == 0) << e;
  }
  return m;
}

__global__ void __launch_bounds__(kPlanThreads, 1) kv_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* row0 = plan_smem;                  // [n_seq + 1] first row of each request
  int32_t* page0 = plan_smem + a.n_seq + 1;   // [n_seq + 1] pages taken before each request
  __shared__ long long tot[2 * kPlanThreads / 32];
  __shared__ int warp_tot[kPlanThreads / 32], my_free;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x, n_cta = cluster_size();   // (the grid is one cluster)
  pdl_wait();
  pdl_launch();
  // ---- this slice's free pages, counted while the lengths arrive
  const int quads = (a.n_pages + 3) / 4, per = (quads + static_cast<int>(n_cta) - 1) / static_cast<int>(n_cta);
  const int q0 = static_cast<int>(rank) * per, q1 = min(quads, q0 + per);
  int mine = 0;
  for (int q = q0 + tid; q < q1; q += kPlanThreads) mine += __popc(free_mask(a, q));
  // ---- prefix sums over the requests
  long long rows = 0, pages = 0;
  bool neg = false, wide = false, bad = false;
  for (int s0 = 0; s0 < a.n_seq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    long long len = 0, add = 0;
    if (s < a.n_seq) {
      len = a.kv_len[s];
      add = a.n_new[s];
      neg |= len < 0 || add < 0;
      wide |= (len + add + kPageTokens - 1) / kPageTokens > a.width;
      // the page that a request's next token goes to is the caller's (the others of
      // a plan come from the pool): out of range, its slot could be another page's
      if (add > 0 && len > 0 && len % kPageTokens && len / kPageTokens < a.width) {
        const int page = a.table[static_cast<int64_t>(s) * a.width + len / kPageTokens];
        bad |= page < 0 || page >= a.n_pages;
      }
    }
    long long r = add, p = (len + add + kPageTokens - 1) / kPageTokens - (len + kPageTokens - 1) / kPageTokens, tr, tp;
    block_scan2(r, p, tot, &tr, &tp);
    if (s < a.n_seq) {
      row0[s + 1] = static_cast<int32_t>(min(rows + r, 0x7fffffffll));
      page0[s + 1] = static_cast<int32_t>(min(pages + p, 0x7fffffffll));
    }
    rows += tr;
    pages += tp;
  }
  if (tid == 0) row0[0] = page0[0] = 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) warp_tot[warp] = mine;
  neg = __syncthreads_or(neg);
  wide = __syncthreads_or(wide);
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    const int v = __reduce_add_sync(0xffffffffu, warp_tot[lane]);
    if (lane == 0) my_free = v;
  }
  cluster_barrier();
  long long before = 0, free_pages = 0;
  for (uint32_t c = 0; c < n_cta; ++c) {
    const int v = cluster_load(&my_free, c);
    if (c < rank) before += v;
    free_pages += v;
  }
  int code = 0;
  if (pages > free_pages) code = 1;
  if (wide) code = 2;
  if (rows > a.max_rows) code = 4;
  if (bad) code = 5;
  if (neg) {
    code = 3;
    rows = pages = 0;
  }
  const bool ok = code == 0;
  if (rank == 0 && tid == 0) {
    a.status[0] = code;
    a.status[1] = static_cast<int32_t>(min(rows, 0x7fffffffll));
    a.status[2] = static_cast<int32_t>(min(pages, 0x7fffffffll));
  }
  if (rank == 0)
    for (int s = tid; s <= a.n_seq; s += kPlanThreads) a.row_start[s] = ok ? row0[s] : 0;
  // ---- the k-th free page goes to the request whose share holds k
  if (ok) {
    for (int b = q0; b < q1 && before < pages; b += kPlanThreads) {
      const int q = b + tid;
      const uint32_t m = q < q1 ? free_mask(a, q) : 0u;
      int incl = __popc(m);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      __syncthreads();
      if (lane == 31) warp_tot[warp] = incl;
      __syncthreads();
      int w = warp_tot[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
      }
      const int all = __shfl_sync(0xffffffffu, w, 31), ahead = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
      long long k = before + (warp > 0 ? ahead : 0) + incl - __popc(m);
      for (uint32_t f = m; f && k < pages; f &= f - 1, ++k) {
        const int p = 4 * q + __ffs(f) - 1;
        const int s = upper_index(page0, a.n_seq, static_cast<int32_t>(k));
        const int had = (a.kv_len[s] + kPageTokens - 1) / kPageTokens;
        a.table[static_cast<int64_t>(s) * a.width + had + (k - page0[s])] = p;
        a.page_refs[p] = 1;
      }
      before += all;
    }
  }
  cluster_barrier();   // the table cells written above are read below; no CTA reads another's memory behind it
  const int stride = static_cast<int>(n_cta) * kPlanThreads;
  for (int r = static_cast<int>(rank) * kPlanThreads + tid; r < a.max_rows; r += stride) {
    int pos = 0, slot = -1;
    if (ok && r < rows) {
      const int s = upper_index(row0, a.n_seq, r);
      pos = a.kv_len[s] + r - row0[s];
      slot = __ldcg(a.table + static_cast<int64_t>(s) * a.width + pos / kPageTokens) * kPageTokens + pos % kPageTokens;
    }
    a.pos[r] = pos;
    a.slot[r] = slot;
  }
  cluster_barrier();   // kv_len may be new_len
  if (rank == 0)
    for (int s = tid; s < a.n_seq; s += kPlanThreads) a.new_len[s] = ok ? a.kv_len[s] + a.n_new[s] : a.kv_len[s];
}

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kv_plan_kernel), 2 * (kMaxPlanSeqs + 1) * 4, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // one CTA reads 4096 pages at a time: alone up to two rounds of them (and of rows)
  const unsigned n = a.n_pages <= 8192 && a.max_rows <= 4096 ? 1 : 8;
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = 2 * (a.n_seq + 1) * sizeof(int32_t);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
}

// ============================================================================
// QK-norm, rotation, append
// ============================================================================
// A CTA per row; HD / 8 lanes per head vector, 8 elements (16 bytes of bf16) each,
// so a warp holds 2 or 4 vectors, and the row's rotation is read once per lane.
// Memory bound: every vector is read once and written once.  The sum of squares,
// the rotation and the scale are fp32; a cell is rounded once, when it is stored.
// Measured: 8001 rows of 32 + 2 x 8 heads of 128, bf16: 46.6 us, 4.2 TB/s (62% of a
// copy's rate: each row is a CTA that waits for its position, its slot and then its
// vectors).  4096 rows to 4-bit cells: 47.5 us, 2.7 TB/s of input and output, bound by
// instructions (the exact rounding of the codes); with 64-bit arithmetic for it, 89 us
// per call instead of 55.
// Few rows: 6.3 us at 8, 17 us at 64 rows to 4 bits, a launch and three dependent
// reads, then (4 bits) fp64 for the few elements next to a rounding border.

// 8 bf16 (one 16-byte word) or 8 fp32 values (two).
template <bool BF16>
DEVI void widen8(const uint4 (&r)[BF16 ? 1 : 2], float (&x)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16lo(w[j]);
      x[2 * j + 1] = bf16hi(w[j]);
    }
  } else {
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
  }
}
template <bool BF16>
DEVI void store8(void* p, int64_t i, const float (&x)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}
// 8 bf16 that are 4-byte aligned.
DEVI void load_table8(const uint16_t* p, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(p)[j];
    x[2 * j] = bf16lo(w);
    x[2 * j + 1] = bf16hi(w);
  }
}

template <bool BF16, int HD, int BITS>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int L = HD / 8, VPC = 256 / L;   // lanes per vector, vectors of a CTA at a time
  constexpr int NW = BF16 ? 1 : 2, NV = 4;   // 16-byte words of a lane's elements, vectors per lane at a time
  const int row = blockIdx.x, l = threadIdx.x % L, v0 = threadIdx.x / L;
  const int hk = a.kv.n_kv_head, n_vec = a.n_head + 2 * hk;
  pdl_wait();
  pdl_launch();
  // the first vectors are on their way before the row's position is known
  uint4 raw[NV][NW];
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.qkv) +
                                                    (static_cast<int64_t>(row) * a.ld + 8 * l) * (BF16 ? 2 : 4));
  auto fetch = [&](int vb) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int h = vb + k * VPC + v0;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        raw[k][w] = make_uint4(0, 0, 0, 0);
        if (h < n_vec) raw[k][w] = src[static_cast<int64_t>(h) * (HD / 8 * NW) + w];
      }
    }
  };
  fetch(0);
  const int pos = a.pos[row], slot = a.slot[row];
  if (pos < 0 || pos >= a.n_pos) {
    if (threadIdx.x == 0) raise_error(a.err, DEV_ERR_BAD_INDEX);
    return;
  }
  const bool far = slot >= a.kv.n_pages * kPageTokens;
  if (far && threadIdx.x == 0) raise_error(a.err, DEV_ERR_BAD_INDEX);
  const bool put = slot >= 0 && !far;
  const int live = put ? n_vec : a.n_head;
  float cs[4], sn[4];
  {
    const int64_t i = static_cast<int64_t>(pos) * (HD / 2) + 4 * l;
    const uint32_t c0 = *reinterpret_cast<const uint32_t*>(a.cos + i), c1 = *reinterpret_cast<const uint32_t*>(a.cos + i + 2);
    const uint32_t s0 = *reinterpret_cast<const uint32_t*>(a.sin + i), s1 = *reinterpret_cast<const uint32_t*>(a.sin + i + 2);
    cs[0] = bf16lo(c0);
    cs[1] = bf16hi(c0);
    cs[2] = bf16lo(c1);
    cs[3] = bf16hi(c1);
    sn[0] = bf16lo(s0);
    sn[1] = bf16hi(s0);
    sn[2] = bf16lo(s1);
    sn[3] = bf16hi(s1);
  }
  const int page = put ? slot / kPageTokens : 0, t = put ? slot % kPageTokens : 0;
  // whole warps go on together: a warp's last vectors may be behind the row's end
  constexpr int VPW = 32 / L;
  const int warp_v0 = v0 / VPW * VPW;
  for (int vb = 0; vb + warp_v0 < live; vb += VPC * NV) {
    if (vb > 0) fetch(vb);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int h = vb + k * VPC + v0;
      if (h - v0 + warp_v0 >= live) break;
      const bool on = h < live;
      const bool is_q = h < a.n_head, is_v = h >= a.n_head + hk;
      float x[8], v[8], g[8];
      widen8<BF16>(raw[k], x);
      const uint16_t* gain = is_q ? a.q_norm : a.k_norm;
      const bool norm = gain != nullptr && !is_v;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.f;
      if (norm) load_table8(gain + 8 * l, g);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
      ss = lanes_sum<L>(ss);
      const float inv = norm ? 1.0f / sqrtf(ss / static_cast<float>(HD) + a.eps) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = norm ? x[j] * inv * g[j] : x[j];
      if (!is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = v[2 * j], q = v[2 * j + 1];
          v[2 * j] = p * cs[j] - q * sn[j];
          v[2 * j + 1] = p * sn[j] + q * cs[j];
        }
      }
      if (is_q && on) store8<BF16>(a.q_out, static_cast<int64_t>(row) * a.ldq + static_cast<int64_t>(h) * HD + 8 * l, v);
      const int kh = h - a.n_head - (is_v ? hk : 0);
      if constexpr (BITS == 16) {
        if (!is_q && on) store8<true>(kv_block(a.kv, page, is_v, kh), t * HD + 8 * l, v);
      } else {
        if (h - v0 + warp_v0 + VPW > a.n_head) {   // some vector of the warp is a key or value
          uint32_t u[8];
          const bool as_is = is_v || is_q;     // (a query's codes are not used)
          const uint16_t sc = quantize_vector<8, L>(x, v, g, cs, sn, as_is, norm, norm ? ss : 1.f, a.eps, u);
          uint32_t code = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) code |= u[j] << (4 * j);
          if (!is_q && on) {
            unsigned char* blk = kv_block(a.kv, page, is_v, kh);
            *reinterpret_cast<uint32_t*>(blk + t * (HD / 2) + 4 * l) = code;
            if (l == 0) reinterpret_cast<uint16_t*>(blk + kPageTokens * HD / 2)[t] = sc;
          }
        }
      }
    }
  }
}

template <bool BF16, int HD>
static cudaError_t norm_rope_one(const NormRopeArgs& a, cudaStream_t st) {
  return launch_pdl(a.kv.bits == 16 ? norm_rope_kernel<BF16, HD, 16> : norm_rope_kernel<BF16, HD, 4>, dim3(a.rows), dim3(256), 0,
                    st, a);
}

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, bool bf16, cudaStream_t st) {
  if (a.kv.head_dim == 128) return bf16 ? norm_rope_one<true, 128>(a, st) : norm_rope_one<false, 128>(a, st);
  return bf16 ? norm_rope_one<true, 64>(a, st) : norm_rope_one<false, 64>(a, st);
}

// ============================================================================
// Read-back
// ============================================================================
// HD / 8 lanes per vector, 8 elements each; exact.  Memory bound, mostly by the fp32
// output: 4096 slots of 2 x 8 heads of 128 from 4 bits: 12 us, 3.2 TB/s.
template <int HD>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvView kv, const int32_t* slots, int n, float* k, float* v,
                                                      uint32_t* err) {
  constexpr int L = HD / 8;
  pdl_wait();
  pdl_launch();
  const int l = threadIdx.x % L;
  const long long id = static_cast<long long>(blockIdx.x) * (256 / L) + threadIdx.x / L;
  if (id >= 2ll * n * kv.n_kv_head) return;
  const int h = static_cast<int>(id % kv.n_kv_head), which = static_cast<int>((id / kv.n_kv_head) & 1);
  const int i = static_cast<int>(id / (2 * kv.n_kv_head));
  const int slot = slots[i];
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = 0.f;
  if (slot >= kv.n_pages * kPageTokens) {
    if (l == 0) raise_error(err, DEV_ERR_BAD_INDEX);
  } else if (slot >= 0) {
    const unsigned char* blk = kv_block(kv, slot / kPageTokens, which, h);
    const int t = slot % kPageTokens;
    if (kv.bits == 16) {
      const uint4 w[1] = {*reinterpret_cast<const uint4*>(blk + (t * HD + 8 * l) * 2)};
      widen8<true>(w, y);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + t * (HD / 2) + 4 * l);
      const float s = bf16bits_to_f32(reinterpret_cast<const uint16_t*>(blk + kPageTokens * HD / 2)[t]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = static_cast<float>(static_cast<int>((w >> (4 * j)) & 15u) - 8) * s;
    }
  }
  store8<false>(which ? v : k, (static_cast<int64_t>(i) * kv.n_kv_head + h) * HD + 8 * l, y);
}

cudaError_t launch_kv_read(const KvView& kv, const int32_t* slot, int n, float* k, float* v, uint32_t* err,
                           cudaStream_t st) {
  const int per = 256 / (kv.head_dim / 8);
  const long long blocks = (2ll * n * kv.n_kv_head + per - 1) / per;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_pdl(kv.head_dim == 128 ? kv_read_kernel<128> : kv_read_kernel<64>, dim3(static_cast<unsigned>(blocks)), dim3(256),
                    0, st, kv, slot, n, k, v, err);
}

// ============================================================================
// The decoder's rows as a step
// ============================================================================
__global__ void decoder_step_kernel(const DevPtrs d, int nrows, int one_sequence, const StepBuffers b) {
  pdl_wait();
  pdl_launch();
  const int r = threadIdx.x;
  if (r < nrows) {
    const RowInfo ri = d.rows[r];
    const int pg = ri.pos / kPageTokens;
    int slot = -1;
    if (ri.active && pg < d.pages_per_seq) {
      const int page = d.page_table[static_cast<size_t>(ri.slot) * d.pages_per_seq + pg];
      if (page >= 0 && page < d.max_pages) slot = page * kPageTokens + ri.pos % kPageTokens;
      else raise_error(d.err, DEV_ERR_BAD_PAGE);
    }
    b.pos[r] = ri.pos;
    b.slot[r] = slot;
    if (!one_sequence || r == nrows - 1) {
      const int s = one_sequence ? 0 : r;
      b.kv_len[s] = ri.pos + 1;
      b.table_row[s] = ri.slot;
      b.row_start[s + 1] = r + 1;
    }
  }
  if (r == 0) b.row_start[0] = 0;
}

cudaError_t launch_decoder_step(const DevPtrs& d, int nrows, bool one_sequence, const StepBuffers& b, cudaStream_t st) {
  static_assert(kMaxRows <= 128, "one thread per row");
  return launch_pdl(decoder_step_kernel, dim3(1), dim3(128), 0, st, d, nrows, one_sequence ? 1 : 0, b);
}

// ============================================================================
// Attention: which kernel
// ============================================================================
// Few (token, head) rows a request on average: the decode kernel.  Both kernels are
// right for any rows; the decode kernel reads a request's cache once per 8 rows, the
// other once per 128 or 256 and pads its tiles to that.  The limits are where the two
// cross for requests of equal rows: 32 of 4000 tokens, 8 heads of 128, us per call
// (decode kernel, other):
//   rows           8          16         24         32         64
//   bf16         89, 178   116, 180   234, 179   214, 180   411, 181
//   bf16, fp32   93, 220   143, 221   237, 221   269, 221   516, 220
//   4 bits       53, 226    86, 227   121, 226   154, 227   290, 228
//   4 bits, fp32 76, 262   126, 262   187, 262   226, 263   432, 264
// One kernel serves the whole call, which costs mixed steps: 500 single tokens beside a
// chunk of 1500 (bf16: 698 and 248 us apart, 2616 together; 64 beside it: 63, 248 and
// 367), and rows are the call's, so those behind the last request count: 64 single
// tokens padded to 1024 rows take 228 us instead of 110 (to 128 rows: 110).
static bool few_rows(int bits, int rows, int group, int n_seq) {
  return static_cast<long long>(rows) * group <= (bits == 4 ? 32ll : 16ll) * n_seq;
}

int64_t paged_attention_workspace(bool bf16, int bits, int rows, int n_head, int n_kv_head, int head_dim, int n_seq) {
  return 4 * (few_rows(bits, rows, n_head / n_kv_head, n_seq) ? decode_workspace_floats(bits, head_dim)
                                                        : prompt_workspace_floats(!bf16, head_dim));
}

cudaError_t launch_paged_attention(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st) {
  const int n = n_sm < kAttnSms ? n_sm : kAttnSms;
  return few_rows(a.kv.bits, a.rows, a.n_head / a.kv.n_kv_head, a.n_seq) ? launch_attn_decode(a, bf16, n, st)
                                                              : launch_attn_prompt(a, bf16, n, st);
}

}  // namespace dualar
