// Device helpers of the paged key/value operators: cached vectors, activation
// vectors, and the exact 4-bit rule.
#pragma once

#include <atomic>

#include "common.cuh"
#include "paged.h"

namespace dualar {

// Lets a kernel use `bytes` of dynamic shared memory on the current device, once
// per device (`allowed`: one bit each).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit & allowed.load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A request's row of the page table.
DEVI const int32_t* table_of(const AttnArgs& a, int seq) {
  return a.table + static_cast<int64_t>(a.table_row ? a.table_row[seq] : seq) * a.width;
}

// First index s in [0, n) with start[s + 1] > x, for a non-decreasing start
// with start[n] > x.
DEVI int upper_index(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid + 1] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

DEVI unsigned char* kv_block(const KvView& kv, int page, int which, int head) {
  return kv.data + static_cast<int64_t>(page) * kv.page_stride +
         static_cast<int64_t>(which * kv.n_kv_head + head) * kv_block_bytes(kv.head_dim, kv.bits);
}

// N = 2 or 4 consecutive activations at element offset i.
template <bool BF16, int N>
DEVI void load_act(const void* p, int64_t i, float (&x)[N]) {
  if constexpr (BF16) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i);
    uint32_t r[N / 2];
    if constexpr (N == 4) {
      const uint2 t = *reinterpret_cast<const uint2*>(w);
      r[0] = t.x;
      r[1] = t.y;
    } else {
      r[0] = w[0];
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      x[2 * j] = bf16lo(r[j]);
      x[2 * j + 1] = bf16hi(r[j]);
    }
  } else if constexpr (N == 4) {
    const float4 t = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    x[0] = t.x;
    x[1] = t.y;
    x[2] = t.z;
    x[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
    x[0] = t.x;
    x[1] = t.y;
  }
}

DEVI float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared; `take` false fills zeros without reading.
DEVI void cp16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
template <int N>
DEVI void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

DEVI uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int N>
DEVI void store_bf16(uint16_t* p, const float (&x)[N]) {
  if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  else *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
}

template <bool BF16, int N>
DEVI void store_act(void* p, int64_t i, const float (&x)[N]) {
  if constexpr (BF16) store_bf16<N>(static_cast<uint16_t*>(p) + i, x);
  else if constexpr (N == 4) *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = make_float2(x[0], x[1]);
}

// ---- the 4-bit rule, exact ---------------------------------------------------
// s = bf16(max|y| / 7), code = rint(y / s), of the real numbers y that a
// vector's inputs define.  The fp32 values decide unless one of them lies next
// to a border, where its rounding could decide otherwise.  A vector that is taken
// as it is (raw: values) is decided by the sign of a fused multiply-add, which is
// exact; for one that was normed and rotated the warp computes its vectors again
// in 64 bits (a few in a thousand).  A vector lies in L lanes of EPL elements.
//
// How far off the fp32 values can be, in units u = 2^-24 of the vector's
// maximum M: the sum of squares has all-positive terms, each through one product
// and at most 8 + 4 additions (8 per lane, 4 across), so it is off by at most 13u
// relative and the root's reciprocal by 6.5u + 3u; x * inv * g adds 2u, the two
// products and the sum of the rotation 3u of at most sqrt(2) M: |error| <= 20u M.  In units
// of s = M/7 (1 +- 2^-8) that is 140u (1.004) + the quotient's own 2u * 7 < 160u
// = 9.6e-6; the margin is 2e-5.  M / 7 is off by at most 22u relative, i.e. 44
// units of the last place of fp32 at the least; the margin is 64 of them.
constexpr float kCodeMargin = 2e-5f;
constexpr uint32_t kScaleMargin = 64;

// Sum and maximum over the L lanes (a power of two) that hold a vector.
template <int L, typename T>
DEVI T lanes_sum(T v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <int L>
DEVI float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <int L>
DEVI double lanes_max(double v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Nearest bf16 of a 64-bit value: rounded to odd in fp32 (two bits and more
// below bf16's last place), then to nearest.
DEVI uint16_t f64_to_bf16bits(double x) {
  float f = __double2float_rz(x);
  if (static_cast<double>(f) != x) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f32_to_bf16bits(f);
}

// The vector again in 64 bits: x the inputs, g the gains, cs/sn the rotation
// (raw: neither).
template <int EPL, int L>
DEVI uint16_t quantize_vector_f64(const float (&x)[EPL], const float (&g)[EPL], const float (&cs)[EPL / 2],
                                  const float (&sn)[EPL / 2], bool raw, bool norm, float eps, uint32_t (&u)[EPL]) {
  double y[EPL];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) y[j] = x[j];
  // (a warp's vectors may be of different kinds: its lanes add up together,
  // whether their vector is normed or not)
  double ss = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) ss += y[j] * y[j];
  ss = lanes_sum<L>(ss);
  if (!raw) {
    if (norm) {
      const double inv = 1.0 / sqrt(ss / (EPL * L) + static_cast<double>(eps));
#pragma unroll
      for (int j = 0; j < EPL; ++j) y[j] = y[j] * inv * static_cast<double>(g[j]);
    }
#pragma unroll
    for (int j = 0; j < EPL / 2; ++j) {
      const double p = y[2 * j], q = y[2 * j + 1], c = cs[j], s = sn[j];
      y[2 * j] = p * c - q * s;
      y[2 * j + 1] = p * s + q * c;
    }
  }
  double m = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    bad |= !(fabs(y[j]) <= 1.7976931348623157e308);
    m = fmax(m, fabs(y[j]));
  }
  m = lanes_max<L>(m);
  bad = lanes_max<L>(bad ? 1.f : 0.f) != 0.f;
  const uint16_t sb = bad ? 0x7FC0 : f64_to_bf16bits(m / 7.0);
  const double s = static_cast<double>(bf16bits_to_f32(sb));
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    double c = s > 0.0 ? rint(y[j] / s) : 0.0;
    c = fmin(fmax(c, -8.0), 7.0);
    u[j] = static_cast<uint32_t>(static_cast<int>(c) + 8);
  }
  return sb;
}

// Codes (as q + 8) and scale bits of a warp's vector.  v: the vector in fp32
// (equal to x when raw); ss: the fp32 sum of squares (1 where there is none).
template <int EPL, int L>
DEVI uint16_t quantize_vector(const float (&x)[EPL], const float (&v)[EPL], const float (&g)[EPL],
                              const float (&cs)[EPL / 2], const float (&sn)[EPL / 2], bool raw, bool norm, float ss,
                              float eps, uint32_t (&u)[EPL]) {
  float m = 0.f;
  bool near = !(ss < 1e30f) || ss < 1e-30f;   // squares that overflow or vanish in fp32
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    near |= !(fabsf(v[j]) <= 1e30f);          // also NaN
    m = fmaxf(m, fabsf(v[j]));
  }
  m = lanes_max<L>(m);
  const float t = m / 7.0f;
  const uint32_t bits = __float_as_uint(t);
  const bool scale_near = (bits & 0xFFFFu) + kScaleMargin - 0x8000u <= 2 * kScaleMargin;
  near |= t < 1e-30f && m > 0.f;
  uint16_t sb = f32_to_bf16bits(t);
  if (scale_near) {
    // raw: m is exact, and so is the sign of m - 7 * (the midpoint)
    const float d = fmaf(-7.f, __uint_as_float((bits & 0xFFFF0000u) | 0x8000u), m);
    const uint32_t low = bits >> 16;
    if (raw) sb = static_cast<uint16_t>(d > 0.f ? low + 1 : d < 0.f ? low : low + (low & 1u));
    else near = true;
  }
  const float s = bf16bits_to_f32(sb), inv = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float y = v[j] * inv;
    float c = rintf(y);
    if (fabsf(fabsf(y - c) - 0.5f) < kCodeMargin) {
      // raw: the sign of v - s (f + 1/2) is exact
      const float f = floorf(y), d = fmaf(-s, f + 0.5f, v[j]);
      if (raw) c = d > 0.f ? f + 1.f : d < 0.f ? f : 2.f * rintf(0.5f * (f + 0.5f));
      else near = true;
    }
    u[j] = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(c, -8.f), 7.f)) + 8);
  }
  if (!__any_sync(0xffffffffu, near)) return sb;
  return quantize_vector_f64<EPL, L>(x, g, cs, sn, raw, norm, eps, u);
}

}  // namespace dualar
