// The 4-bit rule of the paged cache (rule.h: its text from paged.cuh) for one warp
// whose vectors are queries, keys and values side by side.
#include <algorithm>
#include "warp.h"
using std::fabs;
using std::fmax;
using std::fmin;
using std::rint;
using std::sqrt;
#include "rule.h"

template <int L>
static int run(const float* x, const float* v, const float* g, const float* cs, const float* sn, const int* raw,
               const int* norm, const float* ss, float eps, uint8_t* code, uint16_t* scale) {
  return run_warp([&](int lane) {
    const int vec = lane / L, l = lane % L;
    float X[8], V[8], G[8], C[4], S[4];
    for (int j = 0; j < 8; ++j) {
      X[j] = x[vec * 8 * L + 8 * l + j];
      V[j] = v[vec * 8 * L + 8 * l + j];
      G[j] = g[vec * 8 * L + 8 * l + j];
    }
    for (int j = 0; j < 4; ++j) {
      C[j] = cs[4 * l + j];
      S[j] = sn[4 * l + j];
    }
    uint32_t u[8];
    const uint16_t sb = quantize_vector<8, L>(X, V, G, C, S, raw[vec], norm[vec], ss[vec], eps, u);
    for (int j = 0; j < 8; ++j) code[vec * 8 * L + 8 * l + j] = static_cast<uint8_t>(u[j]);
    if (l == 0) scale[vec] = sb;
  }) ? 1 : 0;
}

extern "C" int quantize_warp(int lanes, const float* x, const float* v, const float* g, const float* cs, const float* sn,
                             const int* raw, const int* norm, const float* ss, float eps, uint8_t* code,
                             uint16_t* scale) {
  return lanes == 16 ? run<16>(x, v, g, cs, sn, raw, norm, ss, eps, code, scale)
                     : run<8>(x, v, g, cs, sn, raw, norm, ss, eps, code, scale);
}
