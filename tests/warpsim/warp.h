/* A warp on the host: 32 threads whose shuffles and votes wait for one another,
 * as the full mask of the device's functions asks.  A lane that ends, or calls
 * another function or distance, while others wait in one breaks that rule; it is
 * recorded (where the device's result would be undefined) and nothing waits on. */
#pragma once
#include <cmath>
#include <condition_variable>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#define DEVI static inline

struct WarpSim {
  std::mutex m;
  std::condition_variable cv;
  uint64_t word[2][32];
  int tag[2][32];
  int here = 0, ended = 0, phase = 0;
  bool broken = false;

  // All lanes' words behind the call; this lane's `t` names what it calls.
  const uint64_t* meet(int lane, int t, uint64_t w) {
    std::unique_lock<std::mutex> l(m);
    const int p = phase & 1, mine = phase;
    word[p][lane] = w;
    tag[p][lane] = t;
    if (ended > 0) broken = true;
    if (++here + ended == 32) {
      for (int i = 0; i < 32 && !broken; ++i)
        if (tag[p][i] != t) broken = true;
      here = 0;
      ++phase;
      cv.notify_all();
    } else {
      cv.wait(l, [&] { return phase != mine || broken; });
    }
    return word[p];
  }
  void end() {
    std::unique_lock<std::mutex> l(m);
    ++ended;
    if (here > 0) {
      broken = true;
      cv.notify_all();
    }
  }
};

static WarpSim* g_warp;
static thread_local int t_lane;

template <typename T>
static inline T __shfl_xor_sync(unsigned, T v, int o) {
  uint64_t w = 0;
  std::memcpy(&w, &v, sizeof(T));
  const uint64_t* all = g_warp->meet(t_lane, o * 16 + static_cast<int>(sizeof(T)), w);
  T r;
  std::memcpy(&r, &all[t_lane ^ o], sizeof(T));
  return r;
}
static inline bool __any_sync(unsigned, bool v) {
  const uint64_t* all = g_warp->meet(t_lane, -1, v);
  bool any = false;
  for (int i = 0; i < 32; ++i) any |= all[i] != 0;
  return any;
}
static inline uint32_t __float_as_uint(float f) {
  uint32_t u;
  std::memcpy(&u, &f, 4);
  return u;
}
static inline float __uint_as_float(uint32_t u) {
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
static inline float __double2float_rz(double x) {
  const float f = static_cast<float>(x);
  return std::fabs(static_cast<double>(f)) > std::fabs(x) ? std::nextafterf(f, 0.f) : f;
}
static inline float bf16bits_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
static inline uint16_t f32_to_bf16bits(float f) {
  if (f != f) return 0x7FFF;
  const uint32_t u = __float_as_uint(f);
  return static_cast<uint16_t>((u + 0x7FFF + ((u >> 16) & 1)) >> 16);
}

// Runs f(lane) in every lane; true where all of them kept together.
template <typename F>
static bool run_warp(F f) {
  WarpSim w;
  g_warp = &w;
  std::vector<std::thread> lanes;
  for (int i = 0; i < 32; ++i)
    lanes.emplace_back([&, i] {
      t_lane = i;
      f(i);
      w.end();
    });
  for (auto& t : lanes) t.join();
  return !w.broken;
}
