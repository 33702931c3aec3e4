// Dropout whose kept elements follow from a counter: nothing is stored, the backward pass forms the same choice again.
//
// Element e of a tensor (row-major) has 16 random bits: half-word e mod 8 (a word's low half first) of the four words of
// Philox-4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) at
// counter (e / 8, layer, step low, step high) under key (seed low, seed high).  It is kept where they are at least
// t = round(65536 p), and kept elements are multiplied by 65536 / (65536 - t), the inverse of the chance that sixteen
// bits give them.  Thirty-two bits an element would double the generator's work, which then costs more than the memory
// of a 16-bit tensor.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssc_internal.h"

namespace ssc {
namespace {

struct Drop {
  const int64_t* rng;  // device memory: seed, step
  uint32_t layer, t;
  float scale;
};

// p of a host call: t of p in [0, 1), or -1.  Values that round to one are held below it: something is always kept.
inline int drop_threshold(double p) {
  if (!(p >= 0.0 && p < 1.0)) return -1;
  const int t = int(p * 65536.0 + 0.5);
  return t > 65535 ? 65535 : t;
}
inline float drop_scale(int t) { return float(65536.0 / double(65536 - t)); }

struct DropKey {
  uint32_t k0, k1, s0, s1;
  __device__ __forceinline__ void load(const int64_t* rng) {
    const uint64_t seed = uint64_t(rng[0]), step = uint64_t(rng[1]);
    k0 = uint32_t(seed);
    k1 = uint32_t(seed >> 32);
    s0 = uint32_t(step);
    s1 = uint32_t(step >> 32);
  }
};

// the four words of elements 8 block .. 8 block + 7
__device__ __forceinline__ void philox(uint32_t block, uint32_t layer, const DropKey& key, uint32_t (&w)[4]) {
  uint32_t c0 = block, c1 = layer, c2 = key.s0, c3 = key.s1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0;
  w[1] = c1;
  w[2] = c2;
  w[3] = c3;
}

// f = kept ? f * scale : 0 for N elements from e0 (a multiple of N); what a dropped element held does not matter
template <int N>
__device__ __forceinline__ void drop(float (&f)[N], int64_t e0, const Drop& d, const DropKey& key) {
  uint32_t w[4];
  philox(uint32_t(uint64_t(e0) >> 3), d.layer, key, w);
  // four elements take two of the words: chosen bit by bit, as a choice of addresses would put the words into memory
  if constexpr (N == 4) {
    const uint32_t upper = e0 & 4 ? ~0u : 0u;
    w[0] ^= (w[0] ^ w[2]) & upper;
    w[1] ^= (w[1] ^ w[3]) & upper;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t word = w[j / 2];
    const uint32_t bits = (j & 1) ? word >> 16 : word & 0xFFFFu;
    f[j] = bits >= d.t ? f[j] * d.scale : 0.f;
  }
}

constexpr int64_t kMaxDropElements = int64_t(1) << 35;  // a block's number is one word of the counter

}  // namespace
}  // namespace ssc
