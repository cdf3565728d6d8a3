// Random bits by counter: Philox 4x32 with 10 rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).
//
// Value i of a tensor, in row-major order, takes half i % 8 (low half of a word
// first) of the four words that counter i / 8 gives: 16 bits a value, so that a
// call serves eight of them (20 products of 32 x 32 bits).  The counter's words
// are the low 32 bits of i / 8, its upper 16 with the call's site above them, and
// the step; the key is the seed.  Nothing is stored: a backward pass asks again.
#pragma once

#include <stdint.h>

namespace psgd {

struct Philox {
  uint32_t key[2], step[2], site;  // site: in the upper 16 bits
  __device__ __forceinline__ Philox() {}
  __device__ __forceinline__ Philox(const int64_t* state, uint32_t where) {
    const uint64_t seed = (uint64_t)state[0], at = (uint64_t)state[1];
    key[0] = (uint32_t)seed, key[1] = (uint32_t)(seed >> 32);
    step[0] = (uint32_t)at, step[1] = (uint32_t)(at >> 32);
    site = where << 16;
  }
  // The bits of values 8 group .. + 7, two to a word.
  __device__ __forceinline__ uint4 operator()(uint64_t group) const {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32) | site, c2 = step[0], c3 = step[1];
    uint32_t k0 = key[0], k1 = key[1];
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
      c0 = (uint32_t)(b >> 32) ^ c1 ^ k0, c1 = (uint32_t)b;
      c2 = (uint32_t)(a >> 32) ^ c3 ^ k1, c3 = (uint32_t)a;
      k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
  }
};

// Dropout of eight values: those whose bits are below `cut` become 0, whatever
// they are, the others are scaled.
__device__ __forceinline__ void drop8(float (&v)[8], const uint4& bits, uint32_t cut, float scale) {
  const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (w[j] & 0xFFFFu) >= cut ? v[2 * j] * scale : 0.f;
    v[2 * j + 1] = (w[j] >> 16) >= cut ? v[2 * j + 1] * scale : 0.f;
  }
}

}  // namespace psgd
