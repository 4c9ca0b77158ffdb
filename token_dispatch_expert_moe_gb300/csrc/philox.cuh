// The counter-based generator of the dropout: Philox4x32-10, from its paper
// (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3,
// 2011). One block of four 32-bit words serves eight consecutive elements, 16
// bits each; nothing is stored, every pass that needs the mask makes it again.
// 16 bits an element and not 32: 20 wide multiplications a block are half as
// many per element, which keeps the passes bound by memory.
#pragma once
#include "common.cuh"

namespace moe {

// round(65536 p): an element is kept if its 16 bits are >= this
inline uint32_t drop_threshold(float p) {
  const uint32_t t = (uint32_t)((double)p * 65536.0 + 0.5);
  return t < 65535u ? t : 65535u;
}
inline float drop_scale(uint32_t threshold) { return 65536.0f / (float)(65536u - threshold); }

struct Philox {
  uint32_t key[20];     // of the ten rounds: made once a thread (a block of its own additions would cost a fifth)
  uint32_t c2, c3;
  uint32_t threshold;   // << 16

  // rng: {seed, offset} on the device; NULL beside the threshold 0, which keeps everything
  __device__ __forceinline__ Philox(const uint64_t *rng, uint32_t t) : threshold(t << 16) {
    const uint64_t seed = rng != nullptr ? rng[0] : 0, offset = rng != nullptr ? rng[1] : 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      key[2 * i] = (uint32_t)seed + i * 0x9E3779B9u;
      key[2 * i + 1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
    }
    c2 = (uint32_t)offset;
    c3 = (uint32_t)(offset >> 32);
  }

  __device__ __forceinline__ uint4 block(uint64_t b) const {
    uint32_t x0 = (uint32_t)b, x1 = (uint32_t)(b >> 32), x2 = c2, x3 = c3;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t m0 = (uint64_t)x0 * 0xD2511F53u, m1 = (uint64_t)x2 * 0xCD9E8D57u;
      x0 = (uint32_t)(m1 >> 32) ^ x1 ^ key[2 * i];
      x1 = (uint32_t)m1;
      x2 = (uint32_t)(m0 >> 32) ^ x3 ^ key[2 * i + 1];
      x3 = (uint32_t)m0;
    }
    return make_uint4(x0, x1, x2, x3);
  }

  // whether element j of the block is kept: 16 bits against the threshold, as
  // the upper halves of words
  template <int J> __device__ __forceinline__ bool kept(const uint4 &w) const {
    constexpr int i = J >> 1;
    const uint32_t v = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return ((J & 1) ? v : v << 16) >= threshold;
  }
};

}  // namespace moe
