// drop.hpp - dropout whose mask is computed where it is used and never stored.
//
// Unit u (a value, a channel of a sample or a sample, numbered in memory order) is
// kept where its 16 random bits are not below t = rint(65536 p), and what is kept is
// multiplied by 65536 / (65536 - t), the inverse of the probability that t stands for.
// The bits are half (u % 2) of word (u % 8) / 2 of block u / 8 of the counter-based
// generator Philox 4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy
// as 1, 2, 3, SC 2011), key: the seed, counter: the block and an offset, 64 bits each.
// 16 bits a unit halve the generator's work (20 products of 32 x 32 bits a block, at a
// quarter of the multiply rate): a block serves eight values, so a stream of 16-bit
// values is bound by memory; with 32 bits a value it would not be.
#pragma once

#include "block_ops.hpp"

namespace fno {

struct DropKey {
  uint32_t k0, k1, o0, o1;
};

// the call's key; a step counter in memory moves the offset (a captured graph's replays differ by it)
__device__ __forceinline__ DropKey drop_key(const Drop &d) {
  uint64_t o = d.offset;
  if (d.step) o += *d.step;
  return DropKey{(uint32_t)d.seed, (uint32_t)(d.seed >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

// bit i: unit 8 block + i is kept
__device__ __forceinline__ uint32_t drop_block(const DropKey &key, uint32_t thr, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= ((w[i] & 0xffffu) >= thr ? 1u : 0u) << (2 * i);
    m |= ((w[i] >> 16) >= thr ? 1u : 0u) << (2 * i + 1);
  }
  return m;
}

// bit i < n: unit u + i is kept (n <= 8); a second block only where the units reach into it
__device__ __forceinline__ uint32_t drop_units(const DropKey &key, uint32_t thr, uint64_t u, int n) {
  const int at = (int)(u & 7);
  uint32_t m = drop_block(key, thr, u >> 3) >> at;
  if (at + n > 8) m |= drop_block(key, thr, (u >> 3) + 1) << (8 - at);
  return m;
}

// all bits or none: unit u alone
__device__ __forceinline__ uint32_t drop_one(const DropKey &key, uint32_t thr, uint64_t u) {
  return (drop_block(key, thr, u >> 3) >> (u & 7)) & 1u ? 0xffu : 0u;
}

// v where bit e is set, else 0 (whatever v is, a NaN too), without a branch round what computes v
__device__ __forceinline__ float drop_masked(uint32_t keep, int e, float v) {
  return __uint_as_float(__float_as_uint(v) & (uint32_t)__builtin_amdgcn_sbfe((int)keep, e, 1));
}

}  // namespace fno
