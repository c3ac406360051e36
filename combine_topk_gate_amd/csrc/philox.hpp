// Counter-based random words for the dropout: Philox 4x32 with ten rounds
// (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011).  Element n of a tensor takes word n % 4 of the block
// with counter {n / 4, offset} and key seed, so any kernel that reads seed
// and offset makes the same mask again, in any order, and it is never stored.
//
// One block is 20 products of 32 x 32 to 64 bits, four elements' worth; a
// combine of 8192 x 4096 outputs needs about 26 us of the whole card's
// integer units, beside about 65 us of its HBM traffic.
#pragma once

#include "common.hpp"

namespace moe {

struct Dropout {
  const uint64_t* rng;  // device: {seed, offset}; read by the kernel, so a replayed graph sees new values
  uint32_t threshold;   // an element is kept where its word is at least this: floor(p 2^32)
  float scale;          // of a kept element: 1 / (1 - p)
};

struct Philox {
  uint32_t seed_lo, seed_hi, off_lo, off_hi;

  __device__ __forceinline__ explicit Philox(const uint64_t* rng) {
    const uint64_t s = rng[0], o = rng[1];
    seed_lo = (uint32_t)s;
    seed_hi = (uint32_t)(s >> 32);
    off_lo = (uint32_t)o;
    off_hi = (uint32_t)(o >> 32);
  }

  __device__ __forceinline__ uint4 block(uint64_t i) const {
    uint32_t x0 = (uint32_t)i, x1 = (uint32_t)(i >> 32), x2 = off_lo, x3 = off_hi, k0 = seed_lo, k1 = seed_hi;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
      x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
      x1 = (uint32_t)b;
      x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
      x3 = (uint32_t)a;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
  }
};

// Which of the elements 4 i .. 4 i + 3 the dropout keeps.
struct Kept {
  bool x, y, z, w;
};

__device__ __forceinline__ Kept kept(const Philox& ph, const Dropout& d, uint64_t i) {
  const uint4 v = ph.block(i);
  return {v.x >= d.threshold, v.y >= d.threshold, v.z >= d.threshold, v.w >= d.threshold};
}

// v scale where kept, else 0 (also where v is not finite).
__device__ __forceinline__ float4 dropped(const Kept& keep, float scale, float4 v) {
  return make_float4(keep.x ? v.x * scale : 0.f, keep.y ? v.y * scale : 0.f, keep.z ? v.z * scale : 0.f,
                     keep.w ? v.w * scale : 0.f);
}

}  // namespace moe
