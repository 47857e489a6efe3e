// philox.cuh -- the counter-based generator of the dropout masks: Philox4x32-10 (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
//
// Element i of a tensor takes word i % 4 of the block with counter (i / 4, offset) under
// the key `seed`, whatever kernel, tile or thread asks for it, so a mask is never stored:
// the backward pass draws it again. An element is dropped when its word is below
// floor(p * 2^32).
#pragma once

#include <cstdint>

namespace moe {

struct DropArgs {
    const uint64_t* rng;  // device {seed, offset}; read only when `on`
    uint32_t thr;         // words below are dropped
    float scale;          // 1 / (1 - p)
    int on;               // p > 0
};

struct PhiloxKey {
    uint32_t k0, k1, o0, o1;  // seed, offset
};

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng) {
    const uint64_t s = __ldg(reinterpret_cast<const unsigned long long*>(rng));
    const uint64_t o = __ldg(reinterpret_cast<const unsigned long long*>(rng) + 1);
    return PhiloxKey{(uint32_t)s, (uint32_t)(s >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

// The four words of block `ctr` (element index / 4).
__device__ __forceinline__ uint4 philox4x32_10(const PhiloxKey& key, uint64_t ctr) {
    uint32_t c0 = (uint32_t)ctr, c1 = (uint32_t)(ctr >> 32), c2 = key.o0, c3 = key.o1;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Bit j set: element 4 * ctr + j is kept.
__device__ __forceinline__ uint32_t philox_keep4(const PhiloxKey& key, uint64_t ctr, uint32_t thr) {
    const uint4 w = philox4x32_10(key, ctr);
    return (w.x >= thr ? 1u : 0u) | (w.y >= thr ? 2u : 0u) | (w.z >= thr ? 4u : 0u) | (w.w >= thr ? 8u : 0u);
}

}  // namespace moe
