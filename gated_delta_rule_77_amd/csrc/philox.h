// Random bits of an element from its place alone: Philox4x32-10 (Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), whose ten
// rounds turn a counter of four words and a key of two into four words.  Device
// and host code.  Not a public header.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pdn {

struct Philox {
    uint32_t w[4];
};

// The block of eight elements n / 8 = `block` of the call `stream` under `key`.
__host__ __device__ __forceinline__ Philox philox(uint64_t key, uint64_t stream, uint64_t block) {
    uint32_t a = static_cast<uint32_t>(block), b = static_cast<uint32_t>(block >> 32);
    uint32_t c = static_cast<uint32_t>(stream), d = static_cast<uint32_t>(stream >> 32);
    uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = static_cast<uint64_t>(a) * 0xD2511F53u, q = static_cast<uint64_t>(c) * 0xCD9E8D57u;
        a = static_cast<uint32_t>(q >> 32) ^ b ^ k0;
        c = static_cast<uint32_t>(p >> 32) ^ d ^ k1;
        b = static_cast<uint32_t>(q);
        d = static_cast<uint32_t>(p);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Philox{{a, b, c, d}};
}

// Whether element j (0 .. 7) of a block is kept: its 16 bits reach the threshold.
__host__ __device__ __forceinline__ bool philox_keeps(const Philox& p, int j, uint32_t threshold) {
    return ((p.w[j >> 1] >> (16 * (j & 1))) & 0xffffu) >= threshold;
}

}  // namespace pdn
