// Eight consecutive elements of a row, and sums over the lanes that share a
// row: what the per-head norms and the vector-state scan read, write and
// reduce with.  Not a public header.
#pragma once
#include "common.h"
#include "kernels.h"

namespace pdn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight elements as they lie in memory: 16 bytes of bf16, 32 of fp32.
//
// `stream` loads what a call reads once without keeping it in the caches, which
// then hold more of what the call writes, for the next call to read or to write
// over: q/k norm of B4 T8192 H16 d128 113 -> 82 us and gated output norm of the
// same 106 -> 100 us with the outputs in place, 112 -> 109 and 106 -> 105 us into
// other memory each call.
template <bool BF16>
struct Raw8;

template <>
struct Raw8<true> {
    u32x4 v;
    __device__ __forceinline__ void load(const void* p, long i) {
        v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void stream(const void* p, long i) {
        v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i));
    }
    __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(v[j] << 16);
            f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
        }
    }
    // the same eight elements of another lane's row part
    __device__ __forceinline__ Raw8 from_lane(int lane) const {
        Raw8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.v[j] = __shfl(v[j], lane, 64);
        return r;
    }
};

template <>
struct Raw8<false> {
    f32x4 lo, hi;
    __device__ __forceinline__ void load(const void* p, long i) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        lo = q[0];
        hi = q[1];
    }
    __device__ __forceinline__ void stream(const void* p, long i) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        lo = __builtin_nontemporal_load(q);
        hi = __builtin_nontemporal_load(q + 1);
    }
    __device__ __forceinline__ void zero() { lo = hi = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = lo[j];
            f[4 + j] = hi[j];
        }
    }
    __device__ __forceinline__ Raw8 from_lane(int lane) const {
        Raw8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.lo[j] = __shfl(lo[j], lane, 64);
            r.hi[j] = __shfl(hi[j], lane, 64);
        }
        return r;
    }
};

// Store eight fp32 values as fp32, or rounded to the nearest bf16 (ties to
// even): the one rounding of an output.
template <bool BF16>
__device__ __forceinline__ void store8(void* p, long i, const float (&f)[8]) {
    if constexpr (BF16) {
        f32x8 w;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = f[j];
        *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(p) + i) = __builtin_convertvector(w, bf16x8);
    } else {
        f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        q[0] = f32x4{f[0], f[1], f[2], f[3]};
        q[1] = f32x4{f[4], f[5], f[6], f[7]};
    }
}

// Workgroup i of n in an order in which each XCD's workgroups (every kXcds-th)
// follow one another, so that an XCD works on one stretch of a tensor, not on
// pieces of all of it.  It decides locality only, and pays where many distant
// rows are written: q/k norm of B1 T65536 H16 d128 195 -> 167 us, scan training
// step of B2 T8192 D4096 239 -> 232 us.  Where the distant rows are read it costs
// (q/k norm's backward 211 -> 258 us, output norm 100 -> 113 us).
__device__ __forceinline__ unsigned by_xcd(unsigned i, unsigned n) {
    const unsigned x = i % kXcds, whole = n / kXcds, rest = n % kXcds;
    return x * whole + (x < rest ? x : rest) + i / kXcds;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    const int i = __float_as_int(x);
    return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, true));
}

// Sum over the LPR neighbouring lanes (a power of two up to 32) that hold one
// row, the same bits in each of them.  Within a DPP row of 16 lanes by lane
// swaps inside the vector unit: quads (lane ^ 1, lane ^ 2), then mirrors,
// whose two halves already agree.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
    if constexpr (LPR >= 2) x += dpp<0xB1>(x);   // quad_perm 1,0,3,2
    if constexpr (LPR >= 4) x += dpp<0x4E>(x);   // quad_perm 2,3,0,1
    if constexpr (LPR >= 8) x += dpp<0x141>(x);  // row_half_mirror
    if constexpr (LPR >= 16) x += dpp<0x140>(x); // row_mirror
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16, 64);
    return x;
}

}  // namespace pdn
