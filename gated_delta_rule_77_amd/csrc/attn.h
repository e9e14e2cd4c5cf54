// What the attention kernels share: 32x32 matrix tiles of bf16 or fp32 operands (these
// as sums of bf16 parts), tiles of rows in LDS, and which keys a query sees.  Not a
// public header.
//
// A matrix instruction's operands hold 8 consecutive k-slots to a lane: lane l holds row (or
// column) l % 32 and slots 8 (l / 32) .. + 7.  Which k a slot stands for is free as long as both
// operands agree.  A result's 16 registers
// of lane l are column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4; registers 8 s ..
// 8 s + 7 of a result are therefore an operand of the next product, whose slots
// stand for rows 16 s + 4 (l / 32) + {0 .. 3, 8 .. 11}.  So scores are formed
// transposed (keys down, queries across): a query's sums run over a lane's own
// registers and one other lane, and the probabilities never leave registers.
#pragma once
#include "common.h"
#include "rows.h"

#include <type_traits>

namespace pdn {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) char lds_char;

template <bool BF16>
struct El;

template <>
struct El<true> {
    static constexpr int BYTES = 2;
    typedef bf16x8 Frag;
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ Frag load(const void* p, long i) {
        return *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(p) + i);
    }
    static __device__ __forceinline__ Frag zero() { return __builtin_bit_cast(Frag, u32x4{0u, 0u, 0u, 0u}); }
    // registers 8 s .. 8 s + 7 of a result, to the nearest bf16
    static __device__ __forceinline__ Frag of(const f32x16& r, int s) {
        f32x8 w;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r[8 * s + j];
        return __builtin_convertvector(w, bf16x8);
    }
    static __device__ __forceinline__ bool is_finite(const Frag& f) {
        const u32x4 w = __builtin_bit_cast(u32x4, f);
        bool all = true;
#pragma unroll
        for (int j = 0; j < 4; ++j) all &= (w[j] & 0x7f80u) != 0x7f80u && (w[j] & 0x7f800000u) != 0x7f800000u;
        return all;
    }
    // infinities and NaN to zero
    static __device__ __forceinline__ Frag finite(const Frag& f) {
        u32x4 w = __builtin_bit_cast(u32x4, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if ((w[j] & 0x7f80u) == 0x7f80u) w[j] &= 0xffff0000u;
            if ((w[j] & 0x7f800000u) == 0x7f800000u) w[j] &= 0xffffu;
        }
        return __builtin_bit_cast(Frag, w);
    }
};

template <>
struct El<false> {
    static constexpr int BYTES = 4;
    typedef f32x8 Frag;
    // x = x0 + x1 + x2 in bf16, each the nearest to what is left: 24 bits of a normal x.
    // (|x| from 3.396e38 on rounds to infinity; below 2^-110 the last parts lose bits as
    // bf16 has no more exponents: 2^-133 at the most.)
    static __device__ __forceinline__ void parts(const Frag& f, bf16x8 (&p)[3]) {
        Frag left = f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            p[i] = __builtin_convertvector(left, bf16x8);
            if (i == 2) break;
            const u32x4 w = __builtin_bit_cast(u32x4, p[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                left[2 * j] -= __uint_as_float(w[j] << 16);
                left[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
    // An fp32 product as six of bf16 parts, the smallest first.  |x1| <= 2^-8 |x| and |x2| <=
    // 2^-17 |x| (half steps of 8 bits), so that what is left out, x1 y2 + x2 y1 + x2 y2, is
    // 2^-24 of |x y| at the most: one fp32 rounding.  The fp32 instruction takes 64 cycles
    // for 4096 operations, these 32 for 32768: six take 3/8 of its time, and forming the
    // parts (5.5 operations an element) most of what that leaves (B3 H8/2 T1237 after 100
    // d64: forward 85 -> 58 us, dq 107 -> 94, dk and dv 153 -> 116; error against 64 bits
    // 2.4e-7 -> 2.0e-7).
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c) {
        bf16x8 x[3], y[3];
        parts(a, x);
        parts(b, y);
        c = El<true>::mma(x[2], y[0], c);
        c = El<true>::mma(x[0], y[2], c);
        c = El<true>::mma(x[1], y[1], c);
        c = El<true>::mma(x[1], y[0], c);
        c = El<true>::mma(x[0], y[1], c);
        return El<true>::mma(x[0], y[0], c);
    }
    static __device__ __forceinline__ Frag load(const void* p, long i) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 lo = q[0], hi = q[1];
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ Frag zero() { return Frag{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}; }
    static __device__ __forceinline__ Frag of(const f32x16& r, int s) {
        Frag w;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r[8 * s + j];
        return w;
    }
    static __device__ __forceinline__ bool has_parts(float x) { return (__float_as_uint(x) & 0x7fffffffu) < 0x7f7f8000u; }
    static __device__ __forceinline__ bool is_finite(const Frag& f) {
        bool all = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) all &= has_parts(f[j]);
        return all;
    }
    // what has no finite parts to zero
    static __device__ __forceinline__ Frag finite(Frag f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = has_parts(f[j]) ? f[j] : 0.0f;
        return f;
    }
};

// A tile of rows in LDS, D channels each, as 16-byte chunks: chunk c of row r lies
// at c ^ swizzle(r), so that neither the reads of one chunk of 16 rows nor those of
// four neighbouring chunks of four rows meet in a bank.
template <bool BF16, int D>
struct Tile {
    static constexpr int ROW = D * El<BF16>::BYTES, CHUNKS = ROW / 16;
    static constexpr int ROWS_PER_DMA = 64 / CHUNKS;  // a wave's load of 16 bytes a lane
    typedef typename El<BF16>::Frag Frag;

    static __device__ __forceinline__ int swizzle(int r) {
        if constexpr (CHUNKS >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
        return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);  // two rows share the banks' width
    }
    // A wave's load of 16 bytes a lane fills rows n ROWS_PER_DMA .. of a tile: what lane l
    // takes, row l / CHUNKS of them, chunk lane_chunk(l) ^ swizzle(n ROWS_PER_DMA) (the
    // swizzle moves bits, so that of a sum of rows without carries is its parts').
    static __device__ __forceinline__ uint32_t lane_chunk(int lane) { return (lane % CHUNKS) ^ swizzle(lane / CHUNKS); }
    // its offset from the row n ROWS_PER_DMA, for rows `stride` bytes apart: part = lane / CHUNKS * stride
    static __device__ __forceinline__ uint32_t lane_offset(uint32_t part, uint32_t chunk, int n) {
        return part + ((chunk ^ swizzle(n * ROWS_PER_DMA)) << 4);
    }
    // where chunk c of row r lies
    static __device__ __forceinline__ int at(int r, int chunk) { return r * ROW + ((chunk ^ swizzle(r)) << 4); }

    // Operands are read from LDS addresses tile + base(lane): tiles begin at multiples
    // of 1024 bytes and operands at rows that are multiples of 16, so that the step to
    // another chunk is an exclusive or of the address and to other rows a constant.

    // rows l % 32, slots for channels 16 s + 8 (l / 32) .. + 7
    static __device__ __forceinline__ uint32_t row_base(int lane) {
        return at(lane & 31, (BF16 ? 1 : 2) * (lane >> 5));
    }
    static __device__ __forceinline__ Frag rows(uint32_t p, int r0, int s) {
        if constexpr (BF16) {
            return __builtin_bit_cast(Frag, read<u32x4>((p ^ (s << 5)) + r0 * ROW));
        } else {
            const f32x4 lo = read<f32x4>((p ^ (s << 6)) + r0 * ROW), hi = read<f32x4>((p ^ (s << 6) ^ 16) + r0 * ROW);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // channels 32 c + l % 32, slots for rows 4 (l / 32) + {0 .. 3, 8 .. 11}.  bf16 by
    // transpose reads: of each 16 lanes lane 4 i + j points at row i, channels 4 j .. + 3
    // of 16, and is given channel 4 i + j of the four rows.
    static __device__ __forceinline__ uint32_t column_base(int lane) {
        const int r = 4 * (lane >> 5);
        if constexpr (BF16) return at(r + ((lane >> 2) & 3), ((lane >> 3) & 2) + ((lane >> 1) & 1)) + ((lane & 1) << 3);
        return at(r, (lane & 31) >> 2) + ((lane & 3) << 2);
    }
    static __device__ __forceinline__ Frag columns(uint32_t p, int r0, int c) {
        if constexpr (BF16) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)static_cast<uintptr_t>((p ^ (c << 6)) + r0 * ROW));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)static_cast<uintptr_t>((p ^ (c << 6) ^ 32) + (r0 + 8) * ROW));
            return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            Frag f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = read<float>((p ^ (c << 7) ^ ((j & 3) << 6) ^ ((j >> 2) << 5)) + (r0 + (j & 3) + 8 * (j >> 2)) * ROW);
            return f;
        }
    }

private:
    template <class T>
    static __device__ __forceinline__ T read(uint32_t p) {
        return *(const __attribute__((address_space(3))) T*)static_cast<uintptr_t>(p);
    }
};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char*)(const char*)p));
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// From memory to LDS past the registers: 16 (or 4) bytes a lane, lane l's to LDS address
// dst + 16 l (4 l).  Written out, because the compiler puts a wait for every such load of
// its own before the next read of LDS, also of another buffer.  They have no result
// register.  landed() waits for all of this wave's loads; the compiler takes note of its wait
// (and drops its own for what it loaded before).
// Two things the compiler does not see to in such a block: that m0, which cannot be named as
// overwritten, has no other use, and that five instructions lie between a vector instruction
// that writes a scalar register (as uniform() is) and a load that takes its address from
// there.  tests/test_attn_listing.py holds every build to both: to bring m0 back and the five
// in each block cost 256 single tokens over up to 8192 501 -> 516 us, a windowed step 1%.
__device__ __forceinline__ void to_lds(const void* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uniform(dst)), "v"(src) : "memory");
}
__device__ __forceinline__ const char* uniform(const char* p) {
    const uint64_t x = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = uniform(static_cast<int>(x)), hi = uniform(static_cast<int>(x >> 32));
    return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
}
// the same from a uniform address and 32-bit offsets of the lanes
__device__ __forceinline__ void to_lds(const char* base, uint32_t offset, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform(dst)), "v"(offset), "s"(uniform(base)) : "memory");
}
__device__ __forceinline__ void to_lds4(const void* base, uint32_t offset, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(uniform(dst)), "v"(offset),
                 "s"(uniform(static_cast<const char*>(base)))
                 : "memory");
}
// The same but for the last N loads.  The compiler does not see this wait: its own loads
// have to have landed before.
template <int N>
__device__ __forceinline__ void landed_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void landed() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0), the other counters free
}

// The keys that a query sees: low .. low + count - 1.
struct Seen {
    int low, count;
};

// Query i of nq on nk keys, the queries being the last of them.
__device__ __forceinline__ Seen seen_by(int i, int nq, int nk, int window, int first) {
    const int p = i + nk - nq;
    int low = first > 0 ? min(first, nk) : 0;
    if (window > 0 && p - window + 1 > low) low = p - window + 1;
    const int count = p - low + 1;  // p < nk
    return Seen{low, count > 0 ? count : 0};
}

__device__ __forceinline__ bool sees(const Seen& s, int key) {
    return static_cast<unsigned>(key - s.low) < static_cast<unsigned>(s.count);
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// What a row's exponentials go by, ref being one of its largest scores: those of scores s are
// 2^fma(s, c, -m).  Any m near ref c does, as all of the row's have the same: its rounding is
// off by 32 at most while |ref c| is below 2^30, and the fused product exact but for its one
// rounding.  Beyond, that would soon pass an exponential's range; but two different scores are
// 64 apart there, and all but the largest count for nothing.  A power of two that brings ref to
// 2^30 .. 2^31 keeps them so, and takes ref itself to exactly 0.
constexpr float kFar = 0x1p30f;
struct Shift {
    float c, m;
    bool far;
};
__device__ __forceinline__ Shift shift_of(float ref, float c) {
    const float m = ref * c;
    if (!(fabsf(m) >= kFar && fabsf(ref) < INFINITY)) return Shift{c, m, false};
    const float by = __builtin_amdgcn_ldexpf(1.0f, min(31 - __builtin_amdgcn_frexp_expf(ref), 127));
    return Shift{by, ref * by, true};
}
// What turns sums that went by `from` into such that go by `to`, not below it (-inf: no score yet).
__device__ __forceinline__ float weight(float from, float to, float c) {
    const Shift a = shift_of(from, c), b = shift_of(to, c);
    return from == to || from == -INFINITY ? 1.0f : a.far || b.far ? 0.0f : ex2(a.m - b.m);
}
// The logarithm of the sum of exponentials, `sum` of them going by ref.
__device__ __forceinline__ float log_of(float ref, float sum, float c) {
    const Shift s = shift_of(ref, c);
    return s.far ? fmaf(ref, c * kLn2, lg2(sum) * kLn2) : (s.m + lg2(sum)) * kLn2;
}

// x, of which the compiler knows nothing: keeps what follows from it within a loop,
// where taking it out would cost registers.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// x of the two half waves joined, the same in both: lanes l and l ^ 32 swap theirs.
template <bool MAX>
__device__ __forceinline__ float halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    const float a = __uint_as_float(p[0]), b = __uint_as_float(p[1]);
    return MAX ? fmaxf(a, b) : a + b;
}

__device__ __forceinline__ int wave_min_i(int x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = min(x, __shfl_xor(x, off, 64));
    return x;
}
__device__ __forceinline__ int wave_max_i(int x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = max(x, __shfl_xor(x, off, 64));
    return x;
}

// n / d for n below 2^16 and d up to 2^10, by a product with inverse_of(d).
inline uint32_t inverse_of(uint32_t d) { return d == 1 ? 0u : static_cast<uint32_t>((uint64_t{1} << 32) / d + 1); }
__device__ __forceinline__ int quotient(int n, uint32_t inverse) {
    return inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), inverse)) : n;
}

}  // namespace attn
}  // namespace pdn
