// Where a paged cache holds a sequence's tokens, and which rows of a call are its
// new ones: device and host code, so that numbers that lead nowhere can be tried
// without a device.  Every number that comes from device memory (table, lens,
// starts) is held to the arrays' sizes here.  Not a public header.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pdn {

struct PageMap {
    const int32_t* table;   // [B, width]
    const int32_t* lens;    // [B]
    const int32_t* starts;  // [B + 1], or null
    int B, N, width, pages;
    int shift;              // page_size = 1 << shift
};

// A sequence's new tokens: rows start .. start + n - 1 of N, tokens len - n .. len - 1.
struct Sequence {
    int start, n, len;
};

__host__ __device__ __forceinline__ int held(int x, int low, int high) { return x < low ? low : x > high ? high : x; }

__host__ __device__ __forceinline__ Sequence sequence_of(const PageMap& m, int b) {
    Sequence s;
    if (m.starts) {
        const int from = m.starts[b], to = m.starts[b + 1];
        const bool rows = 0 <= from && from <= to && to <= m.N;  // else it has none
        s.start = rows ? from : 0;
        s.n = rows ? to - from : 0;
    } else {
        s.n = m.N / m.B;
        s.start = b * s.n;
    }
    s.len = static_cast<int>(held(m.lens[b], 0, m.width << m.shift));
    return s;
}

// The page of a sequence's token, 0 <= token < width << shift; an entry outside the
// cache is held to it.
__host__ __device__ __forceinline__ int page_of(const PageMap& m, int b, int token) {
    return held(m.table[static_cast<long>(b) * m.width + (token >> m.shift)], 0, m.pages - 1);
}

}  // namespace pdn
