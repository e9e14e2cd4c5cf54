// How the tiles of a vector-state scan hand the state on: what scan.hip's kernels
// publish, wait for and join along a column of tiles.  Not a public header.  It
// needs the device's atomics and votes only, so that a host program that brings
// its own can run it in any order of workgroups.
//
// A tile publishes its run (A, H) as soon as it has it, then looks back along its
// column for the nearest tile whose state behind it is known, applies the (A, H)
// of the tiles between in their order, and publishes the state behind itself
// (decoupled look-back: "Single-pass Parallel Prefix Scan with Decoupled
// Look-back", Merrill and Garland).  Whichever tile it starts from, that is the
// same chain of operations h_{j+1} = A_j h_j + H_j, so results are the same bits
// whatever the timing.  A column's tiles are dealt by a counter of its own, in the
// order of their tokens: a tile depends only on tiles that started before it and
// publish before they wait, so every wait ends.  (The waits are bounded all the
// same: a call whose workspace another call overwrites gives NaN instead of
// hanging.)
//
// A published pair is one 64-bit word, stored and loaded by relaxed atomics at
// device scope: the word is its own flag (all ones = not there yet, which no
// published word is), so no fence, and no write-back of an L2, is needed.
//
// With few columns each has a carrier besides: its first workgroup, which takes
// the tiles' (A, H) as they come and publishes the states behind them, the same
// chain of operations in one place.  The carrier waits for tiles that start after
// it, which other work on the device can put off, so no tile relies on it: one
// that does not find its state within kPatience loads looks back like any other.
#pragma once

namespace pdn {

typedef unsigned long long u64;

constexpr int kCols = 128;     // channels of a tile
// Predecessors looked at together: 2 and 8 measured 1 to 5% slower (rounds, and
// registers and traffic).
constexpr int kWindow = 4;
// Runs that a carrier takes a round (8, 16 and 32 at one column of 512 tiles:
// 125, 86 and 65 us), and the columns up to which they have carriers.  With few
// columns many of a column's tiles are in flight, and each would look far back;
// with many, the carriers' places are worth more.  Without and with them, bf16,
// T = 65536: forward on tiles of 128 tokens 1 column 88 and 65 us, 4 columns 90
// and 71; as it stands 8 columns 90 and 89 (backward 160 and 142), 16 columns
// 158 and 165 (backward 269 and 279).
constexpr int kCarry = 32;
constexpr int kCarried = 8;
// Loads after which a tile no longer waits for its carrier, some milliseconds: a
// carrier that runs answers within tens of microseconds.
constexpr unsigned kPatience = 1u << 12;
constexpr u64 kEmpty = ~0ull;
constexpr unsigned kPolls = 1u << 21;  // loads before a tile or a carrier gives up: seconds, where thousands are the most that is needed

// Where a launch's tiles meet: the counter that deals each column's, and, for
// every column and tile in processing order, kCols words of each kind.
struct Chain {
    unsigned* counters;
    u64* agg;      // (A, H) of a tile
    u64* inc;      // the state behind it
    int tiles;     // of a column
    int carrier;   // 1: each column's first workgroup carries its state (see carry)
};

__device__ __forceinline__ float apply(float A, float h, float H) { return A == 0.0f ? H : fmaf(A, h, H); }
// the decay of a run `first` followed by one of decay `then`
__device__ __forceinline__ float join(float first, float then) { return then == 0.0f ? 0.0f : first * then; }

__device__ __forceinline__ u64 pair_word(float A, float H) {
    // a NaN from the inputs could have all bits set, and with it the word
    const uint32_t a = A != A ? 0x7fc00000u : __float_as_uint(A);
    return (static_cast<u64>(__float_as_uint(H)) << 32) | a;
}
__device__ __forceinline__ float word_A(u64 w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ __forceinline__ float word_H(u64 w) { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }

template <class T>
__device__ __forceinline__ T peek(const T* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ void publish(T* p, T w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The word at p, once it is there; `polls` counts down over all of a wave's waits.
__device__ __forceinline__ u64 settled(const u64* p, u64 w, unsigned& polls) {
    while (!__all(w != kEmpty) && polls) {
        --polls;
        __builtin_amdgcn_s_sleep(1);
        w = peek(p);
    }
    return w;
}

// The published states behind the kWindow tiles up to `from`.
struct Window {
    u64 w[kWindow];
    __device__ __forceinline__ void load(const u64* first, int from) {
#pragma unroll
        for (int k = 0; k < kWindow; ++k) w[k] = peek(first + static_cast<long>(max(from - k, 0)) * kCols);
    }
};

// The state before tile `at` of this column (at > 0), one channel to a lane of
// one wave; agg and inc point at this lane's word of the column's first tile,
// `inc_words` holds the states behind the tiles up to at - 1.
//
// A load from where other workgroups publish takes 1.5 to 2 us here under the
// tiles' own traffic, so what counts is how many of them follow one another:
// one for the known states, one for the runs behind the nearest of them.  (The
// first is issued before the tile's own run is published: the memory counter is
// in order, so a load behind a store waits for both.)
__device__ __forceinline__ float look_back(const u64* agg, const u64* inc, Window& inc_words, int at) {
    unsigned polls = kPolls;
    int known = -1;
    float h = 0.0f;
    for (int from = at - 1;;) {
#pragma unroll
        for (int k = 0; k < kWindow; ++k)
            if (known < 0 && from - k >= 0 && __all(inc_words.w[k] != kEmpty)) {
                known = from - k;
                h = word_H(inc_words.w[k]);
            }
        if (known >= 0) break;
        if (!--polls) return __uint_as_float(0x7fc00000u);
        if (from >= kWindow) {
            from -= kWindow;
        } else {
            from = at - 1;
            __builtin_amdgcn_s_sleep(1);
        }
        inc_words.load(inc, from);
    }
    for (int j = known + 1; j < at; j += kWindow) {
        u64 r[kWindow];
#pragma unroll
        for (int k = 0; k < kWindow; ++k) r[k] = peek(agg + static_cast<long>(min(j + k, at - 1)) * kCols);
#pragma unroll
        for (int k = 0; k < kWindow; ++k) {
            if (j + k >= at) break;
            r[k] = settled(agg + static_cast<long>(j + k) * kCols, r[k], polls);
            h = apply(word_A(r[k]), h, word_H(r[k]));
        }
    }
    return polls ? h : __uint_as_float(0x7fc00000u);
}

// The carrier's work, a channel to a lane of its first two waves: from the state
// behind the column's first tile, which that tile publishes, the state behind
// each tile but the last, as their runs come in, up to kCarry of them a round.
// Where it gives up, the tiles go on without it.
__device__ inline void carry(const Chain& c, int column, int ch) {
    const long word = static_cast<long>(column) * c.tiles * kCols + ch;
    const int n = c.tiles - 1;
    unsigned polls = kPolls;
    float h = word_H(settled(c.inc + word, peek(c.inc + word), polls));
    for (int next = 1; next < n && polls;) {
        u64 r[kCarry];
#pragma unroll
        for (int k = 0; k < kCarry; ++k) r[k] = peek(c.agg + word + static_cast<long>(min(next + k, n - 1)) * kCols);
        int done = 0;
#pragma unroll
        for (int k = 0; k < kCarry; ++k)
            if (done == k && next + k < n && __all(r[k] != kEmpty)) {
                h = apply(word_A(r[k]), h, word_H(r[k]));
                publish(c.inc + word + static_cast<long>(next + k) * kCols, pair_word(0.0f, h));
                done = k + 1;
            }
        next += done;
        if (!done) {
            --polls;
            __builtin_amdgcn_s_sleep(1);
        }
    }
}

// What waves 0 and 1 do for the tile, a channel to a lane: join the waves'
// runs (totA, totH, in processing order), publish, find the state before the
// tile, publish; the state before the tile's first run, and through `behind` that
// behind its last.
template <int WAVES>
__device__ __forceinline__ float meet(const Chain& c, const float (&totA)[WAVES][kCols],
                                      const float (&totH)[WAVES][kCols], int column, int at, int ch, float start,
                                      float& behind) {
    const long word = static_cast<long>(column) * c.tiles * kCols + ch;
    const long mine = word + static_cast<long>(at) * kCols;
    const bool last = at + 1 == c.tiles;
    Window inc_words;
    if (at > 0 && !c.carrier) inc_words.load(c.inc + word, at - 1);
    float tA = totA[0][ch], tH = totH[0][ch];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        tH = apply(totA[w][ch], tH, totH[w][ch]);
        tA = join(tA, totA[w][ch]);
    }
    float h = start;
    bool carried = false;
    if (at == 0) {
        // the last tile may write over what `start` was read from, and only this
        // order keeps it behind that load
        asm volatile("" : : "v"(start) : "memory");
    } else {
        if (!last) publish(c.agg + mine, pair_word(tA, tH));
        if (c.carrier) {
            unsigned polls = kPatience;
            const u64* from = c.inc + mine - kCols;
            inc_words.w[0] = settled(from, peek(from), polls);
#pragma unroll
            for (int k = 1; k < kWindow; ++k) inc_words.w[k] = kEmpty;
            carried = polls != 0;
        }
        h = look_back(c.agg + word, c.inc + word, inc_words, at);
    }
    behind = apply(tA, h, tH);
    if (!last && !carried) publish(c.inc + mine, pair_word(0.0f, behind));
    return h;
}

}  // namespace pdn
