// The gated linear recurrence with a vector state,
//
//   h_t = a_t h_{t-1} + g(a_t) x_t,  a_t = exp(log_a_t)
//
// over [B,T,D], its backward, and its single-token step.
//
// A run of tokens maps the state before it to the state after it by
// h -> A h + H (per channel), and runs compose:
//   (A2, H2) after (A1, H1) = (A2 A1, A2 H1 + H2).
// Nothing here needs more than a few operations an element, so the bound is
// bytes: every element is read once and written once.  A workgroup takes a tile
// of 64 channels (one 128-byte line of bf16 a token) by R * 32 tokens: a lane
// holds 8 channels of R tokens in registers, reduces them to its (A, H), the
// eight lanes' worth of token groups in a wave are scanned by lane shifts, the
// four waves through LDS.  What is left is the state before the tile:
//
// each tile publishes its (A, H) as soon as it has it, then looks back along
// its column for the nearest tile whose state behind it is known, applies the
// (A, H) of the tiles between in their order, and publishes the state behind
// itself.  Whichever tile it starts from, that is the same chain of operations
// h_{j+1} = A_j h_j + H_j, so results are the same bits whatever the timing.
// Tiles are dealt by a counter, in the order of their tokens: a tile waits only
// for tiles that started before it, so every wait ends.  (The waits are bounded
// all the same: a call whose workspace another call overwrites gives NaN
// instead of hanging.)
//
// A published pair is one 64-bit word, stored and loaded by relaxed atomics at
// device scope: the word is its own flag (all ones = not there yet, which no
// published word is), so no fence, and no write-back of an L2, is needed.
//
// A decay that is zero drops the state before it, infinities and NaN included:
// every "a h + b" below selects b, and every product of decays 0, where the
// later factor is zero.
#include "kernels.h"
#include "rows.h"

namespace pdn {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kCols = 64;    // channels of a tile
constexpr int kFwdR = 8;     // tokens of a lane, forward (256 of a tile)
constexpr int kBwdR = 4;     // backward (128 of a tile: three inputs in registers)
constexpr int kFwdTile = kFwdR * kThreads / 8;
constexpr int kBwdTile = kBwdR * kThreads / 8;
constexpr int kWindow = 8;   // predecessors looked at together
constexpr u64 kEmpty = ~0ull;
constexpr unsigned kPolls = 1u << 21;  // polls before a wait gives up: seconds

static_assert(kBwdTile == PDN_SCAN_MARK, "the backward's tiles start at the marks");
static_assert(kFwdTile % PDN_SCAN_MARK == 0, "marks lie at wave boundaries of the forward's tiles");

struct Rows {
    const void* p;
    long sb, st;
};
struct RowsOut {
    void* p;
    long sb, st;
};

// Where a launch's tiles meet: the counter that deals them and, for every
// column and tile in processing order, 64 words of each kind.
struct Chain {
    unsigned* counter;
    u64* agg;   // (A, H) of a tile
    u64* inc;   // the state behind it
};

struct ScanParams {
    Rows x, la, dh;
    RowsOut h, dx, dla;
    const float* h0;
    float* hT;
    float* marks_out;
    const float* marks;  // backward: the states before its tiles; NULL = one tile, from h0
    const float* dhT;
    float* dh0;
    int T, D;
    int strips;          // 64-channel strips of a row
    int columns;         // B * strips
    int tiles;           // along T
    Chain chain;
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

__device__ __forceinline__ u64 peek(const u64* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(u64* p, u64 w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state before tile `at` of this column (at > 0), one channel to a lane of
// one wave; agg and inc point at this lane's word of the column's first tile.
__device__ float look_back(const u64* agg, const u64* inc, int at) {
    unsigned polls = 0;
    float h = 0.0f;
    int known = -1;
    for (int from = at - 1; known < 0;) {
        u64 w[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i) w[i] = from - i >= 0 ? peek(inc + static_cast<long>(from - i) * kCols) : kEmpty;
#pragma unroll
        for (int i = 0; i < kWindow; ++i)
            if (known < 0 && __all(w[i] != kEmpty)) {
                known = from - i;
                h = word_H(w[i]);
            }
        if (known >= 0) break;
        if (from >= kWindow) {
            from -= kWindow;
        } else {
            from = at - 1;
            if (++polls > kPolls) return __uint_as_float(0x7fc00000u);
            __builtin_amdgcn_s_sleep(1);
        }
    }
    for (int j = known + 1; j < at; j += kWindow) {
        u64 w[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i) w[i] = j + i < at ? peek(agg + static_cast<long>(j + i) * kCols) : 0;
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            if (j + i >= at) break;
            while (!__all(w[i] != kEmpty)) {
                if (++polls > kPolls) return __uint_as_float(0x7fc00000u);
                __builtin_amdgcn_s_sleep(1);
                w[i] = peek(agg + static_cast<long>(j + i) * kCols);
            }
            h = apply(word_A(w[i]), h, word_H(w[i]));
        }
    }
    return h;
}

// The tile of this workgroup, dealt in processing order: all columns' first
// tiles, then their second ones, ..
__device__ __forceinline__ void deal(const ScanParams& p, int* slot, int& column, int& at) {
    if (p.tiles == 1) {
        column = blockIdx.x;
        at = 0;
        return;
    }
    if (threadIdx.x == 0)
        *slot = static_cast<int>(__hip_atomic_fetch_add(p.chain.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    __syncthreads();
    const int n = *slot;
    at = n / p.columns;
    column = n - at * p.columns;
}

__device__ __forceinline__ float decay(float la) { return __builtin_amdgcn_exp2f(la * kLog2e); }

// 1 - e^y for y <= 0 to fp32 accuracy, given e = e^y: the difference where e
// is far from 1 (y < -0.5), else the series of e^y, whose ninth term is below
// 2^-24 of the sum there.
__device__ __forceinline__ float one_minus_exp(float y, float e) {
    float s = 1.0f / 40320.0f;
    s = fmaf(s, y, 1.0f / 5040.0f);
    s = fmaf(s, y, 1.0f / 720.0f);
    s = fmaf(s, y, 1.0f / 120.0f);
    s = fmaf(s, y, 1.0f / 24.0f);
    s = fmaf(s, y, 1.0f / 6.0f);
    s = fmaf(s, y, 0.5f);
    s = fmaf(s, y, 1.0f);
    return y < -0.5f ? 1.0f - e : -y * s;
}

template <int GAIN>
__device__ __forceinline__ float gain(float la, float a) {
    if constexpr (GAIN == PDN_GAIN_COMPLEMENT) return one_minus_exp(la, a);
    if constexpr (GAIN == PDN_GAIN_NORM) return __builtin_amdgcn_sqrtf(one_minus_exp(2.0f * la, a * a));
    return 1.0f;
}
// its derivative by la, given the gain g
template <int GAIN>
__device__ __forceinline__ float gain_slope(float a, float g) {
    if constexpr (GAIN == PDN_GAIN_COMPLEMENT) return -a;
    if constexpr (GAIN == PDN_GAIN_NORM) return -a * a * __builtin_amdgcn_rcpf(g);
    return 0.0f;
}

// Inclusive scan over a wave's eight token groups (lanes 8 apart), forward
// (each lane's run after the lower lanes') or backward (after the higher ones').
template <bool REVERSE>
__device__ __forceinline__ void scan_groups(float (&A)[8], float (&H)[8], int lane) {
#pragma unroll
    for (int off = 8; off < 64; off *= 2) {
        const bool has = REVERSE ? lane + off < 64 : lane >= off;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = REVERSE ? __shfl_down(A[j], off, 64) : __shfl_up(A[j], off, 64);
            const float h = REVERSE ? __shfl_down(H[j], off, 64) : __shfl_up(H[j], off, 64);
            H[j] = has ? apply(A[j], h, H[j]) : H[j];
            A[j] = has ? join(a, A[j]) : A[j];
        }
    }
}

template <bool XBF, bool LBF, int GAIN, bool WRITE_H>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanParams p) {
    constexpr int R = kFwdR;
    __shared__ int slot;
    __shared__ float totA[kWaves][kCols], totH[kWaves][kCols];
    __shared__ float before[kWaves][kCols];  // the state before each wave's tokens
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int column, at;
    deal(p, &slot, column, at);
    const int b = column / p.strips, c0 = (column - b * p.strips) * kCols;
    const int c8 = (lane & 7) * 8, c = c0 + c8;
    const long t0 = static_cast<long>(at) * kFwdTile + (tid >> 3) * R;

    Raw8<XBF> x[R];
    Raw8<LBF> la[R];
    {
        const int cc = c < p.D ? c : 0;
        const long xb = b * p.x.sb + cc, lb = b * p.la.sb + cc;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const long t = t0 + j < p.T ? t0 + j : p.T - 1;
            x[j].load(p.x.p, xb + t * p.x.st);
            la[j].load(p.la.p, lb + t * p.la.st);
        }
        if (static_cast<long>(at + 1) * kFwdTile > p.T) {
            // past the end: a = 1 and nothing added, so the state passes through
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (t0 + j >= p.T) {
                    x[j].zero();
                    la[j].zero();
                }
        }
    }

    float A[8], H[8];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        float xf[8], lf[8];
        x[j].get(xf);
        la[j].get(lf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = decay(lf[i]);
            const float v = xf[i] * gain<GAIN>(lf[i], a);
            H[i] = j ? apply(a, H[i], v) : v;
            A[i] = j ? join(A[i], a) : a;
        }
    }
    scan_groups<false>(A, H, lane);
    if (lane >= 56) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            totA[wave][c8 + i] = A[i];
            totH[wave][c8 + i] = H[i];
        }
    }
    __syncthreads();
    if (wave == 0) {
        const int ch = c0 + lane;  // one channel to a lane here
        const bool in = ch < p.D;
        float tA = totA[0][lane], tH = totH[0][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            tH = apply(totA[w][lane], tH, totH[w][lane]);
            tA = join(tA, totA[w][lane]);
        }
        const long word = (static_cast<long>(column) * p.tiles) * kCols + lane;
        float h;
        if (at == 0) {
            h = p.h0 && in ? p.h0[static_cast<long>(b) * p.D + ch] : 0.0f;
        } else {
            if (at + 1 < p.tiles) publish(p.chain.agg + word + static_cast<long>(at) * kCols, pair_word(tA, tH));
            h = look_back(p.chain.agg + word, p.chain.inc + word, at);
        }
        const float behind = apply(tA, h, tH);
        if (at + 1 < p.tiles) publish(p.chain.inc + word + static_cast<long>(at) * kCols, pair_word(0.0f, behind));
        else if (p.hT && in) p.hT[static_cast<long>(b) * p.D + ch] = behind;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            before[w][lane] = h;
            const int t = w * 8 * R;  // of the tile
            if (p.marks_out && t % PDN_SCAN_MARK == 0) {
                const long tt = static_cast<long>(at) * kFwdTile + t;
                const long marks = (p.T + PDN_SCAN_MARK - 1) / PDN_SCAN_MARK;
                if (tt < p.T && in) p.marks_out[(b * marks + tt / PDN_SCAN_MARK) * p.D + ch] = h;
            }
            h = apply(totA[w][lane], h, totH[w][lane]);
        }
    }
    __syncthreads();
    if constexpr (WRITE_H) {
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = __shfl_up(A[i], 8, 64), v = __shfl_up(H[i], 8, 64);
            h[i] = before[wave][c8 + i];
            if (lane >= 8) h[i] = apply(a, h[i], v);
        }
        const long hb = b * p.h.sb + c;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float xf[8], lf[8];
            x[j].get(xf);
            la[j].get(lf);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = decay(lf[i]);
                h[i] = apply(a, h[i], xf[i] * gain<GAIN>(lf[i], a));
            }
            if (t0 + j < p.T && c < p.D) store8<XBF>(p.h.p, hb + (t0 + j) * p.h.st, h);
        }
    }
}

// Backward: tiles are processed from the last token to the first.  With
// C = a_{t+1} G_{t+1} the gradient that reaches a token from the right (dhT
// behind the last), G = dh + C and the token passes a (dh + C) on: the same
// kind of map, run right to left.  The states h_{t-1} inside a tile come from
// the kept state before it.
template <bool XBF, bool LBF, int GAIN>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(ScanParams p) {
    constexpr int R = kBwdR;
    __shared__ int slot;
    __shared__ float totA[kWaves][kCols], totH[kWaves][kCols];  // the waves' runs, forward
    __shared__ float totB[kWaves][kCols], totG[kWaves][kCols];  // and backward
    __shared__ float before[kWaves][kCols];  // the state before each wave's tokens
    __shared__ float behind[kWaves][kCols];  // what reaches them from the right
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int column, at;
    deal(p, &slot, column, at);
    const int tile = p.tiles - 1 - at;
    const int b = column / p.strips, c0 = (column - b * p.strips) * kCols;
    const int c8 = (lane & 7) * 8, c = c0 + c8;
    const long t0 = static_cast<long>(tile) * kBwdTile + (tid >> 3) * R;

    Raw8<XBF> x[R], dh[R];
    Raw8<LBF> la[R];
    {
        const int cc = c < p.D ? c : 0;
        const long xb = b * p.x.sb + cc, lb = b * p.la.sb + cc, gb = b * p.dh.sb + cc;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const long t = t0 + j < p.T ? t0 + j : p.T - 1;
            x[j].load(p.x.p, xb + t * p.x.st);
            la[j].load(p.la.p, lb + t * p.la.st);
            dh[j].load(p.dh.p, gb + t * p.dh.st);
        }
        if (at == 0) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (t0 + j >= p.T) {
                    x[j].zero();
                    la[j].zero();
                    dh[j].zero();
                }
        }
    }

    float A[8], H[8], AG[8], G[8];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        float xf[8], lf[8];
        x[j].get(xf);
        la[j].get(lf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = decay(lf[i]);
            const float v = xf[i] * gain<GAIN>(lf[i], a);
            H[i] = j ? apply(a, H[i], v) : v;
            A[i] = j ? join(A[i], a) : a;
        }
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
        float gf[8], lf[8];
        dh[j].get(gf);
        la[j].get(lf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = decay(lf[i]);
            const float g = j < R - 1 ? gf[i] + G[i] : gf[i];
            G[i] = join(g, a);
            AG[i] = j < R - 1 ? join(AG[i], a) : a;
        }
    }
    scan_groups<false>(A, H, lane);
    scan_groups<true>(AG, G, lane);
    if (lane >= 56) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            totA[wave][c8 + i] = A[i];
            totH[wave][c8 + i] = H[i];
        }
    }
    if (lane < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            totB[wave][c8 + i] = AG[i];
            totG[wave][c8 + i] = G[i];
        }
    }
    __syncthreads();
    if (wave == 0) {
        const int ch = c0 + lane;
        const bool in = ch < p.D;
        const long state = static_cast<long>(b) * p.D + ch;
        float tA = totB[kWaves - 1][lane], tG = totG[kWaves - 1][lane];
#pragma unroll
        for (int w = kWaves - 2; w >= 0; --w) {
            tG = apply(totB[w][lane], tG, totG[w][lane]);
            tA = join(tA, totB[w][lane]);
        }
        const long word = (static_cast<long>(column) * p.tiles) * kCols + lane;
        float h = 0.0f, g;
        if (in && p.marks) h = p.marks[(static_cast<long>(b) * p.tiles + tile) * p.D + ch];
        else if (in && p.h0) h = p.h0[state];
        if (at == 0) {
            g = p.dhT && in ? p.dhT[state] : 0.0f;
        } else {
            if (at + 1 < p.tiles) publish(p.chain.agg + word + static_cast<long>(at) * kCols, pair_word(tA, tG));
            g = look_back(p.chain.agg + word, p.chain.inc + word, at);
        }
        const float out = apply(tA, g, tG);
        if (at + 1 < p.tiles) publish(p.chain.inc + word + static_cast<long>(at) * kCols, pair_word(0.0f, out));
        else if (p.dh0 && in) p.dh0[state] = out;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            before[w][lane] = h;
            h = apply(totA[w][lane], h, totH[w][lane]);
        }
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
            behind[w][lane] = g;
            g = apply(totB[w][lane], g, totG[w][lane]);
        }
    }
    __syncthreads();
    float h[8], g[8], prev[R][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __shfl_up(A[i], 8, 64), v = __shfl_up(H[i], 8, 64);
        const float ag = __shfl_down(AG[i], 8, 64), vg = __shfl_down(G[i], 8, 64);
        h[i] = before[wave][c8 + i];
        if (lane >= 8) h[i] = apply(a, h[i], v);
        g[i] = behind[wave][c8 + i];
        if (lane < 56) g[i] = apply(ag, g[i], vg);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        float xf[8], lf[8];
        x[j].get(xf);
        la[j].get(lf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = decay(lf[i]);
            prev[j][i] = h[i];
            if (j + 1 < R) h[i] = apply(a, h[i], xf[i] * gain<GAIN>(lf[i], a));
        }
    }
    const long xb = b * p.dx.sb + c, lb = b * p.dla.sb + c;
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
        float xf[8], lf[8], gf[8], dx[8], dl[8];
        x[j].get(xf);
        la[j].get(lf);
        dh[j].get(gf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = decay(lf[i]), k = gain<GAIN>(lf[i], a);
            const float full = gf[i] + g[i];
            dx[i] = GAIN == PDN_GAIN_NONE ? full : k * full;
            dl[i] = join(prev[j][i], a) * full;
            if constexpr (GAIN != PDN_GAIN_NONE) dl[i] = fmaf(gain_slope<GAIN>(a, k) * xf[i], full, dl[i]);
            g[i] = join(full, a);
        }
        if (t0 + j < p.T && c < p.D) {
            store8<XBF>(p.dx.p, xb + (t0 + j) * p.dx.st, dx);
            store8<LBF>(p.dla.p, lb + (t0 + j) * p.dla.st, dl);
        }
    }
}

template <bool XBF, bool LBF, int GAIN>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(pdn_scan_step_args a, int groups, long total) {
    const long n = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (n >= total) return;
    const long b = n / groups;
    const int c = static_cast<int>(n - b * groups) * 8;
    Raw8<XBF> x;
    Raw8<LBF> la;
    Raw8<false> s;
    x.load(a.x, b * a.x_sb + c);
    la.load(a.log_a, b * a.log_a_sb + c);
    s.load(a.h_prev, b * a.D + c);
    float xf[8], lf[8], h[8];
    x.get(xf);
    la.get(lf);
    s.get(h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = decay(lf[i]);
        h[i] = apply(d, h[i], xf[i] * gain<GAIN>(lf[i], d));
    }
    store8<false>(a.h_next, b * a.D + c, h);
    store8<XBF>(a.h, b * a.h_sb + c, h);
}

// Before the tiles: counters to zero, every word to "not there yet".
__global__ void __launch_bounds__(kThreads) scan_reset_kernel(unsigned* counters, u32x4* words, long n) {
    const long step = static_cast<long>(gridDim.x) * kThreads;
    if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0u;
    for (long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step)
        words[i] = u32x4{~0u, ~0u, ~0u, ~0u};
}

// dst = src, or zeros: the state of a call without tokens
__global__ void __launch_bounds__(kThreads) scan_state_kernel(float* dst, const float* src, long n) {
    const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) dst[i] = src ? src[i] : 0.0f;
}

// Workspace: two counters in the first 256 bytes, then the words of the
// forward's tiles, then those of the backward's, then the backward's marks.
constexpr size_t kCounterBytes = 256;

long strips(const pdn_scan_args& a) { return (a.D + kCols - 1L) / kCols; }
long tiles(const pdn_scan_args& a, int tile) { return (a.T + tile - 1L) / tile; }
size_t chain_words(const pdn_scan_args& a, int tile) {
    const long n = tiles(a, tile);
    return n > 1 ? static_cast<size_t>(a.B) * strips(a) * n * kCols * 2 : 0;
}

ScanParams params(const pdn_scan_args& a) {
    ScanParams p = {};
    p.x = Rows{a.x, a.x_sb, a.x_st};
    p.la = Rows{a.log_a, a.log_a_sb, a.log_a_st};
    p.h0 = a.h0;
    p.T = a.T;
    p.D = a.D;
    p.strips = static_cast<int>(strips(a));
    p.columns = a.B * p.strips;
    return p;
}

void set_chain(ScanParams& p, unsigned* counter, u64* words) {
    p.chain.counter = counter;
    p.chain.agg = words;
    p.chain.inc = words + static_cast<long>(p.columns) * p.tiles * kCols;
}

hipError_t reset(void* workspace, size_t words, hipStream_t st) {
    const long n = static_cast<long>(words / 2);  // 16 bytes each
    long blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 2048) blocks = 2048;
    if (blocks < 1) blocks = 1;
    scan_reset_kernel<<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st>>>(
        static_cast<unsigned*>(workspace), reinterpret_cast<u32x4*>(static_cast<char*>(workspace) + kCounterBytes), n);
    return hipGetLastError();
}

template <bool XBF, bool LBF, int GAIN>
void launch_tiles(const ScanParams& p, int kind, dim3 grid, hipStream_t st) {
    if (kind == 0) scan_fwd_kernel<XBF, LBF, GAIN, true><<<grid, dim3(kThreads), 0, st>>>(p);
    else if (kind == 1) scan_fwd_kernel<XBF, LBF, GAIN, false><<<grid, dim3(kThreads), 0, st>>>(p);
    else scan_bwd_kernel<XBF, LBF, GAIN><<<grid, dim3(kThreads), 0, st>>>(p);
}

// kind: 0 forward, 1 forward for the marks alone, 2 backward
hipError_t launch_kind(const ScanParams& p, const pdn_scan_args& a, int kind, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(static_cast<long>(p.columns) * p.tiles));
    const bool xb = a.dtype == PDN_BF16, lb = a.log_dtype == PDN_BF16;
#define PDN_GAINS(X, L)                                                              \
    switch (a.gain) {                                                                \
        case PDN_GAIN_NONE: launch_tiles<X, L, PDN_GAIN_NONE>(p, kind, grid, st); break;            \
        case PDN_GAIN_COMPLEMENT: launch_tiles<X, L, PDN_GAIN_COMPLEMENT>(p, kind, grid, st); break; \
        default: launch_tiles<X, L, PDN_GAIN_NORM>(p, kind, grid, st); break;                       \
    }
    if (xb && lb) { PDN_GAINS(true, true) }
    else if (xb) { PDN_GAINS(true, false) }
    else { PDN_GAINS(false, false) }
#undef PDN_GAINS
    return hipGetLastError();
}

hipError_t copy_state(float* dst, const float* src, const pdn_scan_args& a, hipStream_t st) {
    const long n = static_cast<long>(a.B) * a.D;
    if (!dst || dst == src) return hipSuccess;
    scan_state_kernel<<<dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st>>>(dst, src, n);
    return hipGetLastError();
}

}  // namespace

long scan_blocks(const pdn_scan_args& a) { return a.B * strips(a) * tiles(a, kBwdTile); }

size_t scan_fwd_workspace_bytes(const pdn_scan_args& a) {
    const size_t words = chain_words(a, kFwdTile);
    return words ? kCounterBytes + words * sizeof(u64) : 0;
}

size_t scan_bwd_workspace_bytes(const pdn_scan_bwd_args& b) {
    const pdn_scan_args& a = b.fwd;
    const size_t words = chain_words(a, kBwdTile);
    if (!words) return 0;  // one tile: from h0 to dhT
    size_t n = kCounterBytes + words * sizeof(u64);
    if (!a.marks) n += chain_words(a, kFwdTile) * sizeof(u64) + sizeof(float) * a.B * static_cast<size_t>(tiles(a, kBwdTile)) * a.D;
    return n;
}

hipError_t launch_scan_fwd(const pdn_scan_args& a, hipStream_t st) {
    if (a.T == 0) return copy_state(a.hT, a.h0, a, st);
    ScanParams p = params(a);
    p.h = RowsOut{a.h, a.h_sb, a.h_st};
    p.hT = a.hT;
    p.marks_out = a.marks;
    p.tiles = static_cast<int>(tiles(a, kFwdTile));
    if (p.tiles > 1) {
        const hipError_t e = reset(a.workspace, chain_words(a, kFwdTile), st);
        if (e != hipSuccess) return e;
        set_chain(p, static_cast<unsigned*>(a.workspace), reinterpret_cast<u64*>(static_cast<char*>(a.workspace) + kCounterBytes));
    }
    return launch_kind(p, a, 0, st);
}

hipError_t launch_scan_bwd(const pdn_scan_bwd_args& b, hipStream_t st) {
    const pdn_scan_args& a = b.fwd;
    if (a.T == 0) return copy_state(b.dh0, b.dhT, a, st);
    ScanParams p = params(a);
    p.dh = Rows{b.dh, b.dh_sb, b.dh_st};
    p.dx = RowsOut{b.dx, b.dx_sb, b.dx_st};
    p.dla = RowsOut{b.dlog_a, b.dlog_a_sb, b.dlog_a_st};
    p.dhT = b.dhT;
    p.dh0 = b.dh0;
    p.marks = a.marks;
    p.tiles = static_cast<int>(tiles(a, kBwdTile));
    if (p.tiles > 1) {
        unsigned* counters = static_cast<unsigned*>(b.workspace);
        u64* words = reinterpret_cast<u64*>(static_cast<char*>(b.workspace) + kCounterBytes);
        const size_t fwd = a.marks ? 0 : chain_words(a, kFwdTile), bwd = chain_words(a, kBwdTile);
        hipError_t e = reset(b.workspace, fwd + bwd, st);
        if (e != hipSuccess) return e;
        if (!a.marks) {
            ScanParams f = params(a);
            f.marks_out = reinterpret_cast<float*>(words + fwd + bwd);
            f.tiles = static_cast<int>(tiles(a, kFwdTile));
            set_chain(f, counters + 1, words);
            e = launch_kind(f, a, 1, st);
            if (e != hipSuccess) return e;
            p.marks = f.marks_out;
        }
        set_chain(p, counters, words + fwd);
    }
    return launch_kind(p, a, 2, st);
}

hipError_t launch_scan_step(const pdn_scan_step_args& a, hipStream_t st) {
    const int groups = a.D / 8;
    const long total = static_cast<long>(a.B) * groups;
    const dim3 grid(static_cast<unsigned>((total + kThreads - 1) / kThreads)), block(kThreads);
    const bool xb = a.dtype == PDN_BF16, lb = a.log_dtype == PDN_BF16;
#define PDN_GAINS(X, L)                                                                                                          \
    switch (a.gain) {                                                                                                            \
        case PDN_GAIN_NONE: scan_step_kernel<X, L, PDN_GAIN_NONE><<<grid, block, 0, st>>>(a, groups, total); break;              \
        case PDN_GAIN_COMPLEMENT: scan_step_kernel<X, L, PDN_GAIN_COMPLEMENT><<<grid, block, 0, st>>>(a, groups, total); break;  \
        default: scan_step_kernel<X, L, PDN_GAIN_NORM><<<grid, block, 0, st>>>(a, groups, total); break;                         \
    }
    if (xb && lb) { PDN_GAINS(true, true) }
    else if (xb) { PDN_GAINS(true, false) }
    else { PDN_GAINS(false, false) }
#undef PDN_GAINS
    return hipGetLastError();
}

}  // namespace pdn
