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
// of 128 channels by (waves x R) tokens.  A wave holds R tokens of all 128
// channels in registers, two neighbouring channels to a lane (a row of bf16 is
// one 256-byte access), and reduces them to (A, H) without a word to another
// lane; its row addresses are scalars.  The waves' runs meet in LDS.  What is
// left is the state before the tile:
//
// the tiles hand it on along their column as scan_chain.h says.
//
// Measured on an MI355X, whose large copies reach 5.3 TB/s (counters: 1.02 to
// 1.04 times the bytes that the call cannot do without, the published words
// among them), after the reset of the words (6 us):
//   forward   B4 T8192 D2048, bf16, fp32 decays       98 us   5.5 TB/s
//             B1 T65536 D2048, bf16                  160 us   5.0 TB/s
//             B2 T8192 D4096, bf16, normed gain       86 us   4.7 TB/s
//   backward  of the last, kept states given         142 us   4.7 TB/s
// A tile lives for 8 to 11 us, of which it loads for 3 to 4, waits for its state
// for 2 to 5 and stores for 2; two workgroups to a compute unit cover most of
// that, and what is left is the first round's fill and the last one's drain.
//
// A decay that is zero drops the state before it, infinities and NaN included:
// every "a h + b" below selects b, and every product of decays 0, where the
// later factor is zero.
#include "layer.h"
#include "rows.h"
#include "scan_chain.h"

namespace pdn {
namespace {

constexpr int kThreads = 256;  // of the step, reset and copy kernels
// Waves of a workgroup and tokens of a wave.  Both directions fit 128 registers
// (two workgroups to a compute unit), but for the fp32 backward with the
// complement gain, which spills 20 bytes a lane.  Measured at B2 T8192 D4096 bf16, forward
// 8 x 16 93 us, 16 x 16 101, 4 x 32 104, 8 x 8 108; backward 8 x 12 144, 4 x 16
// 150, 16 x 8 154, 8 x 8 157, 8 x 16 (one workgroup to a compute unit) 177.
// Forward in bf16 24 tokens: 1% slower there, 161 us instead of 176 over 65536 x
// 2048 and 49 instead of 66 over 65536 x 128, where longer tiles mean fewer in a
// chain; in fp32 16: 24 took 77 us instead of 72 at B16 T2048 D1024, 154 instead
// of 147 at B4 T8192 D2048 (159 instead of 169 over 65536 x 1024).
constexpr int kWaves = 8;
constexpr int fwd_r(bool bf16) { return bf16 ? 24 : 16; }
constexpr int kBwdR = 12;
constexpr int kBwdTile = kWaves * kBwdR;
static_assert(kBwdTile == PDN_SCAN_MARK, "the backward's tiles start at the marks");
static_assert(PDN_SCAN_MARK % fwd_r(true) == 0 && PDN_SCAN_MARK % fwd_r(false) == 0, "marks lie at the boundaries of the forward's waves");

struct Rows {
    const void* p;
    long sb, st;
};
struct RowsOut {
    void* p;
    long sb, st;
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
    int strips;          // kCols-channel strips of a row
    int columns;         // B * strips
    Chain chain;
};

// The counters lie a 128-byte line apart and start at all ones, one below 0.
constexpr int kCounterStep = 32;

// This workgroup's column goes by its number (an XCD's workgroups have
// neighbouring columns), its tile by the order in which the column's
// workgroups start.
__device__ __forceinline__ void deal(const ScanParams& p, int* slot, int& column, int& at) {
    column = by_xcd(blockIdx.x % p.columns, p.columns);
    at = 0;
    if (p.chain.tiles == 1) return;
    if (threadIdx.x == 0)
        *slot = static_cast<int>(1u + __hip_atomic_fetch_add(p.chain.counters + static_cast<long>(column) * kCounterStep, 1u,
                                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    __syncthreads();
    at = __builtin_amdgcn_readfirstlane(*slot) - p.chain.carrier;  // -1: this workgroup is the carrier
}

__device__ __forceinline__ float decay(float la) { return __builtin_amdgcn_exp2f(la * kLog2e); }

// 1 - e^y for y <= 0 to fp32 accuracy, given e = e^y: the difference where e
// is far from 1 (y < -0.35: an error of e counts under 2.4 times there), else
// -y times a polynomial for (e^y - 1) / y, fitted to relative error at
// Chebyshev points of [-0.35, 0]: 0.23 x 2^-24 off in exact arithmetic.
__device__ __forceinline__ float one_minus_exp(float y, float e) {
    float s = 0.00720365811f;
    s = fmaf(s, y, 0.0413265228f);
    s = fmaf(s, y, 0.166624129f);
    s = fmaf(s, y, 0.499998122f);
    s = fmaf(s, y, 1.0f);
    return y < -0.35f ? 1.0f - e : -y * s;
}

// The normed gain of a decay of one is +0, whichever zero la is (of la = +0 the
// difference above is -0): the slope divides by it, and tends to -inf there.
template <int GAIN>
__device__ __forceinline__ float gain(float la, float a) {
    if constexpr (GAIN == PDN_GAIN_COMPLEMENT) return one_minus_exp(la, a);
    if constexpr (GAIN == PDN_GAIN_NORM) return fabsf(__builtin_amdgcn_sqrtf(one_minus_exp(2.0f * la, a * a)));
    return 1.0f;
}
// its derivative by la, given the gain g
template <int GAIN>
__device__ __forceinline__ float gain_slope(float a, float g) {
    if constexpr (GAIN == PDN_GAIN_COMPLEMENT) return -a;
    if constexpr (GAIN == PDN_GAIN_NORM) return -a * a * __builtin_amdgcn_rcpf(g);
    return 0.0f;
}

// Two neighbouring channels of a row, as they lie in memory.  What is read once
// is loaded past the caches (STREAM) where rows begin at 128-byte lines: scan
// over 65536 tokens by 2048 channels (128 to a tile) 185 -> 175 us, B16 T2048 D1024 in fp32 86 ->
// 73 us.  Other rows share lines at the strips' borders, which the caches then
// spare: backward of B11 T2346 D2600 in fp32 307 us past them, 288 us through.
// (A template argument: the compiler makes one load of two alike.)
template <bool BF16>
struct Raw2;
template <>
struct Raw2<true> {
    uint32_t v;
    template <bool STREAM>
    __device__ __forceinline__ void load(const void* p, long row, int i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + row + i);
        if constexpr (STREAM) v = __builtin_nontemporal_load(q);
        else v = *q;
    }
    __device__ __forceinline__ void zero() { v = 0u; }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
    static __device__ __forceinline__ void store(void* p, long row, int i, f32x2 f) {
        typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
        *reinterpret_cast<bf16x2*>(static_cast<uint16_t*>(p) + row + i) = __builtin_convertvector(f, bf16x2);
    }
};
template <>
struct Raw2<false> {
    f32x2 v;
    template <bool STREAM>
    __device__ __forceinline__ void load(const void* p, long row, int i) {
        const f32x2* q = reinterpret_cast<const f32x2*>(static_cast<const float*>(p) + row + i);
        if constexpr (STREAM) v = __builtin_nontemporal_load(q);
        else v = *q;
    }
    __device__ __forceinline__ void zero() { v = f32x2{0.f, 0.f}; }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    static __device__ __forceinline__ void store(void* p, long row, int i, f32x2 f) {
        *reinterpret_cast<f32x2*>(static_cast<float*>(p) + row + i) = f;
    }
};

template <bool XBF, bool LBF, int GAIN, bool LINES, bool WRITE_H>
__global__ void __launch_bounds__(64 * kWaves, 4) scan_fwd_kernel(ScanParams p) {
    constexpr int R = fwd_r(XBF), W = kWaves, TILE = W * R;
    __shared__ int slot;
    __shared__ float totA[W][kCols], totH[W][kCols];
    __shared__ float before[W][kCols];  // the state before each wave's tokens
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int column, at;
    deal(p, &slot, column, at);
    const int b = column / p.strips, c0 = (column - b * p.strips) * kCols;
    if (at < 0) {
        if (wave < 2) carry(p.chain, column, tid);
        return;
    }
    const int c2 = 2 * lane, c = c0 + c2;
    const int cc = c < p.D ? c : 0;  // lanes past the last channel read another's
    const int t0 = at * TILE + wave * R;

    Raw2<XBF> x[R];
    Raw2<LBF> la[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const long t = min(t0 + j, p.T - 1);
        x[j].template load<LINES>(p.x.p, b * p.x.sb + t * p.x.st, cc);
        la[j].template load<LINES>(p.la.p, b * p.la.sb + t * p.la.st, cc);
    }
    if (t0 + R > p.T) {
        // past the end: a = 1 and nothing added, so the state passes through
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (t0 + j >= p.T) {
                x[j].zero();
                la[j].zero();
            }
    }

    float a[R][2], v[R][2], A[2], H[2];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float l = la[j].get(i);
            a[j][i] = decay(l);
            v[j][i] = x[j].get(i) * gain<GAIN>(l, a[j][i]);
            H[i] = j ? apply(a[j][i], H[i], v[j][i]) : v[j][i];
            A[i] = j ? join(A[i], a[j][i]) : a[j][i];
        }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        totA[wave][c2 + i] = A[i];
        totH[wave][c2 + i] = H[i];
    }
    __syncthreads();
    if (wave < 2) {
        const int k = wave * 64 + lane, ch = c0 + k;
        const bool in = ch < p.D;
        const long state = static_cast<long>(b) * p.D + ch;
        float behind;
        float h = meet<W>(p.chain, totA, totH, column, at, k, at == 0 && p.h0 && in ? p.h0[state] : 0.0f, behind);
        if (at + 1 == p.chain.tiles && p.hT && in) p.hT[state] = behind;
        const int marks = (p.T + PDN_SCAN_MARK - 1) / PDN_SCAN_MARK;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            before[w][k] = h;
            const int t = at * TILE + w * R;
            if (p.marks_out && t % PDN_SCAN_MARK == 0 && t < p.T && in)
                p.marks_out[(static_cast<long>(b) * marks + t / PDN_SCAN_MARK) * p.D + ch] = h;
            h = apply(totA[w][k], h, totH[w][k]);
        }
    }
    if constexpr (WRITE_H) {
        __syncthreads();
        f32x2 h = {before[wave][c2], before[wave][c2 + 1]};
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) h[i] = apply(a[j][i], h[i], v[j][i]);
            if (t0 + j < p.T && c < p.D)
                Raw2<XBF>::store(p.h.p, b * p.h.sb + static_cast<long>(t0 + j) * p.h.st, c, h);
        }
    }
}

// Backward: tiles are processed from the last token to the first.  With
// C = a_{t+1} G_{t+1} the gradient that reaches a token from the right (dhT
// behind the last), G = dh + C and the token passes a (dh + C) on: the same
// kind of map, run right to left.  The states h_{t-1} inside a tile come from
// the kept state before it.
template <bool XBF, bool LBF, int GAIN, bool LINES>
__global__ void __launch_bounds__(64 * kWaves, 4) scan_bwd_kernel(ScanParams p) {
    constexpr int R = kBwdR, W = kWaves;
    __shared__ int slot;
    __shared__ float totA[W][kCols], totH[W][kCols];  // the waves' runs, forward
    __shared__ float totB[W][kCols], totG[W][kCols];  // and backward, the last wave's first
    __shared__ float before[W][kCols];  // the state before each wave's tokens
    __shared__ float behind[W][kCols];  // what reaches them from the right
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int column, at;
    deal(p, &slot, column, at);
    const int tile = p.chain.tiles - 1 - at;
    const int b = column / p.strips, c0 = (column - b * p.strips) * kCols;
    if (at < 0) {
        if (wave < 2) carry(p.chain, column, tid);
        return;
    }
    const int c2 = 2 * lane, c = c0 + c2;
    const int cc = c < p.D ? c : 0;
    const int t0 = tile * kBwdTile + wave * R;

    Raw2<XBF> x[R], dh[R];
    Raw2<LBF> la[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const long t = min(t0 + j, p.T - 1);
        x[j].template load<LINES>(p.x.p, b * p.x.sb + t * p.x.st, cc);
        la[j].template load<LINES>(p.la.p, b * p.la.sb + t * p.la.st, cc);
        dh[j].template load<LINES>(p.dh.p, b * p.dh.sb + t * p.dh.st, cc);
    }
    if (t0 + R > p.T) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (t0 + j >= p.T) {
                x[j].zero();
                la[j].zero();
                dh[j].zero();
            }
    }

    float a[R][2], g[R][2], A[2], H[2], B[2], G[2];
    {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float l = la[j].get(i);
                a[j][i] = decay(l);
                g[j][i] = gain<GAIN>(l, a[j][i]);
                const float v = x[j].get(i) * g[j][i];
                H[i] = j ? apply(a[j][i], H[i], v) : v;
                A[i] = j ? join(A[i], a[j][i]) : a[j][i];
            }
#pragma unroll
        for (int j = R - 1; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float full = j < R - 1 ? dh[j].get(i) + G[i] : dh[j].get(i);
                G[i] = join(full, a[j][i]);
                B[i] = j < R - 1 ? join(B[i], a[j][i]) : a[j][i];
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        totA[wave][c2 + i] = A[i];
        totH[wave][c2 + i] = H[i];
        totB[W - 1 - wave][c2 + i] = B[i];
        totG[W - 1 - wave][c2 + i] = G[i];
    }
    __syncthreads();
    if (wave < 2) {
        const int k = wave * 64 + lane, ch = c0 + k;
        const bool in = ch < p.D;
        const long state = static_cast<long>(b) * p.D + ch;
        float h = 0.0f, out;
        if (in && p.marks) h = p.marks[(static_cast<long>(b) * p.chain.tiles + tile) * p.D + ch];
        else if (in && p.h0) h = p.h0[state];
        float r = meet<W>(p.chain, totB, totG, column, at, k, at == 0 && p.dhT && in ? p.dhT[state] : 0.0f, out);
        if (at + 1 == p.chain.tiles && p.dh0 && in) p.dh0[state] = out;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            before[w][k] = h;
            h = apply(totA[w][k], h, totH[w][k]);
            behind[W - 1 - w][k] = r;
            r = apply(totB[w][k], r, totG[w][k]);
        }
    }
    __syncthreads();
    // dlog_a = G (a h_{t-1} + g' x): the bracket forward, then G backward
    float q[R][2];
    {
        float h[2] = {before[wave][c2], before[wave][c2 + 1]};
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float xf = x[j].get(i), kept = join(h[i], a[j][i]);
                q[j][i] = GAIN == PDN_GAIN_NONE ? kept : fmaf(gain_slope<GAIN>(a[j][i], g[j][i]), xf, kept);
                h[i] = fmaf(xf, g[j][i], kept);
            }
        }
    }
    float r[2] = {behind[wave][c2], behind[wave][c2 + 1]};
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
        f32x2 dx, dl;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float full = dh[j].get(i) + r[i];
            dx[i] = GAIN == PDN_GAIN_NONE ? full : g[j][i] * full;
            dl[i] = q[j][i] * full;
            r[i] = join(full, a[j][i]);
        }
        if (t0 + j < p.T && c < p.D) {
            Raw2<XBF>::store(p.dx.p, b * p.dx.sb + static_cast<long>(t0 + j) * p.dx.st, c, dx);
            Raw2<LBF>::store(p.dla.p, b * p.dla.sb + static_cast<long>(t0 + j) * p.dla.st, c, dl);
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

// Before the tiles: every word to "not there yet", every counter below 0.
__global__ void __launch_bounds__(kThreads) scan_reset_kernel(u32x4* words, long n) {
    const long step = static_cast<long>(gridDim.x) * kThreads;
    for (long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step)
        words[i] = u32x4{~0u, ~0u, ~0u, ~0u};
}

// dst = src, or zeros: the state of a call without tokens
__global__ void __launch_bounds__(kThreads) scan_state_kernel(float* dst, const float* src, long n) {
    const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n) dst[i] = src ? src[i] : 0.0f;
}

// Workspace: the chain of a backward's tiles, then that of a forward's (each
// its counters, then its words), then the marks that a backward forms.
long strips(const pdn_scan_args& a) { return (a.D + kCols - 1L) / kCols; }
int fwd_tile(const pdn_scan_args& a) { return kWaves * fwd_r(a.dtype == PDN_BF16); }
long tiles(const pdn_scan_args& a, int tile) { return (a.T + tile - 1L) / tile; }
size_t chain_bytes(const pdn_scan_args& a, int tile) {
    const size_t n = tiles(a, tile), columns = a.B * strips(a);
    return n > 1 ? columns * (kCounterStep * sizeof(unsigned) + n * kCols * 2 * sizeof(u64)) : 0;
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

bool has_carriers(long columns, long tiles) { return tiles > 1 && columns <= kCarried; }

void set_chain(ScanParams& p, char* at) {
    p.chain.carrier = has_carriers(p.columns, p.chain.tiles);
    p.chain.counters = reinterpret_cast<unsigned*>(at);
    p.chain.agg = reinterpret_cast<u64*>(at + sizeof(unsigned) * kCounterStep * p.columns);
    p.chain.inc = p.chain.agg + static_cast<long>(p.columns) * p.chain.tiles * kCols;
}

hipError_t reset(void* workspace, size_t bytes, hipStream_t st) {
    const long n = static_cast<long>(bytes / sizeof(u32x4));
    const long blocks = (n + kThreads - 1) / kThreads;
    scan_reset_kernel<<<dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048)), dim3(kThreads), 0, st>>>(
        static_cast<u32x4*>(workspace), n);
    return hipGetLastError();
}

template <bool XBF, bool LBF, int GAIN, bool LINES>
void launch_tiles(const ScanParams& p, int kind, dim3 grid, hipStream_t st) {
    if (kind == 0) scan_fwd_kernel<XBF, LBF, GAIN, LINES, true><<<grid, dim3(64 * kWaves), 0, st>>>(p);
    else if (kind == 1) scan_fwd_kernel<XBF, LBF, GAIN, LINES, false><<<grid, dim3(64 * kWaves), 0, st>>>(p);
    else scan_bwd_kernel<XBF, LBF, GAIN, LINES><<<grid, dim3(64 * kWaves), 0, st>>>(p);
}

template <bool XBF, bool LBF>
void launch_gain(const ScanParams& p, int gain, bool lines, int kind, dim3 grid, hipStream_t st) {
    switch (gain) {
#define PDN_CASE(G)                                                      \
    case G:                                                              \
        if (lines) launch_tiles<XBF, LBF, G, true>(p, kind, grid, st);   \
        else launch_tiles<XBF, LBF, G, false>(p, kind, grid, st);        \
        break;
        PDN_CASE(PDN_GAIN_NONE)
        PDN_CASE(PDN_GAIN_COMPLEMENT)
        PDN_CASE(PDN_GAIN_NORM)
#undef PDN_CASE
    }
}

// whether every row of B x T rows at these strides begins at a 128-byte line
bool whole_lines(const void* p, long sb, long st, int32_t dtype, const pdn_scan_args& a) {
    const long e = dtype == PDN_BF16 ? 2 : 4;
    return reinterpret_cast<uintptr_t>(p) % 128 == 0 && (a.B == 1 || sb * e % 128 == 0) && (a.T == 1 || st * e % 128 == 0);
}

// kind: 0 forward, 1 forward for the marks alone, 2 backward
hipError_t launch_kind(const ScanParams& p, const pdn_scan_args& a, int kind, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(static_cast<long>(p.columns) * (p.chain.tiles + p.chain.carrier)));
    const bool xb = a.dtype == PDN_BF16, lb = a.log_dtype == PDN_BF16;
    const bool lines = whole_lines(p.x.p, p.x.sb, p.x.st, a.dtype, a) && whole_lines(p.la.p, p.la.sb, p.la.st, a.log_dtype, a) &&
                       (kind != 2 || whole_lines(p.dh.p, p.dh.sb, p.dh.st, a.dtype, a));
    if (xb && lb) launch_gain<true, true>(p, a.gain, lines, kind, grid, st);
    else if (xb) launch_gain<true, false>(p, a.gain, lines, kind, grid, st);
    else launch_gain<false, false>(p, a.gain, lines, kind, grid, st);
    return hipGetLastError();
}

hipError_t copy_state(float* dst, const float* src, const pdn_scan_args& a, hipStream_t st) {
    const long n = static_cast<long>(a.B) * a.D;
    if (!dst || dst == src) return hipSuccess;
    scan_state_kernel<<<dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st>>>(dst, src, n);
    return hipGetLastError();
}

}  // namespace

bool scan_fits(const pdn_scan_args& a) {
    static_assert(kBwdR <= fwd_r(false) && kBwdR <= fwd_r(true), "the backward has the most tiles");
    const long columns = a.B * strips(a), n = tiles(a, kBwdTile);
    return columns * (n + has_carriers(columns, n)) <= kMaxGridThreads / (64 * kWaves);
}

size_t scan_fwd_workspace_bytes(const pdn_scan_args& a) { return chain_bytes(a, fwd_tile(a)); }

size_t scan_bwd_workspace_bytes(const pdn_scan_bwd_args& b) {
    const pdn_scan_args& a = b.fwd;
    const size_t n = chain_bytes(a, kBwdTile);
    if (n == 0 || a.marks) return n;  // one tile runs from h0 to dhT
    return n + chain_bytes(a, fwd_tile(a)) + sizeof(float) * a.B * static_cast<size_t>(tiles(a, kBwdTile)) * a.D;
}

hipError_t launch_scan_fwd(const pdn_scan_args& a, hipStream_t st) {
    if (a.T == 0) return copy_state(a.hT, a.h0, a, st);
    ScanParams p = params(a);
    p.h = RowsOut{a.h, a.h_sb, a.h_st};
    p.hT = a.hT;
    p.marks_out = a.marks;
    p.chain.tiles = static_cast<int>(tiles(a, fwd_tile(a)));
    if (p.chain.tiles > 1) {
        const hipError_t e = reset(a.workspace, chain_bytes(a, fwd_tile(a)), st);
        if (e != hipSuccess) return e;
        set_chain(p, static_cast<char*>(a.workspace));
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
    p.chain.tiles = static_cast<int>(tiles(a, kBwdTile));
    if (p.chain.tiles > 1) {
        char* ws = static_cast<char*>(b.workspace);
        const size_t bwd = chain_bytes(a, kBwdTile), fwd = a.marks ? 0 : chain_bytes(a, fwd_tile(a));
        hipError_t e = reset(ws, bwd + fwd, st);
        if (e != hipSuccess) return e;
        set_chain(p, ws);
        if (!a.marks) {
            ScanParams f = params(a);
            f.marks_out = reinterpret_cast<float*>(ws + bwd + fwd);
            f.chain.tiles = static_cast<int>(tiles(a, fwd_tile(a)));
            set_chain(f, ws + bwd);
            e = launch_kind(f, a, 1, st);
            if (e != hipSuccess) return e;
            p.marks = f.marks_out;
        }
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
