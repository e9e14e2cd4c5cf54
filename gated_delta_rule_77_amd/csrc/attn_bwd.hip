// The gradient of causal softmax attention, from q, k, v, dO and what the forward
// left (o and each row's lse):
//
//   P_ij = exp(scale s_ij - lse_i),  D_i = <dO_i, o_i>,  dS_ij = P_ij (<dO_i, v_j> - D_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i
//
// in two passes that each own their sums, so that no atomics decide an order: dq by
// rows of queries over tiles of keys (which also leaves D), then dk and dv by blocks of keys
// over tiles of queries, head after head of those that share them.  P and <dO, v> are
// formed in both: 14 products of d for each pair of a query and a key it sees, where
// one pass would take 10.
//
// Bound as the forward is: in both passes the matrix units take 50 to 57% of the cycles and
// the vector units 40 to 45% (T65536 with a window of 2048, H16/4 d128: dq 1.5 to 1.6 ms,
// 1.03 PFLOP/s; dk and dv 2.2 to 2.3 ms, 0.96), the second also by its reads of LDS, 40 KB a wave
// and block, for which 38% of the cycles go: K stays in registers, V, which would leave no
// second wave to a SIMD, does not.  Even so its kernels of d128 lack some: in bf16 9 vector
// registers (11 with parts) and 28 scalar ones are kept in memory or in other registers, read
// again once a tile and twice a masked block; in fp32 dq's lacks 19.  Two blocks of keys a wave
// lack far more (an early form 1800 us, so 2826).  Packed rows of B2 H32/8 T8192 run at 0.50
// to 0.55 PFLOP/s there: blocks hold ends of sequences, and the longest sequences' workgroups
// end last.
#include "attn.h"
#include "block.h"
#include "layer.h"

namespace pdn {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kQueries = 32;  // of a tile in the pass over keys' gradients

struct View4 {
    const void* p;
    long sb, sh, st;
};
struct Out4 {
    void* p;
    long sb, sh, st;
};

struct BwdParams {
    View4 q, k, v, o, d_o;
    Out4 dq, dk, dv;
    const float* lse;
    const int32_t* first;
    float *delta, *lse2;   // D, and lse in powers of two: [B,H,Tq]
    uint16_t* do16;        // bf16 copy of an fp32 dO, [B,H,Tq,D]; else null
    int* first_least;      // [B][tiles of queries]: least `first`; null without
    int H, Hk, shared;
    uint32_t inverse;
    int Tq, Tk, window;
    float scale, c;        // c: scale * log2(e)
    int o_f32, g_f32;
    int tiles, splits;     // of the launch's own rows or keys; of what each goes over
    float* part;           // splits > 1: sums [splits][rows][D], those of dv behind those of dk
    long rows;             // B H Tq, or B Hk Tk
    int query_tiles;
};

// The least first key of each tile of queries.
__global__ void __launch_bounds__(64) first_least_kernel(const int32_t* first, int Tq, int tiles, int* out) {
    const int b = blockIdx.x / tiles, t = blockIdx.x - b * tiles;
    const int i = min(t * kQueries + static_cast<int>(threadIdx.x % kQueries), Tq - 1);
    const int least = wave_min_i(first[static_cast<long>(b) * Tq + i]);
    if (threadIdx.x == 0) out[blockIdx.x] = least;
}

// Four channels of an output's row.
template <bool BF16>
__device__ __forceinline__ void store4(void* p, long at, int f32, const f32x4& x) {
    if (!BF16 || f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = x;
    else *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(p) + at) = __builtin_convertvector(x, bf16x4);
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, BF16 ? 2 : 1) attn_dq_kernel(BwdParams p) {
    using E = El<BF16>;
    using TL = Tile<BF16, D>;
    typedef typename E::Frag Frag;
    constexpr int ROWS = 128, KT = !BF16 && D == 128 ? 32 : 64;
    constexpr int S = D / 16, C = D / 32, KB = KT / 32;
    constexpr int TILE = KT * TL::ROW, DMAS = KT / TL::ROWS_PER_DMA / 4;
    __shared__ __align__(1024) char smem[4 * TILE];
    __shared__ int bounds[2][4];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int h = lane >> 5;
    const int hk = blockIdx.x % p.Hk, rest = blockIdx.x / p.Hk, batch = gridDim.x / (p.Hk * p.splits * p.tiles);  // as in the forward
    const int b = rest % batch, split = rest / batch % p.splits, tile = p.tiles - 1 - rest / batch / p.splits;
    const int nq = p.Tq, nk = p.Tk;
    const char* kb = static_cast<const char*>(p.k.p) + (b * p.k.sb + hk * p.k.sh) * E::BYTES;
    const char* vb = static_cast<const char*>(p.v.p) + (b * p.v.sb + hk * p.v.sh) * E::BYTES;
    const int row0 = tile * ROWS, nrows = nq * p.shared;

    const int t0 = row0 / p.shared, m0 = row0 - t0 * p.shared;
    const int dr = 32 * wave + (lane & 31);
    const bool stored = row0 + dr < nrows;
    const int r = m0 + (stored ? dr : nrows - 1 - row0), dt = quotient(r, p.inverse), token = t0 + dt, head = hk * p.shared + r - dt * p.shared;
    const Seen seen = seen_by(token, nq, nk, p.window, p.first ? p.first[static_cast<long>(b) * nq + token] : 0);
    int low = INT32_MAX, high = -1, full_low = 0, full_high = INT32_MAX;
    if (seen.count > 0) {
        const int last = seen.low + seen.count - 1;
        low = min(low, seen.low);
        high = max(high, last);
        full_low = max(full_low, seen.low);
        full_high = min(full_high, last);
    }
    const long qa = b * p.q.sb + head * p.q.sh + token * p.q.st;
    const long oa = b * p.o.sb + head * p.o.sh + token * p.o.st;
    const long da = b * p.d_o.sb + head * p.d_o.sh + token * p.d_o.st;
    const long row = (static_cast<long>(b) * p.H + head) * nq + token;
    Frag q[S], dof[S];
    float dot = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int ch = 16 * s + 8 * h;
        q[s] = E::load(p.q.p, qa + ch);
        f32x8 x, y;
        if (!BF16 || p.o_f32) {
            x = El<false>::load(p.o.p, oa + ch);
            y = El<false>::load(p.d_o.p, da + ch);
            if constexpr (BF16) dof[s] = __builtin_convertvector(y, bf16x8);
            else dof[s] = y;
            if constexpr (BF16) {
                if (stored && split == 0) *reinterpret_cast<bf16x8*>(p.do16 + row * D + ch) = dof[s];
            }
        } else if constexpr (BF16) {
            x = __builtin_convertvector(El<true>::load(p.o.p, oa + ch), f32x8);
            dof[s] = E::load(p.d_o.p, da + ch);
            y = __builtin_convertvector(dof[s], f32x8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(x[j], y[j], dot);
    }
    float delta = dot + __shfl_xor(dot, 32, 64);
    // A row without a score above -inf has given 0: all of its probabilities are to be 0.  A
    // query that is not finite may give such scores too (any other makes lse NaN): its
    // probabilities are to be NaN, for all keys that it sees, in whatever tile they lie.
    const float lse = p.lse[row];
    float lse2 = lse * kLog2e;
    if (__ballot(lse == -INFINITY)) {
        bool sound = true;
#pragma unroll
        for (int s = 0; s < S; ++s) sound &= E::is_finite(q[s]);
        const uint64_t sounds = __ballot(sound), both = sounds & (sounds >> 32);
        if (lse == -INFINITY) lse2 = both >> (lane & 31) & 1 ? INFINITY : NAN;
    }
    low = uniform(wave_min_i(low));
    high = uniform(wave_max_i(high));
    full_low = uniform(wave_max_i(full_low));
    full_high = uniform(wave_min_i(full_high));
    if (lane == 0) {
        bounds[0][wave] = low;
        bounds[1][wave] = high;
    }
    __syncthreads();
    const int all_low = uniform(min(min(bounds[0][0], bounds[0][1]), min(bounds[0][2], bounds[0][3])));
    const int all_high = uniform(max(max(bounds[1][0], bounds[1][1]), max(bounds[1][2], bounds[1][3])));
    int first_tile = all_low / KT, end_tile = all_high < 0 ? first_tile : all_high / KT + 1;
    if (p.splits > 1) {
        const int n = (end_tile - first_tile + p.splits - 1) / p.splits;
        first_tile += split * n;
        end_tile = min(end_tile, first_tile + n);
    }

    const uint32_t at = lds_address(smem), row_base = TL::row_base(lane), column_base = TL::column_base(lane);

    // as in the forward
    constexpr int RPD = TL::ROWS_PER_DMA;
    const uint32_t chunk = TL::lane_chunk(lane);
    const uint32_t k_part = static_cast<uint32_t>(lane / TL::CHUNKS * p.k.st * E::BYTES), v_part = static_cast<uint32_t>(lane / TL::CHUNKS * p.v.st * E::BYTES);
    auto load_tile = [&](int t, int buffer) __attribute__((always_inline)) {
        const uint32_t dst = at + buffer * 2 * TILE + wave * DMAS * 1024;
        if (t * KT + KT <= nk) {
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                const int n = wave * DMAS + i;
                const long key = t * KT + n * RPD;
                to_lds(kb + key * p.k.st * E::BYTES, TL::lane_offset(k_part, chunk, n), dst + i * 1024);
                to_lds(vb + key * p.v.st * E::BYTES, TL::lane_offset(v_part, chunk, n), dst + TILE + i * 1024);
            }
        } else {  // keys behind the last repeat it, unseen
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                const int n = wave * DMAS + i;
                const long key = min(t * KT + n * RPD + lane / TL::CHUNKS, nk - 1);
                to_lds(kb + key * p.k.st * E::BYTES + TL::lane_offset(0, chunk, n), dst + i * 1024);
                to_lds(vb + key * p.v.st * E::BYTES + TL::lane_offset(0, chunk, n), dst + TILE + i * 1024);
            }
        }
    };

    f32x16 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] = 0.0f;

    // A block of 32 keys.  `partly`: some rows may not see all of them.  A key that is not
    // finite gives scores that are not: it is taken out of the product for those that do not
    // see it, and those that do have 0 times it from dP.
    auto block = [&](int k0, uint32_t kt, auto partly) __attribute__((always_inline)) {
        constexpr bool PARTLY = decltype(partly)::value;
        const uint32_t kr = kt + row_base, kc = kt + column_base, vr = kr + TILE;
        f32x16 s, dp;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const Frag kf = TL::rows(kr, 0, st);
            s = E::mma(kf, q[st], s);
        }
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const Frag vf = TL::rows(vr, 0, st);
            dp = E::mma(vf, dof[st], dp);
        }
        bool dirty = false;
        if constexpr (PARTLY) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) any |= !(fabsf(s[i]) < INFINITY);
            dirty = __ballot(any) != 0;
            if (dirty) {
#pragma unroll 1  // (rare: unrolled its operands cost the whole kernel registers)
                for (int st = 0; st < S; ++st) dp = E::mma(TL::rows(kr, 0, st), E::zero(), dp);
            }
        }
        Frag df[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = ex2(fmaf(s[i], p.c, -lse2));
        if constexpr (PARTLY) {
            const Seen to = {opaque(seen.low - k0 - 4 * h), seen.count};
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!sees(to, 8 * (i >> 2) + (i & 3))) s[i] = dp[i] = 0.0f;
                dot = fmaf(s[i], dp[i], dot);
            }
            // Where all that a row sees lies in this block, D is formed from it: a row of few
            // keys is where the rounding of o to bf16 would show most (alone it sees itself,
            // and its gradients vanish).
            dot = halves<false>(dot);
            if (seen.low >= k0 && seen.low + seen.count <= k0 + 32) delta = dot;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= dp[i] - delta;
        df[0] = E::of(s, 0);
        df[1] = E::of(s, 1);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Frag kf = TL::columns(kc, 16 * u, c);
                if constexpr (PARTLY)
                    if (dirty) kf = E::finite(kf);
                acc[c] = E::mma(kf, df[u], acc[c]);
            }
    };

    int t = first_tile;
    auto next = [&](uint32_t& kt) __attribute__((always_inline)) {
        const int buffer = (t - first_tile) & 1;
        landed();
        __syncthreads();
        if (t + 1 < end_tile) load_tile(t + 1, buffer ^ 1);
        kt = at + buffer * 2 * TILE;
    };
    auto some = [&](int end) __attribute__((always_inline)) {
        for (; t < end; ++t) {
            uint32_t kt;
            next(kt);
#pragma unroll 1
            for (int e = 0; e < KB; ++e) {
                const int k0 = t * KT + 32 * e;
                if (k0 <= high && k0 + 31 >= low) block(k0, kt + 32 * e * TL::ROW, std::true_type());
            }
        }
    };
    int from = max((full_low + KT - 1) / KT, first_tile), to = min((full_high + 1) / KT, end_tile);  // whole tiles
    if (low == INT32_MAX || from >= to) from = to = end_tile;
    if (first_tile < end_tile) load_tile(first_tile, 0);
    some(min(from, end_tile));
    for (; t < to; ++t) {
        uint32_t kt;
        next(kt);
#pragma unroll
        for (int e = 0; e < KB; ++e) block(0, kt + 32 * e * TL::ROW, std::false_type());
    }
    some(end_tile);
    if (!stored) return;
    // for the pass over the keys, from the one part that begins with what the row sees
    const int first = seen.low / KT;
    if (h == 0 && (seen.count > 0 ? first_tile <= first && first < end_tile : split == 0)) {
        p.delta[row] = delta;
        p.lse2[row] = lse2;
    }
    const long out = p.splits > 1 ? (split * p.rows + row) * D : b * p.dq.sb + head * p.dq.sh + token * p.dq.st;
    const float scale = p.splits > 1 ? 1.0f : p.scale;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = seen.count > 0 ? acc[c][4 * g + i] * scale : 0.0f;
            if (p.splits > 1) store4<false>(p.part, out + 32 * c + 8 * g + 4 * h, 1, x);
            else store4<BF16>(p.dq.p, out + 32 * c + 8 * g + 4 * h, p.g_f32, x);
        }
}

// PARTS: the workgroups of a block of keys are p.splits.
template <bool BF16, int D, bool PARTS>
__global__ void __launch_bounds__(kThreads, BF16 || D == 64 ? 2 : 1) attn_dkv_kernel(BwdParams p) {
    using E = El<BF16>;
    using TL = Tile<BF16, D>;
    typedef typename E::Frag Frag;
    constexpr int KEYS = 128, QT = kQueries;
    constexpr int S = D / 16, C = D / 32;
    constexpr int TILE = QT * TL::ROW, DMAS = QT / TL::ROWS_PER_DMA / 4;
    constexpr int VALUES = KEYS * TL::ROW, V_DMAS = KEYS / TL::ROWS_PER_DMA / 4;
    __shared__ __align__(1024) char smem[4 * TILE + VALUES];  // two tiles of queries and dO, the keys' values
    // Of a tile's queries: lse, D, first key.  A wave's load fills 64 places, of which QT are read
    // (with half of its lanes off for it the pass took 1.6% longer: packed rows of B2 H32/8 T8192
    // d128 850 and 864 us).
    __shared__ __align__(16) float stats[2][3][64];
    __shared__ int range[2][4];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int h = lane >> 5;
    // Heads of all sequences first, so that those of one XCD go through the rows side by side
    // (packed rows of B2 Hk8 T8192 1408 us one after another, 1322 so); then the keys, of which
    // the first have the most queries.
    const int splits = PARTS ? p.splits : 1, heads = static_cast<int>(gridDim.x) / (p.tiles * splits);
    const int bh = blockIdx.x % heads, rest = blockIdx.x / heads, b = bh / p.Hk, hk = bh - b * p.Hk;
    const int split = rest % splits, tile = rest / splits;
    const int nq = p.Tq, nk = p.Tk, off = nk - nq;
    const int key0 = tile * KEYS, key1 = min(key0 + KEYS, nk) - 1;

    // this lane's key; those behind the last repeat it, unstored and unseen
    Frag k[S];
    const int key = key0 + 32 * wave + (lane & 31);
    const long j = min(key, nk - 1);
    const long ka = b * p.k.sb + hk * p.k.sh + j * p.k.st;
#pragma unroll
    for (int s = 0; s < S; ++s) k[s] = E::load(p.k.p, ka + 16 * s + 8 * h);

    // the tiles of queries that see some of these keys
    int begin = max(key0 - off, 0) / QT, end = nq;
    if (p.window > 0 && key1 - off < nq - p.window) end = key1 - off + p.window;  // the last such query + 1
    end = end <= 0 ? begin : (end + QT - 1) / QT;
    if (p.first) {
        int lo = INT32_MAX, hi = -1;
        for (int t = begin + tid; t < end; t += kThreads)
            if (p.first_least[b * p.query_tiles + t] <= key1) {
                lo = min(lo, t);
                hi = t;
            }
        lo = wave_min_i(lo);
        hi = wave_max_i(hi);
        if (lane == 0) {
            range[0][wave] = lo;
            range[1][wave] = hi;
        }
        __syncthreads();
        begin = max(begin, min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3])));
        end = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3])) + 1;
    }
    begin = uniform(begin);
    end = uniform(end);

    if (!p.first && tid < 64) stats[0][2][tid] = stats[1][2][tid] = __int_as_float(INT32_MIN);  // before the first barrier
    f32x16 dk[C], dv[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[c][i] = dv[c][i] = 0.0f;

    const uint32_t at = lds_address(smem), row_base = TL::row_base(lane), column_base = TL::column_base(lane);
    const bool copied = BF16 && p.o_f32;
    constexpr int RPD = TL::ROWS_PER_DMA;
    const long d_st = copied ? D : p.d_o.st;
    auto load_values = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < V_DMAS; ++i) {
            const int n = wave * V_DMAS + i;
            const long j = min(key0 + n * RPD + lane / TL::CHUNKS, nk - 1);
            const char* vb = static_cast<const char*>(p.v.p) + (b * p.v.sb + hk * p.v.sh + j * p.v.st) * E::BYTES;
            to_lds(vb + TL::lane_offset(0, TL::lane_chunk(lane), n), at + 4 * TILE + n * 1024);
        }
    };
    // of the next tile's head: its queries, dO and their sums
    const char* q_head = static_cast<const char*>(p.q.p) + (b * p.q.sb + hk * p.shared * p.q.sh) * E::BYTES;
    const char* d_head = copied ? reinterpret_cast<const char*>(p.do16) + (static_cast<long>(b) * p.H + hk * p.shared) * nq * D * 2
                                : static_cast<const char*>(p.d_o.p) + (b * p.d_o.sb + hk * p.shared * p.d_o.sh) * E::BYTES;
    const long q_step = p.q.sh * E::BYTES, d_step = copied ? static_cast<long>(nq) * D * 2 : p.d_o.sh * E::BYTES;
    const long q_row = p.q.st * E::BYTES, d_row = d_st * E::BYTES;
    // of its sums: this wave's are lse (wave 0), D (1) or first keys (2)
    const long sums = (static_cast<long>(b) * p.H + hk * p.shared) * nq;
    const char* s_head = reinterpret_cast<const char*>(wave == 0 ? p.lse2 + sums : wave == 1 ? p.delta + sums : nullptr);
    const long s_step = wave < 2 ? 4L * nq : 0;
    if (wave == 2 && p.first) s_head = reinterpret_cast<const char*>(p.first + static_cast<long>(b) * nq);
    auto load_tile = [&](int t, int buffer) __attribute__((always_inline)) {
        const uint32_t dst = at + buffer * 2 * TILE + wave * DMAS * 1024;
        const int ln = opaque(lane), r = ln / TL::CHUNKS;
        const uint32_t chunk = TL::lane_chunk(ln), q_part = r * static_cast<uint32_t>(q_row), d_part = r * static_cast<uint32_t>(d_row);
        if (t * QT + QT <= nq) {
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                const int n = wave * DMAS + i;
                const long row = t * QT + n * RPD;
                to_lds(q_head + row * q_row, TL::lane_offset(q_part, chunk, n), dst + i * 1024);
                to_lds(d_head + row * d_row, TL::lane_offset(d_part, chunk, n), dst + TILE + i * 1024);
            }
        } else {  // queries behind the last repeat it, unseen
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                const int n = wave * DMAS + i;
                const long row = min(t * QT + n * RPD + r, nq - 1);
                to_lds(q_head + row * q_row + TL::lane_offset(0, chunk, n), dst + i * 1024);
                to_lds(d_head + row * d_row + TL::lane_offset(0, chunk, n), dst + TILE + i * 1024);
            }
        }
        if (s_head) to_lds4(s_head + 4L * QT * t, 4 * min(ln, nq - 1 - t * QT), lds_address(&stats[buffer][wave][0]));
    };

    // A block of 32 queries from i0.  `partly`: some may not see all of the wave's keys; queries
    // and their dO that are not finite are then taken out of the products for keys that they
    // do not see, and reach the others through P and D.
    auto block = [&](int i0, uint32_t qt, const float* lses, auto partly) __attribute__((always_inline)) {
        constexpr bool PARTLY = decltype(partly)::value;
        // (nothing that follows from the lane stays from block to block: there is no register for it)
        const uint32_t row = opaque(row_base), column = opaque(column_base);
        const uint32_t qr = qt + row, qc = qt + column, dr = qr + TILE, dc = qc + TILE;
        const uint32_t vr = at + 4 * TILE + 32 * wave * TL::ROW + row;
        const float* deltas = lses + 64;
        f32x16 s, dp;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const Frag f = TL::rows(qr, 0, st);
            s = E::mma(f, k[st], s);
        }
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const Frag f = TL::rows(dr, 0, st);
            dp = E::mma(f, TL::rows(vr, 0, st), dp);
        }
        bool dirty = false;
        if constexpr (PARTLY) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) any |= !(fabsf(s[i]) < INFINITY) || !(fabsf(dp[i]) < INFINITY);
            dirty = __ballot(any) != 0;
        }
        Frag pf[2], df[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x4 lse = *reinterpret_cast<const f32x4*>(lses + 8 * e + 4 * h);
            const f32x4 dl = *reinterpret_cast<const f32x4*>(deltas + 8 * e + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = 4 * e + i;
                s[x] = ex2(fmaf(s[x], p.c, -lse[i]));
                dp[x] = s[x] * (dp[x] - dl[i]);
                if constexpr (PARTLY)
                    if (dirty) s[x] += 0.0f * dl[i];
            }
        }
        if constexpr (PARTLY) {
            // query r of the block sees the key from r = from on, to the window's end, and
            // where its first key is not behind it
            const int from = opaque(key - off - i0 - 4 * h);
            int to = nq - i0 - 4 * h;
            if (p.window > 0) to = min(to, from + p.window);
            if (key >= nk) to = INT32_MIN;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 first = *reinterpret_cast<const f32x4*>(deltas + 64 + 8 * e + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 4 * e + i, r = 8 * e + i;
                    const bool seen = (r >= from) & (r < to) & (__float_as_int(first[i]) <= key);
                    if (!seen) s[x] = dp[x] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            pf[u] = E::of(s, u);
            df[u] = E::of(dp, u);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Frag x = TL::columns(dc, 16 * u, c), y = TL::columns(qc, 16 * u, c);
                if constexpr (PARTLY)
                    if (dirty) {
                        x = E::finite(x);
                        y = E::finite(y);
                    }
                dv[c] = E::mma(x, pf[u], dv[c]);
                dk[c] = E::mma(y, df[u], dk[c]);
            }
    };

    // The tiles of each head in turn, QT / 32 blocks each (one: written without these loops the
    // compiler's order of the masked block costs the pass 2%); runs of those whose queries all see
    // all of the wave's keys in a loop of their own.
    const int w0 = key0 + 32 * wave, w1 = w0 + 31;  // this wave's keys
    int count = end > begin ? (end - begin) * p.shared : 0, t = begin;
    if (PARTS && count > 0) {  // this part of them
        const int each = (count + splits - 1) / splits, from = min(split * each, count), g = from / (end - begin);
        count = min(each, count - from);
        t = begin + from - g * (end - begin);
        q_head += g * q_step;
        d_head += g * d_step;
        s_head += g * s_step;
    }
    int n = 0, i0 = 0, buffer = 1;  // tiles begun; the present one's first query and place
    bool partly = false;
    auto next = [&]() __attribute__((always_inline)) {
        landed();
        if (n == count) {
            n = count + 1;  // none is left
            return;
        }
        i0 = t * QT;
        buffer ^= 1;
        __syncthreads();
        if (++t == end) {
            t = begin;
            q_head += q_step;
            d_head += d_step;
            s_head += s_step;
        }
        if (++n < count) load_tile(t, buffer ^ 1);
        const int p0 = i0 + off;
        partly = i0 + QT > nq || p0 < w1 || (p.window > 0 && p0 + QT - 1 - p.window >= w0) ||
                 (p.first && __ballot(__float_as_int(stats[buffer][2][lane % QT]) > w0) != 0);
    };
    if (count > 0) {
        load_values();
        load_tile(t, 0);
    }
    next();
    while (n <= count && count > 0) {
        for (; n <= count && partly; next()) {
#pragma unroll 1
            for (int e = 0; e < QT / 32; ++e) {
                const int i = i0 + 32 * e, p0 = i + off;
                if (i < nq && p0 + 31 >= w0 && !(p.window > 0 && p0 - p.window >= w1))
                    block(i, at + buffer * 2 * TILE + 32 * e * TL::ROW, &stats[buffer][0][32 * e], std::true_type());
            }
        }
        for (; n <= count && !partly; next()) {
#pragma unroll
            for (int e = 0; e < QT / 32; ++e)
                block(0, at + buffer * 2 * TILE + 32 * e * TL::ROW, &stats[buffer][0][32 * e], std::false_type());
        }
    }
    if (key >= nk) return;
    const long row = (static_cast<long>(b) * p.Hk + hk) * nk + key;
    const long ko = !PARTS ? b * p.dk.sb + hk * p.dk.sh + key * p.dk.st : (split * p.rows + row) * D;
    const long vo = !PARTS ? b * p.dv.sb + hk * p.dv.sh + key * p.dv.st : ((splits + split) * p.rows + row) * D;
    const float scale = !PARTS ? p.scale : 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f32x4 x, y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = dk[c][4 * e + i] * scale;
                y[i] = dv[c][4 * e + i];
            }
            if constexpr (!PARTS) {
                store4<BF16>(p.dk.p, ko + 32 * c + 8 * e + 4 * h, p.g_f32, x);
                store4<BF16>(p.dv.p, vo + 32 * c + 8 * e + 4 * h, p.g_f32, y);
            } else {
                store4<false>(p.part, ko + 32 * c + 8 * e + 4 * h, 1, x);
                store4<false>(p.part, vo + 32 * c + 8 * e + 4 * h, 1, y);
            }
        }
}

// The parts' sums of each row added up, in their order: D / 4 lanes to a row.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) attn_add_parts_kernel(const float* part, int splits, long rows, Out4 out, int heads, int T, float scale,
                                                                  int f32) {
    constexpr int LPR = D / 4;
    const long row = (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / LPR;
    if (row >= rows) return;
    const int ch = 4 * (threadIdx.x % LPR);
    const long bh = row / T, b = bh / heads;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) x += *reinterpret_cast<const f32x4*>(part + (s * rows + row) * D + ch);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= scale;
    store4<BF16>(out.p, b * out.sb + (bh - b * heads) * out.sh + (row - bh * T) * out.st + ch, f32, x);
}

size_t up256(size_t n) { return (n + 255) & ~size_t{255}; }

int query_tiles(int Tq) { return (Tq + kQueries - 1) / kQueries; }

// Where the grid of a pass would leave much of the device idle, at its end above all, what
// each of its workgroups goes over (keys for dq, queries of the heads for dk and dv) is dealt
// to `splits` of them: bf16 to four workgroups a compute unit (B2 H16/4 T2048 d128 241 us
// with two, 203 with four, 298 with eight), fp32, whose steps take three times as long, to
// two (B4 H8/2 T1000 d64 148 us, with four 153; B3 T1237 181 and 176) of half the length (B3
// T1000 137 us, 158 of the same length).
constexpr int kMaxSplits = 32;

int splits_of(bool bf16, long groups, long steps) {  // steps: blocks of 32 that a workgroup goes over
    const long fill = bf16 ? 1024 : 512, most = steps / (bf16 ? 16 : 8);
    long n = groups < fill ? (fill + groups - 1) / groups : 1;
    if (n > most) n = most;
    if (n > kMaxSplits) n = kMaxSplits;
    return n > 1 ? static_cast<int>(n) : 1;
}

struct Layout {
    int q_splits, k_splits;
    size_t delta, lse2, do16, first_least, part, bytes;  // offsets in the workspace
};

Layout layout(const pdn_attn_bwd_args& a) {
    const pdn_attn_args& f = a.fwd;
    const size_t rows = static_cast<size_t>(f.B) * f.H * f.Tq, keys = static_cast<size_t>(f.B) * f.Hk * f.Tk;
    const long heads = static_cast<long>(f.B) * f.Hk, shared = f.H / f.Hk, window = f.window > 0 && f.window < f.Tk ? f.window : f.Tk;
    Layout l{};
    l.q_splits = f.Tq > 0 ? splits_of(f.dtype == PDN_BF16, heads * ((f.Tq * shared + 127) / 128), window / 32) : 1;
    l.k_splits = f.Tk > 0 ? splits_of(f.dtype == PDN_BF16, heads * ((f.Tk + 127) / 128), shared * query_tiles(window < f.Tq ? static_cast<int>(window) : f.Tq)) : 1;
    l.lse2 = up256(rows * sizeof(float));
    l.do16 = 2 * l.lse2;
    l.first_least = l.do16 + (f.dtype == PDN_BF16 && f.o_dtype == PDN_F32 ? up256(rows * f.d * 2) : 0);
    l.part = l.first_least + (f.first ? up256(static_cast<size_t>(f.B) * query_tiles(f.Tq) * sizeof(int)) : 0);
    // dq's parts have been added up before dk's and dv's are formed
    const size_t q = l.q_splits > 1 ? l.q_splits * rows * f.d * sizeof(float) : 0;
    const size_t k = l.k_splits > 1 ? 2 * l.k_splits * keys * f.d * sizeof(float) : 0;
    l.bytes = l.part + up256(q > k ? q : k);
    return l;
}

template <bool BF16, int D>
hipError_t add_parts(const BwdParams& p, const float* part, const Out4& out, int heads, int T, float scale, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.rows * (D / 4) + kThreads - 1) / kThreads)), block(kThreads);
    attn_add_parts_kernel<BF16, D><<<grid, block, 0, stream>>>(part, p.splits, p.rows, out, heads, T, scale, p.g_f32);
    return hipGetLastError();
}

template <bool BF16, int D>
hipError_t launch(BwdParams p, int B, const Layout& l, hipStream_t stream) {
    const long heads = static_cast<long>(B) * p.Hk;
    const dim3 block(kThreads);
    hipError_t rc = hipSuccess;
    if (p.Tq > 0) {
        const long rows = static_cast<long>(p.Tq) * p.shared;
        p.tiles = static_cast<int>((rows + 127) / 128);
        p.splits = l.q_splits;
        p.rows = rows * heads;
        attn_dq_kernel<BF16, D><<<dim3(static_cast<unsigned>(heads * p.tiles * p.splits)), block, 0, stream>>>(p);
        rc = hipGetLastError();
        if (rc == hipSuccess && p.splits > 1) rc = add_parts<BF16, D>(p, p.part, p.dq, p.H, p.Tq, p.scale, stream);
    }
    if (p.Tk > 0 && rc == hipSuccess) {
        p.tiles = (p.Tk + 127) / 128;
        p.splits = l.k_splits;
        p.rows = heads * p.Tk;
        const dim3 grid(static_cast<unsigned>(heads * p.tiles * p.splits));
        if (p.splits > 1) attn_dkv_kernel<BF16, D, true><<<grid, block, 0, stream>>>(p);
        else attn_dkv_kernel<BF16, D, false><<<grid, block, 0, stream>>>(p);
        rc = hipGetLastError();
        if (rc == hipSuccess && p.splits > 1) rc = add_parts<BF16, D>(p, p.part, p.dk, p.Hk, p.Tk, p.scale, stream);
        if (rc == hipSuccess && p.splits > 1) rc = add_parts<BF16, D>(p, p.part + p.splits * p.rows * D, p.dv, p.Hk, p.Tk, 1.0f, stream);
    }
    return rc;
}

}  // namespace

size_t attn_bwd_workspace_bytes(const pdn_attn_bwd_args& a) { return layout(a).bytes; }

hipError_t launch_attn_bwd(const pdn_attn_bwd_args& a, hipStream_t stream) {
    const pdn_attn_args& f = a.fwd;
    const Layout l = layout(a);
    char* ws = static_cast<char*>(a.workspace);
    BwdParams p{};
    p.q = {f.q, f.q_sb, f.q_sh, f.q_st};
    p.k = {f.k, f.k_sb, f.k_sh, f.k_st};
    p.v = {f.v, f.v_sb, f.v_sh, f.v_st};
    p.o = {f.o, f.o_sb, f.o_sh, f.o_st};
    p.d_o = {a.d_o, a.do_sb, a.do_sh, a.do_st};
    p.dq = {a.dq, a.dq_sb, a.dq_sh, a.dq_st};
    p.dk = {a.dk, a.dk_sb, a.dk_sh, a.dk_st};
    p.dv = {a.dv, a.dv_sb, a.dv_sh, a.dv_st};
    p.lse = f.lse;
    p.first = f.first;
    p.delta = reinterpret_cast<float*>(ws + l.delta);
    p.lse2 = reinterpret_cast<float*>(ws + l.lse2);
    p.do16 = reinterpret_cast<uint16_t*>(ws + l.do16);
    p.first_least = reinterpret_cast<int*>(ws + l.first_least);
    p.H = f.H;
    p.Hk = f.Hk;
    p.shared = f.H / f.Hk;
    p.inverse = inverse_of(p.shared);
    p.Tq = f.Tq;
    p.Tk = f.Tk;
    p.window = f.window < f.Tk ? f.window : 0;  // as far as there are keys: all of them
    p.scale = f.scale;
    p.c = f.scale * kLog2e;
    p.o_f32 = f.o_dtype == PDN_F32;
    p.g_f32 = a.g_dtype == PDN_F32;
    p.query_tiles = query_tiles(f.Tq);
    if (f.first && f.Tq > 0) {
        first_least_kernel<<<dim3(static_cast<unsigned>(f.B * p.query_tiles)), dim3(64), 0, stream>>>(f.first, f.Tq, p.query_tiles, p.first_least);
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    p.part = reinterpret_cast<float*>(ws + l.part);
    if (f.dtype == PDN_BF16) return f.d == 64 ? launch<true, 64>(p, f.B, l, stream) : launch<true, 128>(p, f.B, l, stream);
    return f.d == 64 ? launch<false, 64>(p, f.B, l, stream) : launch<false, 128>(p, f.B, l, stream);
}

}  // namespace pdn
