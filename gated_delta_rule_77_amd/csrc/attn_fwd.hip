// Causal softmax attention, over contiguous keys and over a paged cache:
//
//   o_i = sum_j exp(c (s_ij - m_i)) v_j / sum_j exp(c (s_ij - m_i)),  s = <q, k>,
//
// one pass over the keys with a running maximum m and sum.  The heads that share a
// key head are rows of one tile beside the tokens (row = token * shared + head), so
// that a tile of keys is read once for all of them and a tile's diagonal is short.
//
// A workgroup is four waves.  WK = 1: each wave holds 32 rows of its own and the
// waves share tiles of KT keys in LDS, loaded one tile ahead past the registers.
// WK > 1 (few rows, a decode step above all): WK waves share the rows, each takes
// its part of every tile's keys, and their sums are joined at the end.  Where the
// grid would not fill the device, the keys are dealt to `splits` workgroups, whose
// sums a second kernel joins.
//
// Many rows are bound by the units that turn scores into probabilities beside those that
// multiply: of the cycles of B4 H16/4 T8192 d128 in bf16 the matrix units take 57%, the
// vector units 52% (1031 us, 1.07 PFLOP/s; a window of 2048 over T65536 0.92 to 0.96).  Two waves a
// SIMD cover each other; 64 rows a wave, which halve the reads of LDS (29% of its cycles),
// leave no registers for a second and ran at 470 TFLOP/s.  fp32 is bound by forming parts
// (vector units 65%, matrix units 37%).  Few rows are bound by the keys' bytes: 256
// sequences of 2048 to 8192 tokens, H16/4 d128, 2.7 GB at 5.4 TB/s.
#include "attn.h"
#include "block.h"
#include "layer.h"
#include "pages.h"

namespace pdn {
namespace {

using namespace attn;

struct FwdParams {
    const void *q, *k, *v;
    void* o;
    float* lse;
    const int32_t* first;
    long q_sb, q_sh, q_st, k_sb, k_sh, k_st, v_sb, v_sh, v_st, o_sb, o_sh, o_st;
    int H, Hk, shared;   // query heads, key heads, H / Hk
    uint32_t inverse;    // of `shared`
    int Tq, Tk;
    int window;
    float c;             // scale * log2(e)
    int o_f32;
    int tiles, splits;   // of rows; of the keys
    float* part;         // splits > 1: [splits][rows][D] sums, then [splits][rows][2] (maximum, sum; kNoPart: no tiles, no sums)
    long rows;           // B H Tq
    // paged: q_st, o_st step rows of N; k_sb, v_sb step pages
    PageMap map;
};

constexpr int kThreads = 256;
constexpr int kMaxSplits = 128;
// Parts that a row's lanes join one after another; more of them are joined by a workgroup a
// row (64 parts of one token, H16: call of 58 and 34 us; 4 parts of 16 tokens the same).
constexpr int kFewParts = 8;
// In the place of a sum of exponentials: the part had no keys, and its sums are unwritten.
// (Sums that are there count however small their weight is, as 0 times a value that is not
// finite does.)
constexpr float kNoPart = -1.0f;
// A row's maximum is moved (and its sums scaled) when a score passes it by this
// much, in powers of two: until then the exponentials stay below 2^8 (times what the
// rounding of the subtrahend makes of it), well inside fp32 for values up to 2^119 / Tk and, as
// bf16 factors, as exact as any (B4 H16/4 T8192 1053 us, 1100 where every larger score moves it).
constexpr float kSlack = 8.0f;

// Chunks of few sequences of a paged cache: the longest sequence's workgroups are dealt
// first, so that the last to start are short ones (8 sequences of up to 512 new and 16384
// tokens 288 us in the given order, 245 so; 16 of up to 256 and 8192 164 and 115; 32 of up
// to 128 and 4096 122 and 106).  Every workgroup finds its sequence by itself, which with
// many of them costs more than it gives (32 of one length 174 and 178 us, 64 of different
// lengths 148 and 156).
constexpr int kRanked = 32;

// Which of the sequences (as many as a wave has lanes at the most) is the r-th longest, the
// earlier first among equals.
__device__ __forceinline__ int by_length(const PageMap& m, int r, int lane) {
    const Sequence s = sequence_of(m, min(lane, m.B - 1));
    const int len = s.n > 0 ? s.len : 0;
    int rank = 0;
    for (int j = 0; j < m.B; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += (other > len) | ((other == len) & (j < lane));
    }
    return __builtin_ctzll(__ballot((lane < m.B) & (rank == r)));
}

template <bool BF16, int D, int WK, int KT, bool PAGED>
__global__ void __launch_bounds__(kThreads, (BF16 || D == 64) && KT * D * El<BF16>::BYTES < 32768 ? 2 : 1) attn_fwd_kernel(FwdParams p) {
    using E = El<BF16>;
    using TL = Tile<BF16, D>;
    typedef typename E::Frag Frag;
    constexpr int WR = 4 / WK;                 // waves with rows of their own
    constexpr int ROWS = 32 * WR;              // of the workgroup
    constexpr int KB = KT / 32 / WK;           // a wave's blocks of 32 keys in a tile
    constexpr int S = D / 16, C = D / 32;
    constexpr int TILE = KT * TL::ROW, DMAS = KT / TL::ROWS_PER_DMA / 4;
    constexpr bool ALONE = WK == 4 && KB == 1;  // a wave reads the 32 rows of each tile that it loads
    static_assert(KB >= 1 && DMAS >= 1, "every wave has keys to read and rows to load");
    __shared__ __align__(1024) char smem[4 * TILE];  // keys and values of two tiles: one being read, one being loaded
    __shared__ int bounds[2][4];
    __shared__ float joined[WK > 1 ? 2 : 1][WK > 1 ? 4 : 1][32];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int h = lane >> 5;
    // Key heads first: their workgroups are dealt over the XCDs, so that every XCD (and every
    // part of it) has its share of each sequence, whatever their lengths, and a head's keys
    // are in as few L2s as that allows.  Then the sequences, the parts of the keys and the tiles
    // of rows, those with the most keys first, so that the last to start are short ones (tiles
    // before sequences: B2 H16/4 T2048 d128 66 us, 56 so; fp32 B2 H8 T2048 d64 152 and 113; B4
    // H16/4 T8192 d128 1036 and 1027; fp32 B3 H8/2 T1237 after 100 d64 79 and 84).  A cache's
    // sequences, of lengths of their own, come one after another.
    const int hk = blockIdx.x % p.Hk, rest = blockIdx.x / p.Hk;
    int b, split, tile;
    if constexpr (PAGED) {
        split = rest % p.splits;
        tile = p.tiles - 1 - rest / p.splits % p.tiles;
        b = rest / p.splits / p.tiles;
    } else {
        const int batch = gridDim.x / (p.Hk * p.splits * p.tiles);
        b = rest % batch;
        split = rest / batch % p.splits;
        tile = p.tiles - 1 - rest / batch / p.splits;
    }
    if constexpr (PAGED && WK == 1)
        if (p.map.B <= kRanked) b = by_length(p.map, b, lane);

    int nq = p.Tq, nk = p.Tk;
    const char *qb = static_cast<const char*>(p.q), *kb = static_cast<const char*>(p.k), *vb = static_cast<const char*>(p.v);
    long orow = 0;   // of the sequence's token 0
    if constexpr (PAGED) {
        const Sequence sq = sequence_of(p.map, b);
        nq = min(sq.n, p.Tq);
        nk = sq.len;
        const int behind = sq.n - nq;  // tokens past what the launch was sized for stay out
        nk = max(nk - behind, 0);
        qb += sq.start * p.q_st * E::BYTES;
        orow = sq.start;
    } else {
        qb += b * p.q_sb * E::BYTES;
        kb += b * p.k_sb * E::BYTES;
        vb += b * p.v_sb * E::BYTES;
    }
    kb += hk * p.k_sh * E::BYTES;
    vb += hk * p.v_sh * E::BYTES;
    const int row0 = tile * ROWS, nrows = nq * p.shared;
    if (row0 >= nrows) return;

    // this lane's row: its token, head and keys; rows behind the last repeat it, unstored
    const int t0 = row0 / p.shared, m0 = row0 - t0 * p.shared;
    const int dr = 32 * (wave / WK) + (lane & 31);
    const bool stored = row0 + dr < nrows;
    const int r = m0 + (stored ? dr : nrows - 1 - row0), dt = quotient(r, p.inverse), token = t0 + dt, head = hk * p.shared + r - dt * p.shared;
    const Seen seen = seen_by(token, nq, nk, p.window, !PAGED && p.first ? p.first[static_cast<long>(b) * p.Tq + token] : 0);
    int low = INT32_MAX, high = -1, full_low = 0, full_high = INT32_MAX;
    if (seen.count > 0) {
        const int last = seen.low + seen.count - 1;
        low = min(low, seen.low);
        high = max(high, last);
        full_low = max(full_low, seen.low);
        full_high = min(full_high, last);
    }
    Frag q[S];
#pragma unroll
    for (int s = 0; s < S; ++s) q[s] = E::load(qb + (token * p.q_st + head * p.q_sh) * E::BYTES, 16 * s + 8 * h);
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

    // A tile's rows to LDS: a wave's loads of RPD rows each, 16 bytes a lane, the source
    // chunk swizzled.  Such rows lie at one stride from a uniform address, on one page of a
    // cache too; those of a tile that passes the last key repeat it, unseen.
    constexpr int RPD = TL::ROWS_PER_DMA;
    const uint32_t chunk = TL::lane_chunk(lane);
    const uint32_t k_part = static_cast<uint32_t>(lane / TL::CHUNKS * p.k_st * E::BYTES), v_part = static_cast<uint32_t>(lane / TL::CHUNKS * p.v_st * E::BYTES);
    // The sequence's pages, 64 a lane at a time and the next 64 behind them, so that no tile
    // waits for the table.  A load's rows lie on one page (16 tokens at the least).
    int pages = 0, ahead = 0, pages_at = 0;
    auto fetch_pages = [&](int at) __attribute__((always_inline)) {
        return page_of(p.map, b, min((at + lane) << p.map.shift, nk - 1));
    };
    auto place = [&](int first, int key, long& ko, long& vo) __attribute__((always_inline)) {  // of a token in the load that begins at `first`
        if constexpr (PAGED) {
            const int n = uniform(min(first, nk - 1) >> p.map.shift);
            if (n >= pages_at + 64) {
                pages_at += 64;
                pages = ahead;
                ahead = fetch_pages(pages_at + 64);
            }
            const long page = __builtin_amdgcn_readlane(pages, n - pages_at);
            const int in = key & ((1 << p.map.shift) - 1);
            ko = page * p.k_sb + in * p.k_st;
            vo = page * p.v_sb + in * p.v_st;
        } else {
            ko = key * p.k_st;
            vo = key * p.v_st;
        }
    };
    auto load_tile = [&](int t, int buffer) __attribute__((always_inline)) {
        const uint32_t dst = at + buffer * 2 * TILE + wave * DMAS * 1024;
        if (t * KT + KT <= nk) {
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                long ko, vo;
                place(t * KT + (wave * DMAS + i) * RPD, t * KT + (wave * DMAS + i) * RPD, ko, vo);
                to_lds(kb + ko * E::BYTES, TL::lane_offset(k_part, chunk, wave * DMAS + i), dst + i * 1024);
                to_lds(vb + vo * E::BYTES, TL::lane_offset(v_part, chunk, wave * DMAS + i), dst + TILE + i * 1024);
            }
        } else {
#pragma unroll
            for (int i = 0; i < DMAS; ++i) {
                const int n = wave * DMAS + i;
                const uint32_t in_row = TL::lane_offset(0, chunk, n);
                long ko, vo;
                place(t * KT + n * RPD, min(t * KT + n * RPD + lane / TL::CHUNKS, nk - 1), ko, vo);
                to_lds(kb + ko * E::BYTES + in_row, dst + i * 1024);
                to_lds(vb + vo * E::BYTES + in_row, dst + TILE + i * 1024);
            }
        }
    };

    // 0 v, summed over the channels, of a block's keys: a result's rows
    auto times_zero = [&](uint32_t vr) __attribute__((always_inline)) {
        f32x16 x;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll
        for (int st = 0; st < S; ++st) x = E::mma(TL::rows(vr, 0, st), E::zero(), x);
        return x;
    };
    auto not_finite = [&](uint32_t vr) __attribute__((always_inline)) {
        const f32x16 x = times_zero(vr);
        bool any = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) any |= x[i] != x[i];
        return __ballot(any);
    };

    f32x16 acc[C];
    // the maximum, and what its exponentials go by; the score that moves it; this half wave's part of the sum
    float ref = -INFINITY, by = p.c, m = 0.0f, limit = -INFINITY, sum = 0.0f;
    const float slack = kSlack / p.c;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] = 0.0f;

    // The maximum moved where a row's scores pass it (each row by itself: what another
    // holds has no part in its rounding either).
    auto move = [&](float top) __attribute__((always_inline)) {
        const bool moves = top > limit;
        if (__ballot(moves) == 0) return;
        const float to = moves ? top : ref, keep = weight(ref, to, p.c);
        const Shift shift = shift_of(to, p.c);
        ref = to;
        limit = to + slack;
        by = shift.c;
        m = to == -INFINITY ? 0.0f : shift.m;
        sum *= keep;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c][i] *= keep;
    };

    // a block of 32 keys of which some rows may not see all
    auto some_seen = [&](int k0, uint32_t kt, uint32_t vt) __attribute__((always_inline)) {
        if (k0 > high || k0 + 31 < low) return;
        const uint32_t kr = kt + row_base, vr = vt + row_base, vc = vt + column_base;
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int st = 0; st < S; ++st) {
            const Frag kf = TL::rows(kr, 0, st);
            s = E::mma(kf, q[st], s);
        }
        // Unseen keys: no part in the maximum, a probability of zero.  Zero times a value
        // that is not finite would still be NaN: such values (which 0 v shows) are taken out
        // of the product, and make the probabilities of those that see them NaN instead.
        const bool dirty = not_finite(vr) != 0;
        const Seen to = {opaque(seen.low - k0 - 4 * h), seen.count};
        float x = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (!sees(to, 8 * (i >> 2) + (i & 3))) s[i] = -INFINITY;
            x = fmaxf(x, s[i]);
        }
        move(halves<true>(x));
        Frag pf[2];
        float add = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = ex2(fmaf(s[i], by, -m));
            add += s[i];
        }
        sum += add;
        if (dirty) {
            const f32x16 poison = times_zero(vr);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (sees(to, 8 * (i >> 2) + (i & 3))) s[i] += poison[i];
        }
        pf[0] = E::of(s, 0);
        pf[1] = E::of(s, 1);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Frag vf = TL::columns(vc, 16 * u, c);
                if (dirty) vf = E::finite(vf);
                acc[c] = E::mma(vf, pf[u], acc[c]);
            }
    };

    // a wave's keys of a tile that all its rows see
    auto all_seen = [&](uint32_t kt, uint32_t vt) __attribute__((always_inline)) {
        const uint32_t kr = kt + row_base, vc = vt + column_base;
        f32x16 s[KB];
#pragma unroll
        for (int e = 0; e < KB; ++e) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[e][i] = 0.0f;
#pragma unroll
            for (int st = 0; st < S; ++st) {
                const Frag kf = TL::rows(kr, 32 * e, st);
                s[e] = E::mma(kf, q[st], s[e]);
            }
        }
        float x = s[0][0];
#pragma unroll
        for (int e = 0; e < KB; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) x = fmaxf(x, s[e][i]);
        move(halves<true>(x));
        Frag pf[KB][2];
#pragma unroll
        for (int e = 0; e < KB; ++e) {
            float add = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[e][i] = ex2(fmaf(s[e][i], by, -m));
                add += s[e][i];
            }
            sum += add;
            pf[e][0] = E::of(s[e], 0);
            pf[e][1] = E::of(s[e], 1);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < KB; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Frag vf = TL::columns(vc, 32 * e + 16 * u, c);
                    acc[c] = E::mma(vf, pf[e][u], acc[c]);
                }
    };

    // The tiles in order; those that all of the wave's rows see whole in a loop of their own.
    const int rw = 32 * KB * (wave % WK);  // the wave's first row of a tile
    int t = first_tile;
    auto next = [&](uint32_t& kt) __attribute__((always_inline)) {
        const int buffer = (t - first_tile) & 1;
        if constexpr (ALONE) {
            if (t + 1 < end_tile) landed_but<2 * DMAS>();
            else landed_but<0>();
        } else {
            landed();
            __syncthreads();  // every wave's part of the tile; and the other buffer has been read
            if (t + 1 < end_tile) load_tile(t + 1, buffer ^ 1);
        }
        kt = at + buffer * 2 * TILE;
    };
    // A wave that reads the rows that it loads itself goes at its own pace, without barriers,
    // and loads two tiles ahead, into the place that it has just read.
    auto done = [&]() __attribute__((always_inline)) {
        if constexpr (ALONE) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (t + 2 < end_tile) load_tile(t + 2, (t - first_tile) & 1);
        }
    };
    auto some = [&](int end) __attribute__((always_inline)) {
        for (; t < end; ++t) {
            uint32_t kt;
            next(kt);
#pragma unroll 1
            for (int e = 0; e < KB; ++e) some_seen(t * KT + rw + 32 * e, kt + (rw + 32 * e) * TL::ROW, kt + TILE + (rw + 32 * e) * TL::ROW);
            done();
        }
    };
    int from = (full_low - rw + KT - 1) / KT, to = (full_high + 1 - rw - 32 * KB) / KT + 1;  // whole tiles from .. to - 1
    from = max(from, first_tile);
    to = min(full_high + 1 < rw + 32 * KB ? first_tile : to, end_tile);
    if (low == INT32_MAX || from >= to) from = to = end_tile;
    if (first_tile < end_tile) {
        if constexpr (PAGED) {
            pages_at = uniform((min(first_tile * KT, nk - 1) >> p.map.shift) & ~63);
            pages = fetch_pages(pages_at);
            ahead = fetch_pages(pages_at + 64);
        }
        landed();
        load_tile(first_tile, 0);
        if (ALONE && first_tile + 1 < end_tile) load_tile(first_tile + 1, 1);
    }
    some(min(from, end_tile));
    for (; t < to; ++t) {
        uint32_t kt;
        next(kt);
        all_seen(kt + rw * TL::ROW, kt + TILE + rw * TL::ROW);
        done();
    }
    some(end_tile);
    sum = halves<false>(sum);

    // a row of the sums
    auto index = [&]() { return (static_cast<long>(b) * p.H + head) * p.Tq + token; };
    auto store4 = [&](int ch, f32x4 x) {  // four channels of one row
        if (p.splits > 1) {
            if (first_tile < end_tile) *reinterpret_cast<f32x4*>(p.part + (split * p.rows + index()) * D + ch) = x;
            return;
        }
        const long at = (PAGED ? (orow + token) * p.o_st : b * p.o_sb + token * p.o_st) + head * p.o_sh + ch;
        if (!BF16 || p.o_f32) {
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.o) + at) = x;
        } else {
            *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(p.o) + at) = __builtin_convertvector(x, bf16x4);
        }
    };
    auto store_sums = [&](float top, float l) {
        if (p.splits > 1) {
            float* ml = p.part + p.splits * p.rows * D + (split * p.rows + index()) * 2;
            ml[0] = seen.count > 0 ? top : -INFINITY;
            ml[1] = first_tile >= end_tile ? kNoPart : seen.count > 0 ? l : 0.0f;
        } else if (p.lse) {
            p.lse[PAGED ? (orow + token) * p.H + head : index()] = seen.count > 0 ? log_of(top, l, p.c) : -INFINITY;
        }
    };
    // what turns a row's sums into its output (or leaves them, for the join)
    auto norm = [&](float l) { return p.splits > 1 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l; };

    if constexpr (WK == 1) {
        if (!stored) return;
        const bool none = seen.count == 0;
        const float n = norm(sum);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = none ? 0.0f : acc[c][4 * g + i] * n;
                store4(32 * c + 8 * g + 4 * h, x);
            }
        if (h == 0) store_sums(ref, sum);
    } else {
        // The WK waves of a row: their maxima and sums, then their scaled sums by channel
        // through the tiles' memory.  A wave adds up D / WK of the channels.
        static_assert(4 * TILE >= 4 * 32 * (D + 4) * 4, "the waves' sums fit the tiles' memory");
        if (h == 0) {
            joined[0][wave][lane & 31] = ref;
            joined[1][wave][lane & 31] = sum;
        }
        __syncthreads();
        const int w0 = wave / WK * WK;
        float top = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < WK; ++w) top = fmaxf(top, joined[0][w0 + w][lane & 31]);
#pragma unroll
        for (int w = 0; w < WK; ++w) l += joined[1][w0 + w][lane & 31] * weight(joined[0][w0 + w][lane & 31], top, p.c);
        const float keep = weight(ref, top, p.c);
        float* mine = reinterpret_cast<float*>(smem) + (wave * 32 + (lane & 31)) * (D + 4);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = acc[c][4 * g + i] * keep;
                *reinterpret_cast<f32x4*>(mine + 32 * c + 8 * g + 4 * h) = x;
            }
        __syncthreads();
        if (!stored) return;
        const bool none = seen.count == 0;
        const float n = norm(l);
        constexpr int PART = D / WK;
#pragma unroll
        for (int j = 0; j < PART / 8; ++j) {
            const int ch = (wave % WK) * PART + 8 * j + 4 * h;
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WK; ++w)
                x += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(smem) + ((w0 + w) * 32 + (lane & 31)) * (D + 4) + ch);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = none ? 0.0f : x[i] * n;
            store4(ch, x);
        }
        if (h == 0 && wave % WK == 0) store_sums(top, l);
    }
}

// The splits' sums of each row joined: D / 4 lanes to a row.
struct JoinParams {
    const float* part;
    void* o;
    float* lse;
    long rows, o_sb, o_sh, o_st;
    int splits, H, Tq;
    int o_f32;
    float c;
    PageMap map;
};

// G = 1: D / 4 lanes to a row, which take its parts one after another.  G > 1: a workgroup
// to a row, G groups of such lanes with every G-th part each.  Bound by latency: 5 us for
// two parts of 4096 rows, 6.5 for 64 of 16, d128.
template <int D, int G, bool PAGED>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(JoinParams p) {
    constexpr int LPR = D / 4;
    static_assert(G == 1 || G * LPR == kThreads, "a row is a workgroup's");
    const long row = G > 1 ? blockIdx.x : (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / LPR;
    if (row >= p.rows) return;
    const int ch = 4 * (threadIdx.x % LPR), group = threadIdx.x / LPR;
    const long bh = row / p.Tq, b = bh / p.H, head = bh - b * p.H;
    long t = row - bh * p.Tq, out = row;  // out: of lse
    if constexpr (PAGED) {
        const Sequence s = sequence_of(p.map, static_cast<int>(b));
        if (t >= s.n) return;
        t += s.start;
        out = t * p.H + head;
    }
    const long at = b * p.o_sb + head * p.o_sh + t * p.o_st + ch;
    const float* ml = p.part + p.splits * p.rows * D + row * 2;
    float m = -INFINITY, l = 0.0f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if constexpr (G > 1) {
        __shared__ float weights[kMaxSplits];
        __shared__ float red[2][4];
        __shared__ f32x4 sums[G][LPR];
        const int tid = threadIdx.x, wave = tid >> 6;
        float ms = -INFINITY, ls = kNoPart;
        if (tid < p.splits) {
            ms = ml[tid * p.rows * 2];
            ls = ml[tid * p.rows * 2 + 1];
        }
        float top = ms;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        if ((tid & 63) == 0) red[0][wave] = top;
        __syncthreads();
        m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        const float w = ls == kNoPart ? kNoPart : weight(ms, m, p.c);
        if (tid < p.splits) weights[tid] = w;
        const float part = wave_sum(ls == kNoPart ? 0.0f : ls * w);
        if ((tid & 63) == 0) red[1][wave] = part;
        __syncthreads();
        l = red[1][0] + red[1][1] + red[1][2] + red[1][3];
#pragma unroll 4
        for (int s = group; s < p.splits; s += G) {
            const float by = weights[s];
            if (by != kNoPart) x += *reinterpret_cast<const f32x4*>(p.part + (s * p.rows + row) * D + ch) * by;
        }
        sums[group][threadIdx.x % LPR] = x;
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < G; ++g) x += sums[g][threadIdx.x];
    } else {
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) m = fmaxf(m, ml[s * p.rows * 2]);
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const float ms = ml[s * p.rows * 2], ls = ml[s * p.rows * 2 + 1];
            const f32x4 y = *reinterpret_cast<const f32x4*>(p.part + (s * p.rows + row) * D + ch);
            const float by = weight(ms, m, p.c);
            if (ls != kNoPart) l = fmaf(ls, by, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] += ls == kNoPart ? 0.0f : y[i] * by;
        }
    }
    const bool none = l == 0.0f;
    const float n = none ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= n;
    if (p.o_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p.o) + at) = x;
    else *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(p.o) + at) = __builtin_convertvector(x, bf16x4);
    if (p.lse && ch == 0) p.lse[out] = none ? -INFINITY : log_of(m, l, p.c);
}

// How a call is laid over the device, by its sizes alone.
struct Plan {
    int wk;             // waves that share rows
    int tiles, splits;
};

constexpr long kUnits = 256;  // compute units

// Waves share rows where a call has no more of them than a wave holds (one token of 256
// sequences 560 us, so 501; of one with 65536 tokens 36.4 and 33.8; of one of 1024 17.6 and
// 14.1).  The keys are then dealt until every unit has a workgroup (twice that: 41.9 us for
// the one of 65536), or, where the heads alone give it one, eight of at least 1024 keys, so
// that unequal sequences end together (four 513 us, sixteen 526).  With more rows each unit
// is given two, four for a cache's chunks, whose lengths differ (8 of up to 512 new and 16384
// tokens: with two 388 us, four 272, eight 269; contiguous 512 of 16384 tokens: one 93, two
// 83, four 94).  A part has 512 keys at least, in fp32, whose tiles take three times as long,
// 256, or with more rows 96 while lanes join the parts (500 tokens of 16384, H4/2 d64 with a
// window of 300: one part 32 us, three 20; T1500 H4/2 d64: five 30 us, eight 28, eleven 34; 113
// of up to 11056, B2 H12 d64: eight 92 us, 43 65).  Keys are those that a workgroup can see:
// with a window that and its tokens (bf16 T4096 H4 d128: a window of 64 in one part 14 us, in
// the four that all keys would give 21; of 300 22 and 24).
Plan plan(bool bf16, int d, long heads, long rows, long shared, long keys, long window, bool ragged) {
    Plan p{};
    const bool wide = !bf16 && d == 128;  // 512-byte rows: half the keys to a tile
    p.wk = rows > (wide ? 64 : 32) ? 1 : wide ? 2 : 4;
    const long tile = 32 * (4 / p.wk);
    p.tiles = static_cast<int>((rows + tile - 1) / tile);
    const long groups = heads * p.tiles;
    const long tokens = (rows < tile ? rows : tile) / shared + 1;
    if (window > 0 && window + tokens < keys) keys = window + tokens;
    long splits = 1, most = keys / (bf16 ? 512 : 256);
    if (p.wk > 1 && groups < kUnits) {
        splits = kUnits / groups;
    } else if (p.wk > 1) {
        splits = (8 * kUnits + groups - 1) / groups;
        most = keys / 1024;
    } else if (groups < (ragged ? 4 : 2) * kUnits) {
        splits = ((ragged ? 4 : 2) * kUnits + groups - 1) / groups;
        if (!bf16 && most < kFewParts) most = keys / 96 < kFewParts ? keys / 96 : kFewParts;
    }
    if (splits > most) splits = most;
    if (splits > kMaxSplits) splits = kMaxSplits;
    p.splits = splits > 1 ? static_cast<int>(splits) : 1;
    return p;
}

size_t part_bytes(const Plan& p, long rows, int d) {
    return p.splits > 1 ? static_cast<size_t>(p.splits) * rows * (d + 2) * sizeof(float) : 0;
}

template <bool BF16, int D, bool PAGED>
hipError_t launch_kind(const FwdParams& p, const Plan& pl, long groups, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(groups)), block(kThreads);
    constexpr bool wide = !BF16 && D == 128;
    constexpr int WK = wide ? 2 : 4, KT_FEW = wide ? 64 : 128, KT = BF16 ? 64 : 32;
    if (pl.wk > 1) attn_fwd_kernel<BF16, D, WK, KT_FEW, PAGED><<<grid, block, 0, stream>>>(p);
    else attn_fwd_kernel<BF16, D, 1, KT, PAGED><<<grid, block, 0, stream>>>(p);
    return hipGetLastError();
}

template <bool PAGED>
hipError_t launch(const FwdParams& p, const Plan& pl, int32_t dtype, int d, long heads, hipStream_t stream) {
    const long groups = heads * pl.tiles * pl.splits;
    if (dtype == PDN_BF16) return d == 64 ? launch_kind<true, 64, PAGED>(p, pl, groups, stream) : launch_kind<true, 128, PAGED>(p, pl, groups, stream);
    return d == 64 ? launch_kind<false, 64, PAGED>(p, pl, groups, stream) : launch_kind<false, 128, PAGED>(p, pl, groups, stream);
}

template <bool PAGED>
hipError_t launch_join(const JoinParams& p, int d, hipStream_t stream) {
    const dim3 block(kThreads);
    if (p.splits > kFewParts) {
        const dim3 grid(static_cast<unsigned>(p.rows));
        if (d == 64) attn_join_kernel<64, 16, PAGED><<<grid, block, 0, stream>>>(p);
        else attn_join_kernel<128, 8, PAGED><<<grid, block, 0, stream>>>(p);
    } else {
        const dim3 grid(static_cast<unsigned>((p.rows * (d / 4) + kThreads - 1) / kThreads));
        if (d == 64) attn_join_kernel<64, 1, PAGED><<<grid, block, 0, stream>>>(p);
        else attn_join_kernel<128, 1, PAGED><<<grid, block, 0, stream>>>(p);
    }
    return hipGetLastError();
}

Plan plan_of(const pdn_attn_args& a) {
    const long shared = a.H / a.Hk;
    return plan(a.dtype == PDN_BF16, a.d, static_cast<long>(a.B) * a.Hk, a.Tq * shared, shared, a.Tk, a.window, false);
}

Plan plan_of(const pdn_attn_paged_args& a) {
    const pdn_cache& c = a.cache;
    const long shared = a.H / c.Hk;
    return plan(c.dtype == PDN_BF16, c.d, static_cast<long>(c.B) * c.Hk, c.max_new * shared, shared,
                static_cast<long>(c.table_width) * c.page_size, a.window, true);
}

}  // namespace

// 128 rows to a workgroup (or one workgroup for fewer), 128 keys in the backward, and 32
// queries to a wave of its range kernel; a call with splits is a small one.
bool attn_fits(const pdn_attn_args& a) {
    const long heads = static_cast<long>(a.B) * a.Hk, rows = static_cast<long>(a.Tq) * (a.H / a.Hk);
    return heads * ((rows + 127) / 128 + 1) * kThreads < kMaxGridThreads && heads * ((a.Tk + 127L) / 128) * kThreads < kMaxGridThreads &&
           static_cast<long>(a.B) * ((a.Tq + 31L) / 32) * 64 < kMaxGridThreads;
}

bool attn_paged_fits(const pdn_attn_paged_args& a) {
    const long heads = static_cast<long>(a.cache.B) * a.cache.Hk, rows = static_cast<long>(a.cache.max_new) * (a.H / a.cache.Hk);
    return heads * ((rows + 127) / 128 + 1) * kThreads < kMaxGridThreads;
}

size_t attn_fwd_workspace_bytes(const pdn_attn_args& a) {
    return a.Tq == 0 ? 0 : part_bytes(plan_of(a), static_cast<long>(a.B) * a.H * a.Tq, a.d);
}

hipError_t launch_attn_fwd(const pdn_attn_args& a, hipStream_t stream) {
    if (a.Tq == 0) return hipSuccess;
    const Plan pl = plan_of(a);
    FwdParams p{};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.o = a.o;
    p.lse = a.lse;
    p.first = a.first;
    p.q_sb = a.q_sb, p.q_sh = a.q_sh, p.q_st = a.q_st;
    p.k_sb = a.k_sb, p.k_sh = a.k_sh, p.k_st = a.k_st;
    p.v_sb = a.v_sb, p.v_sh = a.v_sh, p.v_st = a.v_st;
    p.o_sb = a.o_sb, p.o_sh = a.o_sh, p.o_st = a.o_st;
    p.H = a.H;
    p.Hk = a.Hk;
    p.shared = a.H / a.Hk;
    p.inverse = inverse_of(p.shared);
    p.Tq = a.Tq;
    p.Tk = a.Tk;
    p.window = a.window < a.Tk ? a.window : 0;  // as far as there are keys: all of them
    p.c = a.scale * kLog2e;
    p.o_f32 = a.o_dtype == PDN_F32;
    p.tiles = pl.tiles;
    p.splits = pl.splits;
    p.part = static_cast<float*>(a.workspace);
    p.rows = static_cast<long>(a.B) * a.H * a.Tq;
    const hipError_t rc = launch<false>(p, pl, a.dtype, a.d, static_cast<long>(a.B) * a.Hk, stream);
    if (rc != hipSuccess || pl.splits == 1) return rc;
    JoinParams j{};
    j.part = p.part;
    j.o = a.o;
    j.lse = a.lse;
    j.rows = p.rows;
    j.o_sb = a.o_sb, j.o_sh = a.o_sh, j.o_st = a.o_st;
    j.splits = pl.splits;
    j.H = a.H;
    j.Tq = a.Tq;
    j.o_f32 = p.o_f32;
    j.c = p.c;
    return launch_join<false>(j, a.d, stream);
}

size_t attn_paged_workspace_bytes(const pdn_attn_paged_args& a) {
    return a.cache.N == 0 || a.cache.max_new == 0 ? 0 : part_bytes(plan_of(a), static_cast<long>(a.cache.B) * a.H * a.cache.max_new, a.cache.d);
}

hipError_t launch_attn_paged(const pdn_attn_paged_args& a, hipStream_t stream) {
    const pdn_cache& c = a.cache;
    if (c.N == 0 || c.max_new == 0) return hipSuccess;
    const Plan pl = plan_of(a);
    FwdParams p{};
    p.q = a.q;
    p.k = c.k_pages;
    p.v = c.v_pages;
    p.o = a.o;
    p.lse = a.lse;
    p.q_sh = a.q_sh, p.q_st = a.q_sn;
    p.k_sb = c.k_sp, p.k_sh = c.k_sh, p.k_st = c.k_st;
    p.v_sb = c.v_sp, p.v_sh = c.v_sh, p.v_st = c.v_st;
    p.o_sh = a.o_sh, p.o_st = a.o_sn;
    p.H = a.H;
    p.Hk = c.Hk;
    p.shared = a.H / c.Hk;
    p.inverse = inverse_of(p.shared);
    p.Tq = c.max_new;
    p.window = a.window < c.table_width * c.page_size ? a.window : 0;
    p.c = a.scale * kLog2e;
    p.o_f32 = a.o_dtype == PDN_F32;
    p.tiles = pl.tiles;
    p.splits = pl.splits;
    p.part = static_cast<float*>(a.workspace);
    p.rows = static_cast<long>(c.B) * a.H * c.max_new;
    p.map = page_map(c);
    const hipError_t rc = launch<true>(p, pl, c.dtype, c.d, static_cast<long>(c.B) * c.Hk, stream);
    if (rc != hipSuccess || pl.splits == 1) return rc;
    JoinParams j{};
    j.part = p.part;
    j.o = a.o;
    j.lse = a.lse;
    j.rows = p.rows;
    j.o_sh = a.o_sh, j.o_st = a.o_sn;
    j.splits = pl.splits;
    j.H = a.H;
    j.Tq = c.max_new;
    j.o_f32 = p.o_f32;
    j.c = p.c;
    j.map = p.map;
    return launch_join<true>(j, c.d, stream);
}

}  // namespace pdn
