// Norms of a head's rows on the way into the recurrence and out of it:
//
//   qk_norm   n = x r w s, r = (c sum x^2 + eps)^-1/2, then the rotation of
//             pairs by position * inv_freq, from [B,T,Hx,d] to [B,H,T,d]
//   out_norm  y = o r w act(z), from [B,H,T,dv] to [B,T,H,dv]
//
// and their gradients.  With g the gradient of n (after the rotation is turned
// back and the heads that share a row are summed) and gw = g w s:
//   dw = sum_rows g s x r,   dx = r (gw - x r^2 c sum_row(gw x)).
//
// All four are bound by bytes: some ten operations an element.  A row is held
// by d / 8 lanes, 8 elements (one 16-byte load of bf16) each, so its sums stay
// within a few lanes; the same lanes take the same token's head after head,
// so a token's rows stream in one sweep, its angles are formed once (per lane:
// 8 pairs at most), and the rotation folds into two factors per element,
//   out_i = r (x_i wc_i + x_partner(i) ws_i).
//
// Measured on an MI355X, whose large copies reach 5.3 TB/s (counters: each
// of these moves within 3% of the bytes it cannot do without):
//   q/k norm      B4 T8192 H16 d128 bf16, no rotation      82 us   6.5 TB/s (*)
//                 B1 T65536 Hq16 Hk4 H16, half rotated    165 us   5.3 TB/s
//   its backward  B2 T8192 H32, all rotated, weights      208 us   5.2 TB/s
//   output norm   B4 T8192 H16 dv128, fp32 o, bf16 z, y   100 us   5.4 TB/s
//   its backward  B2 T8192 H32                            186 us   5.1 TB/s
// (*) over the copy's rate: part of the 268 MB written stays in the 256 MB
// cache from one call to the next, where q and k are overwritten in place (109 us
// into other memory each call).
#include "layer.h"
#include "rows.h"

namespace pdn {
namespace {

constexpr int kThreads = 256;
// Heads whose loads are in flight together, forward: 2 and 8 measured 120 and
// 109 us where 4 took 111.  The backward takes two: its gradients are fp32.
constexpr int kUnroll = 4;

enum { ROPE_NONE = 0, ROPE_HALF = 1, ROPE_PAIRS = 2 };

struct Strided {
    const void* p;
    long sb, st, sh;
};
struct StridedOut {
    void* p;
    long sb, st, sh;
};

struct QkSide {
    Strided x;
    StridedOut dx;      // backward
    const float* w;
    const float* g;     // backward: [B,H,T,d] fp32
    void* out;          // forward: [B,H,T,d]
    float scale;
    int heads, rep;     // input heads, outputs that share one
};

struct QkParams {
    QkSide side[2];
    const double* inv_freq;
    const int64_t* positions;
    float* partial;     // backward: [blocks][2][d]
    int tokens, T, H;
    int rot;
    int heads_per_block;
    float mean;         // c: 1/d or 1
    float eps;
    float rope_scale;
    int norm;
};

// The lane that holds this lane's partner elements in the half layout (rot is
// a multiple of 16, so that a lane's eight elements have theirs in one lane);
// itself behind the rotated part.
__device__ __forceinline__ int half_partner(int lane, int e, int rot) {
    const int h8 = rot >> 4;
    return e < h8 ? lane + h8 : e < 2 * h8 ? lane - h8 : lane;
}

// cos and sin of the angles of this lane's eight elements, times rope_scale:
// out_i = n_i c_i + n_partner s_i, so s carries the sign of its element; (1, 0)
// behind the rotated part.  The angle is formed in turns in 64 bits: position
// times frequency keeps its fraction to 1e-9 turns at positions of millions,
// where 32 bits would leave 1e-1.  Two elements share each angle: in the half
// layout the lane `pl` holds the others, and each of the two lanes forms four.
template <int ROPE>
__device__ __forceinline__ void angles(const QkParams& p, int t, int n, int e, int pl, float (&c)[8], float (&s)[8]) {
    const double pos = p.positions ? static_cast<double>(p.positions[n]) : static_cast<double>(t);
    const bool rotated = 8 * e < p.rot;
    const bool second = ROPE == ROPE_HALF && 16 * e >= p.rot;
    const int pair0 = ROPE == ROPE_HALF ? 8 * e - (second ? (p.rot >> 1) - 4 : 0) : 4 * e;
    float cn[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double f = rotated ? p.inv_freq[pair0 + j] : 0.0;
        const double turns = pos * f * 0.15915494309189535;  // 1 / (2 pi)
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn[j], &cn[j]);
        cn[j] = rotated ? cn[j] * p.rope_scale : 1.0f;
        sn[j] = rotated ? sn[j] * p.rope_scale : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (ROPE == ROPE_HALF) {
            const float co = __shfl(cn[j], pl, 64), so = __shfl(sn[j], pl, 64);
            c[j] = second ? co : cn[j];
            c[4 + j] = second ? cn[j] : co;
            s[j] = second ? so : -sn[j];
            s[4 + j] = second ? sn[j] : -so;
        } else {
            c[2 * j] = c[2 * j + 1] = cn[j];
            s[2 * j] = -sn[j];
            s[2 * j + 1] = sn[j];
        }
    }
}

// Zeros behind the rotated part: times a sine of zero an infinity there would
// reach its neighbour, or turn itself into NaN.
template <int ROPE>
__device__ __forceinline__ void partners(const float (&x)[8], int lane, bool rotated, float (&xp)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float other = ROPE == ROPE_HALF ? __shfl(x[j], lane, 64) : x[j ^ 1];
        xp[j] = rotated ? other : 0.0f;
    }
}

// A workgroup takes SLOTS tokens and (unless tokens are few) all their heads:
// splitting the heads costs the angles once more for each part (B1 T65536,
// half rotated: 169, 193 and 251 us in 2, 4 and 8 parts, one 165).  The next heads' loads
// are issued ahead of the present ones' arithmetic, the first ones' ahead of the
// angles.
template <bool BF16, int D, int ROPE>
__global__ void __launch_bounds__(kThreads) qk_norm_fwd_kernel(QkParams p) {
    constexpr int LPR = D / 8, SLOTS = kThreads / LPR;
    const int tid = threadIdx.x, lane = tid & 63, e = tid % LPR;
    const long want = static_cast<long>(by_xcd(blockIdx.x, gridDim.x)) * SLOTS + tid / LPR;
    const bool valid = want < p.tokens;
    const int n = valid ? static_cast<int>(want) : p.tokens - 1;  // idle lanes repeat the last token, unstored
    const int b = n / p.T, t = n - b * p.T;

    const int first = blockIdx.y * p.heads_per_block;
    const int last = min(first + p.heads_per_block, p.side[0].heads + p.side[1].heads);
    // a side's heads in this workgroup, and the loads of its first ones ahead of the angles
    int h0[2], h1[2];
    long row[2];
    Raw8<BF16> raw[2][kUnroll];
    auto load = [&](int k, int h) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) raw[k][u].stream(p.side[k].x.p, row[k] + min(h + u, h1[k] - 1) * p.side[k].x.sh);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int skip = k ? p.side[0].heads : 0;
        h0[k] = max(first - skip, 0);
        h1[k] = min(last - skip, p.side[k].heads);
        row[k] = b * p.side[k].x.sb + t * p.side[k].x.st + 8 * e;
        if (h0[k] < h1[k]) load(k, h0[k]);
    }
    float c[8], s[8];
    int pl = lane;
    const bool rotated = 8 * e < p.rot;  // rot is a multiple of 16: all of a lane's elements, or none
    if constexpr (ROPE == ROPE_HALF) pl = half_partner(lane, e, p.rot);
    if constexpr (ROPE != ROPE_NONE) angles<ROPE>(p, t, n, e, pl, c, s);

#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const QkSide& q = p.side[k];
        if (h0[k] >= h1[k]) continue;
        float wc[8], ws[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) wc[j] = (q.w ? q.w[8 * e + j] : 1.0f) * q.scale;
        if constexpr (ROPE != ROPE_NONE) {
            partners<ROPE>(wc, pl, rotated, ws);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                wc[j] *= c[j];
                ws[j] *= s[j];
            }
        }
        for (int h = h0[k]; h < h1[k]; h += kUnroll) {
            Raw8<BF16> now[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) now[u] = raw[k][u];
            if (h + kUnroll < h1[k]) load(k, h + kUnroll);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (h + u >= h1[k]) break;
                float x[8], y[8];
                now[u].get(x);
                float r = 1.0f;
                if (p.norm) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
                    r = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(sum), p.mean, p.eps));
                }
                if constexpr (ROPE == ROPE_NONE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = x[j] * wc[j] * r;
                } else {
                    float xp[8];
                    if constexpr (ROPE == ROPE_HALF) {
                        Raw8<BF16> other = now[u].from_lane(pl);
                        if (!rotated) other.zero();
                        other.get(xp);
                    } else {
                        partners<ROPE>(x, pl, rotated, xp);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = fmaf(x[j], wc[j], xp[j] * ws[j]) * r;
                }
                if (valid) {
                    const long o = ((static_cast<long>(b) * p.H + static_cast<long>(h + u) * q.rep) * p.T + t) * D + 8 * e;
                    for (int m = 0; m < q.rep; ++m) store8<BF16>(q.out, o + static_cast<long>(m) * p.T * D, y);
                }
            }
        }
    }
}

// Sum of `acc` over the workgroup's rows, 8 columns to a lane, into
// dst[0..width): each column's terms in slot order.
template <int LPR>
__device__ __forceinline__ void sum_slots(const float (&acc)[8], float* red, float* dst, int width) {
    constexpr int SLOTS = kThreads / LPR;
    const int tid = threadIdx.x, e = tid % LPR, slot = tid / LPR;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[slot * (LPR * 8) + 8 * e + j] = acc[j];
    __syncthreads();
    for (int i = tid; i < width; i += kThreads) {
        float s = 0.0f;
        for (int m = 0; m < SLOTS; ++m) s += red[m * (LPR * 8) + i];
        dst[i] = s;
    }
}

// A workgroup takes token groups in strides of the grid, so that a lane's
// weight gradients add up in registers over all its tokens and heads; one
// partial sum per workgroup goes to the workspace (at most kBwdFill of them: the
// kernel that adds them up takes 6 us).  Its loads stay behind the angles: ahead of
// them they cost the registers of a fourth wave (205 -> 212 us, interleaved; the
// half layout takes 131 to 133 registers and has three, 225 us where that takes 217).  They go through
// the caches, where a recurrence's backward has just left some of what they read:
// the same at B2 T8192 H32, 32 us instead of 40 for 6725 tokens of 12 fp32 heads.
template <bool BF16, int D, int ROPE>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(QkParams p) {
    constexpr int LPR = D / 8, SLOTS = kThreads / LPR;
    __shared__ float red[kThreads * 8];
    const int tid = threadIdx.x, lane = tid & 63, e = tid % LPR;
    const int first = blockIdx.y * p.heads_per_block;
    const int last = min(first + p.heads_per_block, p.side[0].heads + p.side[1].heads);
    const int groups = (p.tokens + SLOTS - 1) / SLOTS;
    float dw[2][8] = {};
    int pl = lane;
    const bool rotated = 8 * e < p.rot;
    if constexpr (ROPE == ROPE_HALF) pl = half_partner(lane, e, p.rot);

    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        const long want = static_cast<long>(grp) * SLOTS + tid / LPR;
        const bool valid = want < p.tokens;
        const int n = valid ? static_cast<int>(want) : p.tokens - 1;
        const int b = n / p.T, t = n - b * p.T;
        float c[8], s[8];
        if constexpr (ROPE != ROPE_NONE) angles<ROPE>(p, t, n, e, pl, c, s);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const QkSide& q = p.side[k];
            const int skip = k ? p.side[0].heads : 0;
            const int h0 = max(first - skip, 0), h1 = min(last - skip, q.heads);
            if (h0 >= h1) continue;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = q.w ? q.w[8 * e + j] : 1.0f;
            const long row = b * q.x.sb + t * q.x.st + 8 * e;
            const long drow = b * q.dx.sb + t * q.dx.st + 8 * e;
            for (int h = h0; h < h1; h += 2) {
                Raw8<BF16> raw[2];
                float g[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int hu = min(h + u, h1 - 1);
                    raw[u].load(q.x.p, row + hu * q.x.sh);
                    const long o = ((static_cast<long>(b) * p.H + static_cast<long>(hu) * q.rep) * p.T + t) * D + 8 * e;
                    Raw8<false> gr;
                    gr.load(q.g, o);
                    gr.get(g[u]);
                    for (int m = 1; m < q.rep; ++m) {
                        float more[8];
                        gr.load(q.g, o + static_cast<long>(m) * p.T * D);
                        gr.get(more);
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[u][j] += more[j];
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (h + u >= h1) break;
                    float x[8], y[8];
                    raw[u].get(x);
                    if constexpr (ROPE != ROPE_NONE) {  // the rotation turned back: its transpose
                        float gp[8];
                        partners<ROPE>(g[u], pl, rotated, gp);
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[u][j] = fmaf(g[u][j], c[j], -gp[j] * s[j]);
                    }
                    float r = 1.0f;
                    if (p.norm) {
                        float sum = 0.0f, dot = 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            g[u][j] *= q.scale;
                            sum = fmaf(x[j], x[j], sum);
                            dot = fmaf(g[u][j] * w[j], x[j], dot);
                        }
                        r = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(sum), p.mean, p.eps));
                        const float back = row_sum<LPR>(dot) * r * r * p.mean;
                        const float keep = valid ? r : 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            dw[k][j] = fmaf(g[u][j] * x[j], keep, dw[k][j]);
                            y[j] = r * fmaf(-x[j], back, g[u][j] * w[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = g[u][j] * q.scale;
                    }
                    if (valid) store8<BF16>(q.dx.p, drow + (h + u) * q.dx.sh, y);
                }
            }
        }
    }
    if (p.partial) {
        float* dst = p.partial + (static_cast<long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * D;
        sum_slots<LPR>(dw[0], red, dst, D);
        sum_slots<LPR>(dw[1], red, dst + D, D);
    }
}

struct OutParams {
    const void* o;
    const float* w;
    Strided z;
    StridedOut y;
    Strided dy;         // backward
    float* d_o;
    StridedOut dz;
    float* partial;     // backward: [blocks][dv]
    int tokens, T, H, dv;
    int heads_per_block;
    float mean, eps;
    int act;
};

// The gate's factor and, for the backward, its derivative by z.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

template <bool OBF16, bool BF16, int LPR>
__global__ void __launch_bounds__(kThreads) out_norm_fwd_kernel(OutParams p) {
    constexpr int SLOTS = kThreads / LPR;
    const int tid = threadIdx.x, e = tid % LPR;
    const long want = static_cast<long>(blockIdx.x) * SLOTS + tid / LPR;
    const bool valid = want < p.tokens && 8 * e < p.dv;  // dv / 8 of the LPR lanes hold a row
    const int n = want < p.tokens ? static_cast<int>(want) : p.tokens - 1;
    const int b = n / p.T, t = n - b * p.T;
    const int col = 8 * e < p.dv ? 8 * e : 0;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.H);
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p.w ? p.w[col + j] : 1.0f;
    const long zrow = b * p.z.sb + t * p.z.st + col, yrow = b * p.y.sb + t * p.y.st + col;
    const long step = static_cast<long>(p.T) * p.dv;
    const long orow = (static_cast<long>(b) * p.H * p.T + t) * p.dv + col;
    for (int h = h0; h < h1; h += kUnroll) {
        Raw8<OBF16> o[kUnroll];
        Raw8<BF16> z[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hu = min(h + u, h1 - 1);
            if (valid) o[u].stream(p.o, orow + hu * step);
            else o[u].zero();
            if (p.act && valid) z[u].stream(p.z.p, zrow + hu * p.z.sh);
            else z[u].zero();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h + u >= h1) break;
            float x[8], y[8];
            o[u].get(x);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
            const float r = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(sum), p.mean, p.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[j] * r * w[j];
            if (p.act) {
                float g[8];
                z[u].get(g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = sigmoid(g[j]);
                    y[j] *= p.act == PDN_ACT_SILU ? f * g[j] : f;
                }
            }
            if (valid) store8<BF16>(p.y.p, yrow + (h + u) * p.y.sh, y);
        }
    }
}

// As the q/k norm's backward.  Its loads go through the caches (186 us; past
// them 190).
template <bool OBF16, bool BF16, int LPR>
__global__ void __launch_bounds__(kThreads) out_norm_bwd_kernel(OutParams p) {
    constexpr int SLOTS = kThreads / LPR;
    __shared__ float red[kThreads * 8];
    const int tid = threadIdx.x, e = tid % LPR;
    const bool mine = 8 * e < p.dv;
    const int col = mine ? 8 * e : 0;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.H);
    const int groups = (p.tokens + SLOTS - 1) / SLOTS;
    const long step = static_cast<long>(p.T) * p.dv;
    float w[8], dw[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p.w ? p.w[col + j] : 1.0f;
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        const long want = static_cast<long>(grp) * SLOTS + tid / LPR;
        const bool valid = want < p.tokens && mine;
        const int n = want < p.tokens ? static_cast<int>(want) : p.tokens - 1;
        const int b = n / p.T, t = n - b * p.T;
        const long orow = (static_cast<long>(b) * p.H * p.T + t) * p.dv + col;
        const long zrow = b * p.z.sb + t * p.z.st + col, dzrow = b * p.dz.sb + t * p.dz.st + col;
        const long dyrow = b * p.dy.sb + t * p.dy.st + col;
        for (int h = h0; h < h1; h += 2) {
            Raw8<OBF16> o[2];
            Raw8<BF16> z[2], gy[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int hu = min(h + u, h1 - 1);
                if (valid) {
                    o[u].load(p.o, orow + hu * step);
                    gy[u].load(p.dy.p, dyrow + hu * p.dy.sh);
                } else {
                    o[u].zero();
                    gy[u].zero();
                }
                if (p.act && valid) z[u].load(p.z.p, zrow + hu * p.z.sh);
                else z[u].zero();
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (h + u >= h1) break;
                float x[8], g[8];
                o[u].get(x);
                gy[u].get(g);
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
                const float r = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(sum), p.mean, p.eps));
                if (p.act) {
                    float zf[8], dz[8];
                    z[u].get(zf);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = sigmoid(zf[j]);
                        const float n1 = g[j] * x[j] * r * w[j];
                        if (p.act == PDN_ACT_SILU) {
                            dz[j] = n1 * f * fmaf(zf[j], 1.0f - f, 1.0f);
                            g[j] *= f * zf[j];
                        } else {
                            // 1 - f as it is for -z: where f is near one, the
                            // difference would keep few of its digits
                            dz[j] = n1 * f * sigmoid(-zf[j]);
                            g[j] *= f;
                        }
                    }
                    if (valid) store8<BF16>(p.dz.p, dzrow + (h + u) * p.dz.sh, dz);
                }
                float dot = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[j] = fmaf(g[j] * x[j], r, dw[j]);  // rows past the end hold zeros
                    g[j] *= w[j];
                    dot = fmaf(g[j], x[j], dot);
                }
                const float back = row_sum<LPR>(dot) * r * r * p.mean;
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = r * fmaf(-x[j], back, g[j]);
                if (valid) store8<false>(p.d_o, orow + (h + u) * step, y);
            }
        }
    }
    if (p.partial)
        sum_slots<LPR>(dw, red, p.partial + (static_cast<long>(blockIdx.y) * gridDim.x + blockIdx.x) * p.dv, p.dv);
}

// Column sums of the workgroups' partial sums [blocks][cols], in an order
// fixed by `blocks`: 64 row groups of a 16-column strip, then their sum.
constexpr int kStrip = 16;
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* partial, int blocks, int cols,
                                                            float* dst0, float* dst1, int split) {
    __shared__ float red[64][kStrip];
    const int c = threadIdx.x % kStrip, g = threadIdx.x / kStrip;
    const int col = blockIdx.x * kStrip + c;
    float s = 0.0f;
#pragma unroll 8
    for (int i = g; i < blocks; i += 64) s += partial[static_cast<long>(i) * cols + col];
    red[g][c] = s;
    __syncthreads();
    if (g == 0) {
        s = 0.0f;
        for (int i = 0; i < 64; ++i) s += red[i][c];
        float* dst = col < split ? dst0 : dst1;
        if (dst) dst[col < split ? col : col - split] = s;
    }
}

// Workgroups that fill an MI355X: eight of 256 threads to each of its 256
// compute units.  A constant, not the device's count, so that the workspace
// sizes and the order of the weight gradients' sums go by the arguments alone.
constexpr long kFill = 2048;

// Heads per workgroup: all of a token's (its angles and rows once), unless the
// token groups are too few to fill the device; then the heads are split.
int heads_per_block(long groups, int heads) {
    long parts = groups > 0 ? (kFill + groups - 1) / groups : 1;
    if (parts > heads) parts = heads;
    return static_cast<int>((heads + parts - 1) / parts);
}

// Grid of a backward.  With weight gradients each workgroup leaves a partial sum
// of them, and takes several token groups so that those stay few, the groups
// dealt evenly.  1024, 2048 and 4096 workgroups at B2 T8192 H32: 229, 223 and
// 222 us with the sum of the partial ones.
constexpr long kBwdFill = 2048;
// Heads that a workgroup of the q/k norm's backward takes at most: its streams
// are many (x, its gradient, the heads' gradients), and 8 heads' stay closer
// together than 32's: 215 against 228 us there, 4 heads 221.  The output norm's
// backward does not care.
constexpr int kQkBwdHeads = 8;
struct BwdGrid {
    int x, y, per;
};
BwdGrid bwd_grid(long tokens, int slots, int heads, int most, bool weights) {
    const long groups = (tokens + slots - 1) / slots;
    BwdGrid g;
    g.per = heads_per_block(groups, heads);
    // (but never over kBwdFill parts, whatever the heads)
    const int least = static_cast<int>((heads + kBwdFill - 1) / kBwdFill);
    if (g.per > most) g.per = most > least ? most : least;
    g.y = (heads + g.per - 1) / g.per;
    const long cap = kBwdFill / g.y > 0 ? kBwdFill / g.y : 1;
    const long each = weights && groups > cap ? (groups + cap - 1) / cap : 1;
    g.x = static_cast<int>((groups + each - 1) / each);
    return g;
}

int out_lanes(int dv) {
    int l = 2;
    while (8 * l < dv) l *= 2;
    return l;
}

QkParams qk_params(const pdn_qk_norm_args& a) {
    QkParams p = {};
    p.side[0].x = Strided{a.xq, a.xq_sb, a.xq_st, a.xq_sh};
    p.side[1].x = Strided{a.xk, a.xk_sb, a.xk_st, a.xk_sh};
    p.side[0].w = a.wq;
    p.side[1].w = a.wk;
    p.side[0].out = a.q;
    p.side[1].out = a.k;
    p.side[0].scale = a.q_scale;
    p.side[1].scale = a.k_scale;
    p.side[0].heads = a.Hq;
    p.side[1].heads = a.Hk;
    p.side[0].rep = a.H / a.Hq;
    p.side[1].rep = a.H / a.Hk;
    p.inv_freq = a.inv_freq;
    p.positions = a.positions;
    p.tokens = a.B * a.T;
    p.T = a.T;
    p.H = a.H;
    p.rot = a.rot_dim;
    p.mean = a.norm == PDN_NORM_RMS ? 1.0f / a.d : 1.0f;
    p.eps = a.eps;
    p.rope_scale = a.rope_scale;
    p.norm = a.norm;
    return p;
}

template <bool BF16, int D>
hipError_t qk_launch(const QkParams& p, bool bwd, int layout, dim3 grid, hipStream_t st) {
    const dim3 block(kThreads);
    if (p.rot == 0) {
        if (bwd) qk_norm_bwd_kernel<BF16, D, ROPE_NONE><<<grid, block, 0, st>>>(p);
        else qk_norm_fwd_kernel<BF16, D, ROPE_NONE><<<grid, block, 0, st>>>(p);
    } else if (layout == PDN_ROPE_HALF) {
        if (bwd) qk_norm_bwd_kernel<BF16, D, ROPE_HALF><<<grid, block, 0, st>>>(p);
        else qk_norm_fwd_kernel<BF16, D, ROPE_HALF><<<grid, block, 0, st>>>(p);
    } else {
        if (bwd) qk_norm_bwd_kernel<BF16, D, ROPE_PAIRS><<<grid, block, 0, st>>>(p);
        else qk_norm_fwd_kernel<BF16, D, ROPE_PAIRS><<<grid, block, 0, st>>>(p);
    }
    return hipGetLastError();
}

hipError_t qk_dispatch(const QkParams& p, const pdn_qk_norm_args& a, bool bwd, dim3 grid, hipStream_t st) {
    const bool bf = a.dtype == PDN_BF16;
    if (a.d == 128) return bf ? qk_launch<true, 128>(p, bwd, a.rope_layout, grid, st) : qk_launch<false, 128>(p, bwd, a.rope_layout, grid, st);
    return bf ? qk_launch<true, 64>(p, bwd, a.rope_layout, grid, st) : qk_launch<false, 64>(p, bwd, a.rope_layout, grid, st);
}

template <bool OBF16, bool BF16>
hipError_t out_launch(const OutParams& p, bool bwd, int lanes, dim3 grid, hipStream_t st) {
    const dim3 block(kThreads);
    switch (lanes) {
#define PDN_CASE(L)                                                                       \
    case L:                                                                               \
        if (bwd) out_norm_bwd_kernel<OBF16, BF16, L><<<grid, block, 0, st>>>(p);          \
        else out_norm_fwd_kernel<OBF16, BF16, L><<<grid, block, 0, st>>>(p);              \
        break;
        PDN_CASE(2)
        PDN_CASE(4)
        PDN_CASE(8)
        PDN_CASE(16)
        PDN_CASE(32)
#undef PDN_CASE
        default: return hipErrorNotSupported;
    }
    return hipGetLastError();
}

hipError_t out_dispatch(const OutParams& p, const pdn_out_norm_args& a, bool bwd, dim3 grid, hipStream_t st) {
    const int l = out_lanes(a.dv);
    const bool of = a.o_dtype == PDN_BF16, bf = a.dtype == PDN_BF16;
    if (of) return bf ? out_launch<true, true>(p, bwd, l, grid, st) : out_launch<true, false>(p, bwd, l, grid, st);
    return bf ? out_launch<false, true>(p, bwd, l, grid, st) : out_launch<false, false>(p, bwd, l, grid, st);
}

OutParams out_params(const pdn_out_norm_args& a) {
    OutParams p = {};
    p.o = a.o;
    p.w = a.w;
    p.z = Strided{a.z, a.z_sb, a.z_st, a.z_sh};
    p.y = StridedOut{a.y, a.y_sb, a.y_st, a.y_sh};
    p.tokens = a.B * a.T;
    p.T = a.T;
    p.H = a.H;
    p.dv = a.dv;
    p.mean = 1.0f / a.dv;
    p.eps = a.eps;
    p.act = a.act;
    return p;
}

}  // namespace

bool qk_norm_fits(const pdn_qk_norm_args& a) {
    const int slots = kThreads / (a.d / 8);
    return (static_cast<long>(a.B) * a.T + slots - 1) / slots <= kMaxGridThreads / kThreads;
}

bool out_norm_fits(const pdn_out_norm_args& a) {
    const int slots = kThreads / out_lanes(a.dv);
    return (static_cast<long>(a.B) * a.T + slots - 1) / slots <= kMaxGridThreads / kThreads;
}

hipError_t launch_qk_norm(const pdn_qk_norm_args& a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    QkParams p = qk_params(a);
    const int slots = kThreads / (a.d / 8), heads = a.Hq + a.Hk;
    const long groups = (static_cast<long>(p.tokens) + slots - 1) / slots;
    p.heads_per_block = heads_per_block(groups, heads);
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((heads + p.heads_per_block - 1) / p.heads_per_block));
    return qk_dispatch(p, a, false, grid, st);
}

size_t qk_norm_bwd_workspace_bytes(const pdn_qk_norm_bwd_args& a) {
    if (!a.dwq && !a.dwk) return 0;
    const BwdGrid g = bwd_grid(static_cast<long>(a.fwd.B) * a.fwd.T, kThreads / (a.fwd.d / 8), a.fwd.Hq + a.fwd.Hk, kQkBwdHeads, true);
    return sizeof(float) * 2 * a.fwd.d * static_cast<size_t>(g.x) * g.y;
}

hipError_t launch_qk_norm_bwd(const pdn_qk_norm_bwd_args& a, hipStream_t st) {
    const pdn_qk_norm_args& f = a.fwd;
    const bool weights = a.dwq || a.dwk;
    float* partial = weights ? static_cast<float*>(a.workspace) : nullptr;
    int blocks = 0;
    if (f.T > 0) {
        QkParams p = qk_params(f);
        p.side[0].g = a.dq;
        p.side[1].g = a.dk;
        p.side[0].dx = StridedOut{a.dxq, a.dxq_sb, a.dxq_st, a.dxq_sh};
        p.side[1].dx = StridedOut{a.dxk, a.dxk_sb, a.dxk_st, a.dxk_sh};
        p.partial = partial;
        const BwdGrid g = bwd_grid(p.tokens, kThreads / (f.d / 8), f.Hq + f.Hk, kQkBwdHeads, weights);
        p.heads_per_block = g.per;
        blocks = g.x * g.y;
        const hipError_t e = qk_dispatch(p, f, true, dim3(g.x, g.y), st);
        if (e != hipSuccess) return e;
    }
    if (!weights) return hipSuccess;
    sum_partials_kernel<<<dim3(2 * f.d / kStrip), dim3(1024), 0, st>>>(partial, blocks, 2 * f.d, a.dwq, a.dwk, f.d);
    return hipGetLastError();
}

hipError_t launch_out_norm(const pdn_out_norm_args& a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    OutParams p = out_params(a);
    const int slots = kThreads / out_lanes(a.dv);
    const long groups = (static_cast<long>(p.tokens) + slots - 1) / slots;
    p.heads_per_block = heads_per_block(groups, a.H);
    return out_dispatch(p, a, false, dim3(static_cast<unsigned>(groups), static_cast<unsigned>((a.H + p.heads_per_block - 1) / p.heads_per_block)), st);
}

size_t out_norm_bwd_workspace_bytes(const pdn_out_norm_bwd_args& a) {
    if (!a.dw) return 0;
    const BwdGrid g = bwd_grid(static_cast<long>(a.fwd.B) * a.fwd.T, kThreads / out_lanes(a.fwd.dv), a.fwd.H, a.fwd.H, true);
    return sizeof(float) * a.fwd.dv * static_cast<size_t>(g.x) * g.y;
}

hipError_t launch_out_norm_bwd(const pdn_out_norm_bwd_args& a, hipStream_t st) {
    const pdn_out_norm_args& f = a.fwd;
    float* partial = a.dw ? static_cast<float*>(a.workspace) : nullptr;
    int blocks = 0;
    if (f.T > 0) {
        OutParams p = out_params(f);
        p.dy = Strided{a.dy, a.dy_sb, a.dy_st, a.dy_sh};
        p.d_o = a.d_o;
        p.dz = StridedOut{a.dz, a.dz_sb, a.dz_st, a.dz_sh};
        p.partial = partial;
        const BwdGrid g = bwd_grid(p.tokens, kThreads / out_lanes(f.dv), f.H, f.H, a.dw != nullptr);
        p.heads_per_block = g.per;
        blocks = g.x * g.y;
        const hipError_t e = out_dispatch(p, f, true, dim3(g.x, g.y), st);
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    sum_partials_kernel<<<dim3(f.dv / kStrip), dim3(1024), 0, st>>>(partial, blocks, f.dv, a.dw, nullptr, f.dv);
    return hipGetLastError();
}

}  // namespace pdn
