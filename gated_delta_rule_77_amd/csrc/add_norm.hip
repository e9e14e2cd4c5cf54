// The seam between two sublayers, a token's row of D channels at a time:
//
//   s = res + keep x / (1 - p),   y = s r w,  r = (mean s^2 + eps)^-1/2,
//
// y in fp32, bf16, or 8 bits with a scale a group, and its gradient:
//
//   dres = ds + r (g - s r^2 mean(g s)),  g = dy w,   dx = keep dres / (1 - p),
//   dw = sum_rows dy s r.
//
// Bound by bytes: each tensor once, a row held in registers between its sums and
// its outputs (8 channels a lane and step, TPR lanes to a row).  B4 T8192 D2048 bf16 to
// 8 bits 75 us, 6.3 TB/s; B2 T8192 D4096 with fp32 sums and dropout 145 us forward and
// 211 to 233 backward, 5.5 and 4.9 TB/s.  Dropout's bits are formed from the element's
// place, forward and backward: ten rounds of Philox for eight elements, some 25 issue
// slots an element, beside its 6 to 14 bytes.
#include "block.h"
#include "philox.h"
#include "rows.h"

namespace pdn {
namespace {

struct Rows {
    const void* p;
    long sb, st;
};
struct RowsOut {
    void* p;
    long sb, st;
};

struct AddNormParams {
    Rows x, res;
    RowsOut s, y;
    const float* w;
    float* y_scale;
    const int64_t* seed;
    long rows;
    int T, D, group;      // group: channels of a scale
    uint32_t threshold;   // of 65536; 0 = no dropout
    float factor;         // of what is kept
    float mean, eps;      // mean: 1 / D
};

enum { Y_F32 = 0, Y_BF16 = 1, Y_E4M3 = 2 };

constexpr float kTop8 = 448.0f;            // the largest e4m3
constexpr float kLeast8 = 0x1p-64f;        // the least magnitude that a scale goes by

// Eight values to e4m3, to the nearest (ties to even).
__device__ __forceinline__ uint2 pack8(const float (&f)[8]) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    return uint2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
    return x;
}

// Sum (or maximum) over the TPR lanes of a row, the same bits in each.  More than a
// wave goes through `red`, which the caller does not use again before a barrier.
template <int TPR, bool MAX>
__device__ __forceinline__ float over_row(float x, float* red) {
    x = MAX ? wave_max(x) : wave_sum(x);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) x = MAX ? fmaxf(x, red[i]) : x + red[i];
    }
    return x;
}

// Maximum over the `lanes` (4, 8 or 16) neighbouring lanes that hold a group.
__device__ __forceinline__ float over_group(float x, int lanes) {
    x = fmaxf(x, dpp<0xB1>(x));
    x = fmaxf(x, dpp<0x4E>(x));
    if (lanes > 4) x = fmaxf(x, dpp<0x141>(x));
    if (lanes > 8) x = fmaxf(x, dpp<0x140>(x));
    return x;
}

template <int TPR>
constexpr int kBlock = TPR > 256 ? TPR : 256;

// The product is rounded before the sum, as the formula reads: a fused one would
// give a bf16 residual another neighbour now and then.
__device__ __forceinline__ float kept_times(float x, float factor) { return __fmul_rn(x, factor); }

template <bool XB, bool SB, int YT, int TPR, int C>
__global__ void __launch_bounds__(kBlock<TPR>) add_norm_fwd_kernel(AddNormParams p) {
    constexpr int SLOTS = kBlock<TPR> / TPR;
    __shared__ float red[2][16];
    const int e = threadIdx.x % TPR;
    const long row = static_cast<long>(blockIdx.x) * SLOTS + threadIdx.x / TPR;
    if (SLOTS > 1 && row >= p.rows) return;  // whole waves; those of one row share no barrier
    const long b = row / p.T, t = row - b * p.T;
    const long xr = b * p.x.sb + t * p.x.st, rr = b * p.res.sb + t * p.res.st;
    Raw8<XB> xw[C];
    Raw8<SB> rw[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = 8 * (i * TPR + e);
        if (col < p.D) xw[i].stream(p.x.p, xr + col);
        else xw[i].zero();
        if (p.res.p && col < p.D) rw[i].stream(p.res.p, rr + col);
        else rw[i].zero();
    }
    const long sr = b * p.s.sb + t * p.s.st, yr = b * p.y.sb + t * p.y.st;
    float s[C][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = 8 * (i * TPR + e);
        float x[8], r[8];
        xw[i].get(x);
        rw[i].get(r);
        if (p.threshold) {
            const Philox bits = philox(p.seed[0], p.seed[1], static_cast<uint64_t>(row) * (p.D >> 3) + (col >> 3));
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = philox_keeps(bits, j, p.threshold) ? kept_times(x[j], p.factor) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[i][j] = p.res.p ? __fadd_rn(r[j], x[j]) : x[j];
            if constexpr (SB) s[i][j] = static_cast<float>(static_cast<bf16>(s[i][j]));
            sum = fmaf(s[i][j], s[i][j], sum);
        }
        if (p.s.p && col < p.D) store8<SB>(p.s.p, sr + col, s[i]);
    }
    const float r = __builtin_amdgcn_rsqf(fmaf(over_row<TPR, false>(sum, red[0]), p.mean, p.eps));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = 8 * (i * TPR + e);
        float w[8];
        Raw8<false> ww;
        if (p.w && col < p.D) ww.load(p.w, col);
        else ww.lo = ww.hi = f32x4{1.f, 1.f, 1.f, 1.f};
        ww.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * r * w[j];
        if constexpr (YT != Y_E4M3) {
            if (col < p.D) store8<YT == Y_BF16>(p.y.p, yr + col, s[i]);
        } else {
            float mine = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) mine = fmaxf(mine, fabsf(s[i][j]));
            if (p.group == p.D) {
                top = fmaxf(top, mine);
            } else {
                // a group's lanes lie within a wave, all of them inside the row or none
                const int lanes = p.group >> 3;
                const float m = fmaxf(over_group(mine, lanes), kLeast8);
                const float inv = __fdiv_rn(kTop8, m);
                float q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = s[i][j] * inv;
                if (col < p.D) {
                    *reinterpret_cast<uint2*>(static_cast<char*>(p.y.p) + yr + col) = pack8(q);
                    if (e % lanes == 0) p.y_scale[row * (p.D / p.group) + col / p.group] = __fdiv_rn(m, kTop8);
                }
            }
        }
    }
    if constexpr (YT == Y_E4M3) {
        if (p.group != p.D) return;
        const float m = fmaxf(over_row<TPR, true>(top, red[1]), kLeast8);
        const float inv = __fdiv_rn(kTop8, m);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = 8 * (i * TPR + e);
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = s[i][j] * inv;
            if (col < p.D) *reinterpret_cast<uint2*>(static_cast<char*>(p.y.p) + yr + col) = pack8(q);
        }
        if (e == 0) p.y_scale[row] = __fdiv_rn(m, kTop8);
    }
}

struct AddNormBwdParams {
    Rows s, dy, ds;
    RowsOut dres, dx;
    const float* w;
    float* partial;       // [workgroups][D]
    const int64_t* seed;
    long rows;
    int T, D;
    uint32_t threshold;
    float factor;
    float mean, eps;
};

// A workgroup takes rows in strides of the grid, so that a lane's weight gradients
// add up in registers; one partial sum a workgroup goes to the workspace.
template <bool XB, bool SB, bool YB, int TPR, int C>
__global__ void __launch_bounds__(kBlock<TPR>) add_norm_bwd_kernel(AddNormBwdParams p) {
    constexpr int SLOTS = kBlock<TPR> / TPR;
    __shared__ float red[2][16];
    __shared__ float slots[SLOTS > 1 ? TPR * C * 8 : 1];
    const int e = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    float dw[C][8] = {};
    for (long first = static_cast<long>(blockIdx.x) * SLOTS; first < p.rows; first += static_cast<long>(gridDim.x) * SLOTS) {
        const long row = min(first + slot, p.rows - 1);
        const bool valid = first + slot < p.rows;  // the last workgroup's idle waves repeat a row, unstored
        const long b = row / p.T, t = row - b * p.T;
        const long sr = b * p.s.sb + t * p.s.st, yr = b * p.dy.sb + t * p.dy.st, ur = b * p.ds.sb + t * p.ds.st;
        Raw8<SB> sw[C], uw[C];
        Raw8<YB> yw[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = 8 * (i * TPR + e);
            if (col < p.D) {
                sw[i].load(p.s.p, sr + col);
                yw[i].load(p.dy.p, yr + col);
            } else {
                sw[i].zero();
                yw[i].zero();
            }
            if (p.ds.p && col < p.D) uw[i].load(p.ds.p, ur + col);
            else uw[i].zero();
        }
        float s[C][8], g[C][8], sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = 8 * (i * TPR + e);
            float w[8];
            Raw8<false> ww;
            if (p.w && col < p.D) ww.load(p.w, col);
            else ww.lo = ww.hi = f32x4{1.f, 1.f, 1.f, 1.f};
            ww.get(w);
            sw[i].get(s[i]);
            yw[i].get(g[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum = fmaf(s[i][j], s[i][j], sum);
                dot = fmaf(g[i][j] * w[j], s[i][j], dot);
            }
        }
        // both sums pass over the row's waves with one barrier between
        sum = wave_sum(sum);
        dot = wave_sum(dot);
        if constexpr (TPR > 64) {
            __syncthreads();  // the row before has been read
            if ((threadIdx.x & 63) == 0) {
                red[0][threadIdx.x >> 6] = sum;
                red[1][threadIdx.x >> 6] = dot;
            }
            __syncthreads();
            sum = red[0][0];
            dot = red[1][0];
#pragma unroll
            for (int i = 1; i < TPR / 64; ++i) {
                sum += red[0][i];
                dot += red[1][i];
            }
        }
        const float r = __builtin_amdgcn_rsqf(fmaf(sum, p.mean, p.eps));
        const float back = dot * p.mean * r * r, keep_row = valid ? r : 0.0f;
        const long er = b * p.dres.sb + t * p.dres.st, xr = b * p.dx.sb + t * p.dx.st;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = 8 * (i * TPR + e);
            float w[8], u[8];
            Raw8<false> ww;
            if (p.w && col < p.D) ww.load(p.w, col);
            else ww.lo = ww.hi = f32x4{1.f, 1.f, 1.f, 1.f};
            ww.get(w);
            uw[i].get(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (valid) dw[i][j] = fmaf(g[i][j] * s[i][j], keep_row, dw[i][j]);
                u[j] = fmaf(r, fmaf(-s[i][j], back, g[i][j] * w[j]), u[j]);
            }
            if (valid && col < p.D) {
                store8<SB>(p.dres.p, er + col, u);
                if (p.dx.p) {
                    if (p.threshold) {
                        const Philox bits = philox(p.seed[0], p.seed[1], static_cast<uint64_t>(row) * (p.D >> 3) + (col >> 3));
#pragma unroll
                        for (int j = 0; j < 8; ++j) u[j] = philox_keeps(bits, j, p.threshold) ? kept_times(u[j], p.factor) : 0.0f;
                    }
                    store8<XB>(p.dx.p, xr + col, u);
                }
            }
        }
    }
    if (!p.partial) return;
    float* dst = p.partial + static_cast<long>(blockIdx.x) * p.D;
    if constexpr (SLOTS > 1) {
        for (int k = 0; k < SLOTS; ++k) {  // the waves' sums in their order
            if (slot == k) {
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float& at = slots[8 * (i * TPR + e) + j];
                        at = k == 0 ? dw[i][j] : at + dw[i][j];
                    }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < p.D; i += kBlock<TPR>) dst[i] = slots[i];
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = 8 * (i * TPR + e);
            if (col < p.D) store8<false>(dst, col, dw[i]);
        }
    }
}

// dw from the workgroups' partial sums: 64 columns to a workgroup, its 16 waves a
// stretch of the partial sums each.
__global__ void __launch_bounds__(1024) add_partials_kernel(const float* partial, int n, int D, float* dw) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    float sum = 0.0f;
    if (col < D) {
#pragma unroll 8
        for (int i = wave; i < n; i += 16) sum += partial[static_cast<long>(i) * D + col];
    }
    red[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && col < D) {
#pragma unroll
        for (int i = 1; i < 16; ++i) sum += red[i][lane];
        dw[col] = sum;
    }
}

uint32_t drop_threshold(float p) {
    const double t = nearbyint(static_cast<double>(p) * 65536.0);
    return t > 65535.0 ? 65535u : static_cast<uint32_t>(t);
}
float drop_factor(uint32_t threshold) { return static_cast<float>(65536.0 / (65536.0 - threshold)); }

// Lanes of a row and steps of 8 channels each: a wave while its registers hold the
// row, four waves beyond, and for few rows, where a wave's own latency would show
// (D2048: 256 rows 5.2 us by a wave, 4.1 by four; 4096 rows 12.9 and 14.2).
constexpr long kFewRows = 2048;

template <class F>
hipError_t by_width(int D, long rows, F f) {
    using std::integral_constant;
    if (D <= 512) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (D <= 1024) return f(integral_constant<int, 64>(), integral_constant<int, 2>());
    if (D <= 2048 && rows > kFewRows) return f(integral_constant<int, 64>(), integral_constant<int, 4>());
    if (D <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (D <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (D <= 8192) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    return f(integral_constant<int, 512>(), integral_constant<int, 4>());
}

template <class F>
hipError_t by_types(int32_t dtype, int32_t s_dtype, F f) {
    if (dtype == PDN_F32) return f(std::false_type(), std::false_type());
    if (s_dtype == PDN_F32) return f(std::true_type(), std::false_type());
    return f(std::true_type(), std::true_type());
}

// The backward holds twice as much of a row: more lanes to the widest, two steps each.
template <class F>
hipError_t by_width_bwd(int D, long rows, F f) {
    using std::integral_constant;
    if (D <= 4096) return by_width(D, rows, f);
    if (D <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 2>());
    return f(integral_constant<int, 1024>(), integral_constant<int, 2>());
}

// Workgroups of the backward: four to a compute unit where their registers let four in,
// two otherwise (measured at B2 T8192 D4096, fp32 sums: 218, 211 and 223 us with 512, 1024
// and 2048; at B1 T8192 D8192: 144, 151 and 163).  Each leaves one sum of D.
long bwd_blocks(const pdn_add_norm_bwd_args& a) {
    const long rows = static_cast<long>(a.B) * a.T, slots = a.D <= 1024 || (a.D <= 2048 && rows > kFewRows) ? 4 : 1;
    const long blocks = (rows + slots - 1) / slots, most = a.D > 4096 || (a.D > 1024 && slots == 4) ? 512 : 1024;
    return blocks < most ? blocks : most;
}

}  // namespace

hipError_t launch_add_norm(const pdn_add_norm_args& a, hipStream_t stream) {
    AddNormParams p{};
    p.rows = static_cast<long>(a.B) * a.T;
    if (p.rows == 0) return hipSuccess;
    p.x = {a.x, a.x_sb, a.x_st};
    p.res = {a.res, a.res_sb, a.res_st};
    p.s = {a.s, a.s_sb, a.s_st};
    p.y = {a.y, a.y_sb, a.y_st};
    p.w = a.w;
    p.y_scale = a.y_scale;
    p.seed = a.seed;
    p.T = a.T;
    p.D = a.D;
    p.group = a.group ? a.group : a.D;
    p.threshold = drop_threshold(a.drop_p);
    p.factor = drop_factor(p.threshold);
    p.mean = 1.0f / a.D;
    p.eps = a.eps;
    return by_types(a.dtype, a.s_dtype, [&](auto xb, auto sb) {
        return by_width(a.D, p.rows, [&](auto tpr, auto c) {
            constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value;
            constexpr bool XB = decltype(xb)::value, SB = decltype(sb)::value;
            constexpr int slots = kBlock<TPR> / TPR;
            const dim3 grid(static_cast<unsigned>((p.rows + slots - 1) / slots)), block(kBlock<TPR>);
            if (a.y_dtype == PDN_F32) add_norm_fwd_kernel<XB, SB, Y_F32, TPR, C><<<grid, block, 0, stream>>>(p);
            else if (a.y_dtype == PDN_BF16) add_norm_fwd_kernel<XB, SB, Y_BF16, TPR, C><<<grid, block, 0, stream>>>(p);
            else add_norm_fwd_kernel<XB, SB, Y_E4M3, TPR, C><<<grid, block, 0, stream>>>(p);
            return hipGetLastError();
        });
    });
}

size_t add_norm_bwd_workspace_bytes(const pdn_add_norm_bwd_args& a) {
    return a.dw ? static_cast<size_t>(bwd_blocks(a)) * a.D * sizeof(float) : 0;
}

hipError_t launch_add_norm_bwd(const pdn_add_norm_bwd_args& a, hipStream_t stream) {
    AddNormBwdParams p{};
    p.rows = static_cast<long>(a.B) * a.T;
    const long blocks = bwd_blocks(a);
    p.s = {a.s, a.s_sb, a.s_st};
    p.dy = {a.dy, a.dy_sb, a.dy_st};
    p.ds = {a.ds, a.ds_sb, a.ds_st};
    p.dres = {a.dres, a.dres_sb, a.dres_st};
    p.dx = {a.dx, a.dx_sb, a.dx_st};
    p.w = a.w;
    p.partial = a.dw ? static_cast<float*>(a.workspace) : nullptr;
    p.seed = a.seed;
    p.T = a.T;
    p.D = a.D;
    p.threshold = drop_threshold(a.drop_p);
    p.factor = drop_factor(p.threshold);
    p.mean = 1.0f / a.D;
    p.eps = a.eps;
    if (p.rows > 0) {
        const hipError_t rc = by_types(a.dtype, a.s_dtype, [&](auto xb, auto sb) {
            return by_width_bwd(a.D, p.rows, [&](auto tpr, auto c) {
                constexpr int TPR = decltype(tpr)::value, C = decltype(c)::value;
                constexpr bool XB = decltype(xb)::value, SB = decltype(sb)::value;
                const dim3 grid(static_cast<unsigned>(blocks)), block(kBlock<TPR>);
                if (a.y_dtype == PDN_F32) add_norm_bwd_kernel<XB, SB, false, TPR, C><<<grid, block, 0, stream>>>(p);
                else add_norm_bwd_kernel<XB, SB, true, TPR, C><<<grid, block, 0, stream>>>(p);
                return hipGetLastError();
            });
        });
        if (rc != hipSuccess) return rc;
    }
    if (a.dw) {
        add_partials_kernel<<<dim3(static_cast<unsigned>((a.D + 63) / 64)), dim3(1024), 0, stream>>>(
            static_cast<const float*>(a.workspace), static_cast<int>(blocks), a.D, a.dw);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace pdn
