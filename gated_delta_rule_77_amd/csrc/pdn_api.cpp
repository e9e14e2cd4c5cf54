// Host layer of libpdn.so: the extern "C" entry points declared in pdn.h and
// pdn_layer.h.
// Every entry point validates its arguments before touching the GPU, maps
// HIP errors to PDN_EHIP, and lets no exception escape.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <atomic>
#include <mutex>

#include "kernels.h"
#include "layer.h"
#include "pdn.h"

namespace {

bool valid_dtype(int32_t d) { return d == PDN_F32 || d == PDN_BF16; }
bool valid_alpha(int32_t m) {
    return m == PDN_ALPHA_NONE || m == PDN_ALPHA_SCALAR || m == PDN_ALPHA_VEC;
}
bool valid_beta(int32_t m) { return m == PDN_GATE_SCALAR || m == PDN_GATE_VEC; }
bool valid_gamma(int32_t m) {
    return m == PDN_GATE_SCALAR || m == PDN_GATE_VEC || m == PDN_GAMMA_SAME_AS_BETA;
}
bool valid_key(int32_t m) {
    return m == PDN_KEY_SYMMETRIC || m == PDN_KEY_ERASE_GATE || m == PDN_KEY_WRITE_GATE;
}
// preconditioner mode and bound; x is only read in the stabilised mode
bool valid_precond(float eps, int32_t mode, float x) {
    if (mode != PDN_PRECOND_INVERSE && mode != PDN_PRECOND_STABILISED) return false;
    if (eps >= 0.0f && mode == PDN_PRECOND_STABILISED && !(x > 1.0f && x <= 2.0f)) return false;
    return true;
}

// Largest B*H (and B*H*T) the launch grids and 32/64-bit index math accept.
constexpr long kMaxBH = 1L << 24;
// B * H * T: keeps every launch grid (at most one wave per 32-token chunk and
// (b, h), four per workgroup) below 2^31 workgroups
constexpr long kMaxTokens = 1L << 36;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Gate enums and pointers.  With no tokens to process (need_data false) the
// gate pointers may be NULL.
int check_gates(int32_t amode, const float* la, int32_t bmode, const float* beta,
                int32_t gmode, const float* gamma, float eps, int dk, int dv, bool need_data) {
    if (!valid_alpha(amode) || !valid_beta(bmode) || !valid_gamma(gmode)) return PDN_EINVAL;
    if (need_data) {
        if (amode != PDN_ALPHA_NONE && !la) return PDN_EINVAL;
        if (!beta) return PDN_EINVAL;
        if (gmode != PDN_GAMMA_SAME_AS_BETA && !gamma) return PDN_EINVAL;
    }
    if (gmode == PDN_GAMMA_SAME_AS_BETA && bmode == PDN_GATE_VEC && dk != dv)
        return PDN_EINVAL;
    if (std::isnan(eps)) return PDN_EINVAL;
    return PDN_OK;
}

// check_ws false: everything but the workspace (the size query, made before
// the caller has one)
int check_chunk(const pdn_chunk_fwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    if (a->B < 1 || a->H < 1 || a->T < 0 || a->dk < 1 || a->dv < 1) return PDN_EINVAL;
    if (!valid_dtype(a->qkv_dtype) || !valid_dtype(a->o_dtype)) return PDN_EINVAL;
    if (static_cast<long>(a->B) * a->H > kMaxBH) return PDN_EUNSUPPORTED;
    if (static_cast<long>(a->B) * a->H * a->T > kMaxTokens) return PDN_EUNSUPPORTED;
    int rc = check_gates(a->alpha_mode, a->log_alpha, a->beta_mode, a->beta, a->gamma_mode,
                         a->gamma, a->precond_eps, a->dk, a->dv, a->T > 0);
    if (rc != PDN_OK) return rc;
    if (!valid_key(a->key_mode)) return PDN_EINVAL;
    if (!valid_precond(a->precond_eps, a->precond_mode, a->precond_x)) return PDN_EINVAL;
    if (a->T > 0 && (!a->q || !a->k || !a->v || !a->o)) return PDN_EINVAL;
    // the kernels use 16-byte vector loads and stores
    const void* ptrs[] = {a->q, a->k, a->v, a->o, a->log_alpha, a->beta, a->gamma,
                          a->precond_A0, a->precond_AT, a->S0, a->ST,
                          check_ws ? a->workspace : nullptr};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return PDN_EINVAL;
    if (a->dk != 64 && a->dk != 128) return PDN_EUNSUPPORTED;
    if (a->dv % 16 != 0 || a->dv > 256) return PDN_EUNSUPPORTED;
    const bool vec = a->alpha_mode == PDN_ALPHA_VEC || a->beta_mode == PDN_GATE_VEC ||
                     a->precond_eps >= 0.0f;
    if (vec && a->dv % 32 != 0) return PDN_EUNSUPPORTED;
    // asymmetric keys and the stabilised preconditioner run on the bf16,
    // dk = 128 per-channel-gate kernels only
    const bool stabilised = a->precond_eps >= 0.0f && a->precond_mode == PDN_PRECOND_STABILISED;
    if ((a->key_mode != PDN_KEY_SYMMETRIC || stabilised) &&
        (a->qkv_dtype != PDN_BF16 || a->dk != 128 || a->dv % 32 != 0))
        return PDN_EUNSUPPORTED;
    if (a->S0 && a->ST && a->S0 != a->ST) {
        // distinct state buffers must not overlap
        const long n = static_cast<long>(a->B) * a->H * a->dk * a->dv;
        const float* s0 = a->S0;
        const float* st = a->ST;
        if (s0 < st + n && st < s0 + n) return PDN_EINVAL;
    }
    if (!check_ws) return PDN_OK;
    const size_t need = pdn::chunk_fwd_workspace_bytes(*a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return PDN_EWORKSPACE;
    return PDN_OK;
}

// B * H * T for the backward: its per-chunk grids stay below 2^31 workgroups
constexpr long kMaxBwdTokens = 1L << 35;

int check_bwd(const pdn_chunk_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_chunk_fwd_args& f = a->fwd;
    if (f.B < 1 || f.H < 1 || f.T < 0 || f.dk < 1 || f.dv < 1) return PDN_EINVAL;
    if (!valid_dtype(f.qkv_dtype)) return PDN_EINVAL;
    if (static_cast<long>(f.B) * f.H > kMaxBH) return PDN_EUNSUPPORTED;
    if (static_cast<long>(f.B) * f.H * f.T > kMaxBwdTokens) return PDN_EUNSUPPORTED;
    const bool data = f.T > 0;
    int rc = check_gates(f.alpha_mode, f.log_alpha, f.beta_mode, f.beta, f.gamma_mode, f.gamma,
                         f.precond_eps, f.dk, f.dv, data);
    if (rc != PDN_OK) return rc;
    if (!valid_key(f.key_mode)) return PDN_EINVAL;
    if (!valid_precond(f.precond_eps, f.precond_mode, f.precond_x)) return PDN_EINVAL;
    if (data) {
        if (!f.q || !f.k || !f.v || !a->dO || !a->dq || !a->dk || !a->dv || !a->dbeta)
            return PDN_EINVAL;
        if (f.alpha_mode != PDN_ALPHA_NONE && !a->dlog_alpha) return PDN_EINVAL;
        if (f.gamma_mode != PDN_GAMMA_SAME_AS_BETA && !a->dgamma) return PDN_EINVAL;
    }
    const void* ptrs[] = {f.q, f.k, f.v, f.log_alpha, f.beta, f.gamma, f.precond_A0, f.S0,
                          a->dO, a->dST, a->dq, a->dk, a->dv, a->dlog_alpha, a->dbeta,
                          a->dgamma, a->dS0, a->dA0, check_ws ? a->workspace : nullptr};
    for (const void* ptr : ptrs)
        if (ptr && !aligned16(ptr)) return PDN_EINVAL;
    if (f.dk != 64 && f.dk != 128) return PDN_EUNSUPPORTED;
    if (f.dv % 32 != 0 || f.dv > 256) return PDN_EUNSUPPORTED;
    if (!check_ws) return PDN_OK;
    const size_t need = pdn::chunk_bwd_workspace_bytes(*a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return PDN_EWORKSPACE;
    return PDN_OK;
}

int check_decode(const pdn_decode_args* a) {
    if (!a) return PDN_EINVAL;
    if (a->B < 1 || a->H < 1 || a->dk < 1 || a->dv < 1) return PDN_EINVAL;
    if (!valid_dtype(a->qkv_dtype) || !valid_dtype(a->o_dtype)) return PDN_EINVAL;
    if (!a->q || !a->k || !a->v || !a->o || !a->S) return PDN_EINVAL;
    int rc = check_gates(a->alpha_mode, a->log_alpha, a->beta_mode, a->beta, a->gamma_mode,
                         a->gamma, a->precond_eps, a->dk, a->dv, true);
    if (rc != PDN_OK) return rc;
    if (!valid_key(a->key_mode)) return PDN_EINVAL;
    if (!valid_precond(a->precond_eps, a->precond_mode, a->precond_x)) return PDN_EINVAL;
    if (a->precond_eps >= 0.0f && !a->precond_A) return PDN_EINVAL;
    if (!aligned16(a->S)) return PDN_EINVAL;  // streamed with 16-byte accesses
    if (static_cast<long>(a->B) * a->H > kMaxBH) return PDN_EUNSUPPORTED;
    if ((a->dk != 64 && a->dk != 128) || (a->dv != 64 && a->dv != 128)) return PDN_EUNSUPPORTED;
    return PDN_OK;
}

// ---- the operators around the recurrence ----

// B * T of the strided operators: their kernels index tokens in 32 bits.
constexpr long kMaxRows = 1L << 30;

int elt_bytes(int32_t dtype) { return dtype == PDN_BF16 ? 2 : 4; }

// A strided tensor: a pointer, the sizes of its dimensions but the last (which
// is contiguous, `width` elements) and their strides.
struct View {
    const void* p;
    int64_t size[3], stride[3];
    int64_t width;
    int bytes;
};

View view3(const void* p, int64_t s0, int64_t s1, int64_t s2, int64_t t0, int64_t t1, int64_t t2, int64_t width, int32_t dtype) {
    return View{p, {s0, s1, s2}, {t0, t1, t2}, width, elt_bytes(dtype)};
}

// Strides of a strided tensor (only dimensions longer than 1 are stepped
// over): not negative, every row 16-byte aligned, the whole within 63 bits;
// and, for an output, no row over another.
int check_view(const View& v, bool output) {
    if (!aligned16(v.p)) return PDN_EINVAL;
    constexpr int64_t kMost = int64_t{1} << 56;
    int64_t size[3], stride[3];
    int n = 0;
    __int128 reach = v.width;
    for (int i = 0; i < 3; ++i) {
        if (v.size[i] <= 1) continue;
        if (v.stride[i] < 0 || v.stride[i] > kMost) return PDN_EINVAL;
        if (v.stride[i] * v.bytes % 16 != 0) return PDN_EINVAL;
        reach += static_cast<__int128>(v.stride[i]) * (v.size[i] - 1);
        size[n] = v.size[i];
        stride[n++] = v.stride[i];
    }
    if (reach > kMost) return PDN_EINVAL;
    if (!output) return PDN_OK;
    // from the smallest stride up, each step passes all that lies below it
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (stride[j] < stride[i]) {
                const int64_t a = stride[i], b = size[i];
                stride[i] = stride[j];
                size[i] = size[j];
                stride[j] = a;
                size[j] = b;
            }
    int64_t span = v.width;
    for (int i = 0; i < n; ++i) {
        if (stride[i] < span) return PDN_EINVAL;
        span = stride[i] * (size[i] - 1) + span;
    }
    return PDN_OK;
}

bool valid_eps(float eps) { return std::isnormal(eps) && eps > 0.0f; }

int check_rows(int32_t B, int32_t H, int32_t T) {
    if (B < 1 || H < 1 || T < 0) return PDN_EINVAL;
    if (static_cast<long>(B) * H > kMaxBH) return PDN_EUNSUPPORTED;
    if (static_cast<long>(B) * T > kMaxRows || static_cast<long>(B) * H * T > kMaxTokens) return PDN_EUNSUPPORTED;
    return PDN_OK;
}

// backward: the forward's outputs are not read
int check_qk_norm(const pdn_qk_norm_args* a, bool backward = false) {
    if (!a) return PDN_EINVAL;
    int rc = check_rows(a->B, a->H, a->T);
    if (rc != PDN_OK) return rc;
    if (a->Hq < 1 || a->Hk < 1 || a->H % a->Hq != 0 || a->H % a->Hk != 0) return PDN_EINVAL;
    if (!valid_dtype(a->dtype)) return PDN_EINVAL;
    if (a->norm != PDN_NORM_NONE && a->norm != PDN_NORM_RMS && a->norm != PDN_NORM_L2) return PDN_EINVAL;
    if (a->norm != PDN_NORM_NONE ? !valid_eps(a->eps) : (a->wq || a->wk)) return PDN_EINVAL;
    if (!std::isfinite(a->q_scale) || !std::isfinite(a->k_scale)) return PDN_EINVAL;
    if ((a->d != 64 && a->d != 128) || !pdn::qk_norm_fits(*a)) return PDN_EUNSUPPORTED;
    if (a->rot_dim < 0 || a->rot_dim > a->d) return PDN_EINVAL;
    if (a->rot_dim % 16 != 0) return PDN_EUNSUPPORTED;
    if (a->rot_dim > 0) {
        if (a->rope_layout != PDN_ROPE_HALF && a->rope_layout != PDN_ROPE_INTERLEAVED) return PDN_EINVAL;
        if (!std::isfinite(a->rope_scale) || !a->inv_freq) return PDN_EINVAL;
    }
    if (a->T == 0) return PDN_OK;
    if (!a->xq || !a->xk || (!backward && (!a->q || !a->k))) return PDN_EINVAL;
    const void* ptrs[] = {a->inv_freq, a->positions, a->wq, a->wk, backward ? nullptr : a->q, backward ? nullptr : a->k};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return PDN_EINVAL;
    rc = check_view(view3(a->xq, a->B, a->T, a->Hq, a->xq_sb, a->xq_st, a->xq_sh, a->d, a->dtype), false);
    if (rc != PDN_OK) return rc;
    return check_view(view3(a->xk, a->B, a->T, a->Hk, a->xk_sb, a->xk_st, a->xk_sh, a->d, a->dtype), false);
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need == 0) return PDN_OK;
    if (workspace && !aligned16(workspace)) return PDN_EINVAL;
    return !workspace || bytes < need ? PDN_EWORKSPACE : PDN_OK;
}

int check_qk_norm_bwd(const pdn_qk_norm_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_qk_norm_args& f = a->fwd;
    int rc = check_qk_norm(&f, true);
    if (rc != PDN_OK) return rc;
    if ((f.wq != nullptr) != (a->dwq != nullptr) || (f.wk != nullptr) != (a->dwk != nullptr)) return PDN_EINVAL;
    const void* ptrs[] = {a->dq, a->dk, a->dwq, a->dwk};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return PDN_EINVAL;
    if (f.T > 0) {
        if (!a->dq || !a->dk || !a->dxq || !a->dxk) return PDN_EINVAL;
        rc = check_view(view3(a->dxq, f.B, f.T, f.Hq, a->dxq_sb, a->dxq_st, a->dxq_sh, f.d, f.dtype), true);
        if (rc != PDN_OK) return rc;
        rc = check_view(view3(a->dxk, f.B, f.T, f.Hk, a->dxk_sb, a->dxk_st, a->dxk_sh, f.d, f.dtype), true);
        if (rc != PDN_OK) return rc;
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::qk_norm_bwd_workspace_bytes(*a)) : PDN_OK;
}

int check_out_norm(const pdn_out_norm_args* a, bool backward = false) {
    if (!a) return PDN_EINVAL;
    int rc = check_rows(a->B, a->H, a->T);
    if (rc != PDN_OK) return rc;
    if (!valid_dtype(a->o_dtype) || !valid_dtype(a->dtype) || !valid_eps(a->eps) || a->dv < 1) return PDN_EINVAL;
    if (a->act != PDN_ACT_NONE && a->act != PDN_ACT_SILU && a->act != PDN_ACT_SIGMOID) return PDN_EINVAL;
    if (a->dv % 16 != 0 || a->dv > 256 || !pdn::out_norm_fits(*a)) return PDN_EUNSUPPORTED;
    if (a->w && !aligned16(a->w)) return PDN_EINVAL;
    if (a->T == 0) return PDN_OK;
    if (!a->o || !aligned16(a->o) || (a->z != nullptr) != (a->act != PDN_ACT_NONE)) return PDN_EINVAL;
    if (a->z) {
        rc = check_view(view3(a->z, a->B, a->T, a->H, a->z_sb, a->z_st, a->z_sh, a->dv, a->dtype), false);
        if (rc != PDN_OK) return rc;
    }
    if (backward) return PDN_OK;
    if (!a->y) return PDN_EINVAL;
    return check_view(view3(a->y, a->B, a->T, a->H, a->y_sb, a->y_st, a->y_sh, a->dv, a->dtype), true);
}

int check_out_norm_bwd(const pdn_out_norm_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_out_norm_args& f = a->fwd;
    int rc = check_out_norm(&f, true);
    if (rc != PDN_OK) return rc;
    if ((f.w != nullptr) != (a->dw != nullptr) || (a->dw && !aligned16(a->dw))) return PDN_EINVAL;
    if (f.T > 0) {
        if (!a->dy || !a->d_o || !aligned16(a->d_o) || (a->dz != nullptr) != (f.z != nullptr)) return PDN_EINVAL;
        rc = check_view(view3(a->dy, f.B, f.T, f.H, a->dy_sb, a->dy_st, a->dy_sh, f.dv, f.dtype), false);
        if (rc != PDN_OK) return rc;
        if (a->dz) {
            rc = check_view(view3(a->dz, f.B, f.T, f.H, a->dz_sb, a->dz_st, a->dz_sh, f.dv, f.dtype), true);
            if (rc != PDN_OK) return rc;
        }
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::out_norm_bwd_workspace_bytes(*a)) : PDN_OK;
}

bool valid_gain(int32_t g) { return g == PDN_GAIN_NONE || g == PDN_GAIN_COMPLEMENT || g == PDN_GAIN_NORM; }

// sizes, types and gain of the scan's calls
int check_scan_kind(int32_t B, int32_t T, int32_t D, int32_t dtype, int32_t log_dtype, int32_t gain) {
    if (B < 1 || T < 0 || D < 1) return PDN_EINVAL;
    if (!valid_dtype(dtype) || !valid_dtype(log_dtype) || !valid_gain(gain)) return PDN_EINVAL;
    if (D % 8 != 0 || (dtype == PDN_F32 && log_dtype == PDN_BF16)) return PDN_EUNSUPPORTED;
    if (static_cast<long>(B) * T > kMaxRows || static_cast<long>(B) * D > kMaxRows) return PDN_EUNSUPPORTED;
    return PDN_OK;
}

// a forward's arguments (backward: its outputs are not read)
int check_scan(const pdn_scan_args* a, bool backward = false, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    int rc = check_scan_kind(a->B, a->T, a->D, a->dtype, a->log_dtype, a->gain);
    if (rc != PDN_OK) return rc;
    if (!pdn::scan_fits(*a)) return PDN_EUNSUPPORTED;
    const void* ptrs[] = {a->h0, a->marks, backward ? nullptr : a->hT};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return PDN_EINVAL;
    if (a->T > 0) {
        if (!a->x || !a->log_a || (!backward && !a->h)) return PDN_EINVAL;
        rc = check_view(view3(a->x, a->B, a->T, 1, a->x_sb, a->x_st, 0, a->D, a->dtype), false);
        if (rc != PDN_OK) return rc;
        rc = check_view(view3(a->log_a, a->B, a->T, 1, a->log_a_sb, a->log_a_st, 0, a->D, a->log_dtype), false);
        if (rc != PDN_OK) return rc;
        if (!backward) rc = check_view(view3(a->h, a->B, a->T, 1, a->h_sb, a->h_st, 0, a->D, a->dtype), true);
        if (rc != PDN_OK) return rc;
    }
    if (backward || !check_ws) return PDN_OK;
    return check_workspace(a->workspace, a->workspace_bytes, pdn::scan_fwd_workspace_bytes(*a));
}

int check_scan_bwd(const pdn_scan_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_scan_args& f = a->fwd;
    int rc = check_scan(&f, true);
    if (rc != PDN_OK) return rc;
    if ((a->dhT && !aligned16(a->dhT)) || (a->dh0 && !aligned16(a->dh0))) return PDN_EINVAL;
    if (f.T > 0) {
        if (!a->dh || !a->dx || !a->dlog_a) return PDN_EINVAL;
        rc = check_view(view3(a->dh, f.B, f.T, 1, a->dh_sb, a->dh_st, 0, f.D, f.dtype), false);
        if (rc != PDN_OK) return rc;
        rc = check_view(view3(a->dx, f.B, f.T, 1, a->dx_sb, a->dx_st, 0, f.D, f.dtype), true);
        if (rc != PDN_OK) return rc;
        rc = check_view(view3(a->dlog_a, f.B, f.T, 1, a->dlog_a_sb, a->dlog_a_st, 0, f.D, f.log_dtype), true);
        if (rc != PDN_OK) return rc;
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::scan_bwd_workspace_bytes(*a)) : PDN_OK;
}

int check_scan_step(const pdn_scan_step_args* a) {
    if (!a) return PDN_EINVAL;
    int rc = check_scan_kind(a->B, 1, a->D, a->dtype, a->log_dtype, a->gain);
    if (rc != PDN_OK) return rc;
    if (!a->x || !a->log_a || !a->h_prev || !a->h_next || !a->h) return PDN_EINVAL;
    if (!aligned16(a->h_prev) || !aligned16(a->h_next)) return PDN_EINVAL;
    rc = check_view(view3(a->x, a->B, 1, 1, a->x_sb, 0, 0, a->D, a->dtype), false);
    if (rc != PDN_OK) return rc;
    rc = check_view(view3(a->log_a, a->B, 1, 1, a->log_a_sb, 0, 0, a->D, a->log_dtype), false);
    if (rc != PDN_OK) return rc;
    return check_view(view3(a->h, a->B, 1, 1, a->h_sb, 0, 0, a->D, a->dtype), true);
}

// The extern "C" bodies: an answer, a size or a launch, and no exception out.
template <class F>
int answer(F f) {
    try {
        return f();
    } catch (...) {
        return PDN_EINVAL;
    }
}

template <class A, class Check, class Launch>
int call(const A* args, void* stream, Check check, Launch launch) {
    try {
        const int rc = check(args);
        if (rc != PDN_OK) return rc;
        return launch(*args, static_cast<hipStream_t>(stream)) == hipSuccess ? PDN_OK : PDN_EHIP;
    } catch (...) {
        return PDN_EHIP;
    }
}

template <class A, class Check, class Size>
int size_of(const A* args, size_t* bytes, Check check, Size size) {
    if (!args || !bytes) return PDN_EINVAL;
    return answer([&] {
        const int rc = check(args);
        if (rc == PDN_OK) *bytes = size(*args);
        return rc;
    });
}

// Scratch of pdn_chunk_fwd_noalloc: one copy per GPU, loaded with the code
// object (no allocation call makes it).  In host code `scratch` is a host-side
// stand-in for the symbol, never a device address: every use goes through the
// per-device address from hipGetSymbolAddress below.
static __device__ __align__(256) unsigned char scratch[PDN_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;

// Device address of `scratch` on the current device, looked up once per device
// (with that device current) and kept; nullptr if HIP reports an error.
void* scratch_on_current_device() {
    static std::mutex mu;
    static void* addr[kMaxDevices] = {};
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

}  // namespace

namespace pdn {

int device_cu_count() {
    // queried once per device (decode launches ask on every step)
    static std::atomic<int> cached[kMaxDevices] = {};
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;  // the MI355X count; only grid sizes depend on it
    if (dev < kMaxDevices && (n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) return 256;
    if (dev < kMaxDevices) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace pdn

extern "C" {

int pdn_abi_version(void) { return PDN_ABI_VERSION; }

const char* pdn_strerror(int code) {
    switch (code) {
        case PDN_OK: return "success";
        case PDN_EINVAL: return "invalid argument (null pointer, size or enum value)";
        case PDN_EUNSUPPORTED: return "valid request outside what the kernels support";
        case PDN_EWORKSPACE: return "workspace missing or too small";
        case PDN_EHIP: return "HIP runtime error at launch";
        case PDN_ESCRATCH:
            return "call needs more scratch than pdn_chunk_fwd_noalloc holds "
                   "(PDN_NOALLOC_SCRATCH_BYTES): pass a workspace to pdn_chunk_fwd";
        default: return "unknown error code";
    }
}

int pdn_chunk_fwd_workspace_size(const pdn_chunk_fwd_args* args, size_t* bytes) {
    if (!args || !bytes) return PDN_EINVAL;
    try {
        // validate everything except the workspace itself, then size it (the
        // size arithmetic relies on the validated bounds)
        const int rc = check_chunk(args, false);
        if (rc != PDN_OK) return rc;
        *bytes = pdn::chunk_fwd_workspace_bytes(*args);
        return PDN_OK;
    } catch (...) {
        return PDN_EINVAL;
    }
}

int pdn_chunk_fwd_check(const pdn_chunk_fwd_args* args) {
    try {
        return check_chunk(args);
    } catch (...) {
        return PDN_EINVAL;
    }
}

int pdn_chunk_fwd(const pdn_chunk_fwd_args* args, void* stream) {
    try {
        const int rc = check_chunk(args);
        if (rc != PDN_OK) return rc;
        const hipError_t e = pdn::launch_chunk_fwd(*args, static_cast<hipStream_t>(stream));
        if (e == hipErrorNotSupported) return PDN_EUNSUPPORTED;
        return e == hipSuccess ? PDN_OK : PDN_EHIP;
    } catch (...) {
        return PDN_EHIP;
    }
}

int pdn_chunk_fwd_noalloc(const pdn_chunk_fwd_args* args, void* stream) {
    try {
        int rc = check_chunk(args, false);
        if (rc != PDN_OK) return rc;
        pdn_chunk_fwd_args a = *args;
        const size_t need = pdn::chunk_fwd_workspace_bytes(a);
        if (need > PDN_NOALLOC_SCRATCH_BYTES) return PDN_ESCRATCH;
        a.workspace = nullptr;
        a.workspace_bytes = 0;
        if (need > 0) {
            void* p = scratch_on_current_device();
            if (!p) return PDN_EHIP;
            a.workspace = p;
            a.workspace_bytes = PDN_NOALLOC_SCRATCH_BYTES;
        }
        const hipError_t e = pdn::launch_chunk_fwd(a, static_cast<hipStream_t>(stream));
        if (e == hipErrorNotSupported) return PDN_EUNSUPPORTED;
        return e == hipSuccess ? PDN_OK : PDN_EHIP;
    } catch (...) {
        return PDN_EHIP;
    }
}

int pdn_chunk_bwd_workspace_size(const pdn_chunk_bwd_args* args, size_t* bytes) {
    if (!args || !bytes) return PDN_EINVAL;
    try {
        const int rc = check_bwd(args, false);
        if (rc != PDN_OK) return rc;
        *bytes = pdn::chunk_bwd_workspace_bytes(*args);
        return PDN_OK;
    } catch (...) {
        return PDN_EINVAL;
    }
}

int pdn_chunk_bwd_check(const pdn_chunk_bwd_args* args) {
    try {
        return check_bwd(args);
    } catch (...) {
        return PDN_EINVAL;
    }
}

int pdn_chunk_bwd(const pdn_chunk_bwd_args* args, void* stream) {
    try {
        const int rc = check_bwd(args);
        if (rc != PDN_OK) return rc;
        const hipError_t e = pdn::launch_chunk_bwd(*args, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? PDN_OK : PDN_EHIP;
    } catch (...) {
        return PDN_EHIP;
    }
}

int pdn_decode_check(const pdn_decode_args* args) {
    try {
        return check_decode(args);
    } catch (...) {
        return PDN_EINVAL;
    }
}

int pdn_decode_step(const pdn_decode_args* args, void* stream) {
    try {
        const int rc = check_decode(args);
        if (rc != PDN_OK) return rc;
        const hipError_t e = pdn::launch_decode(*args, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? PDN_OK : PDN_EHIP;
    } catch (...) {
        return PDN_EHIP;
    }
}

int pdn_layer_version(void) { return PDN_LAYER_VERSION; }

int pdn_qk_norm_check(const pdn_qk_norm_args* args) { return answer([&] { return check_qk_norm(args); }); }
int pdn_qk_norm_bwd_check(const pdn_qk_norm_bwd_args* args) { return answer([&] { return check_qk_norm_bwd(args); }); }
int pdn_out_norm_check(const pdn_out_norm_args* args) { return answer([&] { return check_out_norm(args); }); }
int pdn_out_norm_bwd_check(const pdn_out_norm_bwd_args* args) { return answer([&] { return check_out_norm_bwd(args); }); }
int pdn_scan_check(const pdn_scan_args* args) { return answer([&] { return check_scan(args); }); }
int pdn_scan_bwd_check(const pdn_scan_bwd_args* args) { return answer([&] { return check_scan_bwd(args); }); }
int pdn_scan_step_check(const pdn_scan_step_args* args) { return answer([&] { return check_scan_step(args); }); }

int pdn_qk_norm_bwd_workspace_size(const pdn_qk_norm_bwd_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_qk_norm_bwd(a, false); }, pdn::qk_norm_bwd_workspace_bytes);
}
int pdn_out_norm_bwd_workspace_size(const pdn_out_norm_bwd_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_out_norm_bwd(a, false); }, pdn::out_norm_bwd_workspace_bytes);
}
int pdn_scan_fwd_workspace_size(const pdn_scan_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_scan(a, false, false); }, pdn::scan_fwd_workspace_bytes);
}
int pdn_scan_bwd_workspace_size(const pdn_scan_bwd_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_scan_bwd(a, false); }, pdn::scan_bwd_workspace_bytes);
}

int pdn_qk_norm_fwd(const pdn_qk_norm_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_qk_norm(a); }, pdn::launch_qk_norm);
}
int pdn_qk_norm_bwd(const pdn_qk_norm_bwd_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_qk_norm_bwd(a); }, pdn::launch_qk_norm_bwd);
}
int pdn_out_norm_fwd(const pdn_out_norm_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_out_norm(a); }, pdn::launch_out_norm);
}
int pdn_out_norm_bwd(const pdn_out_norm_bwd_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_out_norm_bwd(a); }, pdn::launch_out_norm_bwd);
}
int pdn_scan_fwd(const pdn_scan_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_scan(a); }, pdn::launch_scan_fwd);
}
int pdn_scan_bwd(const pdn_scan_bwd_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_scan_bwd(a); }, pdn::launch_scan_bwd);
}
int pdn_scan_step(const pdn_scan_step_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_scan_step(a); }, pdn::launch_scan_step);
}

int pdn_scan_marks(int32_t T) {
    return T < 0 ? PDN_EINVAL : static_cast<int>((static_cast<long>(T) + PDN_SCAN_MARK - 1) / PDN_SCAN_MARK);
}

int pdn_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, int64_t original_context,
                   double* inv_freq, float* rope_scale) {
    if (!inv_freq || !rope_scale || rot_dim < 2 || rot_dim % 2 != 0) return PDN_EINVAL;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) || original_context < 1)
        return PDN_EINVAL;
    if (scaling < PDN_ROPE_PLAIN || scaling > PDN_ROPE_BY_PARTS) return PDN_EINVAL;
    if (scaling == PDN_ROPE_BASE) {
        if (rot_dim < 4) return PDN_EINVAL;
        base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    }
    constexpr double kFewTurns = 1.0, kManyTurns = 32.0;
    constexpr double kTwoPi = 6.283185307179586;
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        double keep = 1.0;  // share of the frequency that is not divided
        if (scaling == PDN_ROPE_LINEAR) keep = 0.0;
        if (scaling == PDN_ROPE_BY_PARTS) {
            const double turns = static_cast<double>(original_context) * f / kTwoPi;
            keep = (turns - kFewTurns) / (kManyTurns - kFewTurns);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        }
        inv_freq[i] = keep * f + (1.0 - keep) * f / factor;
    }
    *rope_scale = scaling == PDN_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PDN_OK;
}

}  // extern "C"
