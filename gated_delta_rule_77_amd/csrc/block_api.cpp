// Host layer of the operators declared in pdn_block.h: validation before any HIP
// call, then the launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "block.h"
#include "checks.h"
#include "pdn_block.h"

namespace {

using namespace pdn::checks;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// B * T of the seam: a row takes 512 lanes at most, and a launch has 2^32.
constexpr long kMaxSeamRows = 1L << 23;
constexpr int kMaxSeamWidth = 16384;
constexpr int kMaxShared = 1 << 10;   // query heads of a key head
constexpr long kMaxSequences = 1L << 20;
// Elements from one token to the next that the loads of whole tiles take: their lanes'
// offsets are 32 bits, over seven tokens of 2-byte elements or three of 4 bytes.
constexpr int64_t kMaxTokenStep = int64_t{1} << 28;

// the types a call's outputs may have: bf16 only where its inputs do
bool valid_out(int32_t out, int32_t in) { return out == PDN_F32 || (out == PDN_BF16 && in == PDN_BF16); }

// [B,T,D] rows of a type
int rows3(const void* p, int32_t B, int32_t T, int32_t D, int64_t sb, int64_t st, int32_t dtype, bool output) {
    if (!p) return PDN_EINVAL;
    if (dtype != PDN_E4M3) return check_view(view3(p, B, T, 1, sb, st, 0, D, dtype), output);
    // a byte an element, rows at multiples of 8: as pairs, so that the common check's 16 bytes are 8 of them
    if ((B > 1 && sb % 8 != 0) || (T > 1 && st % 8 != 0)) return PDN_EINVAL;
    View v{p, {B, T, 1}, {2 * sb, 2 * st, 0}, 2 * static_cast<int64_t>(D), 1};
    if ((B > 1 && sb > (int64_t{1} << 55)) || (T > 1 && st > (int64_t{1} << 55))) return PDN_EINVAL;
    return check_view(v, output);
}

int check_seam(int32_t B, int32_t T, int32_t D, int32_t dtype, int32_t s_dtype, float eps, float drop_p, const int64_t* seed,
               const float* w) {
    if (B < 1 || T < 0 || D < 1 || !valid_dtype(dtype) || !valid_dtype(s_dtype) || !valid_eps(eps)) return PDN_EINVAL;
    if (!(drop_p >= 0.0f && drop_p < 1.0f) || (drop_p > 0.0f) != (seed != nullptr) || !aligned(seed, 8)) return PDN_EINVAL;
    if (w && !aligned16(w)) return PDN_EINVAL;
    if (D % 8 != 0 || D > kMaxSeamWidth || !valid_out(s_dtype, dtype)) return PDN_EUNSUPPORTED;
    if (static_cast<long>(B) * T >= kMaxSeamRows) return PDN_EUNSUPPORTED;
    return PDN_OK;
}

// one buffer under two names has one set of strides
bool one_buffer(const void* p, int64_t pb, int64_t pt, const void* q, int64_t qb, int64_t qt, int32_t B, int32_t T) {
    return p != q || ((B == 1 || pb == qb) && (T == 1 || pt == qt));
}

int check_add_norm(const pdn_add_norm_args* a) {
    if (!a) return PDN_EINVAL;
    int rc = check_seam(a->B, a->T, a->D, a->dtype, a->s_dtype, a->eps, a->drop_p, a->seed, a->w);
    if (rc != PDN_OK) return rc;
    const bool small = a->y_dtype == PDN_E4M3;
    if (!valid_dtype(a->y_dtype) && !small) return PDN_EINVAL;
    if (small != (a->y_scale != nullptr) || !aligned(a->y_scale, 4)) return PDN_EINVAL;
    if (a->group != 0 && (!small || (a->group != 32 && a->group != 64 && a->group != 128) || a->D % a->group != 0)) return PDN_EINVAL;
    const bool sum = a->res || a->drop_p > 0.0f;
    if (sum != (a->s != nullptr) || (!sum && a->s_dtype != a->dtype)) return PDN_EINVAL;
    if (a->T == 0) return PDN_OK;
    rc = rows3(a->x, a->B, a->T, a->D, a->x_sb, a->x_st, a->dtype, false);
    if (rc == PDN_OK && a->res) rc = rows3(a->res, a->B, a->T, a->D, a->res_sb, a->res_st, a->s_dtype, false);
    if (rc == PDN_OK && a->s) rc = rows3(a->s, a->B, a->T, a->D, a->s_sb, a->s_st, a->s_dtype, true);
    if (rc == PDN_OK) rc = rows3(a->y, a->B, a->T, a->D, a->y_sb, a->y_st, a->y_dtype, true);
    if (rc != PDN_OK) return rc;
    if (a->s && !one_buffer(a->s, a->s_sb, a->s_st, a->res, a->res_sb, a->res_st, a->B, a->T)) return PDN_EINVAL;
    if (a->s && a->s == a->x && (a->res || a->s_dtype != a->dtype)) return PDN_EINVAL;
    if (a->s && !one_buffer(a->s, a->s_sb, a->s_st, a->x, a->x_sb, a->x_st, a->B, a->T)) return PDN_EINVAL;
    return PDN_OK;
}

int check_add_norm_bwd(const pdn_add_norm_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    int rc = check_seam(a->B, a->T, a->D, a->dtype, a->s_dtype, a->eps, a->drop_p, a->seed, a->w);
    if (rc != PDN_OK) return rc;
    if (!valid_dtype(a->y_dtype)) return PDN_EINVAL;
    if ((a->w != nullptr) != (a->dw != nullptr) || !aligned16(a->dw)) return PDN_EINVAL;
    if (a->T > 0) {
        rc = rows3(a->s, a->B, a->T, a->D, a->s_sb, a->s_st, a->s_dtype, false);
        if (rc == PDN_OK) rc = rows3(a->dy, a->B, a->T, a->D, a->dy_sb, a->dy_st, a->y_dtype, false);
        if (rc == PDN_OK && a->ds) rc = rows3(a->ds, a->B, a->T, a->D, a->ds_sb, a->ds_st, a->s_dtype, false);
        if (rc == PDN_OK) rc = rows3(a->dres, a->B, a->T, a->D, a->dres_sb, a->dres_st, a->s_dtype, true);
        if (rc == PDN_OK && a->dx) rc = rows3(a->dx, a->B, a->T, a->D, a->dx_sb, a->dx_st, a->dtype, true);
        if (rc != PDN_OK) return rc;
        if (!one_buffer(a->dres, a->dres_sb, a->dres_st, a->ds, a->ds_sb, a->ds_st, a->B, a->T)) return PDN_EINVAL;
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::add_norm_bwd_workspace_bytes(*a)) : PDN_OK;
}

bool valid_scale(float s) { return std::isfinite(s * 1.4427f) && s > 0.0f; }
bool near(int64_t tokens, int64_t step) { return tokens <= 1 || step <= kMaxTokenStep; }

int check_attn(const pdn_attn_args* a, bool backward = false, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    if (a->B < 1 || a->H < 1 || a->Hk < 1 || a->Tq < 0 || a->Tk < 0 || a->d < 1 || a->H % a->Hk != 0) return PDN_EINVAL;
    if (!valid_dtype(a->dtype) || !valid_dtype(a->o_dtype) || a->window < 0 || !valid_scale(a->scale)) return PDN_EINVAL;
    if ((a->d != 64 && a->d != 128) || !valid_out(a->o_dtype, a->dtype)) return PDN_EUNSUPPORTED;
    if (static_cast<long>(a->B) * a->H > kMaxBH || a->H / a->Hk > kMaxShared) return PDN_EUNSUPPORTED;
    if (static_cast<long>(a->Tq) * (a->H / a->Hk) > kMaxRows || a->Tk > kMaxRows || !pdn::attn_fits(*a)) return PDN_EUNSUPPORTED;
    if (!aligned(a->first, 4) || !aligned(a->lse, 4)) return PDN_EINVAL;
    if (a->Tq > 0) {
        if (!a->q || !a->o || (backward && !a->lse)) return PDN_EINVAL;
        int rc = check_view(view3(a->q, a->B, a->H, a->Tq, a->q_sb, a->q_sh, a->q_st, a->d, a->dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(a->o, a->B, a->H, a->Tq, a->o_sb, a->o_sh, a->o_st, a->d, a->o_dtype), !backward);
        if (rc != PDN_OK) return rc;
    }
    if (a->Tk > 0 && a->Tq > 0) {
        if (!a->k || !a->v) return PDN_EINVAL;
        int rc = check_view(view3(a->k, a->B, a->Hk, a->Tk, a->k_sb, a->k_sh, a->k_st, a->d, a->dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(a->v, a->B, a->Hk, a->Tk, a->v_sb, a->v_sh, a->v_st, a->d, a->dtype), false);
        if (rc != PDN_OK) return rc;
        if (!near(a->Tk, a->k_st) || !near(a->Tk, a->v_st)) return PDN_EUNSUPPORTED;
    }
    if (backward || !check_ws) return PDN_OK;
    return check_workspace(a->workspace, a->workspace_bytes, pdn::attn_fwd_workspace_bytes(*a));
}

int check_attn_bwd(const pdn_attn_bwd_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_attn_args& f = a->fwd;
    int rc = check_attn(&f, true);
    if (rc != PDN_OK) return rc;
    if (!valid_dtype(a->g_dtype)) return PDN_EINVAL;
    if (!valid_out(a->g_dtype, f.dtype)) return PDN_EUNSUPPORTED;
    if (f.Tq > 0) {
        if (!a->d_o || !a->dq) return PDN_EINVAL;
        rc = check_view(view3(a->d_o, f.B, f.H, f.Tq, a->do_sb, a->do_sh, a->do_st, f.d, f.o_dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(a->dq, f.B, f.H, f.Tq, a->dq_sb, a->dq_sh, a->dq_st, f.d, a->g_dtype), true);
        if (rc != PDN_OK) return rc;
        if (!near(f.Tq, f.q_st) || !near(f.Tq, a->do_st)) return PDN_EUNSUPPORTED;
    }
    if (f.Tk > 0) {
        // with no queries their gradients are zeros, and k and v are still read
        if (!a->dk || !a->dv || !f.k || !f.v) return PDN_EINVAL;
        rc = check_view(view3(f.k, f.B, f.Hk, f.Tk, f.k_sb, f.k_sh, f.k_st, f.d, f.dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(f.v, f.B, f.Hk, f.Tk, f.v_sb, f.v_sh, f.v_st, f.d, f.dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(a->dk, f.B, f.Hk, f.Tk, a->dk_sb, a->dk_sh, a->dk_st, f.d, a->g_dtype), true);
        if (rc == PDN_OK) rc = check_view(view3(a->dv, f.B, f.Hk, f.Tk, a->dv_sb, a->dv_sh, a->dv_st, f.d, a->g_dtype), true);
        if (rc != PDN_OK) return rc;
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::attn_bwd_workspace_bytes(*a)) : PDN_OK;
}

// written: the call writes into the pages
int check_cache(const pdn_cache& c, bool written) {
    if (c.B < 1 || c.N < 0 || c.max_new < 0 || c.Hk < 1 || c.d < 1 || c.pages < 1 || c.table_width < 1) return PDN_EINVAL;
    if (!valid_dtype(c.dtype) || c.page_size < 1) return PDN_EINVAL;
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0) return PDN_EUNSUPPORTED;
    if (c.d % 8 != 0) return PDN_EUNSUPPORTED;
    if (!c.starts && (c.N % c.B != 0 || c.max_new < c.N / c.B)) return PDN_EINVAL;
    if (c.B > kMaxSequences || static_cast<long>(c.B) * c.Hk > kMaxBH) return PDN_EUNSUPPORTED;
    if (static_cast<long>(c.table_width) * c.page_size > kMaxRows || c.N > kMaxRows) return PDN_EUNSUPPORTED;
    if (!c.k_pages || !c.v_pages || !c.table || !c.lens) return PDN_EINVAL;
    if (!aligned(c.table, 4) || !aligned(c.lens, 4) || !aligned(c.starts, 4)) return PDN_EINVAL;
    const int rc = check_view(view3(c.k_pages, c.pages, c.page_size, c.Hk, c.k_sp, c.k_st, c.k_sh, c.d, c.dtype), written);
    if (rc != PDN_OK) return rc;
    return check_view(view3(c.v_pages, c.pages, c.page_size, c.Hk, c.v_sp, c.v_st, c.v_sh, c.d, c.dtype), written);
}

int check_append(const pdn_cache_append_args* a) {
    if (!a) return PDN_EINVAL;
    const pdn_cache& c = a->cache;
    int rc = check_cache(c, true);
    if (rc != PDN_OK) return rc;
    if (c.d > 1024) return PDN_EUNSUPPORTED;
    if (static_cast<long>(c.Hk) * c.d > (1L << 24)) return PDN_EUNSUPPORTED;
    if (c.N == 0) return PDN_OK;
    if (!a->k || !a->v) return PDN_EINVAL;
    rc = check_view(view3(a->k, c.N, c.Hk, 1, a->k_sn, a->k_sh, 0, c.d, c.dtype), false);
    if (rc != PDN_OK) return rc;
    return check_view(view3(a->v, c.N, c.Hk, 1, a->v_sn, a->v_sh, 0, c.d, c.dtype), false);
}

int check_paged(const pdn_attn_paged_args* a, bool check_ws = true) {
    if (!a) return PDN_EINVAL;
    const pdn_cache& c = a->cache;
    int rc = check_cache(c, false);
    if (rc != PDN_OK) return rc;
    if (a->H < 1 || a->H % c.Hk != 0 || !valid_dtype(a->o_dtype) || a->window < 0 || !valid_scale(a->scale)) return PDN_EINVAL;
    if ((c.d != 64 && c.d != 128) || !valid_out(a->o_dtype, c.dtype)) return PDN_EUNSUPPORTED;
    if (static_cast<long>(c.B) * a->H > kMaxBH || a->H / c.Hk > kMaxShared) return PDN_EUNSUPPORTED;
    if (static_cast<long>(c.max_new) * (a->H / c.Hk) > kMaxRows || !pdn::attn_paged_fits(*a)) return PDN_EUNSUPPORTED;
    if (!near(c.page_size, c.k_st) || !near(c.page_size, c.v_st)) return PDN_EUNSUPPORTED;
    if (!aligned(a->lse, 4)) return PDN_EINVAL;
    if (c.N > 0) {
        if (!a->q || !a->o) return PDN_EINVAL;
        rc = check_view(view3(a->q, c.N, a->H, 1, a->q_sn, a->q_sh, 0, c.d, c.dtype), false);
        if (rc == PDN_OK) rc = check_view(view3(a->o, c.N, a->H, 1, a->o_sn, a->o_sh, 0, c.d, a->o_dtype), true);
        if (rc != PDN_OK) return rc;
    }
    return check_ws ? check_workspace(a->workspace, a->workspace_bytes, pdn::attn_paged_workspace_bytes(*a)) : PDN_OK;
}

}  // namespace

extern "C" {

int pdn_block_version(void) { return PDN_BLOCK_VERSION; }

int pdn_add_norm_check(const pdn_add_norm_args* args) { return answer([&] { return check_add_norm(args); }); }
int pdn_add_norm_bwd_check(const pdn_add_norm_bwd_args* args) { return answer([&] { return check_add_norm_bwd(args); }); }
int pdn_attn_check(const pdn_attn_args* args) { return answer([&] { return check_attn(args); }); }
int pdn_attn_bwd_check(const pdn_attn_bwd_args* args) { return answer([&] { return check_attn_bwd(args); }); }
int pdn_cache_append_check(const pdn_cache_append_args* args) { return answer([&] { return check_append(args); }); }
int pdn_attn_paged_check(const pdn_attn_paged_args* args) { return answer([&] { return check_paged(args); }); }

int pdn_add_norm_bwd_workspace_size(const pdn_add_norm_bwd_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_add_norm_bwd(a, false); }, pdn::add_norm_bwd_workspace_bytes);
}
int pdn_attn_fwd_workspace_size(const pdn_attn_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_attn(a, false, false); }, pdn::attn_fwd_workspace_bytes);
}
int pdn_attn_bwd_workspace_size(const pdn_attn_bwd_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_attn_bwd(a, false); }, pdn::attn_bwd_workspace_bytes);
}
int pdn_attn_paged_workspace_size(const pdn_attn_paged_args* args, size_t* bytes) {
    return size_of(args, bytes, [](auto* a) { return check_paged(a, false); }, pdn::attn_paged_workspace_bytes);
}

int pdn_add_norm_fwd(const pdn_add_norm_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_add_norm(a); }, pdn::launch_add_norm);
}
int pdn_add_norm_bwd(const pdn_add_norm_bwd_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_add_norm_bwd(a); }, pdn::launch_add_norm_bwd);
}
int pdn_attn_fwd(const pdn_attn_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_attn(a); }, pdn::launch_attn_fwd);
}
int pdn_attn_bwd(const pdn_attn_bwd_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_attn_bwd(a); }, pdn::launch_attn_bwd);
}
int pdn_cache_append(const pdn_cache_append_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_append(a); }, pdn::launch_cache_append);
}
int pdn_attn_paged(const pdn_attn_paged_args* args, void* stream) {
    return call(args, stream, [](auto* a) { return check_paged(a); }, pdn::launch_attn_paged);
}

}  // extern "C"
