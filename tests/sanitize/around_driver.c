/* Drives the validation and workspace sizing of the operators around the
 * recurrence (nothing is launched) under AddressSanitizer and
 * UndefinedBehaviorSanitizer: from valid arguments, random fields set to
 * values from the edges of their ranges or to random bits.  Every answer is
 * one of the library's codes, and a call that a check accepts has a workspace
 * size that the check accepts too, and one byte less that it refuses.
 * Pointers are never dereferenced by these entry points. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "pdn_layer.h"

#define FAKE ((void *)(uintptr_t)0x10000)

/* splitmix64 (Steele, Lea and Flood, "Fast splittable pseudorandom number
 * generators", 2014) */
static uint64_t state = 0xa40dULL;
static uint64_t rnd(void) {
    uint64_t z = (state += 0x9e3779b97f4a7c15ULL);
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ULL;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebULL;
    return z ^ (z >> 31);
}

static long bad, accepted, total;

static int known(int rc) { return rc <= 0 && rc >= -5; }

/* some 4-byte words of a struct set to edges or random bits */
static void mutate(void *p, size_t bytes) {
    static const int32_t pick[] = {0, 1, 2, 3, -1, 8, 12, 16, 64, 72, 96, 128, 256, 1000, 1 << 16, 1 << 20, 1 << 30,
                                   INT32_MAX, INT32_MIN, 0x10000, 0x10004, 0x3f800000, 0x358637bd, 0x7fc00000};
    int n = (int)(rnd() % 5);
    while (n--) {
        int32_t v = rnd() % 8 ? pick[rnd() % (sizeof(pick) / sizeof(pick[0]))] : (int32_t)rnd();
        memcpy((char *)p + 4 * (rnd() % (bytes / 4)), &v, 4);
    }
}

static void fill_qk(pdn_qk_norm_args *a) {
    memset(a, 0, sizeof(*a));
    a->B = 2; a->T = 100; a->H = 8; a->Hq = 8; a->Hk = 2; a->d = 128; a->dtype = PDN_BF16;
    a->norm = PDN_NORM_RMS; a->eps = 1e-6f; a->q_scale = a->k_scale = a->rope_scale = 1.0f;
    a->rot_dim = 64; a->inv_freq = FAKE; a->positions = FAKE; a->wq = a->wk = FAKE;
    a->xq = a->xk = FAKE; a->q = a->k = FAKE;
    a->xq_sb = a->xk_sb = 230400; a->xq_st = a->xk_st = 2304; a->xq_sh = a->xk_sh = 128;
}
static void fill_out(pdn_out_norm_args *a) {
    memset(a, 0, sizeof(*a));
    a->B = 2; a->H = 8; a->T = 100; a->dv = 96; a->dtype = PDN_BF16; a->act = PDN_ACT_SILU; a->eps = 1e-6f;
    a->o = a->w = a->z = FAKE; a->y = FAKE;
    a->z_sb = a->y_sb = 76800; a->z_st = a->y_st = 768; a->z_sh = a->y_sh = 96;
}
static void fill_scan(pdn_scan_args *a) {
    memset(a, 0, sizeof(*a));
    a->B = 2; a->T = 1000; a->D = 72; a->dtype = PDN_BF16; a->gain = PDN_GAIN_NORM;
    a->x = a->log_a = FAKE; a->h0 = FAKE; a->hT = FAKE; a->h = FAKE; a->marks = rnd() % 2 ? FAKE : NULL;
    a->x_sb = a->log_a_sb = a->h_sb = 72000; a->x_st = a->log_a_st = a->h_st = 72;
}

#define SIZED(check, size, a)                                                       \
    do {                                                                            \
        size_t n = 0;                                                               \
        (a).workspace = FAKE;                                                       \
        (a).workspace_bytes = SIZE_MAX;                                             \
        int r1 = check(&(a)), r2 = size(&(a), &n);                                  \
        bad += !known(r1) || r1 != r2;                                              \
        if (r1 == PDN_OK) {                                                         \
            ++accepted;                                                             \
            (a).workspace_bytes = n;                                                \
            bad += check(&(a)) != PDN_OK;                                           \
            (a).workspace_bytes = n - 1;                                            \
            bad += n > 0 && check(&(a)) != PDN_EWORKSPACE;                          \
        }                                                                           \
        ++total;                                                                    \
    } while (0)
#define PLAIN(check, a)                                                             \
    do {                                                                            \
        int r = check(&(a));                                                        \
        bad += !known(r);                                                           \
        accepted += r == PDN_OK;                                                    \
        ++total;                                                                    \
    } while (0)

int main(void) {
    for (int i = 0; i < 100000; ++i) {
        pdn_qk_norm_args q;
        fill_qk(&q);
        mutate(&q, sizeof(q));
        PLAIN(pdn_qk_norm_check, q);
        pdn_qk_norm_bwd_args qb;
        memset(&qb, 0, sizeof(qb));
        fill_qk(&qb.fwd);
        qb.dq = qb.dk = FAKE; qb.dxq = qb.dxk = FAKE; qb.dwq = qb.dwk = FAKE;
        qb.dxq_sb = qb.dxk_sb = 128000; qb.dxq_st = qb.dxk_st = 1280; qb.dxq_sh = qb.dxk_sh = 128;
        mutate(&qb, sizeof(qb));
        SIZED(pdn_qk_norm_bwd_check, pdn_qk_norm_bwd_workspace_size, qb);
        pdn_out_norm_args o;
        fill_out(&o);
        mutate(&o, sizeof(o));
        PLAIN(pdn_out_norm_check, o);
        pdn_out_norm_bwd_args ob;
        memset(&ob, 0, sizeof(ob));
        fill_out(&ob.fwd);
        ob.dy = FAKE; ob.d_o = FAKE; ob.dz = FAKE; ob.dw = FAKE;
        ob.dy_sb = ob.dz_sb = 76800; ob.dy_st = ob.dz_st = 768; ob.dy_sh = ob.dz_sh = 96;
        mutate(&ob, sizeof(ob));
        SIZED(pdn_out_norm_bwd_check, pdn_out_norm_bwd_workspace_size, ob);
        pdn_scan_args s;
        fill_scan(&s);
        mutate(&s, sizeof(s));
        SIZED(pdn_scan_check, pdn_scan_fwd_workspace_size, s);
        pdn_scan_bwd_args sb;
        memset(&sb, 0, sizeof(sb));
        fill_scan(&sb.fwd);
        sb.dh = FAKE; sb.dhT = FAKE; sb.dx = FAKE; sb.dlog_a = FAKE; sb.dh0 = FAKE;
        sb.dh_sb = sb.dx_sb = sb.dlog_a_sb = 72000; sb.dh_st = sb.dx_st = sb.dlog_a_st = 72;
        mutate(&sb, sizeof(sb));
        SIZED(pdn_scan_bwd_check, pdn_scan_bwd_workspace_size, sb);
        pdn_scan_step_args t;
        memset(&t, 0, sizeof(t));
        t.B = 4; t.D = 72; t.dtype = PDN_BF16; t.log_dtype = PDN_BF16; t.gain = PDN_GAIN_COMPLEMENT;
        t.x = t.log_a = FAKE; t.h_prev = FAKE; t.h_next = FAKE; t.h = FAKE;
        t.x_sb = t.log_a_sb = t.h_sb = 72;
        mutate(&t, sizeof(t));
        PLAIN(pdn_scan_step_check, t);
        double f[64];
        float scale;
        int32_t rot = (int32_t)(rnd() % 140) - 4;
        if (rot > 128) rot = INT32_MIN;
        int rc = pdn_rope_freqs(rot, (double)(rnd() % 100000), (int32_t)(rnd() % 6) - 1, (double)(rnd() % 64) / 4.0,
                                (int64_t)(rnd() % 100000) - 10, f, &scale);
        bad += !known(rc);
    }
    printf("%ld argument sets, %ld accepted, %ld inconsistent answers\n", total, accepted, bad);
    return bad != 0;
}
