// New tokens' keys and values into a paged cache: copies of 16 bytes a lane, each
// read and written once.  A sequence's tokens lie in rows of their own here and in
// pages there; both are runs of a head's d channels.  Bound by bytes (16 sequences of
// up to 2048 new tokens, Hk8 d128: 137 MB at 6.2 TB/s), and for single tokens by the
// launch (256 of them 2.8 us).
#include "block.h"
#include "common.h"
#include "pages.h"
#include "rows.h"

namespace pdn {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
    const char *k, *v;
    char *k_pages, *v_pages;
    long k_sn, k_sh, v_sn, v_sh;                // bytes, as all strides here
    long kp_sp, kp_st, kp_sh, vp_sp, vp_st, vp_sh;
    int max_new, Hk, chunks;                    // chunks: 16-byte pieces of a head's row
    int groups;                                 // workgroups of a sequence
    PageMap map;
};

__global__ void __launch_bounds__(kThreads) cache_append_kernel(AppendParams p) {
    const int b = blockIdx.x / p.groups, group = blockIdx.x - b * p.groups;
    const Sequence s = sequence_of(p.map, b);
    const int n = min(s.n, p.max_new);
    const int row = p.Hk * p.chunks;            // pieces of a token's keys
    const long all = static_cast<long>(n) * row;
    for (long i = static_cast<long>(group) * kThreads + threadIdx.x; i < all; i += static_cast<long>(p.groups) * kThreads) {
        const int t = static_cast<int>(i / row), piece = static_cast<int>(i - static_cast<long>(t) * row);
        const int head = piece / p.chunks, c = piece - head * p.chunks;
        // a token or page that is not there is left out, where the reads are held to those that are
        const long want = static_cast<long>(p.map.lens[b]) - s.n + t;
        if (want < 0 || want >= p.map.width << p.map.shift) continue;
        const int token = static_cast<int>(want);
        const int page = p.map.table[static_cast<long>(b) * p.map.width + (token >> p.map.shift)];
        if (page < 0 || page >= p.map.pages) continue;
        const int in = token & ((1 << p.map.shift) - 1);
        const long from = s.start + t;
        const u32x4 k = *reinterpret_cast<const u32x4*>(p.k + from * p.k_sn + head * p.k_sh + 16 * c);
        const u32x4 v = *reinterpret_cast<const u32x4*>(p.v + from * p.v_sn + head * p.v_sh + 16 * c);
        *reinterpret_cast<u32x4*>(p.k_pages + page * p.kp_sp + in * p.kp_st + head * p.kp_sh + 16 * c) = k;
        *reinterpret_cast<u32x4*>(p.v_pages + page * p.vp_sp + in * p.vp_st + head * p.vp_sh + 16 * c) = v;
    }
}

// Pieces that a lane copies, at most, before a sequence gets another workgroup (those 16
// sequences: one 22.7 us, two 22.8, eight 23.6, 32 33.9).
constexpr int kPieces = 2;

}  // namespace

PageMap page_map(const pdn_cache& c) {
    PageMap m{};
    m.table = c.table;
    m.lens = c.lens;
    m.starts = c.starts;
    m.B = c.B;
    m.N = c.N;
    m.width = c.table_width;
    m.pages = c.pages;
    m.shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
    return m;
}

hipError_t launch_cache_append(const pdn_cache_append_args& a, hipStream_t stream) {
    const pdn_cache& c = a.cache;
    if (c.N == 0 || c.max_new == 0) return hipSuccess;
    const long e = c.dtype == PDN_BF16 ? 2 : 4;
    AppendParams p{};
    p.k = static_cast<const char*>(a.k);
    p.v = static_cast<const char*>(a.v);
    p.k_pages = static_cast<char*>(c.k_pages);
    p.v_pages = static_cast<char*>(c.v_pages);
    p.k_sn = a.k_sn * e, p.k_sh = a.k_sh * e, p.v_sn = a.v_sn * e, p.v_sh = a.v_sh * e;
    p.kp_sp = c.k_sp * e, p.kp_st = c.k_st * e, p.kp_sh = c.k_sh * e;
    p.vp_sp = c.v_sp * e, p.vp_st = c.v_st * e, p.vp_sh = c.v_sh * e;
    p.max_new = c.max_new;
    p.Hk = c.Hk;
    p.chunks = static_cast<int>(c.d * e / 16);
    const long most = static_cast<long>(c.max_new) * c.Hk * p.chunks;
    long groups = (most + kThreads * kPieces - 1) / (kThreads * kPieces);
    const long room = (1L << 22) / c.B;  // the launch's limit, far above what fills the device
    if (groups > room) groups = room > 1 ? room : 1;
    p.groups = static_cast<int>(groups);
    p.map = page_map(c);
    cache_append_kernel<<<dim3(static_cast<unsigned>(groups * c.B)), dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace pdn
