// Argument checks that the host layers share: pointers, strided tensors,
// workspaces, and the frame of an extern "C" call.  Host code; not a public header.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "pdn.h"

namespace pdn {
namespace checks {

inline bool valid_dtype(int32_t d) { return d == PDN_F32 || d == PDN_BF16; }

// Largest B*H (and B*H*T) the launch grids and 32/64-bit index math accept.
constexpr long kMaxBH = 1L << 24;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// B * T of the strided operators: their kernels index tokens in 32 bits.
constexpr long kMaxRows = 1L << 30;

inline int elt_bytes(int32_t dtype) { return dtype == PDN_BF16 ? 2 : 4; }

// A strided tensor: a pointer, the sizes of its dimensions but the last (which
// is contiguous, `width` elements) and their strides.
struct View {
    const void* p;
    int64_t size[3], stride[3];
    int64_t width;
    int bytes;
};

inline View view3(const void* p, int64_t s0, int64_t s1, int64_t s2, int64_t t0, int64_t t1, int64_t t2, int64_t width, int32_t dtype) {
    return View{p, {s0, s1, s2}, {t0, t1, t2}, width, elt_bytes(dtype)};
}

// Strides of a strided tensor (only dimensions longer than 1 are stepped
// over): not negative, every row 16-byte aligned, the whole within 63 bits;
// and, for an output, no row over another.
inline int check_view(const View& v, bool output) {
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

inline bool valid_eps(float eps) { return std::isnormal(eps) && eps > 0.0f; }

inline int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need == 0) return PDN_OK;
    if (workspace && !aligned16(workspace)) return PDN_EINVAL;
    return !workspace || bytes < need ? PDN_EWORKSPACE : PDN_OK;
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

}  // namespace checks
}  // namespace pdn
