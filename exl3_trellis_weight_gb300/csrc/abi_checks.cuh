// abi_checks.cuh -- argument checks and workspace layout of the entry points in
// linear_abi.cu and layer_abi.cu.
#pragma once

#include "common.cuh"

namespace exl3 {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = 1ll << 24;
constexpr int64_t kMaxSide = 1ll << 16;

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline exl3_status need(const void *p, const char *name, size_t al) {
    if (!p)
        return set_error(EXL3_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, al))
        return set_error(EXL3_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, al);
    return EXL3_OK;
}

struct Rows {             // [T, n] activations or results of `size`-byte elements
    const void *p;
    int64_t T, n, stride;
    int size = 2;
    size_t bytes() const { return T > 0 ? (size_t)((T - 1) * stride + n) * size : 0; }
};

inline exl3_status check_rows(const Rows &r, const char *name) {
    exl3_status st;
    if (r.T == 0)
        return EXL3_OK;
    if ((st = need(r.p, name, r.size)) != EXL3_OK) return st;
    if (r.stride < r.n || r.stride > (1ll << 32))
        return set_error(EXL3_ERR_INVALID_ARG, "%s: row stride %lld is not in [%lld, 2^32]", name,
                         (long long)r.stride, (long long)r.n);
    return EXL3_OK;
}

inline exl3_status check_apart(const Rows &out, const char *name, const void *p, size_t bytes, const char *other) {
    const uintptr_t a = (uintptr_t)out.p, b = (uintptr_t)p;
    if (p && out.T > 0 && bytes && a < b + bytes && b < a + out.bytes())
        return set_error(EXL3_ERR_INVALID_ARG, "%s overlaps %s", name, other);
    return EXL3_OK;
}

// the same for rows that may stand side by side with the result's: with one stride, rows
// whose columns share no place modulo the stride never meet
inline exl3_status check_apart(const Rows &out, const char *name, const Rows &r, const char *other) {
    if (out.T > 1 && r.T > 1 && out.stride == r.stride && out.size == r.size) {
        const int64_t step = out.stride * out.size, between = (int64_t)((uintptr_t)r.p - (uintptr_t)out.p) % step;
        const int64_t at = between < 0 ? between + step : between;
        if (at >= out.n * out.size && at + r.n * out.size <= step)
            return EXL3_OK;
    }
    return check_apart(out, name, r.p, r.bytes(), other);
}

// workspace: bump allocation at 256-byte boundaries; with a null base it counts
struct Carve {
    unsigned char *p;
    size_t used = 0;
    template <typename T> T *take(size_t n) {
        T *q = p ? reinterpret_cast<T *>(p + used) : nullptr;
        used += align_up(n * sizeof(T), kAlign);
        return q;
    }
};

inline exl3_status check_ws(const void *ws, size_t have, size_t want) {
    if (!ws || !aligned(ws, kAlign))
        return set_error(EXL3_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
    if (have < want)
        return set_error(EXL3_ERR_WORKSPACE, "workspace %zu bytes < %zu", have, want);
    return EXL3_OK;
}

}  // namespace exl3
