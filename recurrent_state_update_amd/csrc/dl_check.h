// dl_check.h -- argument checks shared by the C ABI's host files.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "deltalog.h"

namespace dl::host {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(int t) { return t == DL_F32 || t == DL_BF16; }
inline size_t elem(int t) { return t == DL_BF16 ? 2 : 4; }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// eps > 0 keeps the norm of a zero row finite; NaN is refused
inline bool eps_ok(float eps) { return eps > 0.f && eps < 1e30f; }

struct Span {
    const void *p;
    size_t bytes;
};

inline bool overlap(Span a, Span b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

// Whether a written buffer overlaps another written or a read one.
template <int NW, int NR> bool clash(const Span (&w)[NW], const Span (&r)[NR])
{
    for (int i = 0; i < NW; ++i) {
        for (int j = i + 1; j < NW; ++j)
            if (overlap(w[i], w[j]))
                return true;
        for (int j = 0; j < NR; ++j)
            if (overlap(w[i], r[j]))
                return true;
    }
    return false;
}

} // namespace dl::host
