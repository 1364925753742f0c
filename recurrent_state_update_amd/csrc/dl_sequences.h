// dl_sequences.h -- packed sequences, and rows of channels, as the kernels of state
// space layers read them.
#pragma once

#include <hip/hip_runtime.h>

namespace dl {

// The tokens of sequence n: offsets out of range or out of order give an empty
// or a wrong sequence, and never a row that is not there.
struct Sequences {
    const int *cu;
    int T, N;
    __device__ __forceinline__ int at(int n) const
    {
        if (!cu)
            return n * (T / N);
        const int x = cu[n];
        return x < 0 ? 0 : x > T ? T : x;
    }
    // The sequence that slot `slot` of segments of `seg` tokens belongs to:
    // sequence n has the slots from at(n) / seg + n on, and more than it needs.
    __device__ __forceinline__ int of_slot(int slot, int seg) const
    {
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (at(mid) / seg + mid <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
    // The last sequence that starts at token t or ahead of it (the first, if none does).
    __device__ __forceinline__ int of_token(int t) const
    {
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (at(mid) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

// The first n of V consecutive elements of a row.  VEC: rows are whole vectors, and n
// is V or more, or not above 0.  Loads are not conditional, so that nothing waits for
// them before they are used: p is readable (its first element; VEC: the vector)
// whatever n is, and keep() drops what is not there.
template <int V, typename T, bool VEC> struct Cells {
    using Vec = T __attribute__((ext_vector_type(V)));
    Vec v;
    __device__ __forceinline__ void load(const T *p, int n)
    {
        if constexpr (VEC)
            v = *reinterpret_cast<const Vec *>(p);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = p[i < n ? i : 0];
    }
    __device__ __forceinline__ void keep(int n)
    {
        if constexpr (VEC && V * sizeof(T) >= 4) {
            using Bits = unsigned __attribute__((ext_vector_type(V * sizeof(T) / 4)));
            v = __builtin_bit_cast(Vec, n > 0 ? __builtin_bit_cast(Bits, v) : Bits{});
        } else
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = i < n ? v[i] : static_cast<T>(0.f);
    }
    __device__ __forceinline__ void zero() { keep(0); }
    __device__ __forceinline__ void store(T *p, int n) const
    {
        if constexpr (VEC) {
            if (n > 0)
                *reinterpret_cast<Vec *>(p) = v;
        } else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n)
                    p[i] = v[i];
    }
    __device__ __forceinline__ void get(float (&x)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = static_cast<float>(v[i]);
    }
    __device__ __forceinline__ void put(const float (&x)[V])
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = static_cast<T>(x[i]);
    }
};

} // namespace dl
