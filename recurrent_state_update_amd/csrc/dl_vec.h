// dl_vec.h -- loads and stores of a lane's consecutive elements, and sums over
// lanes, shared by the row kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace dl {

template <typename T> __device__ __forceinline__ float to_f(T x) { return static_cast<float>(x); }

// N consecutive elements from p, as floats (and back).  ALIGNED: p is aligned
// to 16 bytes, or to the N elements where they are fewer.  ONCE: loads that
// leave the caches to others.
template <int N, bool ALIGNED, bool ONCE = false, typename T>
__device__ __forceinline__ void load(float (&x)[N], const T *p)
{
    using V = T __attribute__((ext_vector_type(N)));
    if constexpr (ALIGNED && N > 1) {
        const V v = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const V *>(p)) : *reinterpret_cast<const V *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = to_f(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = to_f(p[i]);
    }
}
template <int N, bool ALIGNED, typename T> __device__ __forceinline__ void store(T *p, const float (&x)[N])
{
    using V = T __attribute__((ext_vector_type(N)));
    if constexpr (ALIGNED && N > 1) {
        V v;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = static_cast<T>(x[i]);
        *reinterpret_cast<V *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[i] = static_cast<T>(x[i]);
    }
}

template <int CTRL> __device__ __forceinline__ float add_dpp(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
// Sum over groups of G consecutive lanes (2 <= G <= 64), in every lane of the
// group: swaps within four lanes, mirrors of 8 and of 16, then across rows.
template <int G> __device__ __forceinline__ float group_sum(float x)
{
    x = add_dpp<0xB1>(x);                        // quad_perm 1 0 3 2
    if constexpr (G >= 4) x = add_dpp<0x4E>(x);  // quad_perm 2 3 0 1
    if constexpr (G >= 8) x = add_dpp<0x141>(x); // row_half_mirror
    if constexpr (G >= 16) x = add_dpp<0x140>(x); // row_mirror
    if constexpr (G >= 32) x += __shfl_xor(x, 16);
    if constexpr (G >= 64) x += __shfl_xor(x, 32);
    return x;
}

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + e^-z), from the exponential and the reciprocal of the hardware (each good to
// two roundings; the exponent's own rounding is |z| 2^-24 of the exponential).
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

} // namespace dl
