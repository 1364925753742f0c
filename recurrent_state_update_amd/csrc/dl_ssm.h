// dl_ssm.h -- the selective state space scan: its mathematics and what its
// kernels share.  The kernels are in dl_ssm.hip (forward, single tokens) and
// dl_ssm_bwd.hip.
//
// Per channel c (in group g = c / (channels / groups)) and state n, with
// delta_t = softplus(dt_t + dt_bias) (or the sum itself):
//   h_t = a_t h_{t-1} + delta_t x_t B_t[n],   a_t = e^{delta_t A[c][n]}
//   y_t = (sum_n C_t[n] h_t + D x_t) silu(z_t)
// and with dy' = dy silu(z) and F_t the gradient of h_t, G_t = a_t F_t that of
// h_{t-1}:
//   F_t = G_{t+1} + dy'_t C_t[n]
//   dB_t[n] = sum_c delta_t x_t F_t,    dC_t[n] = sum_c dy'_t h_t
//   q_t = sum_n F_t B_t[n],             r_t = sum_n A (G_t h_{t-1})
//   dx_t = delta_t q_t + D dy'_t,       ddelta_t = x_t q_t + r_t
//   dA = sum_t delta_t (G_t h_{t-1}),   dD = sum_t dy'_t x_t
//   dz_t = dy_t (sum_n C_t h_t + D x_t) silu'(z_t)
//
// A diagonal recurrence shares nothing between channels that a matrix
// instruction could use: each (token, channel, state) takes an exponential (two
// issue slots on gfx950) and four to fourteen other operations, and the vector
// units are the bound, ahead of memory.  So the layout spends no instruction on
// moving data: the sixteen lanes of a row hold sixteen states of one channel
// (states n, n + 16, ... where there are more), and lane j of the row loads what
// belongs to token j of a block of sixteen (x, delta, the gate: formed once per
// token and channel).  The recurrence reads them as row broadcasts, which are a
// modifier of the multiplication that uses them, and sums over a row end with
// token j's in lane j.
#pragma once

#include <hip/hip_runtime.h>

#include "dl_internal.h"
#include "dl_sequences.h"
#include "dl_vec.h"

namespace dl::ssm {

constexpr int TB = kSsmBlock; // tokens per block: one per lane of a row
static_assert(TB == 16, "a row of lanes");
constexpr float kLog2e = 1.44269504088896340736f;

using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x2 = float __attribute__((ext_vector_type(2)));

// Lane j's value in every lane of the row.
template <int J> __device__ __forceinline__ float row_bcast(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + J, 0xF, 0xF, true));
}
template <int CTRL> __device__ __forceinline__ float dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// for_tokens(f): f(integral constant) for 0 ... 15 (or down from 15), unrolled.
template <int J> struct Int {
    static constexpr int value = J;
};
template <int J = 0, typename F> __device__ __forceinline__ void for_tokens(F &&f)
{
    if constexpr (J < TB) {
        f(Int<J>{});
        for_tokens<J + 1>(f);
    }
}
template <int J = TB - 1, int TO = 0, typename F> __device__ __forceinline__ void for_tokens_down(F &&f)
{
    if constexpr (J >= TO) {
        f(Int<J>{});
        for_tokens_down<J - 1, TO>(f);
    }
}

// Lane j gets the sum over its row of p[j] (lane: its place in the row): halves of
// the row trade what the other half keeps, four times.  The first two are masked
// additions, each writing the half of the lanes that keeps its sum: 33 instructions,
// where selecting ahead of every addition takes 45.  (Two wait states before a row
// operation reads what the instruction ahead may have written, and behind the last
// for what the compiler places there.)
__device__ __forceinline__ float row_sums(float (&p)[TB], int lane)
{
    asm("s_nop 1\n"
        "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %4, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %5, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %6, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %7, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n"
        "v_add_f32_dpp %0, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %4, %12, %12 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %1, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %6, %14, %14 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %7, %15, %15 row_ror:8 row_mask:0xf bank_mask:0xc\n"
        "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0x5\n"
        "v_add_f32_dpp %1, %1, %1 row_half_mirror row_mask:0xf bank_mask:0x5\n"
        "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0x5\n"
        "v_add_f32_dpp %3, %3, %3 row_half_mirror row_mask:0xf bank_mask:0x5\n"
        "v_add_f32_dpp %0, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xa\n"
        "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n"
        "v_add_f32_dpp %2, %6, %6 row_half_mirror row_mask:0xf bank_mask:0xa\n"
        "v_add_f32_dpp %3, %7, %7 row_half_mirror row_mask:0xf bank_mask:0xa\n"
        "s_nop 1"
        : "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]), "+v"(p[4]), "+v"(p[5]), "+v"(p[6]), "+v"(p[7])
        : "v"(p[8]), "v"(p[9]), "v"(p[10]), "v"(p[11]), "v"(p[12]), "v"(p[13]), "v"(p[14]), "v"(p[15]));
    const bool h2 = lane & 2, h1 = lane & 1;
    float c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = (h2 ? p[i + 2] : p[i]) + dpp<0x4E>(h2 ? p[i] : p[i + 2]); // quad_perm 2 3 0 1
    return (h1 ? c[1] : c[0]) + dpp<0xB1>(h1 ? c[0] : c[1]);             // quad_perm 1 0 3 2
}
// The sum over the row, in every lane of it.
__device__ __forceinline__ float row_sum(float x)
{
    return group_sum<16>(x);
}

// softplus(r) = max(r, 0) + log1p(e), e = e^{-|r|}: the logarithm as
// 2 artanh(s), s = e / (2 + e) <= 1/3, so that small results keep all their bits.
// artanh(s) / s is a polynomial in s^2, the best of degree 4 on [0, 1/9] (off by
// 2^-27.9 at the most).
__device__ __forceinline__ float softplus(float r, float &e)
{
    e = __builtin_amdgcn_exp2f(-fabsf(r) * kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), w = s * s;
    float p = 0.140891671f;
    p = fmaf(p, w, 0.139803007f);
    p = fmaf(p, w, 0.200124547f);
    p = fmaf(p, w, 0.333331585f);
    p = fmaf(p, w, 1.f);
    // (r > 0 ? r : 0 would lose a NaN)
    return fmaf(2.f * s, p, r < 0.f ? 0.f : r);
}
// Its derivative, from the same e.
__device__ __forceinline__ float softplus_slope(float r, float e)
{
    return (r < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e);
}
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}
// A as the exponent of 2, for the decay of a token.  -inf (a state that forgets
// all) is kept finite: a token that is not there has delta = 0, and its decay
// has to be 1.
__device__ __forceinline__ float finite_rate(float a)
{
    return a < -1e37f ? -1e37f : a;
}

// What a workgroup works on: tokens [t0, t0 + len) of sequence n, its segment
// `index` of those whose first has slot `base`; last: the sequence ends with it.
struct Piece {
    int n, start, end, t0, len, base, index;
    bool last;
    __device__ __forceinline__ Piece(const Sequences &s, int slot, int seg)
    {
        n = seg ? s.of_slot(slot, seg) : slot;
        start = s.at(n);
        end = s.at(n + 1);
        end = end < start ? start : end;
        base = seg ? start / seg + n : slot;
        index = slot - base;
        t0 = start;
        len = end - start;
        last = true;
        if (seg) {
            const int off = index * seg; // index <= slots <= T / seg + N: checked on the host to fit
            t0 = start + off;
            len = len - off;
            last = len <= seg;
            len = len > seg ? seg : len;
        }
        // an empty sequence is its first segment
        if (index < 0 || (index > 0 && len <= 0))
            n = -1;
    }
    __device__ __forceinline__ bool none() const { return n < 0; }
};

// Work-items of consecutive numbers on one XCD (workgroup b runs on XCD b % 8):
// neighbouring channel tiles share cache lines, which the XCD's L2 then holds once.
__device__ __forceinline__ long xcd_order(long b, long total)
{
    const long q = total / 8, r = total % 8, x = b % 8;
    return x * q + (x < r ? x : r) + b / 8;
}

} // namespace dl::ssm
