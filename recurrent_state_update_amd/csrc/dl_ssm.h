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

// Lane j gets the sum over its row of p[j]: halves of the row trade what the
// other half keeps, four times.  lane: the lane's place in its row.
__device__ __forceinline__ float row_sums(const float (&p)[TB], int lane)
{
    float a[8], b[4], c[2];
    const bool h8 = lane & 8, h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a[i] = (h8 ? p[i + 8] : p[i]) + dpp<0x128>(h8 ? p[i] : p[i + 8]); // row_ror:8
#pragma unroll
    for (int i = 0; i < 4; ++i)
        b[i] = (h4 ? a[i + 4] : a[i]) + dpp<0x141>(h4 ? a[i] : a[i + 4]); // row_half_mirror
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = (h2 ? b[i + 2] : b[i]) + dpp<0x4E>(h2 ? b[i] : b[i + 2]); // quad_perm 2 3 0 1
    return (h1 ? c[1] : c[0]) + dpp<0xB1>(h1 ? c[0] : c[1]);             // quad_perm 1 0 3 2
}
// The sum over the row, in every lane of it.
__device__ __forceinline__ float row_sum(float x)
{
    return group_sum<16>(x);
}

// softplus(r) = max(r, 0) + log1p(e), e = e^{-|r|}: the logarithm as
// 2 artanh(s), s = e / (2 + e) <= 1/3, in odd powers of s up to the 17th (what is
// left out is below 2^-29 of it), so that small results keep all their bits.
__device__ __forceinline__ float softplus(float r, float &e)
{
    e = __builtin_amdgcn_exp2f(-fabsf(r) * kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), w = s * s;
    float p = 1.f / 17;
    p = fmaf(p, w, 1.f / 15);
    p = fmaf(p, w, 1.f / 13);
    p = fmaf(p, w, 1.f / 11);
    p = fmaf(p, w, 1.f / 9);
    p = fmaf(p, w, 1.f / 7);
    p = fmaf(p, w, 1.f / 5);
    p = fmaf(p, w, 1.f / 3);
    p = fmaf(p, w, 1.f);
    // (r > 0 ? r : 0 would lose a NaN)
    return (r < 0.f ? 0.f : r) + 2.f * s * p;
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
