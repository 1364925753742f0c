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
// units are the bound, ahead of memory.  So the layout spends few instructions on
// moving data: the sixteen lanes of a row hold sixteen states of one channel
// (states n, n + 16, ... where there are more), and lane j of the row loads what
// belongs to token j of a block of sixteen (x, delta, the gate: formed once per
// token and channel).  The recurrence reads them as row broadcasts, which are a
// modifier of the multiplication that uses them (backward, dy's are instructions of
// their own: 64 of the 1536 vector instructions of a block of tokens), and sums over a
// row end with token j's in lane j.
#pragma once

#include <hip/hip_runtime.h>

#include "dl_internal.h"
#include "dl_sequences.h"
#include "dl_vec.h"

namespace dl::ssm {

constexpr int TB = kSsmBlock; // tokens per block: one per lane of a row
static_assert(TB == 16, "a row of lanes");

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
        : "+&v"(p[0]), "+&v"(p[1]), "+&v"(p[2]), "+&v"(p[3]), "+&v"(p[4]), "+&v"(p[5]), "+&v"(p[6]), "+&v"(p[7])
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
// artanh(s) / s is a polynomial in s^2, the best of degree 4 on [0, 1/9] with a constant
// term of 1 (off by 2^-27.7 at the most).
__device__ __forceinline__ float softplus(float r, float &e)
{
    e = __builtin_amdgcn_exp2f(-fabsf(r) * kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), w = s * s;
    float p = 0.140032008f;
    p = fmaf(p, w, 0.140015468f);
    p = fmaf(p, w, 0.200107172f);
    p = fmaf(p, w, 0.333332092f);
    p = fmaf(p, w, 1.f);
    // (r > 0 ? r : 0 would lose a NaN)
    return fmaf(2.f * s, p, r < 0.f ? 0.f : r);
}
// Its derivative, from the same e.
__device__ __forceinline__ float softplus_slope(float r, float e)
{
    return (r < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e);
}
// A as the exponent of 2, for the decay of a token.  -inf (a state that forgets
// all) is kept finite: a token that is not there has delta = 0, and its decay
// has to be 1.
__device__ __forceinline__ float finite_rate(float a)
{
    return a < -1e37f ? -1e37f : a;
}
// The state (the adjoint's G) on the other side of a segment whose decays' exponents add
// up to `by`, which adds `add`.  In two halves: where states grow, the whole factor can
// be out of range though a small state's product is not; and a state of zero stays so.
__device__ __forceinline__ float across(float h, float by, float add)
{
    const float half = __builtin_amdgcn_exp2f(0.5f * by);
    return h == 0.f ? add : fmaf(half * h, half, add);
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
            const long off = static_cast<long>(index) * seg; // (offsets out of order can give any index)
            t0 = start + static_cast<int>(off);
            len = off < len ? len - static_cast<int>(off) : 0;
            last = len <= seg;
            len = len > seg ? seg : len;
        }
        // an empty sequence is its first segment
        if (index < 0 || (index > 0 && len <= 0))
            n = -1;
    }
    __device__ __forceinline__ bool none() const { return n < 0; }
};

// The slot and tile of a workgroup, which runs on XCD b % 8: every slot's tiles go to
// the XCDs in runs, since neighbours share cache lines, which the XCD's L2 then holds
// once; all slots alike (sequences differ in length), each a run further, which evens
// out what 8 does not divide.  tile: -1 if there is none.
struct Work {
    int slot, tile;
    __device__ __forceinline__ Work(unsigned b, int tiles)
    {
        const int run = (tiles + 7) / 8, i = b / 8;
        slot = i / run;
        tile = (b + slot) % 8 * run + i % run;
        if (tile >= tiles)
            tile = -1;
    }
};
inline long work_groups(const SsmArgs &a) { return static_cast<long>(a.slots) * ((a.tiles + 7) / 8) * 8; }

// ---- the forward kernels' operands: a stage of TT tokens of a workgroup's channels

constexpr int CH = kSsmTile; // channels per workgroup: four waves of four
constexpr int LOADERS = 256; // threads that bring a stage in
static_assert(CH == 16, "four waves of four rows");

template <int S, int TT> struct Stage {
    static constexpr int XLD = TT + 2, BLD = TT + 4;
    float x[CH][XLD], dt[CH][XLD];
    alignas(16) float b[16 * S][BLD], c[16 * S][BLD];
};

// What it is read from: the adjoint's has dy, times the gate's silu, and C in the
// place of x and B.
struct Sources {
    const void *x, *dt, *z, *b, *c; // z: NULL without a gate
    long xs, dts, zs, bs, cs;
};

// A thread's part: a few channels (states) of one token, next to each other, loaded
// into registers while the stage before is worked on, and put in LDS transposed.
// Every load goes to a row that is there, without a condition, so that nothing waits
// for it early; what is not there is dropped when put.
template <typename T, int S, int TT, bool VEC> struct Loader {
    static constexpr int XV = CH * TT / LOADERS, XPR = CH / XV; // channels, threads per token
    static constexpr int BV = 16 * S * TT / LOADERS < 4 ? 16 * S * TT / LOADERS : 4, BPR = 16 * S / BV, BTOK = LOADERS / BPR, BK = TT / BTOK;
    static_assert(XPR * TT == LOADERS && BK * BTOK == TT && BK > 0, "every thread loads as much");
    Sources s;
    int xt, xc, bt, bn, nx, nb; // token, channel, token, state; channels and states there are
    int col, state;             // the first column of x's and of B's rows
    bool gate;
    long t0;
    int len;
    Cells<XV, T, VEC> rx, rd, rz;
    Cells<BV, T, VEC> rb[BK], rc[BK];

    __device__ __forceinline__ Loader(const Sources &s, int id, int c0, int channels, int b0, int states)
        : s(s), xt(id / XPR), xc(id % XPR * XV), bt(id / BPR), bn(id % BPR * BV), nx(channels - xc), nb(states - bn),
          col(c0 + (nx > 0 ? xc : 0)), state(b0 + (nb > 0 ? bn : 0)), gate(s.z)
    {
    }
    __device__ __forceinline__ void piece(int first, int tokens)
    {
        t0 = first;
        len = tokens;
    }
    // Row `row` of the stage's, at base plus a lane's own columns: the base is the same
    // for all lanes, and what differs fits 32 bits (64 rows of at most 2^22 elements).
    template <typename Cell>
    __device__ __forceinline__ void row(Cell &r, const void *p, long stride, int from, int at, int col, int n)
    {
        const T *const base = static_cast<const T *>(p) + (t0 + from) * stride;
        r.load(base + static_cast<unsigned>(min(at, len - 1 - from) * static_cast<int>(stride) + col), n);
    }
    // Z, C: whether those are ever wanted.  Behind the piece's end: its last row.
    template <bool Z, bool C> __device__ __forceinline__ void read(int from)
    {
        from = min(from, (len - 1) / TT * TT);
        row(rx, s.x, s.xs, from, xt, col, nx);
        row(rd, s.dt, s.dts, from, xt, col, nx);
        if constexpr (Z)
            row(rz, gate ? s.z : s.x, gate ? s.zs : s.xs, from, xt, col, nx);
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            row(rb[k], s.b, s.bs, from, bt + k * BTOK, state, nb);
            if constexpr (C)
                row(rc[k], s.c, s.cs, from, bt + k * BTOK, state, nb);
        }
    }
    // GATED: x times the gate's silu
    template <bool GATED, bool Z, bool C> __device__ __forceinline__ void put(Stage<S, TT> &st, int from)
    {
        const int n = from + xt < len ? nx : 0;
        rx.keep(n);
        rd.keep(n);
        if constexpr (Z)
            rz.keep(gate ? n : 0);
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            float x = to_f(rx.v[i]);
            if constexpr (GATED) {
                const float z = to_f(rz.v[i]);
                x *= fmaf(z, sigmoid(z), gate ? 0.f : 1.f);
            }
            st.x[xc + i][xt] = x;
            st.dt[xc + i][xt] = to_f(rd.v[i]);
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const int m = from + bt + k * BTOK < len ? nb : 0;
            rb[k].keep(m);
            if constexpr (C)
                rc[k].keep(m);
#pragma unroll
            for (int i = 0; i < BV; ++i) {
                st.b[bn + i][bt + k * BTOK] = to_f(rb[k].v[i]);
                if constexpr (C)
                    st.c[bn + i][bt + k * BTOK] = to_f(rc[k].v[i]);
            }
        }
    }
};

// What lane j of a row forms of its tokens at, at + 16, ... of a stage: x and delta.
// Straight code for all blocks of the stage, whose chains of dependent operations then
// overlap; tokens behind the `live` ones have delta 0 and change nothing.
template <int NB> struct Own {
    float x[NB], delta[NB];
    template <typename St>
    __device__ __forceinline__ void form(const St &st, int row, int j, int live, float bias, int softplus_on)
    {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * TB + j;
            float e, raw = st.dt[row][at] + bias, soft = softplus(raw, e);
            asm("" : "+v"(soft)); // a selection, not a branch
            x[i] = st.x[row][at];
            delta[i] = at < live ? softplus_on ? soft : raw : 0.f;
        }
    }
};

// The workgroup's channels: tile `tile` of sixteen, within one group.
struct Tile {
    int g, c0, nc; // group, first channel, channels there are
    __device__ __forceinline__ Tile(const SsmArgs &a, int tile, int width)
    {
        const int per = (a.CG + width - 1) / width;
        g = tile / per;
        c0 = g * a.CG + tile % per * width;
        nc = min(width, (g + 1) * a.CG - c0);
    }
};

} // namespace dl::ssm
