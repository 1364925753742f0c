// dl_scan_carry.h -- the state from chunk to chunk of a scan, forward and (its
// gradient) backward.
//
// One workgroup of four waves per (sequence, head, NC x 16 value columns): the
// columns of the state are independent.  Wave w holds rows 16 w.. of the
// chunk's products and row blocks w, w + 4 of the state, in fp32 registers.
// What one wave's product needs of another's rows passes through LDS as bf16
// planes, already in the order that the matrix instruction reads.  The chunks
// are a chain; what bounds a step is the latency of its three products in a
// row and the reading of the operands (prep's fragments), so each operand of
// the next chunk is loaded into the registers of this one's right behind its
// last use, and the value tiles of one (sequence, head) run on one XCD, whose
// L2 serves all but the first of them.
#pragma once

#include "dl_scan.h"

namespace dl {

constexpr int kXcds = 8; // consecutive workgroups go to consecutive XCDs

// The (sequence, head) and value tile of a workgroup; group >= groups: none.
struct CarryWork {
    int group, tile;
};
__device__ __forceinline__ CarryWork carry_work(int tiles)
{
    const int x = blockIdx.x % kXcds, j = blockIdx.x / kXcds;
    return {j / tiles * kXcds + x, j % tiles};
}

// N planes of 16 columns of a C-layout tile in LDS, as the other operand of a
// product: [16 columns][K], k along the row.
template <int N, int K> struct Planes {
    static constexpr int LD = K + 8;
    __bf16 p[N][16 * LD];
    // the four consecutive k from k0 of column c
    __device__ __forceinline__ void put(int c, int k0, f32x4 x)
    {
        bf16x4 v[N];
        split(x, v);
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x4 *>(&p[i][c * LD + k0]) = v[i];
    }
    template <int M> __device__ __forceinline__ void get(bf16x8 (&f)[M], int ks, int lane) const
    {
#pragma unroll
        for (int i = 0; i < M; ++i)
            f[i] = *reinterpret_cast<const bf16x8 *>(&p[i][(lane & 15) * LD + ks * 32 + (lane >> 4) * 8]);
    }
};

// acc += a b, a row block's fragments of KS steps in registers
template <int ORDER, int KS, int NA, int NB, int K>
__device__ __forceinline__ f32x4 product(const bf16x8 (&a)[KS][NA], const Planes<NB, K> &b, int lane, f32x4 acc)
{
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        constexpr int M = NB < ORDER ? NB : ORDER;
        bf16x8 f[M];
        b.get(f, ks, lane);
        acc = mma<ORDER>(a[ks], f, acc);
    }
    return acc;
}
// The same for a triangular C x C operand: the half that is zero is skipped
// (first: whether k < 32 counts for this row block, second: k >= 32).
template <int ORDER, int NA, int NB>
__device__ __forceinline__ f32x4 product_tri(const bf16x8 (&a)[2][NA], const Planes<NB, C> &b, bool first, bool second,
                                             int lane, f32x4 acc)
{
    constexpr int M = NB < ORDER ? NB : ORDER;
    bf16x8 f[M];
    if (first) {
        b.get(f, 0, lane);
        acc = mma<ORDER>(a[0], f, acc);
    }
    if (second) {
        b.get(f, 1, lane);
        acc = mma<ORDER>(a[1], f, acc);
    }
    return acc;
}
template <int KS, int NP> __device__ __forceinline__ void load_rows(bf16x8 (&f)[KS][NP], const __bf16 *op, int rb, int lane)
{
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        load_frag(f[ks], op, KS, rb, ks, lane);
}
// A row block of a triangular operand; the half that holds nothing is not
// stored, and the other is loaded in its place (the load stays unconditional).
template <int NP> __device__ __forceinline__ void load_tri(bf16x8 (&f)[2][NP], const __bf16 *op, Part part, int rb, int lane)
{
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
        load_frag(f[ks], op, 2, rb, frag_used(part, rb, ks) ? ks : 1 - ks, lane);
}
__device__ __forceinline__ f32x4 ld4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// The state row of a sequence: through a.rows if given; < 0 where the row is
// not one of the caller's a.nrows (nothing is read or written then).
__device__ __forceinline__ long state_row(const ScanArgs &a, int n)
{
    if (!a.rows)
        return n;
    const int r = a.rows[n];
    return r >= 0 && r < a.nrows ? r : -1;
}

// Forward.  SAVE: keeps every chunk's start state and E.
template <int OP, typename TIn, int DKP, int NC, bool SAVE>
__global__ __launch_bounds__(256) void scan_carry_kernel(ScanArgs a)
{
    using P = Plan<OP, TIn>;
    using O = Ops<P::NPX, DKP>;
    constexpr bool DELTA = P::DELTA, ROWS = P::ROWS;
    constexpr int RB = DKP / 64 > 0 ? DKP / 64 : 1, KS = DKP / 32;
    __shared__ Planes<3, DKP> sp[NC];                 // the state
    __shared__ Planes<3, C> rp[DELTA ? NC : 1];       // V - K~ S
    __shared__ Planes<3, C> hp[NC];                   // b (ROWS: P_Ci b), for the state
    __shared__ Planes<P::NPB, C> bp[ROWS ? NC : 1];   // ROWS: b, for o
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, r4 = (lane >> 4) * 4, i0 = w * 16 + r4;
    const CarryWork wk = carry_work(a.dv / (16 * NC));
    if (wk.group >= a.N * a.H)
        return;
    const int h = wk.group % a.H, n = wk.group / a.H;
    const Seq sq = sequence(a, n);
    const int v0 = wk.tile * 16 * NC + col;
    const long row = state_row(a, n);
    const long st0 = (row * a.H + h) * a.dk * a.dv + v0;

    f32x4 S[NC][RB];
#pragma unroll
    for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (w + 4 * r) * 16 + r4 + e;
                S[t][r][e] = a.init && row >= 0 && d < a.dk ? a.init[st0 + static_cast<long>(d) * a.dv + 16 * t] : 0.f;
            }
            if ((w + 4 * r) * 16 < DKP)
                sp[t].put(col, (w + 4 * r) * 16 + r4, S[t][r]);
        }

    const int chunks = (sq.len + C - 1) / C;
    // the operands of a chunk, in the order of their use
    bf16x8 kf[KS][P::NPX], qf[KS][P::NPQ], nf[2][3], bf[2][P::NPB], tf[RB][2][P::NPX];
    f32x4 gi, ge, beta, gam[RB];
    TIn v[NC][4];
    auto ops = [&](int c) { return O(a, static_cast<long>(sq.base + c) * a.H + h); };
    auto load_k = [&](int c) {
        if (DELTA)
            load_rows(kf, ops(c).op(0), w, lane);
        if (ROWS)
            gi = ld4(ops(c).row(0) + i0);
    };
    auto load_v = [&](int c) {
        const long t0 = sq.start + static_cast<long>(c) * C;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long t = t0 + i0 + e, end = static_cast<long>(sq.start) + sq.len - 1;
            const TIn *p = static_cast<const TIn *>(a.v) + (t < end ? t : end) * a.vs + static_cast<long>(h) * a.dv + v0;
#pragma unroll
            for (int x = 0; x < NC; ++x)
                v[x][e] = p[16 * x];
        }
    };
    auto load_q = [&](int c) { load_rows(qf, ops(c).op(1), w, lane); };
    auto load_n = [&](int c) {
        if (DELTA) {
            load_tri(nf, ops(c).mat(0), LOWER, w, lane);
            beta = ld4(ops(c).row(2) + i0);
        }
        if (ROWS)
            ge = ld4(ops(c).row(1) + i0);
    };
    auto load_t = [&](int c) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            // a wave without a row block of the state loads one all the same
            const int rb = (w + 4 * r) * 16 < DKP ? w + 4 * r : 0;
            load_rows(tf[r], ops(c).op(2), rb, lane);
            gam[r] = ld4(ops(c).gam() + rb * 16 + r4);
        }
    };
    auto load_b = [&](int c) { load_tri(bf, ops(c).mat(1), LOWER, w, lane); };
    if (chunks > 0) {
        load_k(0);
        load_v(0);
        load_q(0);
        load_n(0);
        load_t(0);
        load_b(0);
    }
    for (int c = 0; c < chunks; ++c) {
        const int next = c + 1 < chunks ? c + 1 : c;
        const long slot_head = static_cast<long>(sq.base + c) * a.H + h;
        const int rows = sq.len - c * C < C ? sq.len - c * C : C;
        f32x4 x[NC], o[NC];
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) // rows behind the end: zero
                x[t][e] = i0 + e < rows ? from_in(v[t][e]) : 0.f;
        load_v(next);
        if (SAVE) {
#pragma unroll
            for (int t = 0; t < NC; ++t)
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = (w + 4 * r) * 16 + r4 + e;
                        if (d < a.dk)
                            a.save_s[(slot_head * a.dk + d) * a.dv + v0 + 16 * t] = S[t][r][e];
                    }
        }
        __syncthreads(); // the state's planes are complete
        const f32x4 zero = {0, 0, 0, 0};
        if constexpr (DELTA) {
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                f32x4 ks = product<3>(kf, sp[t], lane, zero);
                if (ROWS)
                    ks *= gi;
                rp[t].put(col, i0, x[t] - ks);
            }
        } else {
#pragma unroll
            for (int t = 0; t < NC; ++t)
                hp[t].put(col, i0, x[t]);
        }
#pragma unroll
        for (int t = 0; t < NC; ++t) {
            o[t] = product<P::ORDER_O>(qf, sp[t], lane, zero);
            if (ROWS)
                o[t] *= gi;
        }
        load_k(next);
        load_q(next);
        __syncthreads(); // V - K~ S is complete (RWKV6: b), and the state's planes are read
        if constexpr (DELTA) {
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                x[t] = product_tri<3>(nf, rp[t], true, w >= 2, lane, zero);
                if (SAVE) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a.save_e[(slot_head * C + i0 + e) * a.dv + v0 + 16 * t] = x[t][e];
                }
                x[t] *= beta;
                if (ROWS) {
                    hp[t].put(col, i0, x[t] * ge);
                    bp[t].put(col, i0, x[t]);
                } else {
                    hp[t].put(col, i0, x[t]);
                }
            }
            load_n(next);
            __syncthreads(); // b is complete
        }
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if ((w + 4 * r) * 16 < DKP) {
                    S[t][r] = product<3>(tf[r], hp[t], lane, S[t][r] * gam[r]);
                    sp[t].put(col, (w + 4 * r) * 16 + r4, S[t][r]);
                }
        load_t(next);
#pragma unroll
        for (int t = 0; t < NC; ++t) {
            if constexpr (ROWS)
                o[t] = product_tri<P::ORDER_O>(bf, bp[t], true, w >= 2, lane, o[t]);
            else
                o[t] = product_tri<P::ORDER_O>(bf, hp[t], true, w >= 2, lane, o[t]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + e < rows)
                    static_cast<TIn *>(a.o)[((sq.start + static_cast<long>(c) * C + i0 + e) * a.H + h) * a.dv + v0 + 16 * t] =
                        static_cast<TIn>(o[t][e]);
        }
        load_b(next);
    }
    if (a.fin && row >= 0) {
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = (w + 4 * r) * 16 + r4 + e;
                    if (d < a.dk)
                        a.fin[st0 + static_cast<long>(d) * a.dv + 16 * t] = S[t][r][e];
                }
    }
}

// Backward: chunks from the last to the first, dS in registers.  Writes every
// chunk's dS' and z (delta rule), dv, and per 16 NC value columns the partial
// sums of dbeta; at the end the initial state's gradient.
template <int OP, typename TIn, int DKP, int NC>
__global__ __launch_bounds__(256) void scan_carry_bwd_kernel(ScanArgs a)
{
    using P = Plan<OP, TIn>;
    using O = Ops<P::NPX, DKP>;
    constexpr bool DELTA = P::DELTA, ROWS = P::ROWS;
    constexpr int RB = DKP / 64 > 0 ? DKP / 64 : 1, KS = DKP / 32;
    __shared__ Planes<3, DKP> sp[NC];                   // dS'
    __shared__ Planes<P::NPI, C> gp[2][NC];             // dO (in turn: read to the chunk's end)
    __shared__ Planes<3, C> gg[2][ROWS ? NC : 1];       // ROWS: Gam_i dO
    __shared__ Planes<3, C> wp[DELTA ? NC : 1];         // beta db
    __shared__ Planes<3, C> zp[DELTA ? NC : 1];         // -z
    __shared__ Planes<3, C> zg[ROWS ? NC : 1];          // ROWS: -Gam_i z
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, r4 = (lane >> 4) * 4, i0 = w * 16 + r4;
    const int tiles = a.dv / (16 * NC);
    const CarryWork wk = carry_work(tiles);
    if (wk.group >= a.N * a.H)
        return;
    const int h = wk.group % a.H, n = wk.group / a.H;
    const Seq sq = sequence(a, n);
    const int v0 = wk.tile * 16 * NC + col;
    const long st0 = (static_cast<long>(n) * a.H + h) * a.dk * a.dv + v0;

    f32x4 S[NC][RB]; // dS'
#pragma unroll
    for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (w + 4 * r) * 16 + r4 + e;
                S[t][r][e] = a.dfin && d < a.dk ? a.dfin[st0 + static_cast<long>(d) * a.dv + 16 * t] : 0.f;
            }
            if ((w + 4 * r) * 16 < DKP)
                sp[t].put(col, (w + 4 * r) * 16 + r4, S[t][r]);
        }

    const int chunks = (sq.len + C - 1) / C;
    bf16x8 kf[KS][P::NPX], bt[2][3], nt[2][3], at[2][3], qt[RB][2][P::NPX], kt[RB][2][P::NPX];
    f32x4 gi, ge, beta, gam[RB];
    TIn g[NC][4];
    float E[NC][4];
    auto ops = [&](int c) { return O(a, static_cast<long>(sq.base + c) * a.H + h); };
    auto load_g = [&](int c) {
        const long t0 = sq.start + static_cast<long>(c) * C;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const long t = t0 + i0 + e, end = static_cast<long>(sq.start) + sq.len - 1;
            const long p = ((t < end ? t : end) * a.H + h) * a.dv + v0;
#pragma unroll
            for (int x = 0; x < NC; ++x)
                g[x][e] = a.d_o ? static_cast<const TIn *>(a.d_o)[p + 16 * x] : TIn(0);
        }
        if (ROWS)
            gi = ld4(ops(c).row(0) + i0);
    };
    auto load_db = [&](int c) {
        load_tri(bt, ops(c).mat(1), UPPER, w, lane);
        load_rows(kf, ops(c).op(0), w, lane);
        if (ROWS)
            ge = ld4(ops(c).row(1) + i0);
        if (DELTA)
            beta = ld4(ops(c).row(2) + i0);
    };
    auto load_n = [&](int c) {
        if (DELTA)
            load_tri(nt, ops(c).mat(0), UPPER, w, lane);
    };
    auto load_t = [&](int c) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int rb = (w + 4 * r) * 16 < DKP ? w + 4 * r : 0;
            load_rows(qt[r], ops(c).op(1), rb, lane);
            if (DELTA)
                load_rows(kt[r], ops(c).op(2), rb, lane);
            gam[r] = ld4(ops(c).gam() + rb * 16 + r4);
        }
    };
    auto load_a = [&](int c) {
        if (!DELTA)
            return;
        load_tri(at, ops(c).mat(2), UPPER, w, lane);
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                E[x][e] = a.save_e[((static_cast<long>(sq.base + c) * a.H + h) * C + i0 + e) * a.dv + v0 + 16 * x];
    };
    if (chunks > 0) {
        load_g(chunks - 1);
        load_db(chunks - 1);
        load_n(chunks - 1);
        load_t(chunks - 1);
        load_a(chunks - 1);
    }
    for (int c = chunks - 1; c >= 0; --c) {
        const int next = c > 0 ? c - 1 : 0, turn = c & 1;
        const long slot_head = static_cast<long>(sq.base + c) * a.H + h;
        const int rows = sq.len - c * C < C ? sq.len - c * C : C;
        const f32x4 zero = {0, 0, 0, 0};
        const f32x4 gam_i = gi;
#pragma unroll
        for (int t = 0; t < NC; ++t) {
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = i0 + e < rows ? from_in(g[t][e]) : 0.f;
            gp[turn][t].put(col, i0, x);
            if (ROWS)
                gg[turn][t].put(col, i0, x * gam_i);
        }
        load_g(next);
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = (w + 4 * r) * 16 + r4 + e;
                    if (d < a.dk)
                        a.w_ds[(slot_head * a.dk + d) * a.dv + v0 + 16 * t] = S[t][r][e];
                }
        __syncthreads(); // dO and dS' are complete
        f32x4 db[NC], x[NC];
#pragma unroll
        for (int t = 0; t < NC; ++t) {
            db[t] = product<3>(kf, sp[t], lane, zero);
            if (ROWS)
                db[t] *= ge;
            db[t] = product_tri<3>(bt, gp[turn][t], w < 2, true, lane, db[t]);
            x[t] = db[t];
            if (DELTA)
                wp[t].put(col, i0, db[t] * beta);
        }
        load_db(next);
        __syncthreads(); // beta db is complete; the planes of dS' are read
        if constexpr (DELTA) {
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                x[t] = product_tri<3>(nt, wp[t], w < 2, true, lane, zero);
                zp[t].put(col, i0, -x[t]);
                if (ROWS)
                    zg[t].put(col, i0, -x[t] * gam_i);
            }
            load_n(next);
            __syncthreads(); // z is complete
        }
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if ((w + 4 * r) * 16 < DKP) {
                    f32x4 y = S[t][r] * gam[r];
                    if constexpr (ROWS) {
                        y = product<3>(qt[r], gg[turn][t], lane, y);
                        y = product<3>(kt[r], zg[t], lane, y);
                    } else {
                        y = product<3>(qt[r], gp[turn][t], lane, y);
                        if constexpr (DELTA)
                            y = product<3>(kt[r], zp[t], lane, y);
                    }
                    S[t][r] = y;
                    sp[t].put(col, (w + 4 * r) * 16 + r4, y);
                }
        load_t(next);
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i0 + e < rows)
                    static_cast<TIn *>(a.d_v)[((sq.start + static_cast<long>(c) * C + i0 + e) * a.H + h) * a.dv + v0 + 16 * t] =
                        static_cast<TIn>(x[t][e]);
                if (DELTA)
                    a.w_z[(slot_head * C + i0 + e) * a.dv + v0 + 16 * t] = x[t][e];
            }
        if constexpr (DELTA) {
            f32x4 p = zero;
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                const f32x4 y = product_tri<3>(at, zp[t], w < 2, true, lane, db[t]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] = fmaf(y[e], E[t][e], p[e]);
            }
            load_a(next);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = add_row_ror<1>(p[e]);
                p[e] = add_row_ror<2>(p[e]);
                p[e] = add_row_ror<4>(p[e]);
                p[e] = add_row_ror<8>(p[e]);
                if (col == 0)
                    a.w_db[(slot_head * tiles + wk.tile) * C + i0 + e] = p[e];
            }
        }
    }
    if (a.dinit) {
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = (w + 4 * r) * 16 + r4 + e;
                    if (d < a.dk)
                        a.dinit[st0 + static_cast<long>(d) * a.dv + 16 * t] = S[t][r][e];
                }
    }
}

} // namespace dl
