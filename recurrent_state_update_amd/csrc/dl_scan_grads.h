// dl_scan_grads.h -- per chunk and head of a scan: the gradients of its inputs.
//
// With dS' and z from the backward carry, E and S from the forward one:
//   dQ~ = dO S^T, dK~ = -z S^T, dK^ = b dS'^T        [C][d_k], over d_v
//   dB = dO b^T, dA = -z b^T (lower triangles)       [C][C], over d_v
// on the bf16 matrix instructions from fp32 split into planes, then within the
// chunk (cq, cr: row i's parts through q and k as a reader; cc: through k as
// what is read later)
//   cq_i = Gam_i dQ~_i + sum_j dB_ij P_ij k_j,  cr_i = Gam_i dK~_i + sum_j dA_ij P_ij k_j
//   cc_j = P_Cj dK^_j + sum_i P_ij (dA_ij k_i + dB_ij q_i)
//   dq = cq, dk = cr + cc.  dbeta_j = (db . E)_j - sum_i A_ij z_i . E_j.
// The log-decay's gradient at row t is the sum of what its decay is a factor of,
// per key (GDN: over the keys)
//   Gam_C <S, dS'>                                              for every t
//   reads of S, q_i Gam_i dQ~_i + k_i Gam_i dK~_i              rows i >= t
//   writes into S', k_j P_Cj dK^_j                              rows j < t
//   pairs, P_ij (q_i dB_ij + k_i dA_ij) k_j                     i >= t > j
// (RWKV6's reads and pairs, i > t), and of nothing else.  As a difference of sums
// over all rows or pairs it would carry the rounding of terms that the decay does
// not touch: a strong decay's gradient, which is as small as the decay, would be
// lost in it.
//
// One workgroup per chunk and head, one wave per 16 keys.  Bound by reading S
// and dS' (64 KiB each at d = 128, the largest part of a chunk) and by the
// latency of its phases.
#pragma once

#include <type_traits>

#include "dl_scan_carry.h"
#include "dl_scan_prep.h"

namespace dl {

// dO, -z and E (RWKV6: V) for 32 value columns, as planes.
template <int OP, typename TIn> struct GradStage {
    using P = Plan<OP, TIn>;
    static constexpr int V = 32, LD = V + 8, NE = P::DELTA ? 3 : P::NPI;
    __bf16 g[P::NPI][C * LD], e[NE][C * LD];
    __bf16 z[P::DELTA ? 3 : 1][P::DELTA ? C * LD : 8];
};

template <int OP, typename TIn, int DKP> struct GradLds {
    static constexpr int LD = DKP + 4;
    // GDN: the weights dB P, its transpose and dA P + its transpose (fp32, split
    // when read: in planes they would leave room for one workgroup on a CU)
    struct Rows {
        float x1[C * MLD], x2[C * MLD], x3[C * MLD];
    };
    // per key: keys and queries scaled within their blocks, dA and dB
    struct Keys {
        float kr[C * LD], kl[C * LD], ql[C * LD];
        float dB[C * MLD], dA[C * MLD];
    };
    static constexpr bool ROWS = OP == GDN;
    union {
        GradStage<OP, TIn> st;
        std::conditional_t<ROWS, Rows, Keys> x;
    };
    float gs[DKP];                // sum_v S dS' per key
    float beta[C], dbeta[10][16]; // per pair of blocks: sum_i A_ij (-z_i . E_j)
    // per key
    float eb[ROWS ? 1 : 4 * DKP], pre[ROWS ? 1 : 4 * DKP], suf[ROWS ? 1 : 4 * DKP]; // of, before, behind a block
    float part[ROWS ? 1 : 4 * DKP], cross[ROWS ? 1 : 4 * DKP]; // what crosses all of a block
    // GDN
    float e[C], rpre[C], rsuf[C], reb[4];                      // decays of rows
    float diag[ROWS ? 4 : 1][16 * 16];                         // P_ij of the diagonal blocks
    // sums of W_ij = dB B + dA A: over a row's columns, a column's rows, the
    // pair of blocks; within a block, over the pairs i >= t > j
    float roww[10][16], colw[10][16], allw[10];
    float ra[ROWS ? DKP / 16 : 1][C], rh[ROWS ? DKP / 16 : 1][C]; // per 16 keys: reads of S, writes into S'
};

// x is formed here: the compiler would else move the sums that only a store under
// a condition takes behind that condition, and keep all their terms until then.
__device__ __forceinline__ void formed(float &x) { asm volatile("" : "+v"(x)); }

// Waves to a SIMD that the registers are held to: two workgroups on a CU where
// LDS allows them (GDN, d_k = 128, bf16: 128 registers and 24 bytes a lane in
// scratch, 217 us of a training step over 4096 tokens, 32 heads; with 140 and one
// workgroup 283).
template <int OP, typename TIn, int DKP> constexpr int grad_waves()
{
    return OP == GDN && sizeof(TIn) == 2 ? (DKP == 128 ? 4 : 3) : 2;
}

template <int OP, typename TIn, int DKP>
__global__ __launch_bounds__(DKP * 4, (grad_waves<OP, TIn, DKP>())) void scan_grads_kernel(ScanArgs a, bool vec, int tiles)
{
    using P = Plan<OP, TIn>;
    using G = GradLds<OP, TIn, DKP>;
    using St = GradStage<OP, TIn>;
    constexpr bool DELTA = P::DELTA;
    constexpr int LD = DKP + 4, NT = DKP * 4, NW = NT / 64, TASKS = (10 + NW - 1) / NW;
    extern __shared__ __align__(16) char smem[];
    G &s = *reinterpret_cast<G *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const long slot_head = static_cast<long>(slot) * a.H + h;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0 || ch.behind) {
        if (!DELTA && tid < a.dk)
            a.w_du[slot_head * a.dk + tid] = 0.f;
        return;
    }
    const Ops<P::NPX, DKP> ops(a, slot_head);
    const int c16 = lane & 15, r4 = (lane >> 4) * 4;
    const int d = tid % DKP, I0 = tid / DKP, r0 = I0 * 16; // one thread per (key, block)
    const long t0 = ch.t0;

    // ---- what the chunk itself needs, ahead of the products over d_v
    float kv[16], qv[16], ev[16]; // per key: this thread's rows
    if constexpr (OP == GDN) {
        for (int i = tid; i < C; i += NT)
            s.e[i] = i < ch.rows ? expf(floor_log_decay(a.ld[(t0 + i) * a.H + h])) : 1.f;
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const bool in = r0 + i < ch.rows && d < a.dk;
            const long t = t0 + r0 + i, at = static_cast<long>(h) * a.dk + d;
            kv[i] = in ? from_in(static_cast<const TIn *>(a.k)[t * a.ks + at]) : 0.f;
            qv[i] = in ? from_in(static_cast<const TIn *>(a.q)[t * a.qs + at]) : 0.f;
            ev[i] = in ? a.ld[t * a.H * a.dk + at] : 0.f;
        }
        float p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            ev[i] = expf(floor_log_decay(ev[i]));
            p *= ev[i];
        }
        s.eb[tid] = p;
    }
    for (int i = tid; i < C; i += NT)
        s.beta[i] = !DELTA ? 1.f : i < ch.rows ? a.beta[(t0 + i) * a.H + h] : 0.f;

    // ---- products over d_v, 32 columns at a time
    f32x4 dQ[4], dK[4], dH[4], xB[TASKS], xM[TASKS];
    const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int I = 0; I < 4; ++I)
        dQ[I] = dK[I] = dH[I] = zero;
#pragma unroll
    for (int p = 0; p < TASKS; ++p)
        xB[p] = xM[p] = zero;
    float gs = 0.f;
    auto frag = [&](auto &f, const auto &x, int rb) {
#pragma unroll
        for (int n = 0; n < static_cast<int>(sizeof(f) / sizeof(f[0])); ++n)
            f[n] = *reinterpret_cast<const bf16x8 *>(&x[n][(rb * 16 + c16) * St::LD + (lane >> 4) * 8]);
    };
    for (int v0 = 0; v0 < a.dv; v0 += St::V) {
        f32x8 S = {}, dS = {}; // row d of the state, in the matrix instruction's order
        {
            const int v = v0 + (lane >> 4) * 8, row = w * 16 + c16;
            if (v < a.dv && row < a.dk) {
                S = *reinterpret_cast<const f32x8 *>(&a.save_s[(slot_head * a.dk + row) * a.dv + v]);
                dS = *reinterpret_cast<const f32x8 *>(&a.w_ds[(slot_head * a.dk + row) * a.dv + v]);
            }
        }
        if (v0 > 0)
            __syncthreads(); // the stage before is read
        // pieces of eight columns: 256 of dO, then of E (V), then of z
        constexpr int ARRAYS = DELTA ? 3 : 2;
        for (int it = tid; it < ARRAYS * 256; it += NT) {
            const int i = it / 4 % C, c = it % 4 * 8, v = v0 + c;
            const bool in = i < ch.rows && v < a.dv;
            const long t = t0 + i, at = (slot_head * C + i) * a.dv + v;
            if (it < 256 || (!DELTA && it < 512)) {
                TIn x[8];
                if (it < 256)
                    load_piece(x, static_cast<const TIn *>(a.d_o) + (t * a.H + h) * a.dv + v, in && a.d_o, vec);
                else
                    load_piece(x, static_cast<const TIn *>(a.v) + t * a.vs + static_cast<long>(h) * a.dv + v, in, vec);
                bf16x8 pl[P::NPI];
                if constexpr (P::BF)
                    pl[0] = __builtin_bit_cast(bf16x8, x);
                else
                    split(__builtin_bit_cast(f32x8, x), pl);
#pragma unroll
                for (int n = 0; n < P::NPI; ++n)
                    *reinterpret_cast<bf16x8 *>(it < 256 ? &s.st.g[n][i * St::LD + c] : &s.st.e[n][i * St::LD + c]) = pl[n];
            } else if constexpr (DELTA) {
                f32x8 x = {};
                if (in)
                    x = *reinterpret_cast<const f32x8 *>(it < 512 ? &a.save_e[at] : &a.w_z[at]);
                bf16x8 pl[3];
                split(it < 512 ? x : -x, pl);
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    *reinterpret_cast<bf16x8 *>(it < 512 ? &s.st.e[n][i * St::LD + c] : &s.st.z[n][i * St::LD + c]) = pl[n];
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            gs = fmaf(S[e], dS[e], gs);
        bf16x8 pl[3];
        split(dS, pl);
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            bf16x8 e[St::NE];
            frag(e, s.st.e, I);
            dH[I] = mma(e, pl, dH[I]);
        }
        split(S, pl);
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            bf16x8 g[P::NPI];
            frag(g, s.st.g, I);
            dQ[I] = mma(g, pl, dQ[I]);
            if constexpr (DELTA) {
                bf16x8 z[3];
                frag(z, s.st.z, I);
                dK[I] = mma(z, pl, dK[I]);
            }
        }
#pragma unroll
        for (int p = 0; p < TASKS; ++p) {
            const int b = w + p * NW;
            if (b >= 10)
                break;
            const int I = block_row(b), J = block_col(b);
            bf16x8 g[P::NPI], e[St::NE];
            frag(g, s.st.g, I);
            frag(e, s.st.e, J);
            xB[p] = mma(g, e, xB[p]);
            if constexpr (DELTA) {
                bf16x8 z[3];
                frag(z, s.st.z, I);
                xM[p] = mma(z, e, xM[p]);
            }
        }
    }
    gs = wave_sum_from<16>(gs);
    if (lane < 16)
        s.gs[w * 16 + c16] = gs;
    __syncthreads(); // the stage is read; e, eb, beta and gs are complete

    if constexpr (OP == GDN) {
        // ---- the decays of pairs; zero the weights
        for (int b = w; b < 4; b += NW)
            if (lane < 16) {
                float p = 0.f, pre = 1.f, suf = 1.f, all = 1.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e = s.e[b * 16 + i];
                    p = i == lane ? 1.f : p * e;
                    s.diag[b][i * 16 + lane] = p;
                    pre *= i <= lane ? e : 1.f;
                    suf *= i > lane ? e : 1.f;
                    all *= e;
                }
                s.rpre[b * 16 + lane] = pre;
                s.rsuf[b * 16 + lane] = suf;
                if (lane == 0)
                    s.reb[b] = all;
            }
        constexpr int X = sizeof(typename G::Rows) / 16;
        for (int it = tid; it < X; it += NT)
            reinterpret_cast<f32x4 *>(&s.x)[it] = zero;
        __syncthreads();
#pragma unroll
        for (int p = 0; p < TASKS; ++p) {
            const int b = w + p * NW;
            if (b >= 10)
                break;
            const int I = block_row(b), J = block_col(b);
            const f32x4 *ab = ops.pairs();
            const f32x4 A = ab[b * 64 + lane], B = ab[(10 + b) * 64 + lane];
            const float beta = s.beta[J * 16 + c16];
            float between = 1.f, cm = 0.f, cw = 0.f;
            for (int K = J + 1; K < I; ++K)
                between *= s.reb[K];
            const float right = between * s.rsuf[J * 16 + c16];
            f32x4 w1, w3, W;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = r4 + e;
                const bool below = I > J || i > c16, on = I == J && i == c16;
                const float f = I == J ? s.diag[I][i * 16 + c16] : s.rpre[I * 16 + i] * right;
                const float gb = below || on ? beta * xB[p][e] : 0.f, ga = below ? beta * xM[p][e] : 0.f;
                w1[e] = gb * f;
                w3[e] = ga * f;
                W[e] = below ? gb * B[e] + ga * A[e] : 0.f;
                cw += W[e];
                cm += below ? A[e] * xM[p][e] : 0.f;
            }
            if (I == J) { // of column j's rows, those from row t on, for the t behind j
                const float t1 = __shfl_down(cw, 16), t2 = __shfl_down(cw, 32), t3 = __shfl_down(cw, 48);
                float from = (lane < 48 ? t1 : 0.f) + (lane < 32 ? t2 : 0.f) + (lane < 16 ? t3 : 0.f);
#pragma unroll
                for (int e = 3; e >= 0; --e) {
                    from += W[e];
                    W[e] = r4 + e > c16 ? from : 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float rw = W[e];
                rw = add_row_ror<1>(rw);
                rw = add_row_ror<2>(rw);
                rw = add_row_ror<4>(rw);
                rw = add_row_ror<8>(rw);
                if (c16 == 0)
                    s.roww[b][r4 + e] = rw;
            }
            cm = wave_sum_from<16>(cm);
            cw = wave_sum_from<16>(cw);
            if (lane < 16) {
                s.dbeta[b][lane] = cm;
                s.colw[b][lane] = cw;
            }
            cw = add_row_ror<1>(cw);
            cw = add_row_ror<2>(cw);
            cw = add_row_ror<4>(cw);
            cw = add_row_ror<8>(cw);
            if (lane == 0)
                s.allw[b] = cw;
            *reinterpret_cast<f32x4 *>(&s.x.x2[(J * 16 + c16) * MLD + I * 16 + r4]) = w1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = I * 16 + r4 + e, j = J * 16 + c16;
                s.x.x1[i * MLD + j] = w1[e];
                if (i > j) {
                    s.x.x3[i * MLD + j] = w3[e];
                    s.x.x3[j * MLD + i] = w3[e];
                }
            }
        }
        // ---- wave w: keys 16 w.., all rows
        Operand<2, P::NPX> kt, qt;
        qt.load(ops.op(1), w, lane);
        kt.load(ops.op(2), w, lane);
        TIn kx[4][4], qx[4][4]; // this lane's key in all rows
#pragma unroll
        for (int I = 0; I < 4; ++I)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = I * 16 + r4 + e, key = w * 16 + c16;
                const bool in = i < ch.rows && key < a.dk;
                const long at = static_cast<long>(h) * a.dk + key;
                kx[I][e] = in ? static_cast<const TIn *>(a.k)[(t0 + i) * a.ks + at] : TIn(0);
                qx[I][e] = in ? static_cast<const TIn *>(a.q)[(t0 + i) * a.qs + at] : TIn(0);
            }
        __syncthreads();
        qt.ready();
        kt.ready();
        auto xfrag = [&](bf16x8 (&f)[3], const float (&x)[C * MLD], int rb, int ks) {
            const float *p = &x[(rb * 16 + c16) * MLD + ks * 32 + (lane >> 4) * 8];
            const f32x4 lo = ld4(p), hi = ld4(p + 4);
            split(f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}, f);
        };
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            float bg = 1.f, ag = 1.f; // blocks before, after
            for (int K = 0; K < 4; ++K) {
                bg *= K < I ? s.reb[K] : 1.f;
                ag *= K > I ? s.reb[K] : 1.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = I * 16 + r4 + e;
                const float gam = bg * s.rpre[i], end = ag * s.rsuf[i] * s.beta[i];
                dQ[I][e] *= gam;
                dK[I][e] *= gam;
                dH[I][e] *= end;
                const float k = from_in(kx[I][e]), q = from_in(qx[I][e]);
                float x = fmaf(q, dQ[I][e], k * dK[I][e]), y = k * dH[I][e];
                x = add_row_ror<1>(x);
                y = add_row_ror<1>(y);
                x = add_row_ror<2>(x);
                y = add_row_ror<2>(y);
                x = add_row_ror<4>(x);
                y = add_row_ror<4>(y);
                x = add_row_ror<8>(x);
                y = add_row_ror<8>(y);
                if (c16 == 0) {
                    s.ra[w][i] = x;
                    s.rh[w][i] = y;
                }
                dK[I][e] += dH[I][e];
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8 f[3];
                if (frag_used(LOWER, I, ks)) {
                    xfrag(f, s.x.x1, I, ks);
                    dQ[I] = mma(f, kt.f[ks], dQ[I]);
                }
                xfrag(f, s.x.x3, I, ks);
                dK[I] = mma(f, kt.f[ks], dK[I]);
                if (frag_used(UPPER, I, ks)) {
                    xfrag(f, s.x.x2, I, ks);
                    dK[I] = mma(f, qt.f[ks], dK[I]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = I * 16 + r4 + e, key = w * 16 + c16;
                if (i < ch.rows && key < a.dk) {
                    const long at = ((t0 + i) * a.H + h) * a.dk + key;
                    static_cast<TIn *>(a.d_q)[at] = static_cast<TIn>(dQ[I][e]);
                    static_cast<TIn *>(a.d_k)[at] = static_cast<TIn>(dK[I][e]);
                }
            }
        }
        __syncthreads();
        // ---- one lane per row t
        if (tid < C) {
            const int b = lane >> 4, i = lane & 15;
            // x: reads; y: writes; in: pairs within t's block, of it and earlier
            // ones, of later ones and it; all: of later ones and earlier ones
            float x = 0.f, y = 0.f, g = 0.f, dbeta = 0.f;
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                x += s.ra[n][lane];
                y += s.rh[n][lane];
            }
            for (int K = 0; K < DKP; K += 64)
                g += K + lane < DKP ? s.gs[K + lane] : 0.f;
            g = wave_sum_from<1>(g) * (s.reb[0] * s.reb[1] * s.reb[2] * s.reb[3]);
            const float in = s.roww[b * (b + 3) / 2][i];
            float early = 0.f, late = 0.f;
            for (int K = 0; K < b; ++K)
                early += s.roww[b * (b + 1) / 2 + K][i];
            for (int K = b; K < 4; ++K) {
                late += K > b ? s.colw[K * (K + 1) / 2 + b][i] : 0.f;
                dbeta += s.dbeta[K * (K + 1) / 2 + b][i];
            }
            const float all = b == 1 ? s.allw[3] + s.allw[6] : b == 2 ? s.allw[6] + s.allw[7] : 0.f;
            // rows from t on, rows before t
            y = __shfl_up(y, 1);
            y = lane > 0 ? y : 0.f;
            late = __shfl_up(late, 1);
            late = i > 0 ? late : 0.f;
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const float u = __shfl_up(y, m), v = __shfl_down(x, m);
                y += lane >= m ? u : 0.f;
                x += lane + m < 64 ? v : 0.f;
                if (m < 16) {
                    const float p = __shfl_up(late, m), q = __shfl_down(early, m);
                    late += i >= m ? p : 0.f;
                    early += i + m < 16 ? q : 0.f;
                }
            }
            for (int t = 0; t < tiles; ++t)
                dbeta += a.w_db[(slot_head * tiles + t) * C + lane];
            if (lane < ch.rows) {
                const long at = (t0 + lane) * a.H + h;
                a.d_ld[at] = a.ld[at] < kMinLogDecay ? 0.f : g + x + y + in + early + late + all; // below it the decay is held
                a.d_beta[at] = dbeta;
            }
        }
    } else {
        // ---- dA, dB; keys and queries scaled within their blocks
#pragma unroll
        for (int p = 0; p < TASKS; ++p) {
            const int b = w + p * NW;
            if (b >= 10)
                break;
            const int I = block_row(b), J = block_col(b);
            const float beta = s.beta[J * 16 + c16];
            float cm = 0.f;
            f32x4 A = zero;
            if (DELTA)
                A = ops.pairs()[b * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = I * 16 + r4 + e, j = J * 16 + c16;
                s.x.dB[i * MLD + j] = i >= j ? beta * xB[p][e] : 0.f;
                if (DELTA) {
                    s.x.dA[i * MLD + j] = i > j ? beta * xM[p][e] : 0.f;
                    cm += i > j ? A[e] * xM[p][e] : 0.f;
                }
            }
            if (DELTA) {
                cm = wave_sum_from<16>(cm);
                if (lane < 16)
                    s.dbeta[b][lane] = cm;
            }
        }
        {
            float p = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float before = p;
                p *= ev[i];
                s.x.ql[(r0 + i) * LD + d] = qv[i] * (DELTA ? p : before);
                if (DELTA)
                    s.x.kl[(r0 + i) * LD + d] = kv[i] * p;
            }
            p = 1.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                s.x.kr[(r0 + i) * LD + d] = kv[i] * p;
                p *= ev[i];
            }
            float f = 1.f, g = 1.f;
            for (int K = 0; K < 4; ++K) {
                f *= K < I0 ? s.eb[K * DKP + d] : 1.f;
                g *= K > I0 ? s.eb[K * DKP + d] : 1.f;
            }
            s.pre[tid] = f;
            s.suf[tid] = g;
        }
        __syncthreads();
        // ---- wave w: keys 16 w.., pairs of rows of different blocks, up to
        // the reader's prefix (cq, cr) and the read row's suffix (cc)
        const int key = w * 16 + c16;
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            dQ[I] *= s.pre[I * DKP + key];
            if (DELTA)
                dK[I] *= s.pre[I * DKP + key];
            const f32x4 beta = ld4(&s.beta[I * 16 + r4]);
            dH[I] *= beta * s.suf[I * DKP + key];
        }
        auto column = [&](const float *x, int row, float f) { // four rows of a key
            f32x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = x[(row + r4 + e) * LD + key] * f;
            return y;
        };
        // what crosses whole blocks, per key: the block's reads of S and writes into
        // S', and the pairs of blocks with others between them
        auto rows_sum = [&](f32x4 y) { return wave_sum_from<16>((y[0] + y[1]) + (y[2] + y[3])); };
        auto reads = [&](f32x4 q, f32x4 k, int I) { // by block I, given their parts
            f32x4 y = q * column(s.x.ql, I * 16, 1.f);
            if (DELTA)
                y += k * column(s.x.kl, I * 16, 1.f);
            return y;
        };
        float rs[4], kh[4];
#pragma unroll
        for (int I = 1; I < 4; ++I)
            rs[I] = rows_sum(reads(dQ[I], dK[I], I));
#pragma unroll
        for (int I = 0; I < 3; ++I)
            kh[I] = rows_sum(dH[I] * column(s.x.kr, I * 16, 1.f));
        f32x4 over1 = zero, over2 = zero; // pairs across block 1, across block 2
#pragma unroll
        for (int I = 1; I < 4; ++I) {
            float f = 1.f;
#pragma unroll
            for (int J = I - 1; J >= 0; --J) {
                const f32x4 k = column(s.x.kr, J * 16, f);
                const bool next = J == I - 1;
                const f32x4 q = mfma32x4(ld4(&s.x.dB[(I * 16 + c16) * MLD + J * 16 + r4]), k, next ? dQ[I] : zero);
                f32x4 c = zero;
                if (DELTA)
                    c = mfma32x4(ld4(&s.x.dA[(I * 16 + c16) * MLD + J * 16 + r4]), k, next ? dK[I] : zero);
                if (next) {
                    dQ[I] = q;
                    dK[I] = c;
                } else {
                    const f32x4 y = reads(q, c, I);
                    if (J == 0)
                        over1 += y;
                    if (I == 3)
                        over2 += y;
                    dQ[I] += q;
                    dK[I] += c;
                }
                f *= s.eb[J * DKP + key];
                keep_order(); // (one pair's operands at a time: the registers are full)
            }
        }
        {
            const float all = s.pre[3 * DKP + key] * s.eb[3 * DKP + key] * s.gs[key];
            const float o1 = rows_sum(over1), o2 = rows_sum(over2);
            if (lane < 16) {
                s.cross[key] = all + (rs[1] + rs[2] + rs[3]);
                s.cross[DKP + key] = all + (rs[2] + rs[3]) + kh[0] + o1;
                s.cross[2 * DKP + key] = all + rs[3] + (kh[0] + kh[1]) + o2;
                s.cross[3 * DKP + key] = all + (kh[0] + kh[1] + kh[2]);
            }
        }
#pragma unroll
        for (int J = 0; J < 3; ++J) {
            float f = 1.f;
#pragma unroll
            for (int I = J + 1; I < 4; ++I) {
                f32x4 x, y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = s.x.dB[(I * 16 + r4 + e) * MLD + J * 16 + c16];
                    if (DELTA)
                        y[e] = s.x.dA[(I * 16 + r4 + e) * MLD + J * 16 + c16];
                }
                dH[J] = mfma32x4(x, column(s.x.ql, I * 16, f), dH[J]);
                if (DELTA)
                    dH[J] = mfma32x4(y, column(s.x.kl, I * 16, f), dH[J]);
                f *= s.eb[I * DKP + key];
            }
        }
        // ---- to one thread per (key, block)
        float cq[16], cr[16], cc[16], hb[16];
        auto hand_over = [&](const f32x4 (&x)[4], float (&y)[16]) {
            __syncthreads(); // what is in kr has been read
#pragma unroll
            for (int J = 0; J < 4; ++J)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s.x.kr[(J * 16 + r4 + e) * LD + key] = x[J][e];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                y[i] = s.x.kr[(r0 + i) * LD + d];
        };
        hand_over(dQ, cq);
        hand_over(dH, cc);
        if (DELTA)
            hand_over(dK, cr);
        {
            float p = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float before = p;
                p *= ev[i];
                cq[i] *= DELTA ? p : before;
                cr[i] = DELTA ? cr[i] * p : 0.f;
            }
            p = 1.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                cc[i] *= p;
                p *= ev[i];
            }
        }
        // ---- the log-decay's gradient: reads and writes of the block's rows, across
        // its border
        float gl[16];
        {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                const float before = x;
                x += DELTA ? fmaf(qv[i], cq[i], kv[i] * cr[i]) : qv[i] * cq[i];
                gl[i] = DELTA ? x : before;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                gl[i] += y;
                y = fmaf(kv[i], cc[i], y);
            }
        }
        // ---- pairs inside the block: hb[j] = P_ij of the row i at hand; its pairs
        // with the rows up to j cross row j + 1
        const float ud = !DELTA && d < a.dk ? a.u[static_cast<long>(h) * a.dk + d] : 0.f;
        float du = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            f32x4 gb[4], ga[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q * 4 > i)
                    continue;
                gb[q] = ld4(&s.x.dB[(r0 + i) * MLD + r0 + q * 4]);
                if (DELTA)
                    ga[q] = ld4(&s.x.dA[(r0 + i) * MLD + r0 + q * 4]);
            }
            const float own = gb[i / 4][i % 4]; // dB_ii: the pair (i, i), which no decay touches
            const float f = DELTA ? own : own * ud;
            float pairs = 0.f;
            cq[i] = fmaf(f, kv[i], cq[i]);
            cc[i] = fmaf(f, qv[i], cr[i] + cc[i]);
            du = fmaf(own * qv[i], kv[i], du);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (j >= i)
                    continue;
                const float before = hb[j];
                hb[j] *= ev[i];
                const float b = gb[j / 4][j % 4], pq = DELTA ? hb[j] : before, pk = pq * kv[j];
                cq[i] = fmaf(b, pk, cq[i]);
                float x = b * qv[i];
                if (DELTA) {
                    const float m = ga[j / 4][j % 4];
                    cc[i] = fmaf(m, pk, cc[i]);
                    x = fmaf(m, kv[i], x);
                }
                cc[j] = fmaf(pq, x, cc[j]);
                if (DELTA || j + 1 < i) {
                    pairs = fmaf(pk, x, pairs);
                    gl[j + 1] += pairs;
                }
            }
            hb[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            formed(cq[i]);
            formed(cc[i]);
            formed(gl[i]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (r0 + i < ch.rows && d < a.dk) {
                const long at = ((t0 + r0 + i) * a.H + h) * a.dk + d;
                static_cast<TIn *>(a.d_q)[at] = static_cast<TIn>(cq[i]);
                static_cast<TIn *>(a.d_k)[at] = static_cast<TIn>(cc[i]);
                a.d_ld[at] = a.ld[at] < kMinLogDecay ? 0.f : gl[i] + s.cross[tid]; // below it the decay is held
            }
        }
        if constexpr (!DELTA) {
            s.part[tid] = du;
            __syncthreads();
            if (tid < a.dk)
                a.w_du[slot_head * a.dk + tid] =
                    s.part[tid] + s.part[DKP + tid] + s.part[2 * DKP + tid] + s.part[3 * DKP + tid];
        } else if (tid < C) {
            const int b = lane >> 4, i = lane & 15;
            float dbeta = 0.f;
            for (int K = b; K < 4; ++K)
                dbeta += s.dbeta[K * (K + 1) / 2 + b][i];
            for (int t = 0; t < tiles; ++t)
                dbeta += a.w_db[(slot_head * tiles + t) * C + lane];
            if (lane < ch.rows)
                a.d_beta[(t0 + lane) * a.H + h] = dbeta;
        }
    }
}

// du: the sum over all chunks, as many as a sequence is long, in 64 bits.  16
// columns per workgroup, 16 threads each, which take every 16th chunk.
__global__ inline __launch_bounds__(256) void scan_du_kernel(ScanArgs a)
{
    __shared__ double part[16][17];
    const int c = threadIdx.x % 16, first = threadIdx.x / 16, i = blockIdx.x * 16 + c, n = a.H * a.dk;
    double x = 0.;
    if (i < n)
#pragma unroll 4
        for (int s = first; s < a.slots; s += 16)
            x += a.w_du[static_cast<long>(s) * n + i];
    part[first][c] = x;
    __syncthreads();
    if (first == 0 && i < n) {
        for (int t = 1; t < 16; ++t)
            x += part[t][c];
        a.d_u[i] = static_cast<float>(x);
    }
}

} // namespace dl
