// dl_scan_prep.h -- per chunk and head of a scan: the operands of its carry.
#pragma once

#include <type_traits>

#include "dl_scan.h"

namespace dl {

// Eight elements of an input row (zero where !in); vec: rows and heads start
// on 16-byte boundaries.
template <typename TIn> __device__ __forceinline__ void load_piece(TIn (&x)[8], const TIn *p, bool in, bool vec)
{
    using V = TIn __attribute__((ext_vector_type(8)));
    if (vec) {
        V v = {};
        if (in)
            v = *reinterpret_cast<const V *>(p);
        __builtin_memcpy(x, &v, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = in ? p[e] : TIn(0);
    }
}

template <int DKP> struct PrepLds {
    static constexpr int LD = DKP + 4;
    float k[C * LD], q[C * LD], e[C * LD];
    float A[C * MLD], B[C * MLD];
    float eb[4 * DKP], pre[4 * DKP], suf[4 * DKP]; // per 16-row block: its decay, that of the blocks before, after
    float beta[C];
};

// One chunk of one head: loads q, k and the decays, forms A and B (and N),
// and writes the operands of the forward carry, or (BWD) of the backward one.
//
// The pairs of tokens of one 16 x 16 diagonal block are formed on the vector
// unit (a running product of decays per pair and key); pairs of different
// blocks I > J as products of (prefix in I) and (suffix in J x blocks
// between), both <= 1, on the fp32 matrix instructions.
template <int OP, typename TIn, int DKP, bool BWD>
__global__ __launch_bounds__(256) void scan_prep_kernel(ScanArgs a)
{
    constexpr bool DELTA = OP != RWKV6;
    constexpr int LD = DKP + 4;
    extern __shared__ __align__(16) char smem[];
    PrepLds<DKP> &s = *reinterpret_cast<PrepLds<DKP> *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0)
        return;
    using P = Plan<OP, TIn>;
    const Ops<P::NPX, DKP> ops(a, static_cast<long>(slot) * a.H + h);

    // rows behind the end: k = q = 0, no decay, beta = 0
    for (int it = tid; it < C * DKP; it += 256) {
        const int i = it / DKP, d = it % DKP;
        const bool in = i < ch.rows && d < a.dk;
        const long t = ch.t0 + i;
        float kv = 0.f, qv = 0.f, ev = 1.f;
        if (in) {
            kv = from_in(static_cast<const TIn *>(a.k)[t * a.ks + static_cast<long>(h) * a.dk + d]);
            qv = from_in(static_cast<const TIn *>(a.q)[t * a.qs + static_cast<long>(h) * a.dk + d]);
            const float l = OP == GDN ? a.ld[t * a.H + h] : a.ld[(t * a.H + h) * a.dk + d];
            ev = expf(floor_log_decay(l));
        }
        s.k[i * LD + d] = kv;
        s.q[i * LD + d] = qv;
        s.e[i * LD + d] = ev;
    }
    if (tid < C)
        s.beta[tid] = DELTA && tid < ch.rows ? a.beta[static_cast<long>(ch.t0 + tid) * a.H + h] : 0.f;
    for (int it = tid; it < C * MLD; it += 256)
        s.A[it] = s.B[it] = 0.f;
    __syncthreads();

    // diagonal blocks: wave w takes block w; lane = (column j, quarter of the keys)
    {
        const int j = lane & 15, g = lane >> 4, r0 = w * 16;
        float sa[16], sb[16], su = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sa[i] = sb[i] = 0.f;
        for (int d = g * (DKP / 4); d < (g + 1) * (DKP / 4); ++d) {
            const float kj = s.k[(r0 + j) * LD + d];
            float kd = 0.f; // P_ij k_j
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = s.e[(r0 + i) * LD + d], qi = s.q[(r0 + i) * LD + d];
                if (!DELTA)
                    sb[i] = fmaf(kd, qi, sb[i]); // before the decay of row i
                kd = i == j ? kj : kd * e;
                if (DELTA) {
                    sb[i] = fmaf(kd, qi, sb[i]);
                    sa[i] = fmaf(kd, s.k[(r0 + i) * LD + d], sa[i]);
                }
            }
            if (!DELTA)
                su += d < a.dk ? s.q[(r0 + j) * LD + d] * a.u[static_cast<long>(h) * a.dk + d] * kj : 0.f;
        }
        su = wave_sum_from<16>(su);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float va = DELTA ? wave_sum_from<16>(sa[i]) : 0.f, vb = wave_sum_from<16>(sb[i]);
            if (g == 0) {
                s.A[(r0 + i) * MLD + r0 + j] = i > j ? va : 0.f;
                s.B[(r0 + i) * MLD + r0 + j] = i > j ? vb : i < j ? 0.f : DELTA ? vb : su;
            }
        }
    }
    __syncthreads();

    // in place: k -> k (prefix in its block), q -> q (prefix), e -> k (suffix)
    for (int it = tid; it < 4 * DKP; it += 256) {
        const int d = it % DKP, r0 = it / DKP * 16;
        float kv[16], ev[16], p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            kv[i] = s.k[(r0 + i) * LD + d];
            ev[i] = s.e[(r0 + i) * LD + d];
            const float before = p;
            p *= ev[i];
            s.q[(r0 + i) * LD + d] *= DELTA ? p : before;
            s.k[(r0 + i) * LD + d] = kv[i] * p;
        }
        s.eb[it] = p;
        p = 1.f;
#pragma unroll
        for (int i = 15; i >= 0; --i) {
            s.e[(r0 + i) * LD + d] = kv[i] * p;
            p *= ev[i];
        }
    }
    __syncthreads();
    if (tid < DKP) {
        float p = 1.f, q = 1.f;
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            s.pre[I * DKP + tid] = p;
            p *= s.eb[I * DKP + tid];
            s.suf[(3 - I) * DKP + tid] = q;
            q *= s.eb[(3 - I) * DKP + tid];
        }
        ops.gam()[tid] = p;
    }

    // pairs of different blocks
    for (int pair = w; pair < 6; pair += 4) {
        const int I = pair < 1 ? 1 : pair < 3 ? 2 : 3, J = pair - I * (I - 1) / 2;
        f32x4 ca = {0, 0, 0, 0}, cb = {0, 0, 0, 0};
        for (int ks = 0; ks < DKP / 16; ++ks) {
            const int d = ks * 16 + (lane >> 4) * 4;
            f32x4 r = *reinterpret_cast<const f32x4 *>(&s.e[(J * 16 + (lane & 15)) * LD + d]);
            for (int K = J + 1; K < I; ++K)
                r *= *reinterpret_cast<const f32x4 *>(&s.eb[K * DKP + d]);
            cb = mfma32x4(*reinterpret_cast<const f32x4 *>(&s.q[(I * 16 + (lane & 15)) * LD + d]), r, cb);
            if (DELTA)
                ca = mfma32x4(*reinterpret_cast<const f32x4 *>(&s.k[(I * 16 + (lane & 15)) * LD + d]), r, ca);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = (I * 16 + (lane >> 4) * 4 + e) * MLD + J * 16 + (lane & 15);
            s.B[at] = cb[e];
            if (DELTA)
                s.A[at] = ca[e];
        }
    }
    __syncthreads();

    // operands of C x DKP
    auto kt = [&](int i, int d) { return s.k[i * LD + d] * s.pre[(i >> 4) * DKP + d]; };
    auto qt = [&](int i, int d) { return s.q[i * LD + d] * s.pre[(i >> 4) * DKP + d]; };
    auto kh = [&](int i, int d) { return s.e[i * LD + d] * s.suf[(i >> 4) * DKP + d]; };
    if (!BWD) {
        if (DELTA)
            store_op<P::NPX, C, DKP>(ops.op(0), kt);
        store_op<P::NPQ, C, DKP>(ops.op(1), qt);
        store_op<P::NPX, DKP, C>(ops.op(2), [&](int d, int i) { return kh(i, d); });
        store_op<P::NPB, C, C, LOWER>(ops.mat(1), [&](int i, int j) { return s.B[i * MLD + j]; });
    } else {
        store_op<P::NPX, C, DKP>(ops.op(0), kh);
        store_op<P::NPX, DKP, C>(ops.op(1), [&](int d, int i) { return qt(i, d); });
        if (DELTA)
            store_op<P::NPX, DKP, C>(ops.op(2), [&](int d, int i) { return kt(i, d); });
        store_op<3, C, C, UPPER>(ops.mat(1), [&](int i, int j) { return s.B[j * MLD + i]; });
        if (DELTA)
            store_op<3, C, C, UPPER>(ops.mat(2), [&](int i, int j) { return s.A[j * MLD + i]; });
    }
    if (tid < C)
        ops.row(2)[tid] = s.beta[tid];
    if constexpr (DELTA) {
        // the operands are written: their LDS is free
        float *const area = reinterpret_cast<float *>(smem);
        static_assert(C * MLD + 4 * 16 * 20 <= 3 * C * LD, "N and the scratch of four waves fit");
        float *L = s.A, *N = area;
        __syncthreads();
        for (int it = tid; it < C * C; it += 256) {
            const int i = it / C, j = it % C;
            L[i * MLD + j] *= s.beta[j];
            N[i * MLD + j] = 0.f;
        }
        __syncthreads();
        invert_unit_lower(L, N, area + C * MLD + w * 16 * 20, w, lane);
        if (BWD)
            store_op<3, C, C, UPPER>(ops.mat(0), [&](int i, int j) { return N[j * MLD + i]; });
        else
            store_op<3, C, C, LOWER>(ops.mat(0), [&](int i, int j) { return N[i * MLD + j]; });
    }
}

// GDN: the decay is one number per row, so A and B are K K^T and Q K^T (exact
// products of the inputs' own planes) times the matrix of P_ij, and the keys'
// operands are the inputs themselves.
template <typename TIn, int DKP> struct PrepGdnLds {
    static constexpr int NP = Plan<GDN, TIn>::NPX, LD = DKP + 8;
    __bf16 k[NP][C * LD], q[NP][C * LD];
    float A[C * MLD], N[C * MLD]; // N: first B
    float e[C], beta[C], pre[C], suf[C], eb[4];
    float diag[4][16 * 16]; // P_ij of the diagonal blocks
    float tmp[4][16 * 20];
};

template <typename TIn, int DKP, bool BWD>
__global__ __launch_bounds__(256) void scan_prep_gdn_kernel(ScanArgs a, bool vec)
{
    using P = Plan<GDN, TIn>;
    constexpr int NP = P::NPX, LD = DKP + 8, KS = DKP / 32;
    extern __shared__ __align__(16) char smem[];
    PrepGdnLds<TIn, DKP> &s = *reinterpret_cast<PrepGdnLds<TIn, DKP> *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0)
        return;
    const Ops<NP, DKP> ops(a, static_cast<long>(slot) * a.H + h);

    // eight elements of a row per thread and turn; rows and keys behind the
    // end are zero
    constexpr int PIECES = C * DKP / 8 / 256;
    static_assert(PIECES >= 1, "every thread has a piece");
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const TIn *src = static_cast<const TIn *>(t ? a.q : a.k);
        const long stride = t ? a.qs : a.ks;
        TIn x[PIECES][8];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int i = (p * 256 + tid) / (DKP / 8), d = (p * 256 + tid) % (DKP / 8) * 8;
            load_piece(x[p], src + (ch.t0 + static_cast<long>(i)) * stride + static_cast<long>(h) * a.dk + d,
                       i < ch.rows && d < a.dk, vec);
        }
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int i = (p * 256 + tid) / (DKP / 8), d = (p * 256 + tid) % (DKP / 8) * 8;
            bf16x8 pl[NP];
            if constexpr (P::BF) {
                pl[0] = __builtin_bit_cast(bf16x8, x[p]);
            } else {
                split(__builtin_bit_cast(f32x8, x[p]), pl);
            }
#pragma unroll
            for (int n = 0; n < NP; ++n)
                *reinterpret_cast<bf16x8 *>(&(t ? s.q : s.k)[n][i * LD + d]) = pl[n];
        }
    }
    if (tid < C) {
        const long at = (static_cast<long>(ch.t0) + tid) * a.H + h;
        const bool in = tid < ch.rows;
        s.e[tid] = in ? expf(floor_log_decay(a.ld[at])) : 1.f;
        s.beta[tid] = in ? a.beta[at] : 0.f;
        ops.row(2)[tid] = s.beta[tid];
    }
    for (int it = tid; it < C * MLD; it += 256)
        s.A[it] = s.N[it] = 0.f;
    __syncthreads();
    if (lane < 16) { // products of decays within block w, column lane
        float p = 0.f, pre = 1.f, suf = 1.f, all = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float e = s.e[w * 16 + i];
            p = i == lane ? 1.f : p * e;
            s.diag[w][i * 16 + lane] = p;
            pre *= i <= lane ? e : 1.f;
            suf *= i > lane ? e : 1.f;
            all *= e;
        }
        s.pre[w * 16 + lane] = pre;
        s.suf[w * 16 + lane] = suf;
        if (lane == 0)
            s.eb[w] = all;
    }
    __syncthreads();
    if (tid < C) {
        float g = s.pre[tid], e = s.suf[tid];
        for (int K = 0; K < 4; ++K) {
            g *= K < tid / 16 ? s.eb[K] : 1.f;
            e *= K > tid / 16 ? s.eb[K] : 1.f;
        }
        ops.row(0)[tid] = g;
        ops.row(1)[tid] = e;
    }
    for (int d = tid; d < DKP; d += 256)
        ops.gam()[d] = s.eb[0] * s.eb[1] * s.eb[2] * s.eb[3];

    auto frag = [&](bf16x8 (&f)[NP], const __bf16 (&x)[NP][C * LD], int rb, int ks) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            f[n] = *reinterpret_cast<const bf16x8 *>(&x[n][(rb * 16 + (lane & 15)) * LD + ks * 32 + (lane >> 4) * 8]);
    };
    {
        bf16x8 ka[KS][NP], qa[KS][NP];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            frag(ka[ks], s.k, w, ks);
            frag(qa[ks], s.q, w, ks);
            if (!BWD) { // the rows of this wave are fragments of the operands already
                store_frag(ops.op(0), KS, w, ks, lane, ka[ks]);
                bf16x8 qo[P::NPQ];
#pragma unroll
                for (int n = 0; n < P::NPQ; ++n)
                    qo[n] = qa[ks][n];
                store_frag(ops.op(1), KS, w, ks, lane, qo);
            } else {
                store_frag(ops.op(0), KS, w, ks, lane, ka[ks]);
            }
        }
        float between = 1.f;
        for (int J = w; J >= 0; --J) {
            f32x4 ca = {0, 0, 0, 0}, cb = {0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 kb[NP];
                frag(kb, s.k, J, ks);
                ca = mma<3>(ka[ks], kb, ca);
                cb = mma<3>(qa[ks], kb, cb);
            }
            const int j = lane & 15, i0 = (lane >> 4) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e;
                const float f = J == w ? s.diag[w][i * 16 + j]
                                       : s.pre[w * 16 + i] * (between * s.suf[J * 16 + j]);
                const bool below = J < w || i > j;
                s.A[(w * 16 + i) * MLD + J * 16 + j] = below ? ca[e] * f : 0.f;
                s.N[(w * 16 + i) * MLD + J * 16 + j] = below || i == j ? cb[e] * f : 0.f;
            }
            if (J < w)
                between *= s.eb[J];
        }
    }
    __syncthreads();
    // the operands whose rows are keys: columns of the staged tiles
    auto columns = [&](auto np, __bf16 *op, const __bf16 (&x)[NP][C * LD]) {
        constexpr int N = decltype(np)::value;
        for (int it = tid; it < DKP / 16 * (C / 32) * 64; it += 256) {
            const int l = it & 63, rb = (it >> 6) / (C / 32), ks = (it >> 6) % (C / 32);
            bf16x8 f[N];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[n][e] = x[n][(ks * 32 + (l >> 4) * 8 + e) * LD + rb * 16 + (l & 15)];
            store_frag(op, C / 32, rb, ks, l, f);
        }
    };
    if (!BWD) {
        columns(std::integral_constant<int, NP>(), ops.op(2), s.k);
        store_op<P::NPB, C, C, LOWER>(ops.mat(1), [&](int i, int j) { return s.N[i * MLD + j]; });
    } else {
        columns(std::integral_constant<int, NP>(), ops.op(1), s.q);
        columns(std::integral_constant<int, NP>(), ops.op(2), s.k);
        store_op<3, C, C, UPPER>(ops.mat(1), [&](int i, int j) { return s.N[j * MLD + i]; });
        store_op<3, C, C, UPPER>(ops.mat(2), [&](int i, int j) { return s.A[j * MLD + i]; });
    }
    __syncthreads();
    for (int it = tid; it < C * C; it += 256) {
        const int i = it / C, j = it % C;
        s.A[i * MLD + j] *= s.beta[j];
        s.N[i * MLD + j] = 0.f;
    }
    __syncthreads();
    invert_unit_lower(s.A, s.N, s.tmp[w], w, lane);
    if (BWD)
        store_op<3, C, C, UPPER>(ops.mat(0), [&](int i, int j) { return s.N[j * MLD + i]; });
    else
        store_op<3, C, C, LOWER>(ops.mat(0), [&](int i, int j) { return s.N[i * MLD + j]; });
}

} // namespace dl
