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

// A (and B) in fp32 for grads: the ten blocks of the lower triangle, a lane's
// four rows of its column as in a product's result.
__device__ __forceinline__ void store_pairs(__bf16 *mat, const float *A, const float *B, int n)
{
    for (int it = threadIdx.x; it < n * 640; it += blockDim.x) {
        const int l = it & 63, b = (it >> 6) % 10;
        const float *x = it < 640 ? A : B;
        const int I = b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3, J = b - I * (I + 1) / 2;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = x[(I * 16 + (l >> 4) * 4 + e) * MLD + J * 16 + (l & 15)];
        reinterpret_cast<f32x4 *>(mat)[it] = v;
    }
}

template <int OP, int DKP> struct PrepLds {
    static constexpr int LD = DKP + 4;
    float k[C * LD], q[C * LD], e[C * LD];
    float B[C * MLD], A[OP == RWKV6 ? 4 : C * MLD];
    float eb[4 * DKP], inv[4 * DKP]; // per 16-row block: its decay, and one over it
    float pre[4 * DKP], suf[4 * DKP]; // that of the blocks before, after
    float beta[C], diag[C];
    int strong[4];
};

// One chunk of one head: loads q, k and the decays, forms A and B (and N),
// and writes the operands of the forward carry, or (BWD) of the backward one.
//
// Pairs of tokens of two blocks of 16 rows I >= J are products of rows scaled
// by the decay from I's start (prefix) and to J's end (suffix x the blocks
// between), all <= 1, on the fp32 matrix instructions.  Within a block (I = J)
// that is Gam_C too much, and the suffix is divided by the block's decay:
// relative rounding only, as long as the decay is far from underflow.  Blocks
// where a key decays by more than 2^-40 take the vector unit instead, with a
// running product of decays per pair and key.
//
// Bound by latency (one workgroup of eight waves fits a CU, for its LDS).
template <int DKP> constexpr int prep_threads() { return DKP == 128 ? 512 : 256; }

template <int OP, typename TIn, int DKP, bool BWD>
__global__ __launch_bounds__(prep_threads<DKP>()) void scan_prep_kernel(ScanArgs a, bool vec)
{
    using P = Plan<OP, TIn>;
    constexpr bool DELTA = P::DELTA;
    constexpr int LD = DKP + 4, NT = prep_threads<DKP>(), NW = NT / 64;
    extern __shared__ __align__(16) char smem[];
    PrepLds<OP, DKP> &s = *reinterpret_cast<PrepLds<OP, DKP> *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0)
        return;
    const Ops<P::NPX, DKP> ops(a, static_cast<long>(slot) * a.H + h);

    // rows behind the end: k = q = 0, no decay, beta = 0
    constexpr int PIECES = C * DKP / 8 / NT;
    static_assert(PIECES >= 1, "every thread has a piece");
    {
        TIn xk[PIECES][8], xq[PIECES][8];
        float xl[PIECES][8];
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int i = (p * NT + tid) / (DKP / 8), d = (p * NT + tid) % (DKP / 8) * 8;
            const bool in = i < ch.rows && d < a.dk;
            const long t = static_cast<long>(ch.t0) + i, c = static_cast<long>(h) * a.dk + d;
            load_piece(xk[p], static_cast<const TIn *>(a.k) + t * a.ks + c, in, vec);
            load_piece(xq[p], static_cast<const TIn *>(a.q) + t * a.qs + c, in, vec);
            load_piece(xl[p], a.ld + t * a.H * a.dk + c, in, vec);
        }
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int i = (p * NT + tid) / (DKP / 8), d = (p * NT + tid) % (DKP / 8) * 8;
#pragma unroll
            for (int half = 0; half < 8; half += 4) {
                f32x4 kv, qv, ev;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kv[e] = from_in(xk[p][half + e]);
                    qv[e] = from_in(xq[p][half + e]);
                    ev[e] = expf(floor_log_decay(xl[p][half + e])); // 1 behind the end
                }
                *reinterpret_cast<f32x4 *>(&s.k[i * LD + d + half]) = kv;
                *reinterpret_cast<f32x4 *>(&s.q[i * LD + d + half]) = qv;
                *reinterpret_cast<f32x4 *>(&s.e[i * LD + d + half]) = ev;
            }
        }
    }
    if (tid < C) {
        s.beta[tid] = DELTA && tid < ch.rows ? a.beta[(static_cast<long>(ch.t0) + tid) * a.H + h] : 0.f;
        ops.row(2)[tid] = s.beta[tid];
    }
    if (tid < 4)
        s.strong[tid] = 0;
    for (int it = tid; it < C * MLD; it += NT) {
        s.B[it] = 0.f;
        if (DELTA)
            s.A[it] = 0.f;
    }
    __syncthreads();

    const int d = tid % DKP, I0 = tid / DKP, r0 = I0 * 16; // one thread per (key, block)
    const bool mine = tid < 4 * DKP;
    float ev[16];
    if (mine) {
        float p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            ev[i] = s.e[(r0 + i) * LD + d];
            p *= ev[i];
        }
        s.eb[tid] = p;
        s.inv[tid] = 1.f / p;
        if (!(p >= 0x1p-40f)) // a NaN decay takes the pairwise way as well
            s.strong[I0] = 1;
    }
    if (!DELTA) { // B_ii = sum r u k: NT / 64 lanes per row
        constexpr int G = NT / C;
        const int i = tid / G;
        float x = 0.f;
        for (int c = tid % G; c < a.dk; c += G)
            x = fmaf(s.q[i * LD + c] * a.u[static_cast<long>(h) * a.dk + c], s.k[i * LD + c], x);
#pragma unroll
        for (int m = 1; m < G; m *= 2)
            x += __shfl_xor(x, m);
        if (tid % G == 0)
            s.diag[i] = x;
    }
    __syncthreads();

    const int strong[4] = {s.strong[0], s.strong[1], s.strong[2], s.strong[3]};
    if (strong[0] | strong[1] | strong[2] | strong[3]) {
        // wave w takes block w; lane = (column j, quarter of the keys)
        const int j = lane & 15, g = lane >> 4, b0 = w * 16;
        if (w < 4 && s.strong[w]) {
            float sa[16], sb[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sa[i] = sb[i] = 0.f;
            for (int c = g * (DKP / 4); c < (g + 1) * (DKP / 4); ++c) {
                const float kj = s.k[(b0 + j) * LD + c];
                float kd = 0.f; // P_ij k_j
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e = s.e[(b0 + i) * LD + c], qi = s.q[(b0 + i) * LD + c];
                    if (!DELTA)
                        sb[i] = fmaf(kd, qi, sb[i]); // before the decay of row i
                    kd = i == j ? kj : kd * e;
                    if (DELTA) {
                        sb[i] = fmaf(kd, qi, sb[i]);
                        sa[i] = fmaf(kd, s.k[(b0 + i) * LD + c], sa[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float va = DELTA ? wave_sum_from<16>(sa[i]) : 0.f, vb = wave_sum_from<16>(sb[i]);
                if (g == 0) {
                    if (DELTA)
                        s.A[(b0 + i) * MLD + b0 + j] = i > j ? va : 0.f;
                    s.B[(b0 + i) * MLD + b0 + j] = i > j ? vb : i < j ? 0.f : DELTA ? vb : s.diag[b0 + i];
                }
            }
        }
        __syncthreads();
    }

    // in place: k -> k (prefix in its block), q -> q (prefix), e -> k (suffix)
    if (mine) {
        float kv[16], p = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            kv[i] = s.k[(r0 + i) * LD + d];
            const float before = p;
            p *= ev[i];
            s.q[(r0 + i) * LD + d] *= DELTA ? p : before;
            s.k[(r0 + i) * LD + d] = kv[i] * p;
        }
        p = 1.f;
#pragma unroll
        for (int i = 15; i >= 0; --i) {
            s.e[(r0 + i) * LD + d] = kv[i] * p;
            p *= ev[i];
        }
    }
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
    __syncthreads();

    // pairs of tokens: a wave takes one of the ten block pairs, of A or of B
    for (int task = w; task < (DELTA ? 20 : 10); task += NW) {
        const bool isA = task >= 10;
        const int pair = isA ? task - 10 : task;
        const int I = pair < 1 ? 0 : pair < 3 ? 1 : pair < 6 ? 2 : 3, J = pair - I * (I + 1) / 2;
        if (I == J && strong[I])
            continue;
        const float *left = isA ? s.k : s.q;
        f32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < DKP / 16; ++ks) {
            const int c = ks * 16 + (lane >> 4) * 4;
            f32x4 r = *reinterpret_cast<const f32x4 *>(&s.e[(J * 16 + (lane & 15)) * LD + c]);
            if (I == J)
                r *= *reinterpret_cast<const f32x4 *>(&s.inv[I * DKP + c]);
            for (int K = J + 1; K < I; ++K)
                r *= *reinterpret_cast<const f32x4 *>(&s.eb[K * DKP + c]);
            x = mfma32x4(*reinterpret_cast<const f32x4 *>(&left[(I * 16 + (lane & 15)) * LD + c]), r, x);
        }
        const int j = lane & 15;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = (lane >> 4) * 4 + e;
            float v = x[e];
            if (I == J)
                v = i > j ? v : i < j || isA ? 0.f : DELTA ? v : s.diag[I * 16 + i];
            (isA ? s.A : s.B)[(I * 16 + i) * MLD + J * 16 + j] = v;
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
            store_pairs(ops.mat(2), s.A, s.A, 1);
    }
    if (tid < C)
        ops.row(2)[tid] = s.beta[tid];
    if constexpr (DELTA) {
        // the operands are written: their LDS is free
        float *const area = reinterpret_cast<float *>(smem);
        static_assert(C * MLD + 4 * 16 * 20 <= 3 * C * LD, "N and the scratch of four waves fit");
        float *L = s.A, *N = area;
        __syncthreads();
        for (int it = tid; it < C * C; it += NT) {
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
        store_pairs(ops.mat(2), s.A, s.N, 2);
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
