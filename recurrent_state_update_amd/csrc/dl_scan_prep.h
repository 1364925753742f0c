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

// The outputs' rows of a chunk that belongs to no sequence: zero.
template <typename T> __device__ __forceinline__ void zero_rows(void *p, const ScanArgs &a, const Chunk &ch, int h, int width)
{
    if (!p)
        return;
    for (int it = threadIdx.x; it < ch.rows * width; it += blockDim.x)
        static_cast<T *>(p)[((static_cast<long>(ch.t0) + it / width) * a.H + h) * width + it % width] = T(0);
}
template <int OP, typename TIn, bool BWD> __device__ __forceinline__ void zero_chunk(const ScanArgs &a, const Chunk &ch, int h)
{
    if (!BWD) {
        zero_rows<TIn>(a.o, a, ch, h, a.dv);
        return;
    }
    zero_rows<TIn>(a.d_q, a, ch, h, a.dk);
    zero_rows<TIn>(a.d_k, a, ch, h, a.dk);
    zero_rows<TIn>(a.d_v, a, ch, h, a.dv);
    zero_rows<float>(a.d_beta, a, ch, h, 1);
    zero_rows<float>(a.d_ld, a, ch, h, OP == GDN ? 1 : a.dk);
}

// The chunk of a workgroup that has operands to form (rows > 0); the outputs' rows
// of no sequence, ahead of the first and behind the last, are zeroed here.
template <int OP, typename TIn, bool BWD> __device__ __forceinline__ Chunk prep_chunk(const ScanArgs &a, int slot, int h)
{
    const int before = seq_start(a, 0) - slot * C;
    if (before > 0)
        zero_chunk<OP, TIn, BWD>(a, {slot * C, before < C ? before : C, true}, h);
    Chunk ch = chunk_of(a, slot);
    if (ch.behind && ch.rows > 0) {
        zero_chunk<OP, TIn, BWD>(a, ch, h);
        ch.rows = 0;
    }
    return ch;
}

// The ten 16 x 16 blocks (I, J) of a lower triangle, numbered row by row.
__device__ __forceinline__ int block_row(int b) { return b < 1 ? 0 : b < 3 ? 1 : b < 6 ? 2 : 3; }
__device__ __forceinline__ int block_col(int b)
{
    const int I = block_row(b);
    return b - I * (I + 1) / 2;
}
// A (and B) in fp32 for grads: the ten blocks, a lane's four rows of its
// column as in a product's result; n: block, or 10 + block for B.
__device__ __forceinline__ void store_pair(f32x4 *pairs, int n, int lane, f32x4 v) { pairs[n * 64 + lane] = v; }

// The C x C matrices of a chunk, once the keys' tiles are done with.
struct PrepMats {
    float L[C * MLD], B[C * MLD]; // L = A diag(beta); N takes B's room once B's planes are written
};
// A result block in LDS.
__device__ __forceinline__ void put_block(float *m, int I, int J, int lane, f32x4 v)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        m[(I * 16 + (lane >> 4) * 4 + e) * MLD + J * 16 + (lane & 15)] = v[e];
}
// Zero the six blocks above the diagonal.
__device__ __forceinline__ void zero_above(float *m)
{
    for (int it = threadIdx.x; it < 6 * 64; it += blockDim.x) {
        const int b = it >> 6, J = b < 1 ? 1 : b < 3 ? 2 : 3, I = b - J * (J - 1) / 2;
        *reinterpret_cast<f32x4 *>(&m[(I * 16 + (it & 63) / 4) * MLD + J * 16 + it % 4 * 4]) = f32x4{0, 0, 0, 0};
    }
}
// From L and B in LDS: B's and N's planes.
template <int OP, typename TIn, bool BWD, int NP, int DKP>
__device__ __forceinline__ void store_mats(PrepMats &m, const Ops<NP, DKP> &ops, int w, int lane)
{
    using P = Plan<OP, TIn>;
    if (BWD)
        store_op<3, C, C, UPPER>(ops.mat(1), [&](int i, int j) { return m.B[j * MLD + i]; });
    else
        store_op<3, C, C, LOWER>(ops.mat(1), [&](int i, int j) { return m.B[i * MLD + j]; });
    if constexpr (P::DELTA) {
        __syncthreads(); // B is read (and zero above the diagonal, as N will be)
        invert_unit_lower(m.L, m.B, w, lane);
        if (BWD)
            store_op<3, C, C, UPPER>(ops.mat(0), [&](int i, int j) { return m.B[j * MLD + i]; });
        else
            store_op<3, C, C, LOWER>(ops.mat(0), [&](int i, int j) { return m.B[i * MLD + j]; });
    }
}

// ---- per-key decays (KDA, RWKV6)

// Keys are taken in passes of DP: their tiles then leave LDS for two
// workgroups on a CU.
template <int DKP> constexpr int prep_keys() { return DKP < 64 ? DKP : 64; }
template <int DKP> constexpr int prep_threads() { return 8 * prep_keys<DKP>(); }

template <int OP, int DKP> struct PrepLds {
    static constexpr int DP = prep_keys<DKP>(), LD = DP + 4;
    union {
        struct {
            float k[C * LD], q[C * LD], e[C * LD];
        };
        PrepMats m;
    };
    float eb[4 * DP], inv[4 * DP]; // per 16-row block: its decay, and one over it
    float pre[4 * DP], suf[4 * DP]; // that of the blocks before, after
    float pair[2][4][16 * 16];      // B, A of diagonal blocks formed pair by pair
    float beta[C], diag[C];
    int strong[4];
};

// One chunk of one head: loads q, k and the decays, forms A and B (and N),
// and writes the operands of the forward carry, or (BWD) of the backward one.
//
// Pairs of tokens of two blocks of 16 rows I >= J are products of rows scaled
// by the decay from I's start (prefix) and to J's end (suffix x the blocks
// between), all <= 1, on the fp32 matrix instructions.  Within a block (I = J)
// that is the block's decay too much, and the suffix is divided by it: relative
// rounding only, as long as the decay is far from underflow.  Blocks where a
// key decays by more than 2^-40 take the vector unit instead, with a running
// product of decays per pair and key.
//
// Bound by latency: a handful of short phases between barriers.  Two workgroups
// on a CU at d_k = 128: that holds the registers to 128, with 20 bytes a lane in
// scratch (KDA packed prompts 78 us; with the 152 that it takes unheld, and one
// workgroup, 103).
template <int OP, typename TIn, int DKP, bool BWD>
__global__ __launch_bounds__(prep_threads<DKP>(), 4) void scan_prep_kernel(ScanArgs a, bool vec)
{
    using P = Plan<OP, TIn>;
    constexpr bool DELTA = P::DELTA;
    constexpr int DP = prep_keys<DKP>(), LD = DP + 4, NT = prep_threads<DKP>(), NW = NT / 64;
    constexpr int TASKS = ((DELTA ? 20 : 10) + NW - 1) / NW;
    extern __shared__ __align__(16) char smem[];
    PrepLds<OP, DKP> &s = *reinterpret_cast<PrepLds<OP, DKP> *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const Chunk ch = prep_chunk<OP, TIn, BWD>(a, slot, h);
    if (ch.rows <= 0)
        return;
    const Ops<P::NPX, DKP> ops(a, static_cast<long>(slot) * a.H + h);

    if (tid < C) {
        s.beta[tid] = DELTA && tid < ch.rows ? a.beta[(static_cast<long>(ch.t0) + tid) * a.H + h] : 0.f;
        ops.row(2)[tid] = s.beta[tid];
    }
    for (int it = tid; it < 2 * 4 * 256 / 4; it += NT)
        reinterpret_cast<f32x4 *>(s.pair)[it] = f32x4{0, 0, 0, 0};
    f32x4 acc[TASKS];
#pragma unroll
    for (int p = 0; p < TASKS; ++p)
        acc[p] = f32x4{0, 0, 0, 0};
    float ruk = 0.f; // RWKV6: B_ii = sum r u k, NT / C lanes per row

#pragma unroll 1
    for (int d0 = 0; d0 < DKP; d0 += DP) {
        // rows behind the end: k = q = 0, no decay, beta = 0
        constexpr int PIECES = C * DP / 8 / NT;
        static_assert(PIECES == 1, "one piece per thread");
        const int pi = tid / (DP / 8), pd = tid % (DP / 8) * 8;
        {
            TIn xk[8], xq[8];
            float xl[8];
            const bool in = pi < ch.rows && d0 + pd < a.dk;
            const long t = static_cast<long>(ch.t0) + pi, c = static_cast<long>(h) * a.dk + d0 + pd;
            load_piece(xk, static_cast<const TIn *>(a.k) + t * a.ks + c, in, vec);
            load_piece(xq, static_cast<const TIn *>(a.q) + t * a.qs + c, in, vec);
            load_piece(xl, a.ld + t * a.H * a.dk + c, in, vec);
            if (d0 > 0)
                __syncthreads(); // the pass before is read
            if (tid < 4)
                s.strong[tid] = 0;
#pragma unroll
            for (int half = 0; half < 8; half += 4) {
                f32x4 kv, qv, ev;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kv[e] = from_in(xk[half + e]);
                    qv[e] = from_in(xq[half + e]);
                    ev[e] = expf(floor_log_decay(xl[half + e])); // 1 behind the end
                }
                *reinterpret_cast<f32x4 *>(&s.k[pi * LD + pd + half]) = kv;
                *reinterpret_cast<f32x4 *>(&s.q[pi * LD + pd + half]) = qv;
                *reinterpret_cast<f32x4 *>(&s.e[pi * LD + pd + half]) = ev;
            }
        }
        __syncthreads();

        const int d = tid % DP, I0 = tid / DP, r0 = I0 * 16; // one thread per (key, block)
        const bool mine = tid < 4 * DP;
        if (mine) {
            float p = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                p *= s.e[(r0 + i) * LD + d];
            s.eb[tid] = p;
            s.inv[tid] = 1.f / p;
            if (!(p >= 0x1p-40f)) // a NaN decay takes the pairwise way as well
                s.strong[I0] = 1;
        }
        if (!DELTA) {
            constexpr int G = NT / C;
            for (int c = tid % G; c < DP && d0 + c < a.dk; c += G)
                ruk = fmaf(s.q[tid / G * LD + c] * a.u[static_cast<long>(h) * a.dk + d0 + c], s.k[tid / G * LD + c], ruk);
        }
        __syncthreads();

        const int strong[4] = {s.strong[0], s.strong[1], s.strong[2], s.strong[3]};
        if (strong[0] | strong[1] | strong[2] | strong[3]) {
            // wave w takes block w; lane = (column j, quarter of the keys)
            const int j = lane & 15, g = lane >> 4, b0 = w * 16;
            if (w < 4 && s.strong[w]) {
#pragma unroll 1
                for (int isA = 0; isA < (DELTA ? 2 : 1); ++isA) {
                    const float *left = isA ? s.k : s.q;
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i] = 0.f;
                    for (int c = g * (DP / 4); c < (g + 1) * (DP / 4); ++c) {
                        const float kj = s.k[(b0 + j) * LD + c];
                        float kd = 0.f; // P_ij k_j
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float e = s.e[(b0 + i) * LD + c], l = left[(b0 + i) * LD + c];
                            if (!DELTA)
                                x[i] = fmaf(kd, l, x[i]); // before the decay of row i
                            kd = i == j ? kj : kd * e;
                            if (DELTA)
                                x[i] = fmaf(kd, l, x[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float v = wave_sum_from<16>(x[i]);
                        if (g == 0)
                            s.pair[isA][w][i * 16 + j] += v;
                    }
                }
            }
            __syncthreads();
        }

        // in place: k -> k (prefix in its block), q -> q (prefix), e -> k (suffix)
        if (mine) {
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
            p = 1.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                s.e[(r0 + i) * LD + d] = kv[i] * p;
                p *= ev[i];
            }
        } else if (tid - 4 * DP < DP) {
            const int c = tid - 4 * DP;
            float p = 1.f, q = 1.f;
#pragma unroll
            for (int I = 0; I < 4; ++I) {
                s.pre[I * DP + c] = p;
                p *= s.eb[I * DP + c];
                s.suf[(3 - I) * DP + c] = q;
                q *= s.eb[(3 - I) * DP + c];
            }
            ops.gam()[d0 + c] = p;
        }
        __syncthreads();

        // pairs of tokens: a wave takes blocks of B (0-9) and A (10-19)
#pragma unroll
        for (int p = 0; p < TASKS; ++p) {
            const int task = w + p * NW;
            if (task >= (DELTA ? 20 : 10))
                break;
            const int b = task >= 10 ? task - 10 : task, I = block_row(b), J = block_col(b);
            if (I == J && strong[I])
                continue;
            const float *left = task >= 10 ? s.k : s.q;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                const int c = ks * 16 + (lane >> 4) * 4;
                f32x4 r = *reinterpret_cast<const f32x4 *>(&s.e[(J * 16 + (lane & 15)) * LD + c]);
                if (I == J)
                    r *= *reinterpret_cast<const f32x4 *>(&s.inv[I * DP + c]);
                for (int K = J + 1; K < I; ++K)
                    r *= *reinterpret_cast<const f32x4 *>(&s.eb[K * DP + c]);
                acc[p] = mfma32x4(*reinterpret_cast<const f32x4 *>(&left[(I * 16 + (lane & 15)) * LD + c]), r, acc[p]);
            }
        }

        // operands of C x DKP: this pass's keys
        constexpr int KP = DP / 32, KA = DKP / 32;
        auto rows = [&](auto np, char *op, const float *x, const float *scale) {
            constexpr int NPL = decltype(np)::value;
            for (int it = tid; it < 4 * KP * 64; it += NT) {
                const int l = it & 63, rb = (it >> 6) / KP, ks = (it >> 6) % KP, c = ks * 32 + (l >> 4) * 8;
                f32x8 v;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = x[(rb * 16 + (l & 15)) * LD + c + e] * scale[rb * DP + c + e];
                store_frag<NPL>(op, KA, rb, d0 / 32 + ks, l, v);
            }
        };
        auto columns = [&](auto np, char *op, const float *x, const float *scale) {
            constexpr int NPL = decltype(np)::value;
            for (int it = tid; it < DP / 16 * 2 * 64; it += NT) {
                const int l = it & 63, rb = (it >> 6) / 2, ks = (it >> 6) % 2, c = rb * 16 + (l & 15), i = ks * 32 + (l >> 4) * 8;
                const float f0 = scale[i / 16 * DP + c];
                f32x8 v;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = x[(i + e) * LD + c] * f0;
                store_frag<NPL>(op, 2, d0 / 16 + rb, ks, l, v);
            }
        };
        constexpr std::integral_constant<int, P::NPX> npx;
        if (!BWD) {
            if (DELTA)
                rows(npx, ops.op(0), s.k, s.pre);
            rows(npx, ops.op(1), s.q, s.pre);
            columns(npx, ops.op(2), s.e, s.suf);
        } else {
            rows(npx, ops.op(0), s.e, s.suf);
            columns(npx, ops.op(1), s.q, s.pre);
            if (DELTA)
                columns(npx, ops.op(2), s.k, s.pre);
        }
    }

    if (!DELTA) {
        constexpr int G = NT / C;
#pragma unroll
        for (int m = 1; m < G; m *= 2)
            ruk += __shfl_xor(ruk, m);
        if (tid % G == 0)
            s.diag[tid / G] = ruk;
    }
    __syncthreads(); // the tiles are read
    zero_above(s.m.B);
#pragma unroll
    for (int p = 0; p < TASKS; ++p) {
        const int task = w + p * NW;
        if (task >= (DELTA ? 20 : 10))
            break;
        const bool isA = task >= 10;
        const int b = isA ? task - 10 : task, I = block_row(b), J = block_col(b), j = lane & 15;
        f32x4 v = acc[p];
        if (I == J) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = (lane >> 4) * 4 + e;
                const float x = v[e] + s.pair[isA][I][i * 16 + j];
                v[e] = i > j ? x : i < j || isA ? 0.f : DELTA ? x : s.diag[I * 16 + i];
            }
        }
        if (isA) {
            if (BWD)
                store_pair(ops.pairs(), b, lane, v);
            v *= s.beta[J * 16 + j];
        }
        put_block(isA ? s.m.L : s.m.B, I, J, lane, v);
    }
    __syncthreads();
    store_mats<OP, TIn, BWD>(s.m, ops, w, lane);
}

// ---- one decay per row (GDN)

// A and B are K K^T and Q K^T (exact products of the inputs' own planes) times
// the matrix of P_ij, and the keys' operands are the inputs themselves.
template <typename TIn, int DKP> struct PrepGdnLds {
    static constexpr int NP = Plan<GDN, TIn>::NPX, LD = DKP + 8;
    union {
        struct {
            __bf16 k[NP][C * LD], q[NP][C * LD];
        };
        PrepMats m;
    };
    float e[C], beta[C], pre[C], suf[C], eb[4];
    float diag[4][16 * 16]; // P_ij of the diagonal blocks
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
    const Chunk ch = prep_chunk<GDN, TIn, BWD>(a, slot, h);
    if (ch.rows <= 0)
        return;
    const Ops<NP, DKP> ops(a, static_cast<long>(slot) * a.H + h);

    // eight elements of a row per thread and turn; rows and keys behind the
    // end are zero
    constexpr int PIECES = C * DKP / 8 / 256;
    static_assert(PIECES >= 1, "every thread has a piece");
    {
        TIn x[2][PIECES][8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int i = (p * 256 + tid) / (DKP / 8), d = (p * 256 + tid) % (DKP / 8) * 8;
                load_piece(x[t][p], static_cast<const TIn *>(t ? a.q : a.k) + (ch.t0 + static_cast<long>(i)) * (t ? a.qs : a.ks) +
                                        static_cast<long>(h) * a.dk + d,
                           i < ch.rows && d < a.dk, vec);
            }
        if (tid < C) {
            const long at = (static_cast<long>(ch.t0) + tid) * a.H + h;
            const bool in = tid < ch.rows;
            s.e[tid] = in ? expf(floor_log_decay(a.ld[at])) : 1.f;
            s.beta[tid] = in ? a.beta[at] : 0.f;
            ops.row(2)[tid] = s.beta[tid];
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                const int i = (p * 256 + tid) / (DKP / 8), d = (p * 256 + tid) % (DKP / 8) * 8;
                bf16x8 pl[NP];
                if constexpr (P::BF)
                    pl[0] = __builtin_bit_cast(bf16x8, x[t][p]);
                else
                    split(__builtin_bit_cast(f32x8, x[t][p]), pl);
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    *reinterpret_cast<bf16x8 *>(&(t ? s.q : s.k)[n][i * LD + d]) = pl[n];
            }
    }
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

    // a wave takes five of the twenty blocks of B (0-9) and A (10-19)
    auto frag = [&](bf16x8 (&f)[NP], const __bf16 (&x)[NP][C * LD], int rb, int ks) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
            f[n] = *reinterpret_cast<const bf16x8 *>(&x[n][(rb * 16 + (lane & 15)) * LD + ks * 32 + (lane >> 4) * 8]);
    };
    f32x4 acc[5];
#pragma unroll
    for (int p = 0; p < 5; ++p) {
        const int task = w + p * 4, b = task >= 10 ? task - 10 : task, I = block_row(b), J = block_col(b);
        Acc x;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            bf16x8 l[NP], r[NP];
            if (task >= 10)
                frag(l, s.k, I, ks);
            else
                frag(l, s.q, I, ks);
            frag(r, s.k, J, ks);
            x.add(l, r);
        }
        acc[p] = x.sum();
    }
    // the keys' operands: rows of the tiles, and their columns
    auto rows = [&](char *op, const __bf16 (&x)[NP][C * LD]) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            bf16x8 f[NP];
            frag(f, x, w, ks);
            store_frag<NP>(op, KS, w, ks, lane, f);
        }
    };
    auto columns = [&](char *op, const __bf16 (&x)[NP][C * LD]) {
        for (int it = w; it < DKP / 16 * 2; it += 4) {
            const int rb = it / 2, ks = it % 2;
            bf16x8 f[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[n][e] = x[n][(ks * 32 + (lane >> 4) * 8 + e) * LD + rb * 16 + (lane & 15)];
            store_frag<NP>(op, 2, rb, ks, lane, f);
        }
    };
    rows(ops.op(0), s.k);
    if (!BWD) {
        rows(ops.op(1), s.q);
        columns(ops.op(2), s.k);
    } else {
        columns(ops.op(1), s.q);
        columns(ops.op(2), s.k);
    }
    __syncthreads(); // the tiles are read, the decays complete
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
    zero_above(s.m.B);
#pragma unroll
    for (int p = 0; p < 5; ++p) {
        const int task = w + p * 4, b = task >= 10 ? task - 10 : task, I = block_row(b), J = block_col(b);
        const bool isA = task >= 10;
        const int j = lane & 15, i0 = (lane >> 4) * 4;
        float right = s.suf[J * 16 + j];
        for (int K = J + 1; K < I; ++K)
            right *= s.eb[K];
        f32x4 v = acc[p];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e;
            const float f = I == J ? s.diag[I][i * 16 + j] : s.pre[I * 16 + i] * right;
            v[e] = I > J || i > j || (i == j && !isA) ? v[e] * f : 0.f;
        }
        if (BWD)
            store_pair(ops.pairs(), isA ? b : 10 + b, lane, v);
        if (isA)
            v *= s.beta[J * 16 + j];
        put_block(isA ? s.m.L : s.m.B, I, J, lane, v);
    }
    __syncthreads();
    store_mats<GDN, TIn, BWD>(s.m, ops, w, lane);
}

} // namespace dl
