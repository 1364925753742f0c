// dl_scan.h -- the HIP kernels of the sequence scan (dl_scan, dl_scan_backward)
// for gfx950, instantiated once per operator in dl_scan_gdn.hip,
// dl_scan_kda.hip and dl_scan_rwkv6.hip.
//
// What is computed: the recurrence of the decode step (dl_kernels.h) over
// whole sequences, in chunks of C = 64 tokens.  One (sequence, head), one
// chunk with start state S (d_k x d_v), e_i = e^{ell_i} (per key),
// P_ij = e_{j+1} ... e_i (P_ii = 1), Gam_i = e_1 ... e_i:
//   K~_i = Gam_i (.) k_i       Q~_i = Gam_i (.) q_i      (RWKV6: Gam_{i-1})
//   K^_j = P_Cj (.) k_j
//   A_ij = sum_d P_ij k_i k_j  (j < i)
//   B_ij = sum_d P_ij q_i k_j  (j <= i; RWKV6: P_{i-1,j}, j < i, and
//                               B_ii = sum_d q_i u k_i)
//   delta rule:  E = N (V - K~ S),  N = (I + A diag(beta))^-1,  b = beta E
//   RWKV6:       b = V
//   O  = Q~ S + B b
//   S' = Gam_C (.) S + K^T^ b
// so that all work except the carry from S to S' is matrix products over
// chunks.  Its adjoint (dO, dS' given) has the same shape:
//   db = B^T dO + K^ dS',  z = N^T (beta db),  y = db - A^T z,
//   dbeta = y . E,  dv = z  (RWKV6: dv = db)
//   dS = Gam_C (.) dS' + Q~^T dO - K~^T z
//   dQ~ = dO S^T, dK~ = -z S^T, dK^ = b dS'^T, dB = dO b^T, dA = -z b^T,
// from which dq, dk and the log-decay's gradient follow within the chunk.
//
// Every decay is a product of factors e_m in [0, 1], never a quotient and
// never the exponential of a difference of two cumulative sums: full
// forgetting (e = 0) and any strong decay are exact and cannot overflow.
//
// Kernels: prep (per chunk and head: the scaled operands, B and N, split
// into bf16 planes in the matrix instruction's own register order); the
// forward carry and the backward carry (per sequence, head and 16 value
// columns: the columns of S are independent); grads (per chunk and head).
//
// Precision.  The products run on the bf16 matrix instructions, but state,
// sums and factors are held in 32 bits: an fp32 factor is split into three
// bf16 planes (24 bits) and a product takes the six plane pairs above 2^-24.
#pragma once

#include <hip/hip_runtime.h>

#include "dl_internal.h"
#include "dl_kernels.h"

namespace dl {

constexpr int C = kScanChunk; // tokens per chunk
static_assert(C == 64, "four 16-row blocks, one per wave");

using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x4 = __bf16 __attribute__((ext_vector_type(4)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));

constexpr int MLD = C + 4; // row stride of a C x C fp32 matrix in LDS

__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// One 16-deep step of a 16x16 fp32 product: lane l holds four consecutive k
// (from 4 (l / 16)) of row (column) l % 16.
__device__ __forceinline__ f32x4 mfma32x4(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int t = 0; t < 4; ++t)
        c = mfma32(a[t], b[t], c);
    return c;
}
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// x as a sum of three bf16 values, each the rounding of what is left: the
// planes of an fp32 factor (together its 24 bits).
template <typename V, typename F> __device__ __forceinline__ void split3(F x, V &p0, V &p1, V &p2)
{
    p0 = __builtin_convertvector(x, V);
    F r = x - __builtin_convertvector(p0, F);
    p1 = __builtin_convertvector(r, V);
    r = r - __builtin_convertvector(p1, F);
    p2 = __builtin_convertvector(r, V);
}
using f32x8 = float __attribute__((ext_vector_type(8)));

// c += a b for two factors in three planes each: the pairs whose product is
// at least 2^-24 of the largest, smallest first.
__device__ __forceinline__ f32x4 mfma_split(const bf16x8 (&a)[3], const bf16x8 (&b)[3], f32x4 c)
{
    c = mfma16(a[2], b[0], c);
    c = mfma16(a[0], b[2], c);
    c = mfma16(a[1], b[1], c);
    c = mfma16(a[1], b[0], c);
    c = mfma16(a[0], b[1], c);
    return mfma16(a[0], b[0], c);
}

template <typename TIn> __device__ __forceinline__ float from_in(TIn x);
template <> __device__ __forceinline__ float from_in<float>(float x) { return x; }
template <> __device__ __forceinline__ float from_in<__bf16>(__bf16 x) { return static_cast<float>(x); }

// ---------------------------------------------------------------- sequences --
//
// Chunks are numbered by slots: sequence n owns the slots from
// base(n) = start(n) / C + n on, which leaves every sequence enough of them
// (floor(a / C) + ceil((b - a) / C) <= floor(b / C) + 1) without a prefix sum
// over the lengths; T / C + N slots in all.  Offsets read from cu are clamped
// to [0, T], so a bad array cannot lead an access out of range.
struct Seq {
    int start, len, base;
};
__device__ __forceinline__ int seq_start(const ScanArgs &a, int n)
{
    if (!a.cu)
        return static_cast<int>(static_cast<long>(a.T) * n / a.N);
    const int s = a.cu[n];
    return s < 0 ? 0 : s > a.T ? a.T : s;
}
__device__ __forceinline__ Seq sequence(const ScanArgs &a, int n)
{
    Seq s;
    s.start = seq_start(a, n);
    const int end = seq_start(a, n + 1);
    s.len = end > s.start ? end - s.start : 0;
    s.base = s.start / C + n;
    return s;
}
// The chunk of a slot: its first token and its number of tokens (<= 0: none).
struct Chunk {
    int t0, rows;
};
__device__ __forceinline__ Chunk chunk_of(const ScanArgs &a, int slot)
{
    int lo = 0, hi = a.N - 1; // the last n with base(n) <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (seq_start(a, mid) / C + mid <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Seq s = sequence(a, lo);
    const int c = slot - s.base;
    Chunk r;
    r.t0 = s.start + c * C;
    r.rows = c < 0 ? 0 : s.len - c * C < C ? s.len - c * C : C;
    return r;
}

// -------------------------------------------------------- operands in memory --
//
// Per slot and head, in bf16 planes: three operands of C x DKP elements and
// three of C x C, then Gam_C.  An operand [rows][k] is stored as matrix
// fragments: (16 rows, 32 k, plane) -> 64 lanes x 8 elements, lane l holding
// row l % 16, k from 8 (l / 16): one coalesced 1 KiB load per fragment.
//   forward : op 0 K~ [C][DKP], 1 Q~ [C][DKP], 2 K^ [DKP][C]; mat 0 N, 1 B
//   backward: op 0 K^ [C][DKP], 1 Q~ [DKP][C], 2 K~ [DKP][C]; mat 0 N^T,
//             1 B^T, 2 A^T
template <int DKP> struct Ops {
    static constexpr size_t kOp = size_t(3) * C * DKP, kMat = size_t(3) * C * C; // elements
    static constexpr size_t kBytes = 2 * (3 * kOp + 3 * kMat) + 4 * DKP;
    char *p;
    __device__ Ops(const ScanArgs &a, long slot_head) : p(a.ops + slot_head * kBytes) {}
    __device__ __bf16 *op(int i) const { return reinterpret_cast<__bf16 *>(p) + i * kOp; }
    __device__ __bf16 *mat(int i) const { return reinterpret_cast<__bf16 *>(p) + 3 * kOp + i * kMat; }
    __device__ float *gam() const { return reinterpret_cast<float *>(p + 2 * (3 * kOp + 3 * kMat)); }
};
static_assert(Ops<32>::kBytes == scan_op_bytes(32) && Ops<64>::kBytes == scan_op_bytes(64) &&
                  Ops<128>::kBytes == scan_op_bytes(128),
              "the host sizes the workspace");

__device__ __forceinline__ void load_frag(bf16x8 (&f)[3], const __bf16 *op, int ksteps, int rb, int ks, int lane)
{
    const bf16x8 *p = reinterpret_cast<const bf16x8 *>(op) + ((rb * ksteps + ks) * 3) * 64 + lane;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        f[i] = p[i * 64];
}
__device__ __forceinline__ void store_frag(__bf16 *op, int ksteps, int rb, int ks, int lane, f32x8 x)
{
    bf16x8 f[3];
    split3(x, f[0], f[1], f[2]);
    bf16x8 *p = reinterpret_cast<bf16x8 *>(op) + ((rb * ksteps + ks) * 3) * 64 + lane;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        p[i * 64] = f[i];
}
// Write the fragments of [ROWS][K], element (r, k) given by f.
template <int ROWS, int K, typename F> __device__ __forceinline__ void store_op(__bf16 *op, F f)
{
    for (int it = threadIdx.x; it < ROWS / 16 * (K / 32) * 64; it += blockDim.x) {
        const int lane = it & 63, fr = it >> 6;
        const int r = fr / (K / 32) * 16 + (lane & 15), k = fr % (K / 32) * 32 + (lane >> 4) * 8;
        f32x8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = f(r, k + e);
        store_frag(op, K / 32, fr / (K / 32), fr % (K / 32), lane, x);
    }
}

// --------------------------------------------------------------------- prep --

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
    const Ops<DKP> ops(a, static_cast<long>(slot) * a.H + h);

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
            store_op<C, DKP>(ops.op(0), kt);
        store_op<C, DKP>(ops.op(1), qt);
        store_op<DKP, C>(ops.op(2), [&](int d, int i) { return kh(i, d); });
        store_op<C, C>(ops.mat(1), [&](int i, int j) { return s.B[i * MLD + j]; });
    } else {
        store_op<C, DKP>(ops.op(0), kh);
        store_op<DKP, C>(ops.op(1), [&](int d, int i) { return qt(i, d); });
        if (DELTA)
            store_op<DKP, C>(ops.op(2), [&](int d, int i) { return kt(i, d); });
        store_op<C, C>(ops.mat(1), [&](int i, int j) { return s.B[j * MLD + i]; });
        if (DELTA)
            store_op<C, C>(ops.mat(2), [&](int i, int j) { return s.A[j * MLD + i]; });
    }
    if constexpr (DELTA) {
        // N = (I + L)^-1, L = A diag(beta): the four diagonal blocks by
        // forward substitution, the others block by block,
        // N_IJ = -N_II sum_{J <= K < I} L_IK N_KJ.
        // the operands are written: their LDS is free
        float *const area = reinterpret_cast<float *>(smem);
        static_assert(C * MLD + 4 * 16 * 20 <= 3 * C * LD, "N and the scratch of four waves fit");
        float *L = s.A, *N = area, *tmp = area + C * MLD + w * 16 * 20;
        __syncthreads();
        for (int it = tid; it < C * C; it += 256) {
            const int i = it / C, j = it % C;
            L[i * MLD + j] *= s.beta[j];
            N[i * MLD + j] = 0.f;
        }
        __syncthreads();
        if (lane < 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = i == lane ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < i)
                        v = fmaf(-L[(w * 16 + i) * MLD + w * 16 + j], x[j], v);
                x[i] = v;
                N[(w * 16 + i) * MLD + w * 16 + lane] = v;
            }
        }
        __syncthreads();
        for (int dist = 1; dist < 4; ++dist) {
            if (w + dist < 4) {
                const int J = w, I = w + dist;
                f32x4 t = {0, 0, 0, 0}, c = {0, 0, 0, 0};
                const int r = lane & 15, k0 = (lane >> 4) * 4;
                for (int K = J; K < I; ++K) {
                    f32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = N[(K * 16 + k0 + e) * MLD + J * 16 + r];
                    t = mfma32x4(*reinterpret_cast<const f32x4 *>(&L[(I * 16 + r) * MLD + K * 16 + k0]), x, t);
                }
                // through this wave's own scratch into the other operand's
                // order; one wave's LDS accesses stay in order
                *reinterpret_cast<f32x4 *>(&tmp[r * 20 + k0]) = t;
                __builtin_amdgcn_wave_barrier();
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&tmp[r * 20 + k0]);
                c = mfma32x4(*reinterpret_cast<const f32x4 *>(&N[(I * 16 + r) * MLD + I * 16 + k0]), x, c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    N[(I * 16 + k0 + e) * MLD + J * 16 + r] = -c[e];
            }
            __syncthreads();
        }
        store_op<C, C>(ops.mat(0), [&](int i, int j) { return BWD ? N[j * MLD + i] : N[i * MLD + j]; });
    }
}

// -------------------------------------------------------------------- carry --

// Planes of a C-layout tile in LDS, as the other operand of a product: [16
// columns][K], k along the row.
template <int K> struct Planes {
    static constexpr int LD = K + 8;
    __bf16 p[3][16 * LD];
    // the four consecutive k from k0 of column c
    __device__ __forceinline__ void put(int c, int k0, f32x4 x)
    {
        bf16x4 v[3];
        split3(x, v[0], v[1], v[2]);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<bf16x4 *>(&p[i][c * LD + k0]) = v[i];
    }
    __device__ __forceinline__ void get(bf16x8 (&f)[3], int ks, int lane) const
    {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            f[i] = *reinterpret_cast<const bf16x8 *>(&p[i][(lane & 15) * LD + ks * 32 + (lane >> 4) * 8]);
    }
};

// acc += op[row block rb][K] x planes[K][16]
template <int K> __device__ __forceinline__ f32x4 product(const __bf16 *op, int rb, const Planes<K> &b, int lane, f32x4 acc)
{
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        bf16x8 fa[3], fb[3];
        load_frag(fa, op, K / 32, rb, ks, lane);
        b.get(fb, ks, lane);
        acc = mfma_split(fa, fb, acc);
    }
    return acc;
}

// The state row of a sequence: through a.rows if given; < 0 where the row is
// not one of the caller's a.nrows (nothing is read or written then).
__device__ __forceinline__ long state_row(const ScanArgs &a, int n)
{
    if (!a.rows)
        return n;
    const int r = a.rows[n];
    return r >= 0 && r < a.nrows ? r : -1;
}

// Forward carry: one workgroup per (sequence, head, 16 value columns).  Wave
// w holds rows 16 w.. of the chunk and row blocks w, w + 4 of the state (in
// fp32 registers).  SAVE: keeps every chunk's start state and E.
template <typename TIn, int DKP, bool DELTA, bool SAVE>
__global__ __launch_bounds__(256) void scan_carry_kernel(ScanArgs a)
{
    constexpr int RB = DKP / 64 > 0 ? DKP / 64 : 1;
    __shared__ Planes<DKP> sp;
    __shared__ Planes<C> rp, bp;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int col = lane & 15, r4 = (lane >> 4) * 4;
    const int tiles = a.dv / 16, tile = blockIdx.x % tiles, sh = blockIdx.x / tiles;
    const int h = sh % a.H, n = sh / a.H;
    const Seq sq = sequence(a, n);
    const int v0 = tile * 16 + col;
    const long row = state_row(a, n);
    const long st0 = (row * a.H + h) * a.dk * a.dv + v0;

    f32x4 S[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = (w + 4 * r) * 16 + r4 + e;
            S[r][e] = a.init && row >= 0 && d < a.dk ? a.init[st0 + static_cast<long>(d) * a.dv] : 0.f;
        }

    const int chunks = (sq.len + C - 1) / C;
    for (int c = 0; c < chunks; ++c) {
        const long slot_head = static_cast<long>(sq.base + c) * a.H + h;
        const Ops<DKP> ops(a, slot_head);
        const int rows = sq.len - c * C < C ? sq.len - c * C : C;
        const long t0 = sq.start + static_cast<long>(c) * C;
        f32x4 x, o = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w * 16 + r4 + e;
            x[e] = i < rows ? from_in(static_cast<const TIn *>(a.v)[(t0 + i) * a.vs + static_cast<long>(h) * a.dv + v0])
                            : 0.f;
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int rb = w + 4 * r;
            if (rb * 16 < DKP)
                sp.put(col, rb * 16 + r4, S[r]);
            if (SAVE) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = rb * 16 + r4 + e;
                    if (d < a.dk)
                        a.save_s[(slot_head * a.dk + d) * a.dv + v0] = S[r][e];
                }
            }
        }
        __syncthreads();
        if constexpr (DELTA) {
            rp.put(col, w * 16 + r4, x - product<DKP>(ops.op(0), w, sp, lane, f32x4{0, 0, 0, 0}));
            o = product<DKP>(ops.op(1), w, sp, lane, o);
            __syncthreads();
            x = product<C>(ops.mat(0), w, rp, lane, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = w * 16 + r4 + e;
                if (SAVE)
                    a.save_e[(slot_head * C + i) * a.dv + v0] = x[e];
                x[e] *= i < rows ? a.beta[(t0 + i) * a.H + h] : 0.f;
            }
        } else {
            o = product<DKP>(ops.op(1), w, sp, lane, o);
        }
        bp.put(col, w * 16 + r4, x);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int rb = w + 4 * r;
            if (rb * 16 < DKP)
                S[r] = product<C>(ops.op(2), rb, bp, lane,
                                  S[r] * *reinterpret_cast<const f32x4 *>(ops.gam() + rb * 16 + r4));
        }
        o = product<C>(ops.mat(1), w, bp, lane, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w * 16 + r4 + e;
            if (i < rows)
                static_cast<TIn *>(a.o)[((t0 + i) * a.H + h) * a.dv + v0] = static_cast<TIn>(o[e]);
        }
        // the next chunk writes sp at once: all reads of it lie before the
        // last barrier; bp and rp are rewritten behind further barriers
    }
    if (a.fin && row >= 0) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (w + 4 * r) * 16 + r4 + e;
                if (d < a.dk)
                    a.fin[st0 + static_cast<long>(d) * a.dv] = S[r][e];
            }
    }
}

// Backward carry: chunks from the last to the first, dS in registers.
// Writes every chunk's dS' and z (delta rule), dv, and per 16 value columns
// the partial sums of dbeta; at the end the initial state's gradient.
template <typename TIn, int DKP, bool DELTA>
__global__ __launch_bounds__(256) void scan_carry_bwd_kernel(ScanArgs a)
{
    constexpr int RB = DKP / 64 > 0 ? DKP / 64 : 1;
    __shared__ Planes<DKP> sp;
    __shared__ Planes<C> gp, wp, zp;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int col = lane & 15, r4 = (lane >> 4) * 4;
    const int tiles = a.dv / 16, tile = blockIdx.x % tiles, sh = blockIdx.x / tiles;
    const int h = sh % a.H, n = sh / a.H;
    const Seq sq = sequence(a, n);
    const int v0 = tile * 16 + col;
    const long st0 = (static_cast<long>(n) * a.H + h) * a.dk * a.dv + v0;

    f32x4 S[RB]; // dS
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = (w + 4 * r) * 16 + r4 + e;
            S[r][e] = a.dfin && d < a.dk ? a.dfin[st0 + static_cast<long>(d) * a.dv] : 0.f;
        }

    const int chunks = (sq.len + C - 1) / C;
    for (int c = chunks - 1; c >= 0; --c) {
        const long slot_head = static_cast<long>(sq.base + c) * a.H + h;
        const Ops<DKP> ops(a, slot_head);
        const int rows = sq.len - c * C < C ? sq.len - c * C : C;
        const long t0 = sq.start + static_cast<long>(c) * C;
        f32x4 g;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w * 16 + r4 + e;
            g[e] = i < rows && a.d_o ? from_in(static_cast<const TIn *>(a.d_o)[((t0 + i) * a.H + h) * a.dv + v0]) : 0.f;
        }
        gp.put(col, w * 16 + r4, g);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int rb = w + 4 * r;
            if (rb * 16 < DKP)
                sp.put(col, rb * 16 + r4, S[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = rb * 16 + r4 + e;
                if (d < a.dk)
                    a.w_ds[(slot_head * a.dk + d) * a.dv + v0] = S[r][e];
            }
        }
        __syncthreads();
        f32x4 db = product<C>(ops.mat(1), w, gp, lane, f32x4{0, 0, 0, 0});
        db = product<DKP>(ops.op(0), w, sp, lane, db);
        f32x4 x = db;
        if constexpr (DELTA) {
            f32x4 wb;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = w * 16 + r4 + e;
                wb[e] = i < rows ? db[e] * a.beta[(t0 + i) * a.H + h] : 0.f;
            }
            wp.put(col, w * 16 + r4, wb);
            __syncthreads();
            x = product<C>(ops.mat(0), w, wp, lane, f32x4{0, 0, 0, 0});
            zp.put(col, w * 16 + r4, x);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a.w_z[(slot_head * C + w * 16 + r4 + e) * a.dv + v0] = x[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w * 16 + r4 + e;
            if (i < rows)
                static_cast<TIn *>(a.d_v)[((t0 + i) * a.H + h) * a.dv + v0] = static_cast<TIn>(x[e]);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int rb = w + 4 * r;
            if (rb * 16 < DKP) {
                S[r] *= *reinterpret_cast<const f32x4 *>(ops.gam() + rb * 16 + r4);
                S[r] = product<C>(ops.op(1), rb, gp, lane, S[r]);
                if (DELTA)
                    S[r] -= product<C>(ops.op(2), rb, zp, lane, f32x4{0, 0, 0, 0});
            }
        }
        if constexpr (DELTA) {
            const f32x4 y = db - product<C>(ops.mat(2), w, zp, lane, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = w * 16 + r4 + e;
                float p = y[e] * a.save_e[(slot_head * C + i) * a.dv + v0];
                p = add_row_ror<1>(p);
                p = add_row_ror<2>(p);
                p = add_row_ror<4>(p);
                p = add_row_ror<8>(p);
                if (col == 0)
                    a.w_db[(slot_head * tiles + tile) * C + i] = p;
            }
        }
        __syncthreads(); // gp and sp are rewritten next
    }
    if (a.dinit) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = (w + 4 * r) * 16 + r4 + e;
                if (d < a.dk)
                    a.dinit[st0 + static_cast<long>(d) * a.dv] = S[r][e];
            }
    }
}

// -------------------------------------------------------------------- grads --

template <int DKP> struct GradLds {
    static constexpr int LD = DKP + 4;
    float k[C * LD], q[C * LD], e[C * LD];
    union {
        struct {
            float dA[C * MLD], dB[C * MLD];
        };
        float buf[C * LD]; // one C x DKP product on its way to the keys' threads
    };
    float gam[DKP];     // sum_v S dS' per key
    float part[4 * DKP]; // sums over the rows of a block
};

// One chunk of one head.  Wave w forms the 16 keys w of dQ~, dK~ and dK^ (all
// C rows); then one thread per (key, 16-row block I) walks the rows outside I
// with a running product of decays, and the pairs inside I.
template <int OP, typename TIn, int DKP>
__global__ __launch_bounds__(DKP * 4) void scan_grads_kernel(ScanArgs a)
{
    constexpr bool DELTA = OP != RWKV6;
    constexpr int LD = DKP + 4, NT = DKP * 4, NW = NT / 64;
    extern __shared__ __align__(16) char smem[];
    GradLds<DKP> &s = *reinterpret_cast<GradLds<DKP> *>(smem);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const long slot_head = static_cast<long>(slot) * a.H + h;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0) {
        if (!DELTA && tid < a.dk)
            a.w_du[slot_head * a.dk + tid] = 0.f;
        return;
    }
    for (int it = tid; it < C * DKP; it += NT) {
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

    const int r = lane & 15, k4 = (lane >> 4) * 4;
    // rows of dO, z and b as product operands: four values from v of row i
    auto ld_do = [&](int i, int v) {
        f32x4 x = {0, 0, 0, 0};
        if (i < ch.rows && a.d_o) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = from_in(static_cast<const TIn *>(a.d_o)[((static_cast<long>(ch.t0) + i) * a.H + h) * a.dv + v + e]);
        }
        return x;
    };
    auto ld_b = [&](int i, int v) {
        f32x4 x = {0, 0, 0, 0};
        if (i < ch.rows) {
            if constexpr (DELTA) {
                x = *reinterpret_cast<const f32x4 *>(&a.save_e[(slot_head * C + i) * a.dv + v]) *
                    a.beta[(static_cast<long>(ch.t0) + i) * a.H + h];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = from_in(static_cast<const TIn *>(
                        a.v)[(static_cast<long>(ch.t0) + i) * a.vs + static_cast<long>(h) * a.dv + v + e]);
            }
        }
        return x;
    };
    auto ld_z = [&](int i, int v) {
        return i < ch.rows ? *reinterpret_cast<const f32x4 *>(&a.w_z[(slot_head * C + i) * a.dv + v]) : f32x4{0, 0, 0, 0};
    };

    f32x4 dQ[4], dK[4], dH[4];
#pragma unroll
    for (int I = 0; I < 4; ++I)
        dQ[I] = dK[I] = dH[I] = f32x4{0, 0, 0, 0};
    float gs = 0.f;
    const int kd = w * 16 + r; // the key whose row of S this lane reads
    for (int v = k4; v < a.dv; v += 16) {
        f32x4 S = {0, 0, 0, 0}, dS = {0, 0, 0, 0};
        if (kd < a.dk) {
            S = *reinterpret_cast<const f32x4 *>(&a.save_s[(slot_head * a.dk + kd) * a.dv + v]);
            dS = *reinterpret_cast<const f32x4 *>(&a.w_ds[(slot_head * a.dk + kd) * a.dv + v]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            gs = fmaf(S[e], dS[e], gs);
#pragma unroll
        for (int I = 0; I < 4; ++I) {
            dQ[I] = mfma32x4(ld_do(I * 16 + r, v), S, dQ[I]);
            dH[I] = mfma32x4(ld_b(I * 16 + r, v), dS, dH[I]);
            if (DELTA)
                dK[I] = mfma32x4(ld_z(I * 16 + r, v), S, dK[I]);
        }
    }
    gs = wave_sum_from<16>(gs);
    if (lane < 16)
        s.gam[kd] = gs;

    // to one thread per (key, block of 16 rows)
    const int d = tid % DKP, I = tid / DKP, r0 = I * 16;
    float cq[16], cr[16], cc[16];
    auto hand_over = [&](const f32x4 (&x)[4], float (&y)[16]) {
        __syncthreads();
#pragma unroll
        for (int J = 0; J < 4; ++J)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s.buf[(J * 16 + k4 + e) * LD + w * 16 + r] = x[J][e];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            y[i] = s.buf[(r0 + i) * LD + d];
    };
    hand_over(dQ, cq);
    hand_over(dH, cc);
    if constexpr (DELTA) {
        hand_over(dK, cr);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            cr[i] = -cr[i];
    }
    __syncthreads();

    // dA (strictly lower) and dB (lower)
    for (int p = w; p < 10; p += NW) {
        const int BI = p < 1 ? 0 : p < 3 ? 1 : p < 6 ? 2 : 3, BJ = p - BI * (BI + 1) / 2;
        f32x4 xa = {0, 0, 0, 0}, xb = {0, 0, 0, 0};
        for (int v = k4; v < a.dv; v += 16) {
            const f32x4 b = ld_b(BJ * 16 + r, v);
            xb = mfma32x4(ld_do(BI * 16 + r, v), b, xb);
            if (DELTA)
                xa = mfma32x4(ld_z(BI * 16 + r, v), b, xa);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = BI * 16 + k4 + e, j = BJ * 16 + r;
            s.dA[i * MLD + j] = i > j ? -xa[e] : 0.f;
            s.dB[i * MLD + j] = i >= j ? xb[e] : 0.f;
        }
    }
    __syncthreads();

    // rows of I against the rows before: a running decay downwards
    {
        float tq[16], tr[16], f = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            tq[i] = tr[i] = 0.f;
        for (int j = r0 - 1; j >= 0; --j) {
            const float kj = s.k[j * LD + d] * f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                tq[i] = fmaf(s.dB[(r0 + i) * MLD + j], kj, tq[i]);
                if (DELTA)
                    tr[i] = fmaf(s.dA[(r0 + i) * MLD + j], kj, tr[i]);
            }
            f *= s.e[j * LD + d];
        }
        float p = 1.f; // prefix in the block
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float before = p;
            p *= s.e[(r0 + i) * LD + d];
            cq[i] = (tq[i] + f * cq[i]) * (DELTA ? p : before);
            cr[i] = DELTA ? (tr[i] + f * cr[i]) * p : 0.f;
        }
    }
    // rows of I against the rows behind: a running decay upwards
    float kh = 0.f; // sum over the block of k . (its part of dK^)
    {
        float tc[16], f = 1.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            tc[j] = 0.f;
        for (int m = r0 + 16; m < C; ++m) {
            // RWKV6's row m reads the state before its own decay
            const float qm0 = s.q[m * LD + d] * f;
            f *= s.e[m * LD + d];
            const float km = s.k[m * LD + d] * f, qm = DELTA ? s.q[m * LD + d] * f : qm0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                tc[j] = fmaf(s.dB[m * MLD + r0 + j], qm, tc[j]);
                if (DELTA)
                    tc[j] = fmaf(s.dA[m * MLD + r0 + j], km, tc[j]);
            }
        }
        float p = 1.f; // suffix in the block
#pragma unroll
        for (int j = 15; j >= 0; --j) {
            const float end = f * cc[j] * p;
            kh = fmaf(s.k[(r0 + j) * LD + d], end, kh);
            cc[j] = fmaf(tc[j], p, end);
            p *= s.e[(r0 + j) * LD + d];
        }
    }
    // pairs inside I
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float kj = s.k[(r0 + j) * LD + d];
        float p = 1.f;
#pragma unroll
        for (int i = j + 1; i < 16; ++i) {
            const float before = p;
            p *= s.e[(r0 + i) * LD + d];
            const float gb = s.dB[(r0 + i) * MLD + r0 + j], qi = s.q[(r0 + i) * LD + d];
            const float pq = DELTA ? p : before;
            cq[i] = fmaf(gb * pq, kj, cq[i]);
            cc[j] = fmaf(gb * pq, qi, cc[j]);
            if (DELTA) {
                const float ga = s.dA[(r0 + i) * MLD + r0 + j] * p;
                cr[i] = fmaf(ga, kj, cr[i]);
                cc[j] = fmaf(ga, s.k[(r0 + i) * LD + d], cc[j]);
            }
        }
    }
    // The log-decay's gradient: with G_i = ell_1 + ... + ell_i, row i's
    // gradient by G_i is q cq + k cr - k cc (RWKV6's q reads at G_{i-1}), and
    // G_C's besides that Gam_C sum_v S dS' + sum_j k_j K^'s part; ell_t's is
    // the sum over the G_i, i >= t.
    float gsum = 0.f;
    float gl[16]; // suffix sums over the block
#pragma unroll
    for (int i = 15; i >= 0; --i) {
        const float qi = s.q[(r0 + i) * LD + d], ki = s.k[(r0 + i) * LD + d];
        if (DELTA) {
            gsum += qi * cq[i] + ki * (cr[i] - cc[i]);
            gl[i] = gsum;
        } else {
            gsum -= ki * cc[i];
            gl[i] = gsum;
            gsum += qi * cq[i];
        }
    }
    s.part[I * DKP + d] = gsum + kh;
    float du = 0.f;
    {
        // the pairs (i, i), which no decay touches
        const float ud = !DELTA && d < a.dk ? a.u[static_cast<long>(h) * a.dk + d] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float g = s.dB[(r0 + i) * MLD + r0 + i];
            const float qi = s.q[(r0 + i) * LD + d], ki = s.k[(r0 + i) * LD + d];
            const float f = DELTA ? g : g * ud;
            const float oq = fmaf(f, ki, cq[i]), ok = fmaf(f, qi, cr[i] + cc[i]);
            du = fmaf(g * qi, ki, du);
            if (r0 + i < ch.rows && d < a.dk) {
                const long at = ((static_cast<long>(ch.t0) + r0 + i) * a.H + h) * a.dk + d;
                static_cast<TIn *>(a.d_q)[at] = static_cast<TIn>(oq);
                static_cast<TIn *>(a.d_k)[at] = static_cast<TIn>(ok);
            }
        }
    }
    __syncthreads();
    {
        // behind block I: the sums of the later blocks, every block's share
        // of K^ (those up to I count at G_C), and Gam_C
        float tail = 0.f, all = 1.f;
        for (int J = I + 1; J < 4; ++J)
            tail += s.part[J * DKP + d];
        for (int i = 0; i < C; ++i)
            all *= s.e[i * LD + d];
        __syncthreads();
        s.part[I * DKP + d] = kh;
        __syncthreads();
        for (int J = 0; J <= I; ++J)
            tail += s.part[J * DKP + d];
        tail = fmaf(all, s.gam[d], tail);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            gl[i] += tail;
    }
    if constexpr (OP != GDN) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (r0 + i < ch.rows && d < a.dk) {
                const long at = ((static_cast<long>(ch.t0) + r0 + i) * a.H + h) * a.dk + d;
                a.d_ld[at] = a.ld[at] < kMinLogDecay ? 0.f : gl[i]; // below it the decay is held
            }
    } else {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s.e[(r0 + i) * LD + d] = d < a.dk ? gl[i] : 0.f;
        __syncthreads();
        for (int i = w; i < ch.rows; i += NW) {
            float x = 0.f;
            for (int c = lane; c < DKP; c += 64)
                x += s.e[i * LD + c];
            x = wave_sum_from<1>(x);
            const long at = (static_cast<long>(ch.t0) + i) * a.H + h;
            if (lane == 0)
                a.d_ld[at] = a.ld[at] < kMinLogDecay ? 0.f : x;
        }
    }
    if constexpr (!DELTA) {
        __syncthreads();
        s.part[I * DKP + d] = du;
        __syncthreads();
        if (tid < a.dk)
            a.w_du[slot_head * a.dk + tid] =
                s.part[tid] + s.part[DKP + tid] + s.part[2 * DKP + tid] + s.part[3 * DKP + tid];
    }
    if (DELTA && tid < ch.rows) {
        const int tiles = a.dv / 16;
        float x = 0.f;
        for (int t = 0; t < tiles; ++t)
            x += a.w_db[(slot_head * tiles + t) * C + tid];
        a.d_beta[(static_cast<long>(ch.t0) + tid) * a.H + h] = x;
    }
}

// du: the sum over all chunks, in their order.
__global__ inline __launch_bounds__(256) void scan_du_kernel(ScanArgs a)
{
    const int i = blockIdx.x * 256 + threadIdx.x, n = a.H * a.dk;
    if (i >= n)
        return;
    float x = 0.f;
    for (int s = 0; s < a.slots; ++s)
        x += a.w_du[static_cast<long>(s) * n + i];
    a.d_u[i] = x;
}

// ---------------------------------------------------------------- launchers --

template <typename K> hipError_t set_lds(K *kernel, int bytes)
{
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                               bytes);
}

template <int OP, typename TIn, int DKP> hipError_t scan_forward_t(const ScanArgs &a, hipStream_t st)
{
    constexpr bool DELTA = OP != RWKV6;
    if (a.slots > 0 && a.T > 0) {
        auto *prep = scan_prep_kernel<OP, TIn, DKP, false>;
        if (hipError_t e = set_lds(prep, sizeof(PrepLds<DKP>)); e != hipSuccess)
            return e;
        hipLaunchKernelGGL(prep, dim3(a.slots * a.H), dim3(256), sizeof(PrepLds<DKP>), st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    const dim3 grid(a.N * a.H * (a.dv / 16));
    if (a.save_s)
        hipLaunchKernelGGL((scan_carry_kernel<TIn, DKP, DELTA, true>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((scan_carry_kernel<TIn, DKP, DELTA, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int OP, typename TIn, int DKP> hipError_t scan_backward_t(const ScanArgs &a, hipStream_t st)
{
    constexpr bool DELTA = OP != RWKV6;
    if (a.T > 0) {
        auto *prep = scan_prep_kernel<OP, TIn, DKP, true>;
        if (hipError_t e = set_lds(prep, sizeof(PrepLds<DKP>)); e != hipSuccess)
            return e;
        hipLaunchKernelGGL(prep, dim3(a.slots * a.H), dim3(256), sizeof(PrepLds<DKP>), st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL((scan_carry_bwd_kernel<TIn, DKP, DELTA>), dim3(a.N * a.H * (a.dv / 16)), dim3(256), 0, st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    auto *grads = scan_grads_kernel<OP, TIn, DKP>;
    if (hipError_t e = set_lds(grads, sizeof(GradLds<DKP>)); e != hipSuccess)
        return e;
    hipLaunchKernelGGL(grads, dim3(a.slots * a.H), dim3(DKP * 4), sizeof(GradLds<DKP>), st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (!DELTA) {
        hipLaunchKernelGGL(scan_du_kernel, dim3((a.H * a.dk + 255) / 256), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    return hipSuccess;
}

template <int OP> hipError_t scan_launch(int dtype, bool backward, const ScanArgs &a, hipStream_t st)
{
#define DL_SCAN_CASE(TIN, DKP)                                                                                        \
    return backward ? scan_backward_t<OP, TIN, DKP>(a, st) : scan_forward_t<OP, TIN, DKP>(a, st)
    const int dkp = a.dk < 32 ? 32 : a.dk;
    if (dtype == BF16) {
        if (dkp == 128)
            DL_SCAN_CASE(__bf16, 128);
        if (dkp == 64)
            DL_SCAN_CASE(__bf16, 64);
        DL_SCAN_CASE(__bf16, 32);
    }
    if (dkp == 128)
        DL_SCAN_CASE(float, 128);
    if (dkp == 64)
        DL_SCAN_CASE(float, 64);
    DL_SCAN_CASE(float, 32);
#undef DL_SCAN_CASE
}

} // namespace dl
