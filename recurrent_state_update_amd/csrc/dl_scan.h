// dl_scan.h -- the sequence scan (dl_scan, dl_scan_backward) for gfx950: its
// mathematics and what its kernels share.  The kernels are in dl_scan_prep.h,
// dl_scan_carry.h and dl_scan_grads.h, instantiated once per operator in
// dl_scan_gdn.hip, dl_scan_kda.hip and dl_scan_rwkv6.hip (dl_scan_launch.h).
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
//   db = B^T dO + K^ dS',  z = N^T (beta db),
//   dbeta = (db - A^T z) . E,  dv = z  (RWKV6: dv = db)
//   dS = Gam_C (.) dS' + Q~^T dO - K~^T z
//   dQ~ = dO S^T, dK~ = -z S^T, dK^ = b dS'^T, dB = dO b^T, dA = -z b^T,
// from which dq, dk and the log-decay's gradient follow within the chunk.
//
// Every decay is a product of factors e_m in [0, 1] (prep divides one by its
// block's, where that is far from underflow) and never the exponential of a
// difference of two cumulative sums: full forgetting (e = 0) and strong decays
// neither overflow nor lose what they multiply.
//
// Kernels: prep (per chunk and head: the scaled operands, B and N, in the matrix
// instruction's own register order); the forward carry and the backward carry
// (per sequence, head and 16 or 32 value columns: the columns of S are
// independent; long sequences with few heads in segments, which a small kernel
// joins); grads (per chunk and head).
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
using f32x8 = float __attribute__((ext_vector_type(8)));
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

// A sum of products of factors in planes.  The pairs of planes i + j < 3 count:
// what is left out is below 2^-24 of the largest product.  One accumulator per
// order: their chains overlap, and small sums stay apart from large ones until
// the end.
constexpr int ORDER = 3;
struct Acc {
    f32x4 c[ORDER];
    __device__ __forceinline__ explicit Acc(f32x4 x = f32x4{0, 0, 0, 0})
    {
        c[0] = x;
#pragma unroll
        for (int s = 1; s < ORDER; ++s)
            c[s] = f32x4{0, 0, 0, 0};
    }
    template <int NA, int NB> __device__ __forceinline__ void add(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB])
    {
#pragma unroll
        for (int i = 0; i < ORDER; ++i) // in turn over the accumulators
#pragma unroll
            for (int s = ORDER - 1; s >= i; --s)
                if (i < NA && s - i < NB)
                    c[s] = mfma16(a[i], b[s - i], c[s]);
    }
    __device__ __forceinline__ f32x4 sum() const
    {
        f32x4 x = c[ORDER - 1];
#pragma unroll
        for (int s = ORDER - 2; s >= 0; --s)
            x += c[s];
        return x;
    }
};
// The same with one accumulator, where registers are short and the products
// of several sums overlap anyway.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c)
{
#pragma unroll
    for (int s = ORDER - 1; s >= 0; --s)
#pragma unroll
        for (int i = s; i >= 0; --i)
            if (i < NA && s - i < NB)
                c = mfma16(a[i], b[s - i], c);
    return c;
}
// x as a sum of N bf16 values, each the rounding of what is left: the planes of
// an fp32 factor (three hold its 24 bits).  In pairs: one conversion packs
// two values, whose fp32 forms are its halves.
template <int N, typename V, typename F> __device__ __forceinline__ void split(F x, V (&p)[N])
{
    using f32x2 = float __attribute__((ext_vector_type(2)));
    using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
    constexpr int E = sizeof(F) / 4;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float u = x[e], v = x[e + 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bf16x2 b = __builtin_convertvector((f32x2{u, v}), bf16x2);
            p[i][e] = b[0];
            p[i][e + 1] = b[1];
            if (i + 1 < N) {
                const unsigned raw = __builtin_bit_cast(unsigned, b);
                u -= __uint_as_float(raw << 16);
                v -= __uint_as_float(raw & 0xffff0000u);
            }
        }
    }
}
// Keeps the loads before it ahead of those behind it.  The counter that a wait
// for a load compares counts in order, and where the loads ahead of a loop come
// in another order than at its end, every wait in it is for the worse of both.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// How an operator with inputs of a type runs.
template <int OP, typename TIn> struct Plan {
    static constexpr bool DELTA = OP != RWKV6;
    static constexpr bool BF = sizeof(TIn) == 2;
    // one decay per row: kept out of the keys' operands and applied to the
    // rows of the products
    static constexpr bool ROWS = OP == GDN;
    static constexpr int NPX = scan_planes(OP, BF ? BF16 : F32); // planes of the keys' operands
    static constexpr int NPI = BF ? 1 : 3; // planes of an input
    static constexpr int NPB = DELTA ? 3 : NPI; // planes of b
};

template <typename TIn> __device__ __forceinline__ float from_in(TIn x);
template <> __device__ __forceinline__ float from_in<float>(float x) { return x; }
template <> __device__ __forceinline__ float from_in<__bf16>(__bf16 x) { return static_cast<float>(x); }

// ---------------------------------------------------------------- sequences --
//
// Chunks are numbered by slots: sequence n owns the slots from
// base(n) = start(n) / C + n on, which leaves every sequence enough of them
// (floor(a / C) + ceil((b - a) / C) <= floor(b / C) + 1) without a prefix sum
// over the lengths.  The rows behind the last sequence, T / C + N + 1 slots in
// all, count as sequence N here: no carry has it, and prep zeroes the outputs'
// rows (those ahead of the first sequence too, C of them at slot 0 and so on).
// Offsets read from cu are clamped to [0, T], so a bad array cannot lead
// an access out of range.
struct Seq {
    int start, len, base;
};
__device__ __forceinline__ int seq_start(const ScanArgs &a, int n)
{
    if (!a.cu)
        return n >= a.N ? a.T : static_cast<int>(static_cast<long>(a.T) * n / a.N);
    const int s = n > a.N ? a.T : a.cu[n];
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
// The chunk of a slot: its first token, its number of tokens (<= 0: none), and
// whether it lies behind the last sequence.
struct Chunk {
    int t0, rows;
    bool behind;
};
__device__ __forceinline__ Chunk chunk_of(const ScanArgs &a, int slot)
{
    int lo = 0, hi = a.N; // the last n with base(n) <= slot
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
    r.behind = lo == a.N;
    return r;
}

// -------------------------------------------------------- operands in memory --
//
// Per slot and head: three operands of C x DKP elements, two of C x C, A and B
// in blocks (backward), Gam_C, and per row i Gam_i, P_Ci (used where
// Plan::ROWS) and beta_i (zero behind the end).  An operand [rows][k] is stored
// as the fragments that the matrix instruction reads: of 16 rows x 32 k lane l
// holds row l % 16, k from 8 (l / 16).  One or two planes are stored as such
// (64 lanes x 8 bf16 each: one coalesced 1 KiB load); three are stored as the
// fp32 values (four bytes, not six), 64 lanes x 4 twice, and split when read.
//   forward : op 0 K~ [C][DKP], 1 Q~ [C][DKP], 2 K^T^ [DKP][C]; mat 0 N, 1 B
//   backward: op 0 K^ [C][DKP], 1 Q~^T [DKP][C], 2 K~^T [DKP][C]; mat 0 N^T,
//             1 B^T; pairs: A and (GDN) B, fp32 (store_pair)
// (ROWS: K and Q without their decays.)  Of the triangular C x C operands the
// fragments of zeros are neither written nor read.
template <int NP, int DKP> struct Ops {
    static constexpr size_t kOp = size_t(C) * DKP * (NP == 1 ? 2 : 4), kMat = size_t(C) * C * 4; // bytes
    static constexpr size_t kBytes = scan_op_bytes(NP, DKP);
    char *p;
    __device__ __forceinline__ Ops(const ScanArgs &a, long slot_head) : p(a.ops + slot_head * kBytes) {}
    __device__ __forceinline__ char *op(int i) const { return p + i * kOp; }
    __device__ __forceinline__ char *mat(int i) const { return p + 3 * kOp + i * kMat; }
    __device__ __forceinline__ f32x4 *pairs() const { return reinterpret_cast<f32x4 *>(p + 3 * kOp + 2 * kMat); }
    __device__ __forceinline__ float *gam() const { return reinterpret_cast<float *>(p + 3 * kOp + 2 * kMat + 20 * 1024); }
    __device__ __forceinline__ float *row(int i) const { return gam() + DKP + i * C; } // 0 Gam_i, 1 P_Ci, 2 beta
};

// A fragment in memory: its size, and a lane's loads and stores.
template <int N> constexpr int frag_bytes() { return N == 3 ? 2048 : N * 1024; }
// (uniform base + 32-bit lane offset: the load's scalar-address form)
template <int N>
__device__ __forceinline__ void load_frag(bf16x8 (&f)[N], const char *op, int ksteps, int rb, int ks, int lane)
{
    static_assert(N < 3, "three planes are read as fp32");
    const char *base = op + (rb * ksteps + ks) * frag_bytes<N>();
    const unsigned off = lane * 16;
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = *reinterpret_cast<const bf16x8 *>(base + (off + i * 1024));
}
__device__ __forceinline__ f32x8 load_frag32(const char *op, int ksteps, int rb, int ks, int lane)
{
    const char *base = op + (rb * ksteps + ks) * frag_bytes<3>();
    const unsigned off = lane * 16;
    const f32x4 x = *reinterpret_cast<const f32x4 *>(base + off), y = *reinterpret_cast<const f32x4 *>(base + (off + 1024));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Store x in N planes (three: as it is).
template <int N> __device__ __forceinline__ void store_frag(char *op, int ksteps, int rb, int ks, int lane, f32x8 x)
{
    char *p = op + (rb * ksteps + ks) * frag_bytes<N>() + lane * 16;
    if constexpr (N == 3) {
        *reinterpret_cast<f32x4 *>(p) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
        *reinterpret_cast<f32x4 *>(p + 1024) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
    } else {
        bf16x8 f[N];
        split(x, f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x8 *>(p + i * 1024) = f[i];
    }
}
// The same of planes in registers.
template <int N, int M>
__device__ __forceinline__ void store_frag(char *op, int ksteps, int rb, int ks, int lane, const bf16x8 (&f)[M])
{
    if constexpr (N == 3) {
        store_frag<3>(op, ksteps, rb, ks, lane,
                      __builtin_convertvector(f[0], f32x8) + __builtin_convertvector(f[1], f32x8) +
                          __builtin_convertvector(f[2], f32x8));
    } else {
        char *p = op + (rb * ksteps + ks) * frag_bytes<N>() + lane * 16;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x8 *>(p + i * 1024) = f[i];
    }
}
// Whether fragment (rb, ks) of a triangular C x C operand holds anything.
enum Part { ALL, LOWER, UPPER };
__device__ __forceinline__ bool frag_used(Part part, int rb, int ks)
{
    return part == ALL || (part == LOWER ? ks == 0 || rb >= 2 : ks == 1 || rb < 2);
}
// Write the fragments of [ROWS][K] in N planes, element (r, k) given by f.
template <int N, int ROWS, int K, Part PART = ALL, typename F> __device__ __forceinline__ void store_op(char *op, F f)
{
    for (int it = threadIdx.x; it < ROWS / 16 * (K / 32) * 64; it += blockDim.x) {
        const int lane = it & 63, rb = (it >> 6) / (K / 32), ks = (it >> 6) % (K / 32);
        if (!frag_used(PART, rb, ks))
            continue;
        f32x8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = f(rb * 16 + (lane & 15), ks * 32 + (lane >> 4) * 8 + e);
        store_frag<N>(op, K / 32, rb, ks, lane, x);
    }
}

// N = (I + L)^-1 for a unit lower triangular I + L of C x C fp32 in LDS (row
// stride MLD; of L only what is below the diagonal is read, and of N the
// blocks above it are zero beforehand): the four diagonal blocks by
// forward substitution, wave w taking block w, one column per lane; then
// N_IJ = -N_II sum_{J <= K < I} L_IK N_KJ by block diagonals on the fp32
// matrix instructions.  For whole workgroups of four waves or more.
__device__ __forceinline__ void invert_unit_lower(const float *L, float *N, int w, int lane)
{
    if (w < 4 && lane < 16) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                if (j >= i)
                    continue;
                const f32x4 l = *reinterpret_cast<const f32x4 *>(&L[(w * 16 + i) * MLD + w * 16 + j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < i)
                        v = fmaf(-l[e], x[j + e], v);
            }
            x[i] = v;
            N[(w * 16 + i) * MLD + w * 16 + lane] = v;
        }
    }
    __syncthreads();
    const int r = lane & 15, k0 = (lane >> 4) * 4;
    for (int dist = 1; dist < 4; ++dist) {
        if (w + dist < 4) {
            const int J = w, I = w + dist;
            f32x4 t = {0, 0, 0, 0}, c = {0, 0, 0, 0};
            for (int K = J; K < I; ++K) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = N[(K * 16 + k0 + e) * MLD + J * 16 + r];
                t = mfma32x4(*reinterpret_cast<const f32x4 *>(&L[(I * 16 + r) * MLD + K * 16 + k0]), x, t);
            }
            // a product's result is in the second operand's order
            c = mfma32x4(*reinterpret_cast<const f32x4 *>(&N[(I * 16 + r) * MLD + I * 16 + k0]), t, c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                N[(I * 16 + k0 + e) * MLD + J * 16 + r] = -c[e];
        }
        __syncthreads();
    }
}

} // namespace dl
