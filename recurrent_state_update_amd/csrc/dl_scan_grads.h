// dl_scan_grads.h -- per chunk and head of a scan: the gradients of its inputs.
#pragma once

#include "dl_scan.h"

namespace dl {

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


} // namespace dl
