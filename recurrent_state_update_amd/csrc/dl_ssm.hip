// dl_ssm.hip -- the selective state space scan forward, over sequences and for
// single tokens (the mathematics is in dl_ssm.h).
#include "dl_ssm.h"

namespace dl {

using namespace ssm;

namespace {

// ------------------------------------------------------------------- scan --

// What a pass of a piece of a sequence is for.
enum Pass {
    MAIN,     // y, from the state ahead of the piece
    AHEAD,    // the state behind it from zero, and its sum of delta
    BACKWARD, // the same of the adjoint: G ahead of it, from zero behind it
};

// Tokens per stage: a stage's operands are loaded while the one before is worked
// on, and pass through LDS once.
constexpr int stage_tokens(int S) { return S == 1 ? 64 : 32; }
constexpr int CH = kSsmTile; // channels per workgroup: four waves of four
constexpr int NT = 256;
static_assert(CH == 16, "four waves of four rows");

template <int S> struct Stage {
    static constexpr int TT = stage_tokens(S), XLD = TT + 2, BLD = TT + 4;
    float x[CH][XLD], dt[CH][XLD], z[CH][XLD];
    alignas(16) float b[16 * S][BLD], c[16 * S][BLD];
};
template <int S> struct Shared {
    Stage<S> in[2];
    float y[2][CH][Stage<S>::XLD];
};

// One workgroup per channel tile and piece.  A wave's row of lanes is a channel,
// with S states per lane.
template <typename T, int S, Pass PASS, bool VEC, bool SAVE> __global__ __launch_bounds__(NT) void ssm_kernel(SsmArgs a)
{
    constexpr int TT = Stage<S>::TT, XV = CH * TT / NT, XPR = CH / XV; // a thread's channels, threads per token
    constexpr int BV = 4, BPR = 16 * S / BV, BTOK = NT / BPR, BK = TT / BTOK; // its states, threads per token, turns
    static_assert(XPR * TT == NT && BK * BTOK == TT, "every thread loads as much");
    __shared__ Shared<S> sh;

    const long work = xcd_order(blockIdx.x, gridDim.x);
    const int slot = work / a.tiles, tile = work % a.tiles;
    const int per = (a.CG + CH - 1) / CH, g = tile / per, c0 = g * a.CG + tile % per * CH;
    const int nc = min(CH, (g + 1) * a.CG - c0); // channels there are
    const Sequences seqs{a.cu, a.T, a.N};
    const int tid = threadIdx.x, lane = tid % 64, j = lane % 16, row = tid / 16;
    const int xt = tid / XPR, xc = tid % XPR * XV, bt = tid / BPR, bn = tid % BPR * BV;

    if constexpr (PASS == MAIN) {
        // rows of no sequence, a share for every piece
        const int first = seqs.at(0), behind = seqs.at(a.N), zeros = first + a.T - behind;
        Cells<XV, T, VEC> zero;
        zero.zero();
        for (int i = slot * TT + xt; i < zeros; i += a.slots * TT) {
            const long t = i < first ? i : behind + i - first;
            zero.store(static_cast<T *>(a.y) + t * a.C + c0 + xc, nc - xc);
        }
    }
    const Piece p(seqs, slot, a.seg);
    if (p.none())
        return;
    if (PASS == AHEAD && p.last)
        return;
    if (PASS == BACKWARD && p.index == 0)
        return;

    const int c = c0 + min(row, nc - 1); // this row's channel
    const bool there = row < nc;
    float rate[S], h[S];
    bool has[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        has[s] = there && j + 16 * s < a.S;
        rate[s] = has[s] ? finite_rate(a.A[static_cast<long>(c) * a.S + j + 16 * s] * kLog2e) : 0.f;
        h[s] = 0.f;
    }
    const long of_c = static_cast<long>(c) * a.S + j, states = static_cast<long>(a.C) * a.S;
    if constexpr (PASS == MAIN) {
        if (a.init)
#pragma unroll
            for (int s = 0; s < S; ++s)
                h[s] = has[s] ? a.init[p.n * states + of_c + 16 * s] : 0.f;
        for (int i = 0; i < p.index; ++i) { // the segments ahead
            const float sum = a.seg_d[static_cast<long>(p.base + i) * a.C + c];
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (has[s])
                    h[s] = fmaf(__builtin_amdgcn_exp2f(sum * rate[s]), h[s], a.seg_h[(p.base + i) * states + of_c + 16 * s]);
        }
    }
    float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = PASS == MAIN && a.D ? a.D[c] : 0.f;
    // what a stage is made of: x and B, or for the adjoint dy and C.  (Loads beyond the
    // channels, states or tokens there are go to the first or last that is, and are dropped.)
    const int col = c0 + (xc < nc ? xc : 0), bcol = bn < a.S ? bn : 0;
    const T *const px = static_cast<const T *>(PASS == BACKWARD ? a.dy : a.x) + col,
            *const pd = static_cast<const T *>(a.dt) + col;
    const T *const pb = static_cast<const T *>(PASS == BACKWARD ? a.c : a.b) + static_cast<long>(g) * a.S + bcol,
            *const pc = static_cast<const T *>(a.c) + static_cast<long>(g) * a.S + bcol;
    const long xs = PASS == BACKWARD ? a.C : a.xs, bs = PASS == BACKWARD ? a.cs : a.bs;
    const bool gate = PASS != AHEAD && a.z;
    const float no_gate = gate ? 0.f : 1.f;
    const T *const pz = gate ? static_cast<const T *>(a.z) + col : px;
    const long zs = gate ? a.zs : xs;

    Cells<XV, T, VEC> rx, rd, rz;
    Cells<BV, T, VEC> rb[BK], rc[BK];
    const auto read = [&](int t0) { // the stage from token t0 of the piece on
        const long t = p.t0 + min(t0 + xt, p.len - 1);
        rx.load(px + t * xs, nc - xc);
        rd.load(pd + t * a.dts, nc - xc);
        if constexpr (PASS != AHEAD)
            rz.load(pz + t * zs, nc - xc);
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const long u = p.t0 + min(t0 + bt + k * BTOK, p.len - 1);
            rb[k].load(pb + u * bs, a.S - bn);
            if constexpr (PASS == MAIN)
                rc[k].load(pc + u * a.cs, a.S - bn);
        }
    };
    const auto put = [&](Stage<S> &st, int t0) {
        const int n = t0 + xt < p.len ? nc - xc : 0;
        rx.keep(n);
        rd.keep(n);
        if constexpr (PASS != AHEAD)
            rz.keep(gate ? n : 0);
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            st.x[xc + i][xt] = to_f(rx.v[i]);
            st.dt[xc + i][xt] = to_f(rd.v[i]);
            if constexpr (PASS != AHEAD)
                st.z[xc + i][xt] = to_f(rz.v[i]);
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const int m = t0 + bt + k * BTOK < p.len ? a.S - bn : 0;
            rb[k].keep(m);
            if constexpr (PASS == MAIN)
                rc[k].keep(m);
#pragma unroll
            for (int i = 0; i < BV; ++i) {
                st.b[bn + i][bt + k * BTOK] = to_f(rb[k].v[i]);
                if constexpr (PASS == MAIN)
                    st.c[bn + i][bt + k * BTOK] = to_f(rc[k].v[i]);
            }
        }
    };

    const int stages = (p.len + TT - 1) / TT;
    const auto from = [&](int k) { return (PASS == BACKWARD ? stages - 1 - k : k) * TT; };
    float sum = 0.f; // of delta, this lane's tokens
    // What was loaded above is here before the loop: its first use would wait for the
    // loop's own loads, too.
    asm volatile("" : "+v"(bias), "+v"(skip));
#pragma unroll
    for (int s = 0; s < S; ++s)
        asm volatile("" : "+v"(rate[s]), "+v"(h[s]));
    if (stages > 0) {
        read(from(0));
        put(sh.in[0], from(0));
    }
    __syncthreads();
    for (int k = 0; k < stages; ++k) {
        const Stage<S> &st = sh.in[k % 2];
        const int t0 = from(k);
        // (behind the last stage that one again: a condition here would have every load
        // waited for at once)
        const int next = from(min(k + 1, stages - 1));
        read(next);
        // All blocks of the stage, whatever tokens are there (the others change nothing),
        // in straight code: what belongs to a lane's own tokens first, whose chains of
        // dependent operations then overlap.
        constexpr int NB = TT / TB;
        float x[NB], delta[NB], u[NB], z[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * TB + j;
            const bool live = t0 + at < p.len;
            float e, raw = st.dt[row][at] + bias, soft = softplus(raw, e);
            asm("" : "+v"(soft)); // a selection, not a branch
            x[i] = st.x[row][at];
            delta[i] = live ? a.softplus ? soft : raw : 0.f;
            z[i] = 1.f;
            if constexpr (PASS != AHEAD) {
                const float v = st.z[row][at]; // 0 without a gate
                z[i] = fmaf(v, sigmoid(v), no_gate);
            }
            // what the state takes of B (or C)
            u[i] = PASS == BACKWARD ? x[i] * z[i] : delta[i] * x[i];
        }
        // B and C are read from LDS a block ahead
        f32x4 Bn[S][TB / 4], Cn[S][TB / 4];
        const auto fetch = [&](int at) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int q = 0; q < TB / 4; ++q) {
                    Bn[s][q] = *reinterpret_cast<const f32x4 *>(&st.b[j + 16 * s][at + 4 * q]);
                    if constexpr (PASS == MAIN)
                        Cn[s][q] = *reinterpret_cast<const f32x4 *>(&st.c[j + 16 * s][at + 4 * q]);
                }
        };
        fetch(PASS == BACKWARD ? (NB - 1) * TB : 0);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int i = PASS == BACKWARD ? NB - 1 - n : n, at = i * TB;
            f32x4 B[S][TB / 4], C[S][TB / 4];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int q = 0; q < TB / 4; ++q) {
                    B[s][q] = Bn[s][q];
                    if constexpr (PASS == MAIN)
                        C[s][q] = Cn[s][q];
                }
            if (n + 1 < NB)
                fetch(PASS == BACKWARD ? at - TB : at + TB);
            __builtin_amdgcn_sched_barrier(0x1F); // (LDS reads stay above it)
            if constexpr (SAVE)
                if (t0 + at < p.len) {
                    float *const to = a.saved + (p.start / TB + p.n + (p.t0 - p.start + t0 + at) / TB) * states + of_c;
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        if (has[s])
                            to[16 * s] = h[s];
                }
            float y[TB], d[S][TB], v[S][TB];
            for_tokens([&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    d[s][t] = __builtin_amdgcn_exp2f(row_bcast<t>(delta[i]) * rate[s]);
                    v[s][t] = row_bcast<t>(u[i]) * B[s][t / 4][t % 4];
                }
            });
            const auto token = [&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    h[s] = PASS == BACKWARD ? d[s][t] * (h[s] + v[s][t]) : fmaf(d[s][t], h[s], v[s][t]);
                    if constexpr (PASS == MAIN)
                        y[t] = s ? fmaf(C[s][t / 4][t % 4], h[s], y[t]) : C[s][t / 4][t % 4] * h[s];
                }
            };
            if constexpr (PASS == BACKWARD)
                for_tokens_down(token);
            else
                for_tokens(token);
            if constexpr (PASS == MAIN)
                sh.y[k % 2][row][at + j] = fmaf(skip, x[i], row_sums(y, j)) * z[i];
            else
                sum += delta[i];
        }
        put(sh.in[(k + 1) % 2], next);
        __syncthreads();
        if constexpr (PASS == MAIN)
            if (t0 + xt < p.len) {
                Cells<XV, T, VEC> ry;
#pragma unroll
                for (int i = 0; i < XV; ++i)
                    ry.v[i] = static_cast<T>(sh.y[k % 2][xc + i][xt]);
                ry.store(static_cast<T *>(a.y) + static_cast<long>(p.t0 + t0 + xt) * a.C + c0 + xc, nc - xc);
            }
    }
    if constexpr (PASS == MAIN) {
        if (a.fin && p.last)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (has[s])
                    a.fin[p.n * states + of_c + 16 * s] = h[s];
    } else {
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (has[s])
                a.seg_h[slot * states + of_c + 16 * s] = h[s];
        sum = row_sum(sum);
        if (there && j == 0)
            a.seg_d[static_cast<long>(slot) * a.C + c] = sum;
    }
}

template <typename T, int S, bool VEC> hipError_t scan_v(const SsmArgs &a, Pass pass, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(static_cast<long>(a.slots) * a.tiles));
    if (pass == AHEAD)
        hipLaunchKernelGGL((ssm_kernel<T, S, AHEAD, VEC, false>), grid, dim3(NT), 0, st, a);
    else if (pass == BACKWARD)
        hipLaunchKernelGGL((ssm_kernel<T, S, BACKWARD, VEC, false>), grid, dim3(NT), 0, st, a);
    else if (a.saved)
        hipLaunchKernelGGL((ssm_kernel<T, S, MAIN, VEC, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((ssm_kernel<T, S, MAIN, VEC, false>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T, int S> hipError_t scan_s(const SsmArgs &a, Pass pass, hipStream_t st)
{
    return a.vec_x && a.vec_b ? scan_v<T, S, true>(a, pass, st) : scan_v<T, S, false>(a, pass, st);
}
template <typename T> hipError_t scan_t(const SsmArgs &a, Pass pass, hipStream_t st)
{
    return a.S <= 16 ? scan_s<T, 1>(a, pass, st) : a.S <= 32 ? scan_s<T, 2>(a, pass, st) : scan_s<T, 4>(a, pass, st);
}
hipError_t scan_pass(int dtype, const SsmArgs &a, Pass pass, hipStream_t st)
{
    return dtype == F32 ? scan_t<float>(a, pass, st) : scan_t<__bf16>(a, pass, st);
}

// ---------------------------------------------------------- single tokens --

// Four states per lane, L = 1 ... 16 lanes (a power of two) per channel; the
// state's 8 bytes per element are all of the traffic that counts.  VEC: its rows
// are whole vectors.
template <typename T, int L, bool VEC> __global__ __launch_bounds__(NT) void ssm_step_kernel(SsmArgs a)
{
    const long unit = (static_cast<long>(blockIdx.x) * NT + threadIdx.x) / L; // row and channel
    const int n0 = threadIdx.x % L * 4;
    if (unit >= static_cast<long>(a.T) * a.C) // whole groups of lanes
        return;
    const int t = unit / a.C, c = unit % a.C, g = c / a.CG, m = a.S - n0; // states of this lane, if positive
    const int r = a.rows ? a.rows[t] : t;
    float *const state = a.state + (static_cast<long>(r) * a.C + c) * a.S + n0;
    const bool known = r >= 0 && r < a.n_rows;
    Cells<4, float, VEC> h, rate;
    Cells<4, T, VEC> b, k;
    // (lanes beyond the states there are read the first ones, and drop them)
    const int at = m > 0 ? n0 : 0;
    h.load(a.state + (static_cast<long>(known ? r : 0) * a.C + c) * a.S + at, m);
    rate.load(a.A + static_cast<long>(c) * a.S + at, m);
    b.load(static_cast<const T *>(a.b) + t * a.bs + static_cast<long>(g) * a.S + at, m);
    k.load(static_cast<const T *>(a.c) + t * a.cs + static_cast<long>(g) * a.S + at, m);
    h.keep(known ? m : 0);
    rate.keep(m);
    b.keep(m);
    k.keep(m);
    const float x = to_f(static_cast<const T *>(a.x)[t * a.xs + c]);
    float delta = to_f(static_cast<const T *>(a.dt)[t * a.dts + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f), e;
    delta = a.softplus ? softplus(delta, e) : delta;
    const float u = delta * x;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h.v[i] = fmaf(__builtin_amdgcn_exp2f(delta * finite_rate(rate.v[i] * kLog2e)), h.v[i], u * to_f(b.v[i]));
        y = fmaf(to_f(k.v[i]), h.v[i], y);
    }
    if (known)
        h.store(state, m);
    if constexpr (L > 1)
        y = group_sum<L>(y);
    if (n0 == 0) {
        y = a.D ? fmaf(a.D[c], x, y) : y;
        if (a.z) {
            const float z = to_f(static_cast<const T *>(a.z)[t * a.zs + c]);
            y *= z * sigmoid(z);
        }
        static_cast<T *>(a.y)[static_cast<long>(t) * a.C + c] = static_cast<T>(y);
    }
}

template <typename T, int L> hipError_t step_l(const SsmArgs &a, hipStream_t st)
{
    const long lanes = static_cast<long>(a.T) * a.C * L;
    const dim3 grid(static_cast<unsigned>((lanes + NT - 1) / NT));
    if (a.vec_s && a.vec_b)
        hipLaunchKernelGGL((ssm_step_kernel<T, L, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((ssm_step_kernel<T, L, false>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T> hipError_t step_t(const SsmArgs &a, hipStream_t st)
{
    return a.S <= 4    ? step_l<T, 1>(a, st)
           : a.S <= 8  ? step_l<T, 2>(a, st)
           : a.S <= 16 ? step_l<T, 4>(a, st)
           : a.S <= 32 ? step_l<T, 8>(a, st)
                       : step_l<T, 16>(a, st);
}

} // namespace

hipError_t launch_ssm_scan(int dtype, const SsmArgs &a, hipStream_t st)
{
    if (a.seg)
        if (hipError_t e = scan_pass(dtype, a, AHEAD, st); e != hipSuccess)
            return e;
    return scan_pass(dtype, a, MAIN, st);
}

hipError_t launch_ssm_ahead_of_adjoint(int dtype, const SsmArgs &a, hipStream_t st)
{
    return scan_pass(dtype, a, BACKWARD, st);
}

hipError_t launch_ssm_step(int dtype, const SsmArgs &a, hipStream_t st)
{
    return dtype == F32 ? step_t<float>(a, st) : step_t<__bf16>(a, st);
}

} // namespace dl
