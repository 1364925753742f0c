// dl_ssm.hip -- the selective state space scan forward, over sequences and for
// single tokens (the mathematics is in dl_ssm.h).
#include "dl_ssm.h"

namespace dl {

using namespace ssm;

namespace {

// ------------------------------------------------------------------- scan --

constexpr int NT = 2 * LOADERS;

// Tokens per stage (TT, times S): the decays and inputs of 64 are 64 registers each, of
// which a SIMD holds the waves of one workgroup; of 32 those of two.  Where there is a
// workgroup per CU at the most, the fewest barriers; where there are more, two at a time,
// which hide each other's; and 16 for short sequences, whose stages are not full.  us,
// bf16, 16 states, sequences x tokens x channels (4096 and 2 x 2048 x 2048: 256
// workgroups, one per CU):
//                          16     32     64
//   1024 x 8 x 512         161           576
//   256 x 32 x 512        52.7           149
//   16 x 128 x 2048       33.2   35.1   53.7
//   8 x 256 x 2048        31.4   30.5   40.0
//   8 x 1024 x 2048        111   99.9    110
//   4 x 2048 x 4096        198    177    189
//   2 x 2048 x 2048       73.9   62.9   51.8
//   4096 x 4096            143    119   95.8
constexpr int CUS = 256, SHORT = 128;

template <int S, int TT> struct Shared {
    using In = Stage<S, TT>;
    In in[3];
    float y[2][CH][In::XLD];
    float h[S][LOADERS];
};

// One workgroup per channel tile and piece.  A wave's row of lanes is a channel, with S
// states per lane.  Two sets of four waves share the channels and take turns, a stage
// each: while one takes the states through its stage (a chain of dependent operations,
// whose latency is twice its issue), forms y and loads, the other forms the decays and
// inputs of the next, which need no state.  So a sequence of a few thousand channels,
// one wave of states per SIMD, has two to issue from.
//
// Bound by the vector units: 4096 tokens x 4096 channels, 16 states, bf16: 102 us, of
// which they are busy 85%.  Of a stage's 714 issue slots per wave 516 are an exponential
// (two), the products for its exponent, the input and C, the recurrence and a sixteenth
// of the sums over states for each state and token; the others load, convert and store,
// and form softplus and gate.  A copy of its 134 MB takes 26.  With the states of every
// block saved, 2 x 2048 x 2048: 63 us.
template <typename T, int S, int TT, bool VEC, bool SAVE> __global__ __launch_bounds__(NT, 2) void ssm_kernel(SsmArgs a)
{
    constexpr int NB = TT / TB;
    using Load = Loader<T, S, TT, VEC>;
    __shared__ Shared<S, TT> sh;

    const Work work(blockIdx.x, a.tiles);
    if (work.tile < 0)
        return;
    const int slot = work.slot;
    const Tile tile(a, work.tile, CH);
    const Sequences seqs{a.cu, a.T, a.N};
    const int tid = threadIdx.x % LOADERS, set = __builtin_amdgcn_readfirstlane(threadIdx.x / LOADERS);
    const int j = tid % 16, row = tid / 16;
    Load load(Sources{a.x, a.dt, a.z, a.b, a.c, a.xs, a.dts, a.zs, a.bs, a.cs}, tid, tile.c0, tile.nc,
              tile.g * a.S, a.S);

    {   // rows of no sequence, a share for every piece
        const int first = seqs.at(0), behind = seqs.at(a.N), zeros = first + a.T - behind;
        Cells<Load::XV, T, VEC> zero;
        zero.zero();
        for (int i = (slot * 2 + set) * TT + load.xt; i < zeros; i += a.slots * 2 * TT) {
            const long t = i < first ? i : behind + i - first;
            zero.store(static_cast<T *>(a.y) + t * a.C + tile.c0 + load.xc, load.nx);
        }
    }
    const Piece p(seqs, slot, a.seg);
    if (p.none())
        return;
    load.piece(p.t0, p.len);

    const int c = tile.c0 + min(row, tile.nc - 1); // this row's channel
    const long of_c = static_cast<long>(c) * a.S + j, states = static_cast<long>(a.C) * a.S;
    float rate[S], h[S], bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    bool has[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        has[s] = row < tile.nc && j + 16 * s < a.S;
        rate[s] = has[s] ? finite_rate(a.A[of_c + 16 * s] * kLog2e) : 0.f;
        h[s] = a.init && has[s] ? a.init[p.n * states + of_c + 16 * s] : 0.f;
    }
    // The segments ahead, a few of them loaded at a time.
    constexpr int JOIN = 8;
    for (int i0 = 0; i0 < p.index; i0 += JOIN) {
        float sum[JOIN], add[JOIN][S];
#pragma unroll
        for (int i = 0; i < JOIN; ++i) {
            const long at = static_cast<long>(p.base + min(i0 + i, p.index - 1)) * a.C + c;
            sum[i] = a.seg_d[at];
#pragma unroll
            for (int s = 0; s < S; ++s)
                add[i][s] = a.seg_h[at * a.S + min(j + 16 * s, a.S - 1)];
        }
#pragma unroll
        for (int i = 0; i < JOIN; ++i)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (i0 + i < p.index && has[s])
                    h[s] = across(h[s], sum[i] * rate[s], add[i][s]);
    }
    if (set == 0)
#pragma unroll
        for (int s = 0; s < S; ++s)
            sh.h[s][tid] = h[s];
    float skip[Load::XV]; // D, of the channels that this thread loads and stores
#pragma unroll
    for (int i = 0; i < Load::XV; ++i)
        skip[i] = a.D && i < load.nx ? a.D[load.col + i] : 0.f;
    const float no_gate = a.z ? 0.f : 1.f;
    // What was loaded above is here before the loop: its first use would wait for the
    // loop's own loads, too.
    asm volatile("" : "+v"(bias));
#pragma unroll
    for (int s = 0; s < S; ++s)
        asm volatile("" : "+v"(rate[s]));
#pragma unroll
    for (int i = 0; i < Load::XV; ++i)
        asm volatile("" : "+v"(skip[i]));

    const int stages = (p.len + TT - 1) / TT;
    // What needs no state: of the stage's own tokens, and the decays and inputs.
    Own<NB> own;
    float d[NB][S][TB], v[NB][S][TB];
    const auto ahead = [&](int k) {
        const typename Shared<S, TT>::In &st = sh.in[k % 3];
        own.form(st, row, j, p.len - k * TT, bias, a.softplus);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const float u = own.delta[i] * own.x[i];
            __builtin_amdgcn_sched_barrier(0x1F); // (LDS reads stay below it: all at once are too many registers)
            for_tokens([&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    d[i][s][t] = __builtin_amdgcn_exp2f(row_bcast<t>(own.delta[i]) * rate[s]);
                    v[i][s][t] = row_bcast<t>(u) * st.b[j + 16 * s][i * TB + t];
                }
            });
#pragma unroll
            for (int t = 0; t < TB; ++t) // formed here, and not where they are used
#pragma unroll
                for (int s = 0; s < S; ++s)
                    asm volatile("" : "+v"(d[i][s][t]), "+v"(v[i][s][t]));
        }
    };
    // The states through the stage, and its y.
    const auto chain = [&](int k) {
        const typename Shared<S, TT>::In &st = sh.in[k % 3];
#pragma unroll
        for (int s = 0; s < S; ++s)
            h[s] = sh.h[s][tid];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if constexpr (SAVE)
                if (k * TT + i * TB < p.len) {
                    float *const to = a.saved + (p.start / TB + p.n + (p.t0 - p.start + k * TT) / TB + i) * states + of_c;
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        if (has[s])
                            to[16 * s] = h[s];
                }
            for_tokens([&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s)
                    h[s] = v[i][s][t] = fmaf(d[i][s][t], h[s], v[i][s][t]);
            });
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
            sh.h[s][tid] = h[s];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float y[TB];
            __builtin_amdgcn_sched_barrier(0x1F);
            for_tokens([&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float w = st.c[j + 16 * s][i * TB + t];
                    y[t] = s ? fmaf(w, v[i][s][t], y[t]) : w * v[i][s][t];
                }
            });
            sh.y[k % 2][row][i * TB + j] = row_sums(y, j);
        }
    };
    // y of the stage, by the threads that loaded its x and z.
    Cells<Load::XV, T, VEC> kx, kz;
    const auto store = [&](int k) {
        if (k * TT + load.xt < p.len) {
            Cells<Load::XV, T, VEC> out;
            Cells<Load::XV, float, VEC> plain;
#pragma unroll
            for (int i = 0; i < Load::XV; ++i) {
                const float z = to_f(kz.v[i]), y = fmaf(skip[i], to_f(kx.v[i]), sh.y[k % 2][load.xc + i][load.xt]);
                plain.v[i] = y;
                out.v[i] = static_cast<T>(y * fmaf(z, sigmoid(z), no_gate));
            }
            const long at = static_cast<long>(p.t0 + k * TT + load.xt) * a.C + tile.c0 + load.xc;
            out.store(static_cast<T *>(a.y) + at, load.nx);
            if (SAVE && a.z)
                plain.store(a.plain + at, load.nx);
        }
    };
    // Slot t, which ends at a barrier: chain(t) by one set, ahead(t + 1) by the other.
    // (Loads behind the last stage take the last token's row again: a condition would
    // have every load waited for at once.)
    if (stages > 0) {
        load.template read<true, true>(set * TT);
        load.template put<false, true, true>(sh.in[set], set * TT);
    }
    __syncthreads();
    int slots = stages + 1; // from -1 on
    if (set == 1 && slots > 0) {
        __syncthreads();
        --slots;
    }
    for (int k = set; k < stages; k += 2) {
        ahead(k);
        __syncthreads();
        kx = load.rx;
        kz = load.rz;
        load.template read<true, true>((k + 2) * TT);
        __builtin_amdgcn_s_setprio(2); // its chain is what the other set's next waits for (4096 x 4096: 113 -> 104 us)
        chain(k);
        __builtin_amdgcn_s_setprio(0);
        load.template put<false, true, true>(sh.in[(k + 2) % 3], (k + 2) * TT);
        __syncthreads();
        slots -= 2;
        store(k);
    }
    if (slots > 0)
        __syncthreads();
    if (a.fin && p.last && set == 0)
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (has[s])
                a.fin[p.n * states + of_c + 16 * s] = sh.h[s][tid];
}

template <typename T, int S, int TT, bool VEC> hipError_t scan_v(const SsmArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(work_groups(a)));
    if (a.saved)
        hipLaunchKernelGGL((ssm_kernel<T, S, TT, VEC, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((ssm_kernel<T, S, TT, VEC, false>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T, int S, int TT> hipError_t scan_l(const SsmArgs &a, hipStream_t st)
{
    return a.vec_x && a.vec_b ? scan_v<T, S, TT, true>(a, st) : scan_v<T, S, TT, false>(a, st);
}
template <typename T, int S> hipError_t scan_s(const SsmArgs &a, hipStream_t st)
{
    if (a.T <= static_cast<long>(SHORT) * a.N)
        return scan_l<T, S, TB>(a, st);
    const long pieces = a.seg ? a.T / a.seg : a.N;
    if (pieces * a.tiles > CUS)
        return scan_l<T, S, S == 1 ? 32 : TB>(a, st);
    return scan_l<T, S, 64 / S>(a, st);
}
template <typename T> hipError_t scan_t(const SsmArgs &a, hipStream_t st)
{
    return a.S <= 16 ? scan_s<T, 1>(a, st) : a.S <= 32 ? scan_s<T, 2>(a, st) : scan_s<T, 4>(a, st);
}

// ---------------------------------------------------------- single tokens --

constexpr int STEP = 256;

// Four states per lane, L = 1 ... 16 lanes (a power of two) per channel; the
// state's 8 bytes per element are all of the traffic that counts.  VEC: its rows
// are whole vectors.  64 requests x 4096 channels x 16 states: 9.0 us for 36 MB, 4.0
// TB/s (a copy of as much takes 7.6 from memory, 4.9 from the caches).
template <typename T, int L, bool VEC> __global__ __launch_bounds__(STEP) void ssm_step_kernel(SsmArgs a)
{
    // workgroups of a row: `wide`
    const int wide = (a.C * L + STEP - 1) / STEP, t = blockIdx.x / wide, c = (blockIdx.x % wide * STEP + threadIdx.x) / L;
    const int n0 = threadIdx.x % L * 4;
    if (c >= a.C) // whole groups of lanes
        return;
    const int g = a.G == 1 ? 0 : c / a.CG, m = a.S - n0; // states of this lane, if positive
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
    const dim3 grid(static_cast<unsigned>(static_cast<long>(a.T) * ((a.C * L + STEP - 1) / STEP)));
    if (a.vec_s && a.vec_b)
        hipLaunchKernelGGL((ssm_step_kernel<T, L, true>), grid, dim3(STEP), 0, st, a);
    else
        hipLaunchKernelGGL((ssm_step_kernel<T, L, false>), grid, dim3(STEP), 0, st, a);
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
        if (hipError_t e = launch_ssm_ahead(dtype, false, a, st); e != hipSuccess)
            return e;
    return dtype == F32 ? scan_t<float>(a, st) : scan_t<__bf16>(a, st);
}

hipError_t launch_ssm_step(int dtype, const SsmArgs &a, hipStream_t st)
{
    return dtype == F32 ? step_t<float>(a, st) : step_t<__bf16>(a, st);
}

} // namespace dl
