// dl_ssm_ahead.hip -- what a segment of a sequence that is cut adds to the state
// behind it (the adjoint: to the gradient ahead of it), for dl_ssm.hip and
// dl_ssm_bwd.hip (the mathematics is in dl_ssm.h).
#include "dl_ssm.h"

namespace dl {

using namespace ssm;

namespace {

constexpr int NT = LOADERS;
constexpr int stage_tokens(int S) { return S == 1 ? 64 : 32; }

// One workgroup per channel tile and segment.  A wave's row of lanes is a channel, with
// S states per lane.  From a state of zero: the end state and the sum of delta (which
// gives the segment's decay); ADJOINT: G ahead of the segment from zero behind it.
// Bound by the vector units, 90% busy: 2 x 2048 x 2048, 16 states, bf16, the adjoint: 36
// us.
template <typename T, int S, bool ADJOINT, bool VEC> __global__ __launch_bounds__(NT) void ssm_ahead_kernel(SsmArgs a)
{
    constexpr int TT = stage_tokens(S), NB = TT / TB;
    __shared__ Stage<S, TT> in[2];

    const Work work(blockIdx.x, a.tiles);
    if (work.tile < 0)
        return;
    const int slot = work.slot;
    const Tile tile(a, work.tile, CH);
    const Piece p(Sequences{a.cu, a.T, a.N}, slot, a.seg);
    // nothing comes behind a sequence's last segment (ahead of its first)
    if (p.none() || (ADJOINT ? p.index == 0 : p.last))
        return;
    const int tid = threadIdx.x, j = tid % 16, row = tid / 16;
    const int c = tile.c0 + min(row, tile.nc - 1); // this row's channel
    const bool there = row < tile.nc;
    float rate[S], h[S], bias = a.dt_bias ? a.dt_bias[c] : 0.f, sum = 0.f;
    bool has[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        has[s] = there && j + 16 * s < a.S;
        rate[s] = has[s] ? finite_rate(a.A[static_cast<long>(c) * a.S + j + 16 * s] * kLog2e) : 0.f;
        h[s] = 0.f;
    }
    const Sources from = ADJOINT ? Sources{a.dy, a.dt, a.z, a.c, nullptr, a.C, a.dts, a.zs, a.cs, 0}
                                 : Sources{a.x, a.dt, nullptr, a.b, nullptr, a.xs, a.dts, 0, a.bs, 0};
    Loader<T, S, TT, VEC> load(from, tid, tile.c0, tile.nc, tile.g * a.S, a.S);
    load.piece(p.t0, p.len);
    // What was loaded above is here before the loop: its first use would wait for the
    // loop's own loads, too.
    asm volatile("" : "+v"(bias));
#pragma unroll
    for (int s = 0; s < S; ++s)
        asm volatile("" : "+v"(rate[s]));

    const int stages = (p.len + TT - 1) / TT;
    const auto at_stage = [&](int k) { return (ADJOINT ? stages - 1 - k : k) * TT; };
    load.template read<ADJOINT, false>(at_stage(0));
    load.template put<ADJOINT, ADJOINT, false>(in[0], at_stage(0));
    __syncthreads();
    for (int k = 0; k < stages; ++k) {
        const Stage<S, TT> &st = in[k % 2];
        const int t0 = at_stage(k), next = at_stage(min(k + 1, stages - 1));
        load.template read<ADJOINT, false>(next);
        Own<NB> own;
        own.form(st, row, j, p.len - t0, bias, a.softplus);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int i = ADJOINT ? NB - 1 - n : n;
            const float u = ADJOINT ? own.x[i] : own.x[i] * own.delta[i];
            float d[S][TB], v[S][TB];
            for_tokens([&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    d[s][t] = __builtin_amdgcn_exp2f(row_bcast<t>(own.delta[i]) * rate[s]);
                    v[s][t] = row_bcast<t>(u) * st.b[j + 16 * s][i * TB + t];
                }
            });
            const auto token = [&](auto J) {
                constexpr int t = decltype(J)::value;
#pragma unroll
                for (int s = 0; s < S; ++s)
                    h[s] = ADJOINT ? d[s][t] * (h[s] + v[s][t]) : fmaf(d[s][t], h[s], v[s][t]);
            };
            if constexpr (ADJOINT)
                for_tokens_down(token);
            else
                for_tokens(token);
            sum += own.delta[i];
        }
        load.template put<ADJOINT, ADJOINT, false>(in[(k + 1) % 2], next);
        __syncthreads();
    }
    const long at = static_cast<long>(slot) * a.C + c;
#pragma unroll
    for (int s = 0; s < S; ++s)
        if (has[s])
            a.seg_h[at * a.S + j + 16 * s] = h[s];
    sum = row_sum(sum);
    if (there && j == 0)
        a.seg_d[at] = sum;
}

template <typename T, int S, bool ADJOINT> hipError_t ahead_s(const SsmArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(work_groups(a)));
    if (a.vec_x && a.vec_b)
        hipLaunchKernelGGL((ssm_ahead_kernel<T, S, ADJOINT, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((ssm_ahead_kernel<T, S, ADJOINT, false>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T, bool ADJOINT> hipError_t ahead_t(const SsmArgs &a, hipStream_t st)
{
    return a.S <= 16 ? ahead_s<T, 1, ADJOINT>(a, st) : a.S <= 32 ? ahead_s<T, 2, ADJOINT>(a, st) : ahead_s<T, 4, ADJOINT>(a, st);
}

} // namespace

hipError_t launch_ssm_ahead(int dtype, bool adjoint, const SsmArgs &a, hipStream_t st)
{
    if (dtype == F32)
        return adjoint ? ahead_t<float, true>(a, st) : ahead_t<float, false>(a, st);
    return adjoint ? ahead_t<__bf16, true>(a, st) : ahead_t<__bf16, false>(a, st);
}

} // namespace dl
