// dl_ssm_bwd.hip -- the selective state space scan backward (the mathematics is
// in dl_ssm.h).
#include "dl_ssm.h"

namespace dl {

using namespace ssm;

namespace {

constexpr int NT = 256, WAVES = 4;
constexpr int GC = kSsmGradTile; // channels per workgroup
constexpr int R = GC / (WAVES * 4); // channels of a row of lanes, one after the other
constexpr int LD = TB + 1, BLD = TB + 4;
static_assert(GC * TB == NT * 4, "four channels of a token per thread");

// dy: times the gate's silu; slope: delta's, by dt.
template <int S> struct GradStage {
    float x[GC][LD], delta[GC][LD], slope[GC][LD], dy[GC][LD];
    alignas(16) float b[16 * S][BLD], c[16 * S][BLD];
};
// A lane puts dx and ddt where x and slope were, which nothing else reads: three
// stages, so that one can be stored while the next but one is put in.
template <int S> struct Shared {
    GradStage<S> in[3];
    alignas(16) float db[2][WAVES][16 * S][TB], dc[2][WAVES][16 * S][TB];
};

// x[0 ... 3] of row r: the sums over the wave's four rows of x[4 r ... 4 r + 3].
__device__ __forceinline__ void rows_sum(float (&x)[TB])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[i]), __float_as_uint(x[i + 8]), false, false);
        x[i] = __uint_as_float(v[0]) + __uint_as_float(v[1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(x[i + 4]), false, false);
        x[i] = __uint_as_float(v[0]) + __uint_as_float(v[1]);
    }
}

// What is above is done before what is below: else the compiler works on all of a
// wave's channels at once, and their registers are more than there are.
template <int N> __device__ __forceinline__ void in_order(float *const (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+v"(*x[i]));
}

// acc[i] += (lane T0 + i's x) * v[i]: the broadcast as the multiplication's own
// modifier, which the compiler does not find for sums of products (it spends an
// instruction and a register on each).  Two wait states before a row broadcast
// reads what the instruction ahead may have written, and after the last for one
// that the compiler may place behind.
template <int T0> __device__ __forceinline__ void fma_bcast(float *acc, float x, const float *v)
{
    asm("s_nop 1\n"
        "v_fmac_f32_dpp %0, %8, %9 row_newbcast:%c17 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %8, %10 row_newbcast:%c18 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %2, %8, %11 row_newbcast:%c19 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %3, %8, %12 row_newbcast:%c20 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %4, %8, %13 row_newbcast:%c21 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %5, %8, %14 row_newbcast:%c22 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %6, %8, %15 row_newbcast:%c23 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %7, %8, %16 row_newbcast:%c24 row_mask:0xf bank_mask:0xf\n"
        "s_nop 1"
        : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3]), "+&v"(acc[4]), "+&v"(acc[5]), "+&v"(acc[6]), "+&v"(acc[7])
        : "v"(x), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "n"(T0),
          "n"(T0 + 1), "n"(T0 + 2), "n"(T0 + 3), "n"(T0 + 4), "n"(T0 + 5), "n"(T0 + 6), "n"(T0 + 7));
}
// The same into two sums.
template <int T0> __device__ __forceinline__ void fma_bcast_sum(float &even, float &odd, float x, const float *v)
{
    asm("s_nop 1\n"
        "v_fmac_f32_dpp %0, %2, %3 row_newbcast:%c11 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %2, %4 row_newbcast:%c12 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %2, %5 row_newbcast:%c13 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %2, %6 row_newbcast:%c14 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %2, %7 row_newbcast:%c15 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %2, %8 row_newbcast:%c16 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %2, %9 row_newbcast:%c17 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %2, %10 row_newbcast:%c18 row_mask:0xf bank_mask:0xf\n"
        "s_nop 1"
        : "+&v"(even), "+&v"(odd)
        : "v"(x), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "n"(T0),
          "n"(T0 + 1), "n"(T0 + 2), "n"(T0 + 3), "n"(T0 + 4), "n"(T0 + 5), "n"(T0 + 6), "n"(T0 + 7));
}

// Where token t of state n is in a row of db or dc: its fours in another order for
// every other state, so that states in step do not meet in the same banks.
__device__ __forceinline__ int swizzle(int n, int t) { return t ^ (n / 2 % 4 * 4); }

// One workgroup per tile of 64 channels and piece of a sequence: blocks of
// sixteen tokens from its end.  Per block the states are formed anew from the
// saved one ahead of it, sixteen in registers with their decays; then the adjoint
// goes back over them.  A wave takes four channels at a time, four times: what
// it adds up of dB and dC over channels stays in registers meanwhile, B and C too.
//
// Bound by the vector units, 84% busy at two waves per SIMD: 2 x 2048 x 2048, 16 states,
// bf16: 120 us (218 MB; at the 5.1 TB/s of a copy of as much 43).  64 channels: fewer leave more sums of dB
// and dC to memory (a tile's are 256 bytes a token), more do not fill the GPU.
template <typename T, int S, bool VEC> __global__ __launch_bounds__(NT, S == 1 ? 2 : 1) void ssm_bwd_kernel(SsmArgs a)
{
    constexpr int XV = 4, XPR = GC / XV;
    constexpr int BN = 16 * S * TB / NT; // states of a token per thread
    __shared__ Shared<S> sh;

    const Work work(blockIdx.x, a.tiles);
    if (work.tile < 0)
        return;
    const int slot = work.slot, of_group = work.tile % ((a.CG + GC - 1) / GC);
    const Tile tile(a, work.tile, GC);
    const int g = tile.g, c0 = tile.c0, nc = tile.nc;
    const Sequences seqs{a.cu, a.T, a.N};
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, j = lane % 16, row = lane / 16;
    const int xt = tid / XPR, xc = tid % XPR * XV, bt = tid / 16, bn = tid % 16 * BN;
    const bool gate = a.z;
    const long states = static_cast<long>(a.C) * a.S;

    {   // rows of no sequence, a share for every piece
        const int first = seqs.at(0), behind = seqs.at(a.N), zeros = first + a.T - behind;
        Cells<XV, T, VEC> zero;
        zero.zero();
        for (int i = slot * TB + xt; i < zeros; i += a.slots * TB) {
            const long to = static_cast<long>(i < first ? i : behind + i - first) * a.C + c0 + xc;
            zero.store(static_cast<T *>(a.dx) + to, nc - xc);
            zero.store(static_cast<T *>(a.ddt) + to, nc - xc);
            if (gate)
                zero.store(static_cast<T *>(a.dz) + to, nc - xc);
        }
    }
    const Piece p(seqs, slot, a.seg);
    const int len = p.none() ? 0 : p.len; // a slot of no piece adds zeros to the sums

    // this row's channels are ch(0) ... ch(R - 1)
    const auto in_tile = [&](int i) { return wave * 4 * R + i * 4 + row; };
    float rate[R][S], G[R][S], dA[R][S], skip[R], dD[R], dbias[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = c0 + min(in_tile(i), nc - 1);
        skip[i] = a.D ? a.D[c] : 0.f;
        dD[i] = dbias[i] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool has = in_tile(i) < nc && j + 16 * s < a.S;
            const long at = static_cast<long>(c) * a.S + j + 16 * s;
            rate[i][s] = has ? finite_rate(a.A[at] * kLog2e) : 0.f;
            dA[i][s] = 0.f;
            G[i][s] = 0.f;
            if (has && !p.none() && a.dfin)
                G[i][s] = a.dfin[p.n * states + at];
        }
    }
    if (len > 0 && a.seg) { // the segments behind, a few of them loaded at a time
        constexpr int JOIN = 4;
        const int count = (p.end - p.start + a.seg - 1) / a.seg;
        for (int k0 = count - 1; k0 > p.index; k0 -= JOIN)
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = c0 + min(in_tile(i), nc - 1);
                float sum[JOIN], add[JOIN][S];
#pragma unroll
                for (int k = 0; k < JOIN; ++k) {
                    const long at = static_cast<long>(p.base + max(k0 - k, p.index + 1)) * a.C + c;
                    sum[k] = a.seg_d[at];
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        add[k][s] = a.seg_h[at * a.S + min(j + 16 * s, a.S - 1)];
                }
#pragma unroll
                for (int k = 0; k < JOIN; ++k)
#pragma unroll
                    for (int s = 0; s < S; ++s)
                        if (k0 - k > p.index && in_tile(i) < nc && j + 16 * s < a.S)
                            G[i][s] = across(G[i][s], sum[k] * rate[i][s], add[k][s]);
            }
    }

    // Loads beyond the channels, states or tokens there are go to the first or last that
    // is, and are dropped.  The state ahead of a block is loaded with the rest.
    Cells<XV, T, VEC> rx, rd, rz, ry;
    Cells<XV, float, VEC> rp;
    Cells<BN, T, VEC> rb, rc;
    float bias[XV];
#pragma unroll
    for (int i = 0; i < XV; ++i)
        bias[i] = a.dt_bias && i < nc - xc ? a.dt_bias[c0 + xc + i] : 0.f;
    float ahead[S][R];
    const int col = c0 + (xc < nc ? xc : 0), bcol = g * a.S + (bn < a.S ? bn : 0);
    const float *const saved = a.saved + (p.none() ? 0 : p.start / TB + p.n + (p.t0 - p.start) / TB) * states;
    const auto read = [&](int t0) {
        const long t = p.t0 + min(t0 + xt, len - 1);
        rx.load(static_cast<const T *>(a.x) + t * a.xs + col, nc - xc);
        rd.load(static_cast<const T *>(a.dt) + t * a.dts + col, nc - xc);
        ry.load(static_cast<const T *>(a.dy) + t * a.C + col, nc - xc);
        rz.load(gate ? static_cast<const T *>(a.z) + t * a.zs + col : static_cast<const T *>(a.x) + t * a.xs + col, nc - xc);
        rp.load((gate ? a.plain + t * a.C : a.saved) + col, nc - xc);
        const long u = p.t0 + min(t0 + bt, len - 1);
        rb.load(static_cast<const T *>(a.b) + u * a.bs + bcol, a.S - bn);
        rc.load(static_cast<const T *>(a.c) + u * a.cs + bcol, a.S - bn);
        const float *const from = saved + t0 / TB * states;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < R; ++i)
                ahead[s][i] = from[static_cast<long>(c0 + min(in_tile(i), nc - 1)) * a.S + min(j + 16 * s, a.S - 1)];
    };
    const auto put = [&](GradStage<S> &st, int t0) {
        const int n = t0 + xt < len ? nc - xc : 0, m = t0 + bt < len ? a.S - bn : 0;
        rx.keep(n);
        rd.keep(n);
        ry.keep(n);
        rz.keep(gate ? n : 0);
        rb.keep(m);
        rc.keep(m);
        Cells<XV, T, VEC> dz;
#pragma unroll
        for (int i = 0; i < XV; ++i) {
            float e, raw = to_f(rd.v[i]) + bias[i], soft = softplus(raw, e), slope = softplus_slope(raw, e);
            asm("" : "+v"(soft), "+v"(slope)); // selections, not branches
            const bool there = i < n;
            st.x[xc + i][xt] = to_f(rx.v[i]);
            st.delta[xc + i][xt] = there ? a.softplus ? soft : raw : 0.f;
            st.slope[xc + i][xt] = there ? a.softplus ? slope : 1.f : 0.f;
            const float z = to_f(rz.v[i]), sg = sigmoid(z), dy = to_f(ry.v[i]);
            st.dy[xc + i][xt] = dy * fmaf(z, sg, gate ? 0.f : 1.f);
            dz.v[i] = static_cast<T>(dy * rp.v[i] * sg * fmaf(z, 1.f - sg, 1.f));
        }
        if (gate && t0 + xt < len)
            dz.store(static_cast<T *>(a.dz) + static_cast<long>(p.t0 + t0 + xt) * a.C + c0 + xc, nc - xc);
#pragma unroll
        for (int i = 0; i < BN; ++i) {
            st.b[bn + i][bt] = to_f(rb.v[i]);
            st.c[bn + i][bt] = to_f(rc.v[i]);
        }
    };

    const int blocks = (len + TB - 1) / TB;
    float start[S][R]; // the states ahead of the block
    const auto take = [&] {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < R; ++i)
                start[s][i] = in_tile(i) < nc && j + 16 * s < a.S ? ahead[s][i] : 0.f;
    };
    if (blocks > 0) {
        read((blocks - 1) * TB);
        put(sh.in[0], (blocks - 1) * TB);
        take();
    }
    __syncthreads();
    for (int k = 0; k < blocks; ++k) {
        GradStage<S> &st = sh.in[k % 3];
        const int t0 = (blocks - 1 - k) * TB;
        if (k + 1 < blocks)
            read(t0 - TB);
        float sq[R], sr[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            sq[i] = sr[i] = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float B[TB], C[TB], dB[TB], dC[TB];
#pragma unroll
            for (int t = 0; t < TB; t += 4) {
                const f32x4 b = *reinterpret_cast<const f32x4 *>(&st.b[j + 16 * s][t]),
                            c = *reinterpret_cast<const f32x4 *>(&st.c[j + 16 * s][t]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    B[t + i] = b[i];
                    C[t + i] = c[i];
                    dB[t + i] = dC[t + i] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = in_tile(i);
                float delta = st.delta[c][j], dy = st.dy[c][j], u = delta * st.x[c][j];
                in_order({&delta, &u, &dy, &start[s][i]});
                // forward over the block
                float d[TB], h[TB + 1], f = G[i][s];
                h[0] = start[s][i];
                for_tokens([&](auto J) {
                    constexpr int t = decltype(J)::value;
                    d[t] = __builtin_amdgcn_exp2f(row_bcast<t>(delta) * rate[i][s]);
                    h[t + 1] = fmaf(d[t], h[t], row_bcast<t>(u) * B[t]);
                });
                fma_bcast<0>(dC, dy, h + 1);
                fma_bcast<8>(dC + 8, dy, h + 9);
                in_order({&f});
                // and back
                float q[TB], r[TB], F[TB], moved[TB], odd = 0.f;
                const auto back = [&](auto J) {
                    constexpr int t = decltype(J)::value;
                    F[t] = f + row_bcast<t>(dy) * C[t];
                    q[t] = F[t] * B[t];
                    f = F[t] * d[t];
                    moved[t] = f * h[t];
                    r[t] = moved[t] * rate[i][s];
                };
                for_tokens_down<15, 8>(back);
                fma_bcast<8>(dB + 8, u, F + 8);
                fma_bcast_sum<8>(dA[i][s], odd, delta, moved + 8);
                for_tokens_down<7, 0>(back);
                fma_bcast<0>(dB, u, F);
                fma_bcast_sum<0>(dA[i][s], odd, delta, moved);
                dA[i][s] += odd;
                G[i][s] = f;
                sq[i] += row_sums(q, j);
                sr[i] += row_sums(r, j);
                in_order({&G[i][s], &dA[i][s], &sq[i], &sr[i]});
            }
            rows_sum(dB);
            rows_sum(dC);
            *reinterpret_cast<f32x4 *>(&sh.db[k % 2][wave][j + 16 * s][swizzle(j, 4 * row)]) = f32x4{dB[0], dB[1], dB[2], dB[3]};
            *reinterpret_cast<f32x4 *>(&sh.dc[k % 2][wave][j + 16 * s][swizzle(j, 4 * row)]) = f32x4{dC[0], dC[1], dC[2], dC[3]};
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = in_tile(i);
            const float x = st.x[c][j], dy = st.dy[c][j];
            const float dt = fmaf(x, sq[i], sr[i] * (1.f / kLog2e)) * st.slope[c][j];
            st.x[c][j] = fmaf(st.delta[c][j], sq[i], skip[i] * dy);
            st.slope[c][j] = dt;
            dD[i] = fmaf(dy, x, dD[i]);
            dbias[i] += dt;
        }
        if (k + 1 < blocks) {
            put(sh.in[(k + 1) % 3], t0 - TB);
            take();
        }
        __syncthreads();
        if (t0 + xt < len) {
            const long to = static_cast<long>(p.t0 + t0 + xt) * a.C + c0 + xc;
            Cells<XV, T, VEC> v;
            const auto out = [&](void *dst, const float (&src)[GC][LD]) {
#pragma unroll
                for (int i = 0; i < XV; ++i)
                    v.v[i] = static_cast<T>(src[xc + i][xt]);
                v.store(static_cast<T *>(dst) + to, nc - xc);
            };
            out(a.dx, st.x);
            out(a.ddt, st.slope);
        }
        if (t0 + bt < len) {
            // [tile of the group][token][group][B's states, C's states]
            float *to = a.part_bc + ((static_cast<long>(of_group) * a.T + p.t0 + t0 + bt) * a.G + g) * 2 * a.S;
#pragma unroll
            for (int i = 0; i < BN; ++i) {
                const int n = bn + i;
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    x += sh.db[k % 2][w][n][swizzle(n, bt)];
                    y += sh.dc[k % 2][w][n][swizzle(n, bt)];
                }
                if (n < a.S) {
                    to[n] = x;
                    to[a.S + n] = y;
                }
            }
        }
    }
    float *const sums = a.part_a + slot * (states + 2 * a.C);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long c = c0 + in_tile(i);
        const bool there = in_tile(i) < nc;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (there && j + 16 * s < a.S) {
                sums[c * a.S + j + 16 * s] = dA[i][s];
                if (!p.none() && p.index == 0 && a.dinit)
                    a.dinit[p.n * states + c * a.S + j + 16 * s] = G[i][s];
            }
        const float x = row_sum(dD[i]), y = row_sum(dbias[i]);
        if (there && j == 0) {
            sums[states + c] = x;
            sums[states + a.C + c] = y;
        }
    }
}

// What is summed over workgroups, in 64 bits and in a fixed order (up to hundreds are
// added, and the time is the loads').  The first `first` workgroups: dA, dD and
// dt_bias's gradient, columns of [slots][C S + 2 C], sixteen columns a workgroup and
// every sixteenth row a thread.  The others: dB and dC from the tiles' sums, zero for
// tokens of no sequence.  7.0 us of 22 MB for 2 x 2048 x 2048.
template <typename T> __global__ __launch_bounds__(NT) void ssm_sums_kernel(SsmArgs a, int first, int tiles)
{
    constexpr int U = 8; // loads at a time
    if (static_cast<int>(blockIdx.x) < first) {
        __shared__ double part[16][17];
        const int c = threadIdx.x % 16, s = threadIdx.x / 16;
        const long CS = static_cast<long>(a.C) * a.S, n = CS + 2 * a.C, col = blockIdx.x * 16L + c;
        double x = 0.;
        if (col < n)
            for (int r0 = s; r0 < a.slots; r0 += 16 * U) {
                float v[U];
#pragma unroll
                for (int i = 0; i < U; ++i)
                    v[i] = a.part_a[min(r0 + 16 * i, a.slots - 1) * n + col];
#pragma unroll
                for (int i = 0; i < U; ++i)
                    x += r0 + 16 * i < a.slots ? v[i] : 0.f;
            }
        part[s][c] = x;
        __syncthreads();
        if (s > 0 || col >= n)
            return;
        for (int t = 1; t < 16; ++t)
            x += part[t][c];
        float *const out = col < CS ? a.d_A + col : col < CS + a.C ? a.d_D ? a.d_D + (col - CS) : nullptr
                                                  : a.d_bias ? a.d_bias + (col - CS - a.C) : nullptr;
        if (out)
            *out = static_cast<float>(x);
        return;
    }
    const long width = 2L * a.G * a.S, all = a.T * width, i = static_cast<long>(blockIdx.x - first) * NT + threadIdx.x;
    if (i >= all)
        return;
    const int t = i / width, k = i % width, g = k / (2 * a.S), n = k % (2 * a.S);
    const Sequences seqs{a.cu, a.T, a.N};
    double x = 0.;
    if (t >= seqs.at(0) && t < seqs.at(a.N))
        for (int p0 = 0; p0 < tiles; p0 += U) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = a.part_bc[min(p0 + u, tiles - 1) * all + i];
#pragma unroll
            for (int u = 0; u < U; ++u)
                x += p0 + u < tiles ? v[u] : 0.f;
        }
    T *const out = static_cast<T *>(n < a.S ? a.db : a.dc);
    out[(static_cast<long>(t) * a.G + g) * a.S + (n < a.S ? n : n - a.S)] = static_cast<T>(static_cast<float>(x));
}

template <typename T, int S, bool VEC> void launch(const SsmArgs &a, dim3 grid, hipStream_t st)
{
    hipLaunchKernelGGL((ssm_bwd_kernel<T, S, VEC>), grid, dim3(NT), 0, st, a);
}
template <typename T> hipError_t bwd_t(const SsmArgs &a, hipStream_t st)
{
    const dim3 grid(static_cast<unsigned>(work_groups(a)));
    const bool vec = a.vec_x && a.vec_b;
    if (a.S <= 16)
        vec ? launch<T, 1, true>(a, grid, st) : launch<T, 1, false>(a, grid, st);
    else if (a.S <= 32)
        vec ? launch<T, 2, true>(a, grid, st) : launch<T, 2, false>(a, grid, st);
    else
        vec ? launch<T, 4, true>(a, grid, st) : launch<T, 4, false>(a, grid, st);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    const long columns = static_cast<long>(a.C) * (a.S + 2), bc = static_cast<long>(a.T) * 2 * a.G * a.S;
    const int first = static_cast<int>((columns + 15) / 16);
    hipLaunchKernelGGL((ssm_sums_kernel<T>), dim3(static_cast<unsigned>(first + (bc + NT - 1) / NT)), dim3(NT), 0, st, a,
                       first, (a.CG + GC - 1) / GC);
    return hipGetLastError();
}

} // namespace

hipError_t launch_ssm_backward(int dtype, const SsmArgs &ahead, const SsmArgs &a, hipStream_t st)
{
    hipError_t e = hipSuccess;
    if (a.seg)
        e = launch_ssm_ahead(dtype, true, ahead, st);
    if (e == hipSuccess)
        e = dtype == F32 ? bwd_t<float>(a, st) : bwd_t<__bf16>(a, st);
    return e;
}

} // namespace dl
