// dl_conv.hip -- the short causal convolution in front of a recurrence, forward,
// backward and for single tokens.  Per channel, with W taps, x_{-1}, x_{-2}, ...
// of a sequence being its initial state's last rows (or zero):
//   s_t = bias + sum_j w_j x_{t-W+1+j},   y_t = s_t sigmoid(s_t)  (or s_t)
//   ds = dy silu'(s),  dx_t = sum_k w_{W-1-k} ds_{t+k},
//   dw_j = sum_t ds_t x_{t-W+1+j},  dbias = sum_t ds_t
// A few operations per byte, bound by HBM: a lane walks down a run of tokens with
// a few channels (one vector load and store a token), the last W - 1 inputs and
// the weights in registers, and re-reads the W - 1 tokens ahead of its run
// (backward: behind it).  8192 tokens x 4096 channels, four taps, bf16: forward 28.8
// us, 134 MB at 4.7 TB/s (a copy of as much from memory: 5.1); backward 49.8 us, 201 MB at
// 4.0 (its 32 instructions an element keep the vector units 78% busy); 2756 x 12288,
// six prompts in slices of wider rows, 34.6 us, 4.0 TB/s.  fp32, 8192 x 4096: 48.9 and
// 81.9 us, 5.5 and 4.9 TB/s.  Rows that are not whole vectors take four-byte accesses:
// 777 x 1531, three taps, fp32: 11.0 and 18.6 us for 9.5 and 14.3 MB.
#include "dl_vec.h"

#include "dl_internal.h"
#include "dl_sequences.h"

namespace dl {

namespace {

constexpr int NT = 256;

// What a lane works on: channels c ... c + V - 1 (m of them there), and a walk over
// tokens in ascending order that knows each one's sequence.
template <typename T, int W, int V, bool VEC> struct Lane {
    const ConvArgs &a;
    const Sequences seqs;
    const int c, m;
    float w[W][V], bias[V];
    float x[W][V]; // x[W - 1]: the token's own, x[W - 1 - k]: k tokens back
    int n, start, end;

    __device__ __forceinline__ Lane(const ConvArgs &a, int c)
        : a(a), seqs{a.cu, a.T, a.N}, c(c), m(min(V, a.C - c))
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias && i < m ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j)
                w[j][i] = i < m ? a.weight[static_cast<long>(c + i) * W + j] : 0.f;
        }
    }
    __device__ __forceinline__ void row(float (&out)[V], const void *base, long at) const
    {
        Cells<V, T, VEC> r;
        r.load(static_cast<const T *>(base) + at + c, m);
        r.keep(m);
        r.get(out);
    }
    // row j of sequence n's initial state
    __device__ __forceinline__ void initial(float (&out)[V], int j) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            out[i] = 0.f;
        if (a.init)
            row(out, a.init, (static_cast<long>(n) * (W - 1) + j) * a.C);
    }
    __device__ __forceinline__ void sequence(int k)
    {
        n = k;
        start = seqs.at(k);
        end = seqs.at(k + 1);
    }
    // The sequence of token t, and the tokens ahead of it.
    __device__ __forceinline__ void begin(int t)
    {
        sequence(seqs.of_token(t));
        if (t != start)
            window(t);
    }
    __device__ __forceinline__ void window(int t)
    {
#pragma unroll
        for (int k = 1; k < W; ++k) {
            const int pos = t - start;
            if (pos >= k)
                row(x[W - 1 - k], a.x, (t - k) * a.xs);
            else if (pos >= 0)
                initial(x[W - 1 - k], W - 1 - k + pos);
            else
#pragma unroll
                for (int i = 0; i < V; ++i)
                    x[W - 1 - k][i] = 0.f;
        }
    }
    // Goes on to token t, the next one; whether it is a sequence's.
    __device__ __forceinline__ bool enter(int t)
    {
        while (t >= end && n + 1 < a.N)
            sequence(n + 1);
        if (t == start)
            window(t);
        return t >= start && t < end;
    }
    __device__ __forceinline__ void sums(float (&s)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j)
                s[i] = fmaf(w[j][i], x[j][i], s[i]);
        }
    }
    __device__ __forceinline__ void leave() // the token joins those behind it
    {
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[j][i] = x[j + 1][i];
    }
    // ds of the token from dy
    __device__ __forceinline__ void slope(float (&ds)[V], const float (&dy)[V]) const
    {
        float s[V];
        sums(s);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float sig = sigmoid(s[i]);
            ds[i] = a.silu ? dy[i] * sig * fmaf(s[i], 1.f - sig, 1.f) : dy[i];
        }
    }
};

// Units of V channels: first `runs` runs of tokens, then (fin) the N end states.
template <typename T, int W, int V, bool VEC> __global__ __launch_bounds__(NT) void conv_kernel(ConvArgs a)
{
    constexpr int U = 4; // tokens loaded ahead
    const long unit = static_cast<long>(blockIdx.x) * NT + threadIdx.x;
    const int groups = (a.C + V - 1) / V, run = unit / groups, c = unit % groups * V;
    if (run >= a.runs) {
        const int n = run - a.runs;
        if (n >= a.N || !a.fin)
            return;
        const Sequences seqs{a.cu, a.T, a.N};
        const int start = seqs.at(n), end = max(start, seqs.at(n + 1)), m = min(V, a.C - c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int pos = end - start - (W - 1) + j;
            Cells<V, T, VEC> r;
            if (pos >= 0)
                r.load(static_cast<const T *>(a.x) + (start + pos) * a.xs + c, m);
            else if (a.init)
                r.load(static_cast<const T *>(a.init) + (static_cast<long>(n) * (W - 1) + pos + W - 1) * a.C + c, m);
            else
                r.zero();
            r.store(static_cast<T *>(a.fin) + (static_cast<long>(n) * (W - 1) + j) * a.C + c, m);
        }
        return;
    }
    const int t0 = run * a.run, t1 = min(t0 + a.run, a.T);
    if (t0 >= t1)
        return;
    Lane<T, W, V, VEC> l(a, c);
    // rows as offsets from the run's first (of at most 64 rows): the last one again behind it
    const T *const x = static_cast<const T *>(a.x) + t0 * a.xs + c;
    T *const y = static_cast<T *>(a.y) + static_cast<long>(t0) * a.C + c;
    const unsigned xs = a.xs, last = (t1 - 1 - t0) * xs;
    unsigned from = 0;
    Cells<V, T, VEC> next[U];
    const auto read = [&] {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            next[i].load(x + min(from, last), l.m);
            from += xs;
        }
    };
    read();
    l.begin(t0);
    for (int t = t0; t < t1; t += U) {
        Cells<V, T, VEC> now[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            now[i] = next[i];
        read();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool live = l.enter(t + i);
            now[i].get(l.x[W - 1]);
            float s[V];
            l.sums(s);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (a.silu)
                    s[e] *= sigmoid(s[e]);
                s[e] = live ? s[e] : 0.f;
            }
            Cells<V, T, VEC> out;
            out.put(s);
            if (t + i < t1)
                out.store(y + static_cast<unsigned>(t + i - t0) * static_cast<unsigned>(a.C), l.m);
            l.leave();
        }
    }
}

// Runs as above; then the N initial states' gradients.  dx of a token is done W - 1
// tokens behind it, or at its sequence's end: g[k] is what is gathered of that k
// tokens back.
template <typename T, int W, int V, bool VEC> __global__ __launch_bounds__(NT) void conv_bwd_kernel(ConvArgs a)
{
    const long unit = static_cast<long>(blockIdx.x) * NT + threadIdx.x;
    const int groups = (a.C + V - 1) / V, run = unit / groups, c = unit % groups * V;
    if (run >= a.runs + (a.dinit ? a.N : 0))
        return;
    Lane<T, W, V, VEC> l(a, c);
    const auto add_final = [&](float (&x)[V], int j) { // row j of the end state's gradient
        float d[V];
        l.row(d, a.dfin, (static_cast<long>(l.n) * (W - 1) + j) * a.C);
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] += d[i];
    };
    if (run >= a.runs) {
        l.sequence(run - a.runs);
        const int len = max(l.end - l.start, 0);
        float d[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                d[j][i] = 0.f;
        l.window(l.start);
#pragma unroll
        for (int p = 0; p < W - 1; ++p) {
            if (p >= len)
                break;
            float dy[V], ds[V];
            l.row(l.x[W - 1], a.x, (l.start + p) * a.xs);
            for (int i = 0; i < V; ++i)
                dy[i] = 0.f;
            if (a.dy)
                l.row(dy, a.dy, static_cast<long>(l.start + p) * a.C);
            l.slope(ds, dy);
#pragma unroll
            for (int j = p; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    d[j][i] = fmaf(l.w[j - p][i], ds[i], d[j][i]);
            l.leave();
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (a.dfin && j >= len)
                add_final(d[j], j - len);
            Cells<V, T, VEC> r;
            r.put(d[j]);
            r.store(static_cast<T *>(a.dinit) + (static_cast<long>(l.n) * (W - 1) + j) * a.C + c, l.m);
        }
        return;
    }
    const int t0 = run * a.run, t1 = min(t0 + a.run, a.T);
    float g[W][V], dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j)
            g[j][i] = dw[j][i] = 0.f;
    }
    const auto done = [&](float (&x)[V], int t) { // token t of the sequence
        if (t < t0 || t >= t1 || t < l.start)
            return;
        if (a.dfin && t >= l.end - (W - 1))
            add_final(x, t - (l.end - (W - 1)));
        Cells<V, T, VEC> r;
        r.put(x);
        r.store(static_cast<T *>(a.dx) + static_cast<long>(t) * a.C + c, l.m);
    };
    if (t0 < t1) {
        constexpr int U = 4; // tokens loaded ahead
        const int stop = min(t1 + W - 1, a.T);
        const T *const x = static_cast<const T *>(a.x) + t0 * a.xs + c,
                *const dy = static_cast<const T *>(a.dy ? a.dy : a.x) + t0 * (a.dy ? a.C : a.xs) + c;
        const unsigned xs = a.xs, ys = a.dy ? a.C : a.xs, xlast = (stop - 1 - t0) * xs, ylast = (stop - 1 - t0) * ys;
        unsigned xfrom = 0, yfrom = 0;
        Cells<V, T, VEC> nx[U], ny[U];
        const auto read = [&] {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                nx[i].load(x + min(xfrom, xlast), l.m);
                ny[i].load(dy + min(yfrom, ylast), l.m);
                xfrom += xs;
                yfrom += ys;
            }
        };
        // Tokens t ... t + U - 1 of one sequence, and of this run: nothing to look at but
        // where the run or the sequence begins.
        const auto inner = [&](int t, const Cells<V, T, VEC> (&cx)[U], const Cells<V, T, VEC> (&cy)[U]) {
            const int first = max(t0, l.start);
            T *const to = static_cast<T *>(a.dx) + static_cast<long>(t) * a.C + c;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float dyv[V], ds[V];
                cx[i].get(l.x[W - 1]);
                cy[i].get(dyv);
                l.slope(ds, dyv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        g[k][e] = fmaf(l.w[W - 1 - k][e], ds[e], g[k][e]);
                    db[e] += ds[e];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        dw[j][e] = fmaf(ds[e], l.x[j][e], dw[j][e]);
                }
                if (t + i - (W - 1) >= first) {
                    Cells<V, T, VEC> r;
                    r.put(g[W - 1]);
                    r.store(to + (i - (W - 1)) * a.C, l.m);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
#pragma unroll
                    for (int k = W - 1; k > 0; --k)
                        g[k][e] = g[k - 1][e];
                    g[0][e] = 0.f;
                }
                l.leave();
            }
        };
        // Token t; whether there are more of use.
        const auto token = [&](int t, const Cells<V, T, VEC> &cx, Cells<V, T, VEC> &cy) {
            if (t == l.end) // behind a sequence's last token: what is gathered is whole
#pragma unroll
                for (int k = 1; k < W; ++k) {
                    done(g[k], t - k);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        g[k][i] = 0.f;
                }
            if (t >= stop || (t >= t1 && t >= l.end))
                return false;
            const bool live = l.enter(t);
            float dyv[V], ds[V];
            cx.get(l.x[W - 1]);
            cy.keep(a.dy && live ? l.m : 0);
            cy.get(dyv);
            l.slope(ds, dyv);
            const bool own = live && t < t1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ds[i] = live ? ds[i] : 0.f; // (of no sequence)
#pragma unroll
                for (int k = 0; k < W; ++k)
                    g[k][i] = fmaf(l.w[W - 1 - k][i], ds[i], g[k][i]);
                const float mine = own ? ds[i] : 0.f;
                db[i] += mine;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    dw[j][i] = own ? fmaf(mine, l.x[j][i], dw[j][i]) : dw[j][i];
            }
            if (live) {
                done(g[W - 1], t - (W - 1));
            } else if (t < t1) {
                Cells<V, T, VEC> zero;
                zero.zero();
                zero.store(static_cast<T *>(a.dx) + static_cast<long>(t) * a.C + c, l.m);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int k = W - 1; k > 0; --k)
                    g[k][i] = g[k - 1][i];
                g[0][i] = 0.f;
            }
            l.leave();
            return true;
        };
        read();
        l.begin(t0);
        bool more = true;
        for (int t = t0; more; t += U) {
            Cells<V, T, VEC> cx[U], cy[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                cx[i] = nx[i];
                cy[i] = ny[i];
            }
            read();
            // (the sequence of the token before: its window is the one at hand)
            if (a.dy && t > l.start && t + U <= min(l.end, t1))
                inner(t, cx, cy);
            else
#pragma unroll
                for (int i = 0; i < U; ++i)
                    more = more && token(t + i, cx[i], cy[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < l.m) {
            if (a.part_w)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    a.part_w[(static_cast<long>(run) * a.C + c + i) * W + j] = dw[j][i];
            if (a.part_b)
                a.part_b[static_cast<long>(run) * a.C + c + i] = db[i];
        }
}

// One token each: state row r = [W - 1][C] moves up by one and takes x.  64 x 12288,
// four taps, bf16: 5.7 us for 13 MB, most of it the latency of two loads in a row (the
// state's row, then what is in it) and the launch.
template <typename T, int W, int V, bool VEC> __global__ __launch_bounds__(NT) void conv_step_kernel(ConvArgs a)
{
    // workgroups of a row: `wide`
    const int wide = ((a.C + V - 1) / V + NT - 1) / NT, t = blockIdx.x / wide, c = (blockIdx.x % wide * NT + threadIdx.x) * V;
    if (c >= a.C)
        return;
    Lane<T, W, V, VEC> l(a, c);
    const int r = a.rows ? a.rows[t] : t;
    const bool known = r >= 0 && r < a.n_rows;
    T *const state = static_cast<T *>(a.state) + static_cast<long>(r) * (W - 1) * a.C + c;
    Cells<V, T, VEC> seen[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        seen[j].load((known ? state : static_cast<const T *>(a.state) + c) + j * a.C, l.m);
    seen[W - 1].load(static_cast<const T *>(a.x) + t * a.xs + c, l.m);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        seen[j].keep(known ? l.m : 0);
#pragma unroll
    for (int j = 0; j < W; ++j)
        seen[j].get(l.x[j]);
    float s[V];
    l.sums(s);
    if (a.silu)
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i] *= sigmoid(s[i]);
    Cells<V, T, VEC> y;
    y.put(s);
    y.store(static_cast<T *>(a.y) + static_cast<long>(t) * a.C + c, l.m);
    if (known)
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            seen[j + 1].store(state + j * a.C, l.m);
}

enum Kind { FORWARD, BACKWARD, STEP };

template <typename T, int W, int V, bool VEC> hipError_t conv_v(Kind kind, const ConvArgs &a, hipStream_t st)
{
    const long groups = (a.C + V - 1) / V;
    const long units = groups * (a.runs + ((kind == FORWARD ? a.fin : a.dinit) ? a.N : 0));
    const long blocks = kind == STEP ? a.T * ((groups + NT - 1) / NT) : (units + NT - 1) / NT;
    if (blocks == 0)
        return hipSuccess;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (kind == FORWARD)
        hipLaunchKernelGGL((conv_kernel<T, W, V, VEC>), grid, dim3(NT), 0, st, a);
    else if (kind == BACKWARD)
        hipLaunchKernelGGL((conv_bwd_kernel<T, W, V, VEC>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((conv_step_kernel<T, W, V, VEC>), grid, dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T, int W, int V> hipError_t conv_w(Kind kind, const ConvArgs &a, hipStream_t st)
{
    return a.vec ? conv_v<T, W, V, true>(kind, a, st) : conv_v<T, W, V, false>(kind, a, st);
}
template <typename T, int V> hipError_t conv_t(Kind kind, const ConvArgs &a, hipStream_t st)
{
    return a.W == 2 ? conv_w<T, 2, V>(kind, a, st) : a.W == 3 ? conv_w<T, 3, V>(kind, a, st) : conv_w<T, 4, V>(kind, a, st);
}
hipError_t conv(Kind kind, int dtype, const ConvArgs &a, hipStream_t st)
{
    static_assert(kConvChannels == 4, "every kernel's");
    return dtype == F32 ? conv_t<float, kConvChannels>(kind, a, st) : conv_t<__bf16, kConvChannels>(kind, a, st);
}

} // namespace

hipError_t launch_short_conv(int dtype, const ConvArgs &a, hipStream_t st) { return conv(FORWARD, dtype, a, st); }

hipError_t launch_short_conv_backward(int dtype, const ConvArgs &a, hipStream_t st)
{
    hipError_t e = conv(BACKWARD, dtype, a, st);
    if (e == hipSuccess && a.d_weight)
        e = column_sum(a.part_w, a.runs, a.C * a.W, a.d_weight, a.C, a.d_bias, st);
    else if (e == hipSuccess && a.d_bias)
        e = column_sum(a.part_b, a.runs, a.C, a.d_bias, 0, nullptr, st);
    return e;
}

hipError_t launch_short_conv_step(int dtype, const ConvArgs &a, hipStream_t st) { return conv(STEP, dtype, a, st); }

} // namespace dl
