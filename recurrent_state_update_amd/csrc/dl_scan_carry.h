// dl_scan_carry.h -- the state from chunk to chunk of a scan, forward and (its
// gradient) backward.
//
// One workgroup of eight waves per (sequence, head, NC x 16 value columns): the
// columns of the state are independent.  The chunks are a chain, and with few
// sequences and heads its latency is the time.  Two waves share a SIMD: waves
// 0-3 hold rows 16 w.. of the chunk's products, waves 4-7 the row blocks of the
// state (w - 4, w), in fp32 registers, and while the first form b, the chunk
// before's o.  What a wave's product needs of another's rows
// passes through LDS as bf16 planes, already in the order that the matrix
// instruction reads; LDS bandwidth is most of a step, so what is read from it
// serves every product that the wave forms with it.  Each operand of the next
// chunk is loaded into the registers of this one's right behind its last use,
// and ahead of the stores of the same phase (waits count in order);
// the value tiles of one (sequence, head) run on one XCD, whose L2 serves all
// but the first of them.
#pragma once

#include "dl_scan.h"

namespace dl {

constexpr int kXcds = 8; // consecutive workgroups go to consecutive XCDs

// The (sequence, head) and value tile of a workgroup; group >= groups: none.
struct CarryWork {
    int group, tile;
};
__device__ __forceinline__ CarryWork carry_work(int tiles)
{
    const int x = blockIdx.x % kXcds, j = blockIdx.x / kXcds;
    return {j / tiles * kXcds + x, j % tiles};
}

// N planes of 16 columns of a C-layout tile in LDS, as the other operand of a
// product: [16 columns][K], k along the row.
template <int N, int K> struct Planes {
    static constexpr int LD = K + 8;
    __bf16 p[N][16 * LD];
    // the four consecutive k from k0 of column c
    __device__ __forceinline__ void put(int c, int k0, f32x4 x)
    {
        bf16x4 v[N];
        split(x, v);
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x4 *>(&p[i][c * LD + k0]) = v[i];
    }
    template <int M> __device__ __forceinline__ void get(bf16x8 (&f)[M], int ks, int lane) const
    {
#pragma unroll
        for (int i = 0; i < M; ++i)
            f[i] = *reinterpret_cast<const bf16x8 *>(&p[i][(lane & 15) * LD + ks * 32 + (lane >> 4) * 8]);
    }
};

// The fragments of planes in registers (the first M planes)
template <int KS, int M, int N, int K> __device__ __forceinline__ void get_all(bf16x8 (&f)[KS][M], const Planes<N, K> &b, int lane)
{
    static_assert(KS * 32 == K && M <= N, "all of it");
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        b.get(f[ks], ks, lane);
}
// acc + a b, a row block's fragments and the columns' in registers
template <int KS, int NA, int NB>
__device__ __forceinline__ f32x4 product(const bf16x8 (&a)[KS][NA], const bf16x8 (&b)[KS][NB], f32x4 acc)
{
    Acc c(acc);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        c.add(a[ks], b[ks]);
    return c.sum();
}
// The same for a triangular C x C operand: the half that is zero is skipped
// (first: whether k < 32 counts for this row block, second: k >= 32).
template <int NA, int NB>
__device__ __forceinline__ f32x4 product_tri(const bf16x8 (&a)[2][NA], const Planes<NB, C> &b, bool first, bool second,
                                             int lane, f32x4 acc)
{
    Acc c(acc);
    bf16x8 f[NB];
    if (first) {
        b.get(f, 0, lane);
        c.add(a[0], f);
    }
    if (second) {
        b.get(f, 1, lane);
        c.add(a[1], f);
    }
    return c.sum();
}
// A row block's fragments of an operand in N planes: loaded some phases ahead,
// and, where they come as fp32, split (ready) while the wave has nothing else
// to do.
template <int KS, int N> struct Operand {
    bf16x8 f[KS][N];
    f32x8 raw[N == 3 ? KS : 1];
    __device__ __forceinline__ void one(const char *op, int rb, int at, int ks, int lane)
    {
        if constexpr (N == 3)
            raw[at] = load_frag32(op, KS, rb, ks, lane);
        else
            load_frag(f[at], op, KS, rb, ks, lane);
    }
    __device__ __forceinline__ void load(const char *op, int rb, int lane)
    {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            one(op, rb, ks, ks, lane);
    }
    // Of a triangular operand; the half that holds nothing is not stored, and
    // the other is loaded in its place (the load stays unconditional).
    __device__ __forceinline__ void load_tri(const char *op, Part part, int rb, int lane)
    {
        static_assert(KS == 2, "C x C");
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            one(op, rb, ks, frag_used(part, rb, ks) ? ks : 1 - ks, lane);
    }
    __device__ __forceinline__ void ready()
    {
        if constexpr (N == 3) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                split(raw[ks], f[ks]);
        }
    }
};
__device__ __forceinline__ f32x4 ld4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// The state row of a sequence: through a.rows if given; < 0 where the row is
// not one of the caller's a.nrows (nothing is read or written then).
__device__ __forceinline__ long state_row(const ScanArgs &a, int n)
{
    if (!a.rows)
        return n;
    const int r = a.rows[n];
    return r >= 0 && r < a.nrows ? r : -1;
}

// The row blocks of the state that waves 4-7 hold: RB each, the r-th of wave
// 4 + wb being wb + 4 r.
template <int DKP> struct Holder {
    static constexpr int RB = DKP == 128 ? 2 : 1;
    static __device__ __forceinline__ bool has(int wb) { return DKP >= 64 || wb < DKP / 16; }
    static __device__ __forceinline__ int block(int wb, int r) { return has(wb) ? wb + 4 * r : 0; }
};

// Rows of one chunk of a matrix of inputs, as a buffer of the rows that there
// are: a load behind the end gives zero, a store there is dropped, so both
// stay unconditional (and countable by the waits).
template <typename TIn> struct ChunkRows {
    rsrc_t r;
    // p: row 0 of the sequence at the workgroup's first column
    __device__ __forceinline__ ChunkRows(const TIn *p, unsigned stride, int c, int len, int width)
        : r(make_rsrc(p + static_cast<long>(c) * C * stride,
                      static_cast<unsigned>((((len - c * C < C ? len - c * C : C) - 1) * stride + width) * sizeof(TIn))))
    {
    }
    __device__ __forceinline__ TIn load(unsigned at) const
    {
        if constexpr (sizeof(TIn) == 2)
            return __builtin_bit_cast(TIn, __builtin_amdgcn_raw_buffer_load_b16(r, at * 2u, 0, 0));
        else
            return __builtin_bit_cast(TIn, __builtin_amdgcn_raw_buffer_load_b32(r, at * 4u, 0, 0));
    }
    __device__ __forceinline__ void store(unsigned at, float x) const
    {
        const TIn v = static_cast<TIn>(x);
        if constexpr (sizeof(TIn) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, at * 2u, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, at * 4u, 0, 0);
    }
};

// What only the backward pass reads, stored past the caches, where it would push
// out the operands that the value tiles share (4096 tokens, 32 heads, GDN: 203
// -> 172 us.  The same for dS' and z, which the next kernel reads: no change).
__device__ __forceinline__ void keep_for_backward(float *p, float x) { __builtin_nontemporal_store(x, p); }

// Long sequences with few heads leave most CUs idle while their chunks pass one
// by one.  There they are cut into segments of a.seg chunks (scan_segment):
// over a segment the end state is linear in the start state, S' = M S + L.
//   LOCAL  per segment but the last of its sequence, side by side: L, the carry
//          from a zero state (from the initial one in the first segment), and
//          M, the carry from each column of the identity with V = 0, as d_k more
//          columns
//   join   per sequence and head, over its segments: S = M S + L in fp32
//   PLAIN (or SAVE), the carry itself, segment by segment from these states
// and the same backward, for the gradients of the end states.
// A whole forward scan, d = 128, bf16, us (uncut, cut):
//   tokens, heads   2600, 1     2600, 8     8192, 1     8192, 8     32768, 4
//   GDN             86.4, 56.5  89.8, 83.8  232, 88     246, 159    920, 306
//   KDA             136, 75.2   140, 116    372, 114    402, 262    1636, 551
//   RWKV6           89.3, 56.7  91.4, 74.5  240, 88     258, 150    1130, 323
// forward and backward (below 210 the host is the longer):
//   GDN             234, 206    260, 230    597, 222    746, 541    2600, 1051
//   KDA             317, 206    373, 340    816, 273    1097, 863   3989, 1745
//   RWKV6           198, 204    237, 211    483, 208    713, 504    2469, 1025
// A segment's slot is found as a chunk's: sequence n's first is
// start / (64 a.seg) + n; a sequence without tokens has one too.
struct Segment {
    Seq s;
    int n;
    bool none, first, last;
};
__device__ __forceinline__ Segment segment_of(const ScanArgs &a, int slot)
{
    const int rows = C * a.seg;
    int lo = 0, hi = a.N;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (seq_start(a, mid) / rows + mid <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    Segment g;
    g.n = lo;
    g.s = sequence(a, lo);
    const int k = slot - (g.s.start / rows + lo), t0 = k * rows;
    g.none = lo == a.N || k < 0 || (k > 0 && t0 >= g.s.len);
    g.first = k == 0;
    g.last = t0 + rows >= g.s.len;
    g.s.start += t0;
    g.s.len = g.s.len - t0 < rows ? g.s.len - t0 : rows;
    g.s.base += k * a.seg;
    return g;
}

// Forward.  SAVE: keeps every chunk's start state and E.
enum CarryMode { PLAIN, SAVE, LOCAL };
template <int OP, typename TIn, int DKP, int NC, CarryMode MODE>
__global__ __launch_bounds__(512) void scan_carry_kernel(ScanArgs a)
{
    static_assert(MODE != LOCAL || NC == 1, "tiles of 16 keys");
    using P = Plan<OP, TIn>;
    using O = Ops<P::NPX, DKP>;
    using Own = Holder<DKP>;
    constexpr bool DELTA = P::DELTA, ROWS = P::ROWS;
    constexpr int KS = DKP / 32, RB = Own::RB;
    // Delta rule: three barriers a chunk, every buffer rewritten two behind its
    // readers.  RWKV6's b is known ahead: one barrier, two buffers each.
    constexpr int TWO = DELTA ? 1 : 2;
    __shared__ Planes<3, DKP> sp[TWO][NC];        // the state
    __shared__ Planes<3, C> rp[DELTA ? NC : 1];   // V - K~ S
    __shared__ Planes<P::NPB, C> bp[2][NC];       // b (in turn: the delta rule's o reads it a chunk later)
    __shared__ Planes<3, C> hp[ROWS ? NC : 1];    // P_Ci b, for the state
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, r4 = (lane >> 4) * 4, i0 = (w & 3) * 16 + r4;
    const int tiles = a.dv / (16 * NC);
    const CarryWork wk = carry_work(MODE == LOCAL ? tiles + a.dk / 16 : tiles);
    if (wk.group >= (a.seg ? a.segments : a.N) * a.H)
        return;
    const int h = wk.group % a.H, item = wk.group / a.H; // a sequence or a segment
    Segment sg = {{}, item, false, true, true};
    if (MODE == LOCAL || a.seg)
        sg = segment_of(a, item);
    else
        sg.s = sequence(a, item);
    if (sg.none)
        return;
    const Seq sq = sg.s;
    const bool unit = MODE == LOCAL && wk.tile >= tiles; // a transition's columns
    if (MODE == LOCAL && (sg.last || (unit && sg.first)))
        return;
    const int tile = unit ? wk.tile - tiles : wk.tile, v0 = tile * 16 * NC + col;
    const long first = static_cast<long>(h) * a.dv + (unit ? 0 : v0 - col); // of a row, this workgroup's
    const unsigned width = a.H * a.dv;
    const int chunks = (sq.len + C - 1) / C;
    const f32x4 zero = {0, 0, 0, 0};
    auto ops = [&](int c) { return O(a, static_cast<long>(sq.base + c) * a.H + h); };

    // o = Q~ S + B b of rows i0..
    Operand<KS, P::NPX> qf;
    Operand<2, 3> bf;
    TIn *op = static_cast<TIn *>(a.o) + static_cast<long>(sq.start) * width + first;
    auto load_q = [&](int c) { qf.load(ops(c).op(1), w & 3, lane); };
    auto load_b = [&](int c) { bf.load_tri(ops(c).mat(1), LOWER, w & 3, lane); };
    auto with_b = [&](f32x4 o, const Planes<P::NPB, C> &b) {
        return product_tri(bf.f, b, true, (w & 3) >= 2, lane, o);
    };
    auto store_o = [&](int c, const f32x4 (&o)[NC]) {
        const ChunkRows<TIn> rows(op, width, c, sq.len, 16 * NC);
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                rows.store((i0 + e) * width + col + 16 * t, o[t][e]);
    };

    if (w < 4) {
        if (chunks == 0)
            return; // barriers count the waves that are left
        TIn v[NC][4];
        const TIn *vp = static_cast<const TIn *>(a.v) + static_cast<long>(sq.start) * a.vs + first;
        auto load_v = [&](int c) {
            const ChunkRows<TIn> rows(vp, static_cast<unsigned>(a.vs), c, sq.len, 16 * NC);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    v[t][e] = rows.load((i0 + e) * static_cast<unsigned>(a.vs) + col + 16 * t);
        };
        auto take_v = [&](int t) {
            if (MODE == LOCAL && unit)
                return zero;
            return f32x4{from_in(v[t][0]), from_in(v[t][1]), from_in(v[t][2]), from_in(v[t][3])};
        };
        load_v(0);
        keep_order();
        if constexpr (DELTA) {
            Operand<KS, P::NPX> kf;
            Operand<2, 3> nf;
            f32x4 gi, ge, beta;
            auto load_k = [&](int c) {
                kf.load(ops(c).op(0), w, lane);
                if (ROWS)
                    gi = ld4(ops(c).row(0) + i0);
            };
            auto load_n = [&](int c) {
                nf.load_tri(ops(c).mat(0), LOWER, w, lane);
                beta = ld4(ops(c).row(2) + i0);
                if (ROWS)
                    ge = ld4(ops(c).row(1) + i0);
            };
            load_k(0);
            keep_order();
            load_n(0);
            keep_order();
            kf.ready();
            nf.ready();
            for (int c = 0; c < chunks; ++c) {
                const int next = c + 1 < chunks ? c + 1 : c;
                f32x4 x[NC];
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    x[t] = take_v(t);
                load_v(next);
                __syncthreads(); // the state's planes are complete
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    bf16x8 f[KS][3];
                    get_all(f, sp[0][t], lane);
                    f32x4 ks = product(kf.f, f, zero);
                    if (ROWS)
                        ks *= gi;
                    rp[t].put(col, i0, x[t] - ks);
                }
                load_k(next);
                __syncthreads(); // V - K~ S is complete, and the state's planes are read
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    x[t] = product_tri(nf.f, rp[t], true, w >= 2, lane, zero);
                    const f32x4 b = x[t] * beta;
                    if (ROWS)
                        hp[t].put(col, i0, b * ge);
                    bp[c & 1][t].put(col, i0, b);
                }
                load_n(next);
                if (MODE == SAVE) {
                    const long sh = static_cast<long>(sq.base + c) * a.H + h;
#pragma unroll
                    for (int t = 0; t < NC; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            keep_for_backward(&a.save_e[(sh * C + i0 + e) * a.dv + v0 + 16 * t], x[t][e]);
                }
                __syncthreads(); // b is complete
                kf.ready();
                nf.ready();
            }
        } else {
            auto put_v = [&](int c) {
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    bp[c & 1][t].put(col, i0, take_v(t));
            };
            put_v(0);
            load_v(chunks > 1 ? 1 : 0);
            keep_order();
            if (MODE != LOCAL) {
                load_q(0);
                keep_order();
                load_b(0);
                keep_order();
                qf.ready();
                bf.ready();
            }
            for (int c = 0; c < chunks; ++c) {
                __syncthreads(); // state and b are complete
                const int next = c + 1 < chunks ? c + 1 : c, after = c + 2 < chunks ? c + 2 : next;
                f32x4 o[NC];
                if (MODE != LOCAL)
#pragma unroll
                    for (int t = 0; t < NC; ++t) {
                        bf16x8 f[KS][3];
                        get_all(f, sp[c & 1][t], lane);
                        o[t] = with_b(product(qf.f, f, zero), bp[c & 1][t]);
                    }
                put_v(c + 1); // (behind the last chunk: read by nobody)
                load_v(after);
                if (MODE != LOCAL) {
                    load_q(next);
                    load_b(next);
                    store_o(c, o);
                    qf.ready();
                    bf.ready();
                }
            }
        }
        return;
    }

    const int wb = w - 4;
    const bool has = Own::has(wb);
    // where the state comes from and goes to (NULL: zero, nowhere)
    const long row = state_row(a, sg.n), mat = static_cast<long>(a.dk) * a.dv, caller = (row * a.H + h) * mat + v0;
    const long here = (static_cast<long>(item) * a.H + h) * mat + v0;
    const float *from = sg.first ? (a.init && row >= 0 ? a.init + caller : nullptr) : nullptr;
    float *to = a.fin && row >= 0 ? a.fin + caller : nullptr;
    if (MODE == LOCAL)
        to = unit ? a.seg_m + (static_cast<long>(item + 1) * a.H + h) * a.dk * a.dk + v0 : a.seg_s + here + a.H * mat;
    else if (!sg.first || !sg.last) {
        from = a.seg_s + here; // (the first's too: the caller's state may be overwritten by now)
        to = sg.last ? to : nullptr;
    }
    const long ldw = unit ? a.dk : a.dv;
    f32x4 S[NC][RB], gam[RB];
    Operand<2, P::NPX> tf[RB];
    auto load_t = [&](int c) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            tf[r].load(ops(c).op(2), Own::block(wb, r), lane);
            gam[r] = ld4(ops(c).gam() + Own::block(wb, r) * 16 + r4);
        }
    };
    auto put_state = [&](int c) { // the planes of chunk c's start state
        if (!has)
            return;
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int d0 = Own::block(wb, r) * 16 + r4;
                sp[DELTA ? 0 : c & 1][t].put(col, d0, S[t][r]);
                if (MODE == SAVE && c < chunks) {
                    const long sh = static_cast<long>(sq.base + c) * a.H + h;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (DKP > 32 || d0 + e < a.dk)
                            keep_for_backward(&a.save_s[(sh * a.dk + d0 + e) * a.dv + v0 + 16 * t], S[t][r][e]);
                }
            }
    };
#pragma unroll
    for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = Own::block(wb, r) * 16 + r4 + e;
                const bool in = has && d < a.dk;
                S[t][r][e] = unit ? (in && d == v0 ? 1.f : 0.f) : from && in ? from[static_cast<long>(d) * a.dv + 16 * t] : 0.f;
                if (MODE == LOCAL && sg.first && in)
                    a.seg_s[here + static_cast<long>(d) * a.dv] = S[t][r][e];
            }
    put_state(0);
    if (chunks > 0) {
        f32x4 gi = zero, o[NC], last[NC]; // delta rule: rows' decays, Q~ S of this chunk and the one before
#pragma unroll
        for (int t = 0; t < NC; ++t)
            last[t] = zero;
        auto load_gi = [&](int c) {
            if (ROWS)
                gi = ld4(ops(c).row(0) + i0);
        };
        if (DELTA && MODE != LOCAL) {
            load_q(0);
            load_gi(0);
            keep_order();
            load_b(0);
            keep_order();
        }
        load_t(0);
        keep_order();
        if (DELTA && MODE != LOCAL) {
            qf.ready();
            bf.ready();
        }
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            __syncthreads();
            if constexpr (DELTA && MODE == LOCAL) {
                __syncthreads();
            } else if constexpr (DELTA) {
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    bf16x8 f[KS][3];
                    get_all(f, sp[0][t], lane);
                    o[t] = product(qf.f, f, zero);
                    if (ROWS)
                        o[t] *= gi;
                }
                load_q(next);
                load_gi(next);
                __syncthreads();
                // the chunk before is finished while waves 0-3 form b; the first
                // turn has none (what it writes is written again)
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    last[t] = with_b(last[t], bp[(c + 1) & 1][t]);
                bf.ready(); // this chunk's, loaded a turn ago, for the next turn
                load_b(next);
                store_o(c > 0 ? c - 1 : 0, last);
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    last[t] = o[t];
                qf.ready();
            }
#pragma unroll
            for (int r = 0; r < RB; ++r)
                tf[r].ready();
            if constexpr (DELTA)
                __syncthreads();
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                bf16x8 f[2][P::NPB];
                if constexpr (ROWS)
                    get_all(f, hp[t], lane);
                else
                    get_all(f, bp[c & 1][t], lane);
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    S[t][r] = product(tf[r].f, f, S[t][r] * gam[r]);
            }
            load_t(next);
            put_state(c + 1);
        }
        if constexpr (DELTA && MODE != LOCAL) {
#pragma unroll
            for (int t = 0; t < NC; ++t)
                last[t] = with_b(last[t], bp[(chunks - 1) & 1][t]);
            store_o(chunks - 1, last);
        }
    }
    if (to && has) {
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = Own::block(wb, r) * 16 + r4 + e;
                    if (d < a.dk)
                        to[d * ldw + 16 * t] = S[t][r][e];
                }
    }
}

// The start states of a sequence's segments from the third on (the first two come
// from LOCAL as they are): S = M S + L; BACK: the gradients of their end
// states, from the third last on.  16 value columns per workgroup, a wave per
// 16 keys.  Products on the fp32 matrix instruction; the next transition is
// loaded a turn ahead.
template <int DKP, bool BACK> __global__ __launch_bounds__(DKP * 4) void scan_join_kernel(ScanArgs a)
{
    __shared__ float x[2][16][DKP + 4]; // S by column
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, r4 = (lane >> 4) * 4;
    const int tiles = a.dv / 16, tile = blockIdx.x % tiles, h = blockIdx.x / tiles % a.H, n = blockIdx.x / tiles / a.H;
    const Seq sq = sequence(a, n);
    const int rows = C * a.seg, slot = sq.start / rows + n, count = (sq.len + rows - 1) / rows;
    if (count < 3)
        return;
    const bool in = w * 16 < a.dk;
    const long mat = static_cast<long>(a.dk) * a.dv;
    auto at = [&](int k) { return static_cast<long>(slot + (BACK ? count - 1 - k : k)) * a.H + h; };
    auto state = [&](int k) { return a.seg_s + at(k) * mat + (w * 16 + r4) * a.dv + tile * 16 + col; };
    f32x4 m[DKP / 16], l;
    auto load = [&](int k) {
        const float *p = a.seg_m + (at(k) * a.dk + w * 16 + col) * a.dk + r4, *s = state(k);
#pragma unroll
        for (int j = 0; j < DKP / 16; ++j)
            m[j] = in && j * 16 < a.dk ? *reinterpret_cast<const f32x4 *>(p + j * 16) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            l[e] = in ? s[e * a.dv] : 0.f;
    };
    load(1);
    *reinterpret_cast<f32x4 *>(&x[1][col][w * 16 + r4]) = l;
    load(2);
    for (int k = 2; k < count; ++k) {
        __syncthreads();
        f32x4 y = l;
#pragma unroll
        for (int j = 0; j < DKP / 16; ++j)
            y = mfma32x4(m[j], *reinterpret_cast<const f32x4 *>(&x[(k - 1) & 1][col][j * 16 + r4]), y);
        load(k + 1 < count ? k + 1 : k);
        *reinterpret_cast<f32x4 *>(&x[k & 1][col][w * 16 + r4]) = y;
        if (in) {
            float *s = state(k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e * a.dv] = y[e];
        }
    }
}

// Backward: chunks from the last to the first, dS in registers.  Writes every
// chunk's dS' and z (delta rule), dv, and per 16 NC value columns the partial
// sums of db . E (of dbeta; grads adds the rest); at the end the initial
// state's gradient.
template <int OP, typename TIn, int DKP, int NC, CarryMode MODE>
__global__ __launch_bounds__(512) void scan_carry_bwd_kernel(ScanArgs a)
{
    static_assert(MODE == PLAIN || (MODE == LOCAL && NC == 1), "tiles of 16 keys");
    using P = Plan<OP, TIn>;
    using O = Ops<P::NPX, DKP>;
    using Own = Holder<DKP>;
    constexpr bool DELTA = P::DELTA, ROWS = P::ROWS;
    constexpr int KS = DKP / 32, RB = Own::RB;
    constexpr int TWO = DELTA ? 1 : 2;                  // RWKV6: dS does not wait for db, one barrier a chunk
    __shared__ Planes<3, DKP> sp[TWO][NC];              // dS'
    __shared__ Planes<P::NPI, C> gp[2][NC];             // dO (in turn: put a chunk ahead)
    __shared__ Planes<3, C> gg[2][ROWS ? NC : 1];       // ROWS: Gam_i dO
    __shared__ Planes<3, C> wp[DELTA ? NC : 1];         // beta db
    __shared__ Planes<3, C> zp[DELTA ? NC : 1];         // -z (ROWS: -Gam_i z)
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, r4 = (lane >> 4) * 4, i0 = (w & 3) * 16 + r4;
    const int tiles = a.dv / (16 * NC);
    const CarryWork wk = carry_work(MODE == LOCAL ? tiles + a.dk / 16 : tiles);
    if (wk.group >= (a.seg ? a.segments : a.N) * a.H)
        return;
    const int h = wk.group % a.H, item = wk.group / a.H; // a sequence or a segment
    Segment sg = {{}, item, false, true, true};
    if (MODE == LOCAL || a.seg)
        sg = segment_of(a, item);
    else
        sg.s = sequence(a, item);
    if (sg.none)
        return;
    const Seq sq = sg.s;
    const bool unit = MODE == LOCAL && wk.tile >= tiles; // a transition's columns
    if (MODE == LOCAL && (sg.first || (unit && sg.last)))
        return;
    const int tile = unit ? wk.tile - tiles : wk.tile, v0 = tile * 16 * NC + col;
    const long first = static_cast<long>(h) * a.dv + (unit ? 0 : v0 - col); // of a row, this workgroup's
    const unsigned width = a.H * a.dv;
    const int chunks = (sq.len + C - 1) / C;
    const f32x4 zero = {0, 0, 0, 0};
    auto ops = [&](int c) { return O(a, static_cast<long>(sq.base + c) * a.H + h); };

    if (w < 4) {
        if (chunks == 0 || (MODE == LOCAL && !DELTA))
            return; // barriers count the waves that are left
        Operand<KS, P::NPX> kf;
        Operand<2, 3> bt, nt;
        f32x4 gi, ge, beta;
        float E[NC][4];
        TIn *dvp = static_cast<TIn *>(a.d_v) + static_cast<long>(sq.start) * width + first;
        auto load_db = [&](int c) {
            bt.load_tri(ops(c).mat(1), UPPER, w, lane);
            kf.load(ops(c).op(0), w, lane);
            if (ROWS)
                ge = ld4(ops(c).row(1) + i0);
            if (DELTA)
                beta = ld4(ops(c).row(2) + i0);
        };
        auto load_n = [&](int c) {
            if (DELTA)
                nt.load_tri(ops(c).mat(0), UPPER, w, lane);
            if (ROWS)
                gi = ld4(ops(c).row(0) + i0);
        };
        auto load_e = [&](int c) {
            if (!DELTA || MODE == LOCAL)
                return;
#pragma unroll
            for (int t = 0; t < NC; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    E[t][e] = a.save_e[((static_cast<long>(sq.base + c) * a.H + h) * C + i0 + e) * a.dv + v0 + 16 * t];
        };
        load_db(chunks - 1);
        keep_order();
        load_n(chunks - 1);
        keep_order();
        load_e(chunks - 1);
        keep_order();
        auto ready = [&]() __attribute__((always_inline)) { // (the operands live in registers)
            kf.ready();
            bt.ready();
            if (DELTA)
                nt.ready();
        };
        ready();
        for (int c = chunks - 1; c >= 0; --c) {
            const int next = c > 0 ? c - 1 : 0;
            const long sh = static_cast<long>(sq.base + c) * a.H + h;
            __syncthreads(); // dO and dS' are complete
            f32x4 db[NC], x[NC];
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                bf16x8 f[KS][3];
                get_all(f, sp[DELTA ? 0 : c & 1][t], lane);
                db[t] = product(kf.f, f, zero);
                if (ROWS)
                    db[t] *= ge;
                db[t] = product_tri(bt.f, gp[c & 1][t], w < 2, true, lane, db[t]);
                x[t] = db[t];
                if (DELTA)
                    wp[t].put(col, i0, db[t] * beta);
            }
            load_db(next);
            if constexpr (DELTA) {
                __syncthreads(); // beta db is complete; the planes of dS' are read
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    x[t] = product_tri(nt.f, wp[t], w < 2, true, lane, zero);
                    zp[t].put(col, i0, ROWS ? -x[t] * gi : -x[t]);
                }
                load_n(next);
                __syncthreads(); // z is complete
            }
            if constexpr (MODE != LOCAL) {
                f32x4 p = zero;
                if constexpr (DELTA) {
#pragma unroll
                    for (int t = 0; t < NC; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p[e] = fmaf(db[t][e], E[t][e], p[e]);
                    load_e(next);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = add_row_ror<1>(p[e]);
                        p[e] = add_row_ror<2>(p[e]);
                        p[e] = add_row_ror<4>(p[e]);
                        p[e] = add_row_ror<8>(p[e]);
                    }
                }
                const ChunkRows<TIn> rows(dvp, width, c, sq.len, 16 * NC);
#pragma unroll
                for (int t = 0; t < NC; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rows.store((i0 + e) * width + col + 16 * t, x[t][e]);
                        if (DELTA)
                            a.w_z[(sh * C + i0 + e) * a.dv + v0 + 16 * t] = x[t][e];
                    }
                if (DELTA && col == 0)
                    *reinterpret_cast<f32x4 *>(&a.w_db[(sh * tiles + wk.tile) * C + i0]) = p;
            }
            ready();
        }
        return;
    }

    const int wb = w - 4;
    const bool has = Own::has(wb);
    // where the end state's gradient comes from and the start state's goes to
    const long mat = static_cast<long>(a.dk) * a.dv, caller = (static_cast<long>(sg.n) * a.H + h) * mat + v0;
    const long here = (static_cast<long>(item) * a.H + h) * mat + v0;
    const float *from = sg.last ? (a.dfin ? a.dfin + caller : nullptr) : MODE == LOCAL ? nullptr : a.seg_s + here;
    float *to = sg.first && a.dinit ? a.dinit + caller : nullptr;
    if (MODE == LOCAL)
        to = unit ? a.seg_m + (static_cast<long>(item - 1) * a.H + h) * a.dk * a.dk + v0 : a.seg_s + here - a.H * mat;
    const long ldw = unit ? a.dk : a.dv;
    const bool with_g = a.d_o && !unit;
    f32x4 S[NC][RB], gam[RB], gi; // S: dS'
    Operand<2, P::NPX> qt[RB], kt[RB];
    TIn g[NC][4];
    const TIn *gbase = static_cast<const TIn *>(a.d_o) + static_cast<long>(sq.start) * width + first;
    auto load_g = [&](int c) {
        if (with_g) {
            const ChunkRows<TIn> rows(gbase, width, c, sq.len, 16 * NC);
#pragma unroll
            for (int t = 0; t < NC; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    g[t][e] = rows.load((i0 + e) * width + col + 16 * t);
        }
        if (ROWS)
            gi = ld4(ops(c).row(0) + i0);
    };
    auto put_g = [&](int c) {
#pragma unroll
        for (int t = 0; t < NC; ++t) {
            const f32x4 x = with_g ? f32x4{from_in(g[t][0]), from_in(g[t][1]), from_in(g[t][2]), from_in(g[t][3])} : zero;
            gp[c & 1][t].put(col, i0, x);
            if (ROWS)
                gg[c & 1][t].put(col, i0, x * gi);
        }
    };
    auto load_q = [&](int c) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            qt[r].load(ops(c).op(1), Own::block(wb, r), lane);
            gam[r] = ld4(ops(c).gam() + Own::block(wb, r) * 16 + r4);
        }
    };
    auto load_k = [&](int c) {
        if (!DELTA)
            return;
#pragma unroll
        for (int r = 0; r < RB; ++r)
            kt[r].load(ops(c).op(2), Own::block(wb, r), lane);
    };
    auto put_state = [&](int c) { // the planes of the gradient of chunk c's end state
        if (!has)
            return;
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int d0 = Own::block(wb, r) * 16 + r4;
                sp[DELTA ? 0 : c & 1][t].put(col, d0, S[t][r]);
                if (MODE != LOCAL && c >= 0) {
                    const long sh = static_cast<long>(sq.base + c) * a.H + h;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (DKP > 32 || d0 + e < a.dk)
                            a.w_ds[(sh * a.dk + d0 + e) * a.dv + v0 + 16 * t] = S[t][r][e];
                }
            }
    };
#pragma unroll
    for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = Own::block(wb, r) * 16 + r4 + e;
                const bool in = has && d < a.dk;
                S[t][r][e] = unit ? (in && d == v0 ? 1.f : 0.f) : from && in ? from[static_cast<long>(d) * a.dv + 16 * t] : 0.f;
            }
    put_state(chunks - 1);
    if (chunks > 0) {
        load_g(chunks - 1);
        put_g(chunks - 1);
        keep_order();
        load_g(chunks > 1 ? chunks - 2 : 0);
        keep_order();
        load_q(chunks - 1);
        keep_order();
        load_k(chunks - 1);
        keep_order();
        for (int c = chunks - 1; c >= 0; --c) {
            const int next = c > 0 ? c - 1 : 0;
            __syncthreads();
            put_g(c - 1); // (ahead of the first chunk: read by nobody)
            load_g(c > 1 ? c - 2 : 0);
            if constexpr (DELTA)
                __syncthreads();
            // dS = Gam_C dS' + Q~^T dO - K~^T z, all but the last ahead of z
#pragma unroll
            for (int r = 0; r < RB; ++r)
                qt[r].ready();
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                bf16x8 f[2][ROWS ? 3 : P::NPI];
                if constexpr (ROWS)
                    get_all(f, gg[c & 1][t], lane);
                else
                    get_all(f, gp[c & 1][t], lane);
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    S[t][r] = product(qt[r].f, f, S[t][r] * gam[r]);
            }
            load_q(next);
            if constexpr (DELTA) {
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    kt[r].ready();
                __syncthreads();
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    bf16x8 f[2][3];
                    get_all(f, zp[t], lane);
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        S[t][r] = product(kt[r].f, f, S[t][r]);
                }
            }
            load_k(next);
            put_state(c - 1);
        }
    }
    if (to && has) {
#pragma unroll
        for (int t = 0; t < NC; ++t)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = Own::block(wb, r) * 16 + r4 + e;
                    if (d < a.dk)
                        to[d * ldw + 16 * t] = S[t][r][e];
                }
    }
}

} // namespace dl
