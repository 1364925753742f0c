// dl_layer_api.hip -- the C ABI of the state space layer's operators (short
// convolution, selective scan, their single-token forms, the norm with 8-bit
// output; include/deltalog.h): argument validation, workspace layouts, dispatch.
// Plain host code: kernels are reached only through the launchers declared in
// dl_internal.h.
#include "deltalog.h"
#include "dl_check.h"
#include "dl_internal.h"

namespace {

using namespace dl::host;

// Launches count work-items in 32 bits, 256 a workgroup.
constexpr long long kMostBlocks = 1LL << 24;
constexpr int kMostStates = 64, kMostChannels = 1 << 20;
constexpr long long kMostStride = 1LL << 22;

dl_status status(hipError_t e) { return e == hipSuccess ? DL_OK : DL_E_HIP; }

// The bytes of `rows` rows of `width` elements, `stride` apart.
size_t rows_bytes(long long rows, long long stride, long long width, size_t es)
{
    return rows > 0 ? static_cast<size_t>((rows - 1) * stride + width) * es : 0;
}

// Whether rows of `width` elements can be read four at a time.
bool vectors(const void *p, long long stride, size_t es) { return aligned(p, 4 * es) && stride % 4 == 0; }

// -------------------------------------------------------------- convolution --

dl_status check_conv(const dl_conv_desc *d)
{
    if (!d || !dtype_ok(d->dtype) || d->tokens < 0 || d->seqs < 1 || d->channels < 1)
        return DL_E_INVALID;
    if (d->taps < 2 || d->taps > 4 || d->channels > kMostChannels || d->tokens > (1 << 30) || d->seqs > (1 << 30))
        return DL_E_SHAPE;
    const long long groups = (d->channels + dl::kConvChannels - 1) / dl::kConvChannels;
    // (a step's rows are whole workgroups)
    if ((static_cast<long long>(d->tokens) + d->seqs) * ((groups + 255) / 256) >= kMostBlocks)
        return DL_E_SHAPE;
    return DL_OK;
}

// Tokens per run: long ones re-read less at their ends (W - 1 tokens of each) and
// leave fewer partial sums, short ones give more lanes.  us by the run's length, bf16,
// four taps, tokens x channels:
//                       4     8    16    32    64   128
//   forward 2048 x 2048 9.4   8.1  9.5  14.9  23.3
//          2756 x 12288 49.9  34.9 31.0 30.8  35.2
//          8192 x 4096  48.2  34.3 30.3 28.9  30.7
//         16384 x 4096  89.6  60.1 52.0 55.8  50.5
//   training 2048 x 2048 44.1 32.8 29.7 33.9  41.6  60.9   (forward by the rule)
//          2756 x 12288  254  171  128  111   108   98.5
//          8192 x 4096   256  165  118  99.8  84.8  93.1
//         16384 x 4096   465  326  234  193   170   155
int conv_run(const dl_conv_desc *d, bool backward)
{
    const long groups = (d->channels + dl::kConvChannels - 1) / dl::kConvChannels, lanes = backward ? 1 << 16 : 1 << 17;
    int run = backward ? 8 : 4, most = d->tokens * groups > 1L << 23 ? 64 : 32;
    most *= backward ? 2 : 1;
    while (run < most && d->tokens / (2 * run) * groups >= lanes)
        run *= 2;
    return run;
}
int conv_runs(const dl_conv_desc *d, bool backward)
{
    const int run = conv_run(d, backward);
    return (d->tokens + run - 1) / run;
}

dl_status conv_inputs(const dl_conv_desc *d, bool step, dl::ConvArgs &a, Span (&r)[4])
{
    const dl_status st = check_conv(d);
    if (st != DL_OK)
        return st;
    const long long C = d->channels, xs = d->x_stride ? d->x_stride : C;
    if ((d->tokens > 0 && !d->x) || !d->weight || xs < C)
        return DL_E_INVALID;
    if (!step && !d->cu_seqlens && d->tokens % d->seqs != 0)
        return DL_E_INVALID;
    if (xs > kMostStride) // a run's rows are addressed in 32 bits
        return DL_E_SHAPE;
    const size_t es = elem(d->dtype);
    if (!aligned(d->x, es) || !aligned(d->weight, 4) || !aligned(d->bias, 4) || !aligned(d->cu_seqlens, 4))
        return DL_E_ALIGN;
    a = dl::ConvArgs{};
    a.T = d->tokens;
    a.N = d->seqs;
    a.C = d->channels;
    a.W = d->taps;
    a.silu = d->silu != 0;
    a.cu = step ? nullptr : d->cu_seqlens;
    a.x = d->x;
    a.xs = xs;
    a.weight = d->weight;
    a.bias = d->bias;
    a.vec = vectors(d->x, xs, es) && d->channels % 4 == 0;
    r[0] = {d->x, rows_bytes(d->tokens, xs, C, es)};
    r[1] = {d->weight, static_cast<size_t>(C) * d->taps * 4};
    r[2] = {d->bias, static_cast<size_t>(C) * 4};
    r[3] = {a.cu, (static_cast<size_t>(d->seqs) + 1) * 4};
    return DL_OK;
}

// --------------------------------------------------------------------- scan --

dl_status check_ssm(const dl_ssm_desc *d)
{
    if (!d || !dtype_ok(d->dtype) || d->tokens < 0 || d->seqs < 1 || d->channels < 1 || d->states < 1 || d->groups < 1 ||
        d->channels % d->groups != 0)
        return DL_E_INVALID;
    if (d->states > kMostStates || d->channels > kMostChannels || d->tokens > (1 << 30) || d->seqs > (1 << 30))
        return DL_E_SHAPE;
    const long long tiles = static_cast<long long>(d->groups) *
                            ((d->channels / d->groups + dl::kSsmTile - 1) / dl::kSsmTile);
    // a workgroup (of 512) per sequence and tile, of which cuts add no more than a few
    // thousand; in one launch a thread per element of dB and dC and sixteen per one of
    // dA, dD and ddt_bias
    if (d->seqs * ((tiles + 7) / 8 * 8) >= kMostBlocks / 4 ||
        2LL * d->tokens * d->groups * d->states + 16LL * d->channels * (d->states + 2) >= kMostBlocks * 256 - 4096)
        return DL_E_SHAPE;
    return DL_OK;
}

int tiles_of(const dl_ssm_desc *d, int tile)
{
    return d->groups * ((d->channels / d->groups + tile - 1) / tile);
}

// Tokens per segment, or 0: sequences uncut.  Cut, every token is gone over twice
// (once for what its segment adds to the state), which pays where uncut ones leave
// most of the GPU idle.
//
// Forward: where the sequences' mean length says so, which one long sequence among short
// ones does not reach: 4096 tokens of 512 channels take 33 us alone, among fifteen
// sequences of 17 tokens 113, among 255 of them 182.  us, 16 states, bf16, by segment
// (uncut first):
//                     uncut   64   128   256   512  1024
//   512 x 64 channels  15.4  10.6  12.9  18.0
//   1024 x 512         26.1  18.0  13.8  18.4  28.2
//   1024 x 2048        27.2  59.8  40.1  31.4  29.4
//   4096 x 512         97               32.8  29.8
//   4096 x 2048       101                      95    89
//   2 x 2048 x 2048    52.4       159   114    90    78.3
//   16384 x 256       375     best 55
int ssm_forward_segment(const dl_ssm_desc *d)
{
    const long want = 256, wgs = static_cast<long>(tiles_of(d, dl::kSsmTile)) * d->seqs, each = d->tokens / d->seqs;
    if (wgs * 2 > want || each < 256)
        return 0;
    const long n = want / wgs < each / 64 ? want / wgs : each / 64;
    return static_cast<int>(((each + n - 1) / n + 63) / 64 * 64);
}

// Backward: a wave has four times the channels and eight times the work of a token, so
// that one long sequence among short ones is what a batch waits for.  As many tokens as
// fill the GPU if all are as long, whatever their lengths are (they are known on the
// device only: where none is longer the cut costs 5 to 15 us, where one is it gains most
// of the time), and not less than about sqrt(1.5 T), where a sequence's joins begin to
// cost more than its segments.  us of both passes:
//                           uncut    32    64    96   128   256   512
//   128 x 64 channels        45.8  27.9  35.7
//   512 x 64                  144  37.5  41.4  50.5  56.6  90.6
//   512 x 1024, 64 states     481   108   125   148   169   287
//   3 x 200 x 512, 64 states  206  85.8   106   132   157
//   4096 x 512               1067   162   107   110   107   131   189
//   1024 x 2048               301   120  95.2   105  99.8   126   189
//   2 x 2048 x 2048           583               255   227   219   302
//   40 x 100 + 2000, x 2048   800               473   423   423   478
//   255 x 17 + 4096, x 512   1330         420   423   420   428   487
//   16 x 64 x 512            35.9  45.3  41.4  41.3  40.9  40.5  40.8
//   16 x 300 x 2048           237               311   303   299   252
int ssm_backward_segment(const dl_ssm_desc *d)
{
    const long want = 512, T = d->tokens, tiles = tiles_of(d, dl::kSsmGradTile);
    const long full = (T * tiles + want - 1) / want;
    long seg = (full + 31) / 32 * 32;
    seg = seg < 32 ? 32 : seg;
    while (2 * seg * seg < 3 * T)
        seg += 32;
    return T < 128 || 2 * seg > T ? 0 : static_cast<int>(seg);
}

struct SsmSizes {
    int seg, bseg, slots, bslots;
    size_t states, sums, ahead, plain, bstates, bsums, part, bc;
    explicit SsmSizes(const dl_ssm_desc *d)
        : seg(ssm_forward_segment(d)), bseg(ssm_backward_segment(d)),
          slots(seg ? static_cast<int>(dl::ssm_slots(d->tokens, d->seqs, seg)) : d->seqs),
          bslots(bseg ? static_cast<int>(dl::ssm_slots(d->tokens, d->seqs, bseg)) : d->seqs)
    {
        const size_t C = d->channels, state = C * d->states * 4;
        states = seg ? up256(slots * state) : 0;
        sums = seg ? up256(slots * C * 4) : 0;
        ahead = up256(dl::ssm_slots(d->tokens, d->seqs, dl::kSsmBlock) * state);
        plain = d->z ? up256(d->tokens * C * 4) : 0;
        bstates = bseg ? up256(bslots * state) : 0;
        bsums = bseg ? up256(bslots * C * 4) : 0;
        part = up256(bslots * (state + 2 * C * 4));
        bc = up256(static_cast<size_t>(tiles_of(d, dl::kSsmGradTile) / d->groups) * d->tokens * d->groups * 2 * d->states * 4);
    }
    size_t forward() const { return states + sums + 256; } // never 0
    // the state ahead of every block, and y ahead of the gate
    size_t saved() const { return ahead + plain; }
    // dB and dC of every tile; dA, dD and dt_bias's gradient of every piece; the
    // segments' G and sums of delta
    size_t backward() const { return bc + part + bstates + bsums; }
};

dl_status ssm_inputs(const dl_ssm_desc *d, bool step, dl::SsmArgs &a, Span (&r)[9])
{
    const dl_status st = check_ssm(d);
    if (st != DL_OK)
        return st;
    const bool any = d->tokens > 0;
    if ((any && (!d->x || !d->dt || !d->b || !d->c)) || !d->a)
        return DL_E_INVALID;
    if (!step && !d->cu_seqlens && d->tokens % d->seqs != 0)
        return DL_E_INVALID;
    const long long C = d->channels, GS = static_cast<long long>(d->groups) * d->states;
    const long long xs = d->x_stride ? d->x_stride : C, dts = d->dt_stride ? d->dt_stride : C,
                    zs = d->z_stride ? d->z_stride : C, bs = d->b_stride ? d->b_stride : GS,
                    cs = d->c_stride ? d->c_stride : GS;
    if (xs < C || dts < C || zs < C || bs < GS || cs < GS)
        return DL_E_INVALID;
    // a stage's rows are addressed in 32 bits
    for (long long stride : {xs, dts, zs, bs, cs})
        if (stride > kMostStride)
            return DL_E_SHAPE;
    const size_t es = elem(d->dtype);
    for (const void *p : {d->x, d->dt, d->z, d->b, d->c})
        if (!aligned(p, es))
            return DL_E_ALIGN;
    if (!aligned(d->a, 4) || !aligned(d->d, 4) || !aligned(d->dt_bias, 4) || !aligned(d->cu_seqlens, 4))
        return DL_E_ALIGN;
    a = dl::SsmArgs{};
    a.T = d->tokens;
    a.N = d->seqs;
    a.C = d->channels;
    a.S = d->states;
    a.G = d->groups;
    a.CG = d->channels / d->groups;
    a.softplus = d->softplus != 0;
    a.cu = step ? nullptr : d->cu_seqlens;
    a.x = d->x;
    a.dt = d->dt;
    a.z = d->z;
    a.b = d->b;
    a.c = d->c;
    a.xs = xs;
    a.dts = dts;
    a.zs = zs;
    a.bs = bs;
    a.cs = cs;
    a.A = d->a;
    a.D = d->d;
    a.dt_bias = d->dt_bias;
    a.vec_x = vectors(d->x, xs, es) && vectors(d->dt, dts, es) && (!d->z || vectors(d->z, zs, es)) && a.CG % 4 == 0;
    a.vec_b = vectors(d->b, bs, es) && vectors(d->c, cs, es) && d->states % 4 == 0;
    r[0] = {d->x, rows_bytes(d->tokens, xs, C, es)};
    r[1] = {d->dt, rows_bytes(d->tokens, dts, C, es)};
    r[2] = {d->z, rows_bytes(d->tokens, zs, C, es)};
    r[3] = {d->b, rows_bytes(d->tokens, bs, GS, es)};
    r[4] = {d->c, rows_bytes(d->tokens, cs, GS, es)};
    r[5] = {d->a, static_cast<size_t>(C) * d->states * 4};
    r[6] = {d->d, static_cast<size_t>(C) * 4};
    r[7] = {d->dt_bias, static_cast<size_t>(C) * 4};
    r[8] = {a.cu, (static_cast<size_t>(d->seqs) + 1) * 4};
    return DL_OK;
}

} // namespace

extern "C" {

dl_status dl_short_conv(const dl_conv_desc *d, const void *initial, void *final_state, void *y, void *stream)
{
    dl::ConvArgs a;
    Span in[4];
    const dl_status st = conv_inputs(d, false, a, in);
    if (st != DL_OK)
        return st;
    if (d->tokens > 0 && !y)
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), row = static_cast<size_t>(d->channels) * es;
    if (!aligned(initial, es) || !aligned(final_state, es) || !aligned(y, es))
        return DL_E_ALIGN;
    const size_t states = static_cast<size_t>(d->seqs) * (d->taps - 1) * row;
    const Span w[2] = {{y, d->tokens * row}, {final_state, states}};
    const Span r[5] = {in[0], in[1], in[2], in[3], {initial, states}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.init = initial;
    a.fin = final_state;
    a.y = y;
    a.vec = a.vec && aligned(initial, 4 * es) && aligned(final_state, 4 * es) && aligned(y, 4 * es);
    a.run = conv_run(d, false);
    a.runs = conv_runs(d, false);
    return status(dl::launch_short_conv(d->dtype, a, static_cast<hipStream_t>(stream)));
}

size_t dl_short_conv_workspace_bytes(const dl_conv_desc *d)
{
    if (check_conv(d) != DL_OK)
        return 0;
    return up256(static_cast<size_t>(conv_runs(d, true)) * d->channels * (d->taps + 1) * 4) + 256; // never 0
}

dl_status dl_short_conv_backward(const dl_conv_desc *d, const void *initial, const void *dy, const void *d_final,
                                 void *dx, float *dweight, float *dbias, void *d_initial, void *workspace, void *stream)
{
    dl::ConvArgs a;
    Span in[4];
    const dl_status st = conv_inputs(d, false, a, in);
    if (st != DL_OK)
        return st;
    if ((d->tokens > 0 && !dx) || ((dweight || dbias) && !workspace))
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), row = static_cast<size_t>(d->channels) * es;
    if (!aligned(initial, es) || !aligned(dy, es) || !aligned(d_final, es) || !aligned(dx, es) || !aligned(dweight, 4) ||
        !aligned(dbias, 4) || !aligned(d_initial, es) || !aligned(workspace, 256))
        return DL_E_ALIGN;
    const size_t states = static_cast<size_t>(d->seqs) * (d->taps - 1) * row;
    const Span w[5] = {{dx, d->tokens * row},
                       {dweight, in[1].bytes},
                       {dbias, in[2].bytes},
                       {d_initial, states},
                       {dweight || dbias ? workspace : nullptr, dl_short_conv_workspace_bytes(d)}};
    const Span r[7] = {in[0], in[1], in[2], in[3], {initial, states}, {dy, d->tokens * row}, {d_final, states}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.init = initial;
    a.dy = dy;
    a.dfin = d_final;
    a.dx = dx;
    a.dinit = d_initial;
    a.d_weight = dweight;
    a.d_bias = dbias;
    for (const void *p : {initial, dy, d_final, static_cast<const void *>(dx), static_cast<const void *>(d_initial)})
        a.vec = a.vec && aligned(p, 4 * es);
    a.run = conv_run(d, true);
    a.runs = conv_runs(d, true);
    if (dweight)
        a.part_w = static_cast<float *>(workspace);
    if (dbias)
        a.part_b = static_cast<float *>(workspace) + static_cast<size_t>(a.runs) * d->channels * d->taps;
    return status(dl::launch_short_conv_backward(d->dtype, a, static_cast<hipStream_t>(stream)));
}

dl_status dl_short_conv_step(const dl_conv_desc *d, void *state, const int *state_rows, int n_state_rows, void *y,
                             void *stream)
{
    dl::ConvArgs a;
    Span in[4];
    const dl_status st = conv_inputs(d, true, a, in);
    if (st != DL_OK)
        return st;
    if (d->tokens == 0)
        return DL_OK;
    if (!y || !state || n_state_rows < 1 || (!state_rows && n_state_rows < d->tokens))
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), row = static_cast<size_t>(d->channels) * es;
    if (!aligned(state, es) || !aligned(y, es) || !aligned(state_rows, 4))
        return DL_E_ALIGN;
    const Span w[2] = {{y, d->tokens * row}, {state, static_cast<size_t>(n_state_rows) * (d->taps - 1) * row}};
    const Span r[4] = {in[0], in[1], in[2], {state_rows, static_cast<size_t>(d->tokens) * 4}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.state = state;
    a.rows = state_rows;
    a.n_rows = n_state_rows;
    a.y = y;
    a.vec = a.vec && aligned(state, 4 * es) && aligned(y, 4 * es);
    return status(dl::launch_short_conv_step(d->dtype, a, static_cast<hipStream_t>(stream)));
}

size_t dl_ssm_workspace_bytes(const dl_ssm_desc *d) { return check_ssm(d) == DL_OK ? SsmSizes(d).forward() : 0; }

size_t dl_ssm_saved_bytes(const dl_ssm_desc *d) { return check_ssm(d) == DL_OK ? SsmSizes(d).saved() : 0; }

size_t dl_ssm_backward_workspace_bytes(const dl_ssm_desc *d)
{
    return check_ssm(d) == DL_OK ? SsmSizes(d).backward() : 0;
}

dl_status dl_ssm_scan(const dl_ssm_desc *d, const float *initial, float *final_state, void *y, void *saved,
                      void *workspace, void *stream)
{
    dl::SsmArgs a;
    Span in[9];
    const dl_status st = ssm_inputs(d, false, a, in);
    if (st != DL_OK)
        return st;
    if (!workspace || (d->tokens > 0 && !y))
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), C = d->channels;
    if (!aligned(initial, 4) || !aligned(final_state, 4) || !aligned(y, es) || !aligned(saved, 256) ||
        !aligned(workspace, 256))
        return DL_E_ALIGN;
    const SsmSizes z(d);
    const size_t states = d->seqs * C * d->states * 4;
    const Span w[4] = {{y, d->tokens * C * es}, {final_state, states}, {saved, z.saved()}, {workspace, z.forward()}};
    const Span r[10] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], {initial, states}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.init = initial;
    a.fin = final_state;
    a.y = y;
    a.vec_x = a.vec_x && aligned(y, 4 * es) && d->channels % 4 == 0;
    a.saved = static_cast<float *>(saved);
    a.plain = saved ? reinterpret_cast<float *>(static_cast<char *>(saved) + z.ahead) : nullptr;
    a.seg = z.seg;
    a.slots = z.slots;
    a.tiles = tiles_of(d, dl::kSsmTile);
    a.seg_h = static_cast<float *>(workspace);
    a.seg_d = reinterpret_cast<float *>(static_cast<char *>(workspace) + z.states);
    return status(dl::launch_ssm_scan(d->dtype, a, static_cast<hipStream_t>(stream)));
}

dl_status dl_ssm_scan_backward(const dl_ssm_desc *d, const void *saved, const void *dy, const float *d_final, void *dx,
                               void *ddt, void *dz, void *db, void *dc, float *da, float *dd, float *ddt_bias,
                               float *d_initial, void *workspace, void *stream)
{
    dl::SsmArgs a;
    Span in[9];
    const dl_status st = ssm_inputs(d, false, a, in);
    if (st != DL_OK)
        return st;
    const bool any = d->tokens > 0;
    if (!workspace || !saved || !da || (any && (!dy || !dx || !ddt || !db || !dc || (d->z && !dz))) || (!d->z && dz) ||
        (!d->d && dd) || (!d->dt_bias && ddt_bias))
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), C = d->channels, T = d->tokens;
    for (const void *p : {dy, static_cast<const void *>(dx), static_cast<const void *>(ddt), static_cast<const void *>(dz),
                          static_cast<const void *>(db), static_cast<const void *>(dc)})
        if (!aligned(p, es))
            return DL_E_ALIGN;
    if (!aligned(d_final, 4) || !aligned(da, 4) || !aligned(dd, 4) || !aligned(ddt_bias, 4) || !aligned(d_initial, 4) ||
        !aligned(saved, 256) || !aligned(workspace, 256))
        return DL_E_ALIGN;
    const SsmSizes z(d);
    const size_t states = d->seqs * C * d->states * 4, bc = T * d->groups * d->states * es;
    const Span w[10] = {{dx, T * C * es}, {ddt, T * C * es}, {dz, T * C * es}, {db, bc}, {dc, bc}, {da, in[5].bytes},
                        {dd, C * 4}, {ddt_bias, C * 4}, {d_initial, states}, {workspace, z.backward()}};
    const Span r[12] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], {saved, z.saved()},
                        {dy, T * C * es}, {d_final, states}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.saved = static_cast<float *>(const_cast<void *>(saved));
    a.plain = reinterpret_cast<float *>(static_cast<char *>(const_cast<void *>(saved)) + z.ahead);
    a.dy = dy;
    a.dfin = d_final;
    a.dx = dx;
    a.ddt = ddt;
    a.dz = dz;
    a.db = db;
    a.dc = dc;
    a.d_A = da;
    a.d_D = dd;
    a.d_bias = ddt_bias;
    a.dinit = d_initial;
    a.vec_x = a.vec_x && aligned(dy, 4 * es) && aligned(dx, 4 * es) && aligned(ddt, 4 * es) && aligned(dz, 4 * es) &&
              d->channels % 4 == 0;
    a.seg = z.bseg;
    a.slots = z.bslots;
    a.tiles = tiles_of(d, dl::kSsmGradTile);
    char *p = static_cast<char *>(workspace);
    a.part_bc = reinterpret_cast<float *>(p);
    a.part_a = reinterpret_cast<float *>(p += z.bc);
    a.seg_h = reinterpret_cast<float *>(p += z.part);
    a.seg_d = reinterpret_cast<float *>(p + z.bstates);
    dl::SsmArgs ahead = a;
    ahead.tiles = tiles_of(d, dl::kSsmTile);
    return status(dl::launch_ssm_backward(d->dtype, ahead, a, static_cast<hipStream_t>(stream)));
}

dl_status dl_ssm_step(const dl_ssm_desc *d, float *state, const int *state_rows, int n_state_rows, void *y, void *stream)
{
    dl::SsmArgs a;
    Span in[9];
    const dl_status st = ssm_inputs(d, true, a, in);
    if (st != DL_OK)
        return st;
    // up to sixteen lanes a channel, whole workgroups a row
    if (static_cast<long long>(d->tokens) * ((16LL * d->channels + 255) / 256) >= kMostBlocks)
        return DL_E_SHAPE;
    if (d->tokens == 0)
        return DL_OK;
    if (!y || !state || n_state_rows < 1 || (!state_rows && n_state_rows < d->tokens))
        return DL_E_INVALID;
    const size_t es = elem(d->dtype), C = d->channels;
    if (!aligned(state, 4) || !aligned(y, es) || !aligned(state_rows, 4))
        return DL_E_ALIGN;
    const Span w[2] = {{y, d->tokens * C * es}, {state, n_state_rows * C * d->states * 4}};
    const Span r[9] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7],
                       {state_rows, static_cast<size_t>(d->tokens) * 4}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.state = state;
    a.rows = state_rows;
    a.n_rows = n_state_rows;
    a.y = y;
    a.vec_s = aligned(state, 16) && aligned(d->a, 16) && d->states % 4 == 0;
    return status(dl::launch_ssm_step(d->dtype, a, static_cast<hipStream_t>(stream)));
}

dl_status dl_residual_norm_quant(int rows, int D, dl_dtype dtype, const float *x, const void *y, const float *scale,
                               const float *weight, float eps, float *x_out, int group, void *h, float *h_scale,
                               void *stream)
{
    if (rows < 0 || !dtype_ok(dtype) || !eps_ok(eps))
        return DL_E_INVALID;
    if (D < 1 || D > 16384 || (group != 0 && (group != 128 || D % 128 != 0)))
        return DL_E_SHAPE;
    if (rows == 0)
        return DL_OK;
    if (!x || !h || !h_scale || (y && !x_out) || (!y && (x_out || scale)))
        return DL_E_INVALID;
    if (!aligned(x, 4) || !aligned(x_out, 4) || !aligned(scale, 4) || !aligned(weight, 4) || !aligned(h_scale, 4) ||
        !aligned(y, elem(dtype)))
        return DL_E_ALIGN;
    // whole groups are a wave's vectors
    if (group && (!aligned(x, 16) || !aligned(x_out, 16) || !aligned(y, 16) || !aligned(h, 16)))
        return DL_E_ALIGN;
    const size_t n = static_cast<size_t>(rows) * D;
    const Span w[3] = {{x_out, n * 4}, {h, n}, {h_scale, static_cast<size_t>(rows) * (group ? D / group : 1) * 4}};
    const Span r[4] = {{x_out == x ? nullptr : x, n * 4},
                       {y, n * elem(dtype)},
                       {scale, static_cast<size_t>(D) * 4},
                       {weight, static_cast<size_t>(D) * 4}};
    if (clash(w, r))
        return DL_E_INVALID;
    dl::NormFp8Args a{};
    a.rows = rows;
    a.D = D;
    a.group = group ? group : D;
    a.x = x;
    a.y = y;
    a.scale = scale;
    a.weight = weight;
    a.eps = eps;
    a.x_out = x_out;
    a.h = static_cast<unsigned char *>(h);
    a.h_scale = h_scale;
    return status(dl::launch_residual_norm_fp8(dtype, a, static_cast<hipStream_t>(stream)));
}

} // extern "C"
