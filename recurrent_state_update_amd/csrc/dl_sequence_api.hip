// dl_sequence_api.hip -- the C ABI of the sequence operators (the scan and the
// norms around it, include/deltalog.h): argument validation, workspace
// layouts, dispatch.  Plain host code, like dl_api.hip: kernels are reached
// only through the launchers declared in dl_internal.h.
#include "deltalog.h"
#include "dl_check.h"
#include "dl_internal.h"

namespace {

using namespace dl::host;

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Launches count work-items in 32 bits: at most 512 per chunk and head, and
// 32 d_v per sequence and head.
constexpr long long kMostStride = 1LL << 22;
constexpr long kMostSlotHeads = 1L << 22, kMostSeqHeads = 1L << 19;

dl_status check_sizes(const dl_scan_desc *d)
{
    if (!d || d->op < DL_OP_GDN || d->op > DL_OP_RWKV6 || !dtype_ok(d->in_dtype) || d->tokens < 0 || d->seqs < 1 ||
        d->H < 1)
        return DL_E_INVALID;
    if (!dim_ok(d->d_k) || !dim_ok(d->d_v))
        return DL_E_SHAPE;
    if (static_cast<long>(d->seqs) * d->H > kMostSeqHeads ||
        dl::scan_slots(d->tokens, d->seqs) * d->H > kMostSlotHeads)
        return DL_E_SHAPE;
    return DL_OK;
}

struct ScanSizes {
    size_t slot_heads, ops, states, rows_dv, db, du;
    long segment, segments; // of the carries; 0: uncut
    size_t seg_s, seg_m;
    explicit ScanSizes(const dl_scan_desc *d)
        : slot_heads(static_cast<size_t>(dl::scan_slots(d->tokens, d->seqs)) * d->H),
          ops(up256(slot_heads * dl::scan_op_bytes(dl::scan_planes(d->op, d->in_dtype), dl::scan_keys(d->d_k)))),
          states(up256(slot_heads * d->d_k * d->d_v * 4)),
          rows_dv(d->op == DL_OP_RWKV6 ? 0 : up256(slot_heads * dl::kScanChunk * d->d_v * 4)),
          db(d->op == DL_OP_RWKV6 ? 0 : up256(slot_heads * (d->d_v / 16) * dl::kScanChunk * 4)),
          du(d->op == DL_OP_RWKV6 ? up256(slot_heads * d->d_k * 4) : 0),
          segment(dl::scan_segment(d->tokens, d->seqs, d->H, d->d_v)),
          segments(segment ? dl::scan_segments(d->tokens, d->seqs, segment) : 0),
          seg_s(up256(static_cast<size_t>(segments) * d->H * d->d_k * d->d_v * 4)),
          seg_m(up256(static_cast<size_t>(segments) * d->H * d->d_k * d->d_k * 4))
    {
    }
    size_t forward() const { return ops + seg_s + seg_m; }
    size_t saved() const { return states + rows_dv; }
    // What both passes keep at the workspace's front; returns its end.
    char *place(dl::ScanArgs &a, void *workspace) const
    {
        a.ops = static_cast<char *>(workspace);
        a.seg = static_cast<int>(segment);
        a.segments = static_cast<int>(segments);
        a.seg_s = reinterpret_cast<float *>(a.ops + ops);
        a.seg_m = reinterpret_cast<float *>(a.ops + ops + seg_s);
        return a.ops + forward();
    }
    size_t backward() const { return forward() + states + rows_dv + db + du; }
};

// Checks what both directions read, and fills their part of `a`.
dl_status scan_inputs(const dl_scan_desc *d, dl::ScanArgs &a, Span (&r)[7])
{
    const dl_status st = check_sizes(d);
    if (st != DL_OK)
        return st;
    const bool any = d->tokens > 0, delta = d->op != DL_OP_RWKV6;
    if (any && (!d->q || !d->k || !d->v || !d->log_decay || (delta && !d->beta)))
        return DL_E_INVALID;
    if (!delta && !d->u)
        return DL_E_INVALID;
    if (!d->cu_seqlens && d->tokens % d->seqs != 0)
        return DL_E_INVALID;
    const long long kw = static_cast<long long>(d->H) * d->d_k, vw = static_cast<long long>(d->H) * d->d_v;
    const long long qs = d->q_stride ? d->q_stride : kw, ks = d->k_stride ? d->k_stride : kw,
                    vs = d->v_stride ? d->v_stride : vw;
    if (qs < kw || ks < kw || vs < vw)
        return DL_E_INVALID;
    // a chunk's rows are addressed in 32 bits
    if (qs > kMostStride || ks > kMostStride || vs > kMostStride)
        return DL_E_SHAPE;
    const size_t es = elem(d->in_dtype), T = d->tokens, last = any ? T - 1 : 0;
    if (!aligned(d->q, es) || !aligned(d->k, es) || !aligned(d->v, es) || !aligned(d->beta, 4) ||
        !aligned(d->log_decay, 4) || !aligned(d->u, 4) || !aligned(d->cu_seqlens, 4))
        return DL_E_ALIGN;
    a = dl::ScanArgs{};
    a.T = d->tokens;
    a.N = d->seqs;
    a.H = d->H;
    a.dk = d->d_k;
    a.dv = d->d_v;
    a.slots = static_cast<int>(dl::scan_slots(d->tokens, d->seqs));
    a.cu = d->cu_seqlens;
    a.q = d->q;
    a.k = d->k;
    a.v = d->v;
    a.qs = qs;
    a.ks = ks;
    a.vs = vs;
    a.beta = delta ? d->beta : nullptr;
    a.ld = d->log_decay;
    a.u = delta ? nullptr : d->u;
    r[0] = {d->q, any ? (last * qs + kw) * es : 0};
    r[1] = {d->k, any ? (last * ks + kw) * es : 0};
    r[2] = {d->v, any ? (last * vs + vw) * es : 0};
    r[3] = {a.beta, T * d->H * 4};
    r[4] = {d->log_decay, T * (d->op == DL_OP_GDN ? d->H : kw) * 4};
    r[5] = {a.u, static_cast<size_t>(kw) * 4};
    r[6] = {d->cu_seqlens, (static_cast<size_t>(d->seqs) + 1) * 4};
    return DL_OK;
}

dl_status launch_scan(const dl_scan_desc *d, bool backward, const dl::ScanArgs &a, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch (d->op) {
    case DL_OP_GDN: e = dl::launch_scan_gdn(d->in_dtype, backward, a, st); break;
    case DL_OP_KDA: e = dl::launch_scan_kda(d->in_dtype, backward, a, st); break;
    default: e = dl::launch_scan_rwkv6(d->in_dtype, backward, a, st); break;
    }
    return e == hipSuccess ? DL_OK : DL_E_HIP;
}

// Elements that the gated norm takes, below 2^33.  (rows and H have 31 bits each:
// their product with d would pass 64.)
bool gated_size_ok(int rows, int H, int d) { return static_cast<long long>(rows) * H < (1LL << 33) / d; }

constexpr long kNormBlocks = 1024; // of a backward pass: four workgroups per CU, and as many partial sums per column

int gated_blocks(long rows, long H, int d)
{
    const long b = (rows * H * (d / 8) + 255) / 256;
    return static_cast<int>(b < 1 ? 1 : b < kNormBlocks ? b : kNormBlocks);
}

int residual_blocks(long rows) { return static_cast<int>(rows < 1 ? 1 : rows < kNormBlocks ? rows : kNormBlocks); }

dl_status gated_inputs(int rows, int H, int d, int o_dtype, int dtype, const void *o, const void *gate,
                       long long gate_stride, const float *weight, float eps, dl::GatedNormArgs &a, Span (&r)[3])
{
    if (rows < 0 || H < 1 || !dtype_ok(o_dtype) || !dtype_ok(dtype) || !eps_ok(eps))
        return DL_E_INVALID;
    if (!dim_ok(d) || !gated_size_ok(rows, H, d))
        return DL_E_SHAPE;
    const long long width = static_cast<long long>(H) * d, gs = gate_stride ? gate_stride : width;
    if ((rows > 0 && (!o || !gate)) || gs < width)
        return DL_E_INVALID;
    if (!aligned(o, elem(o_dtype)) || !aligned(gate, elem(dtype)) || !aligned(weight, 4))
        return DL_E_ALIGN;
    a = dl::GatedNormArgs{};
    a.units = static_cast<long>(rows) * H;
    a.H = H;
    a.d = d;
    a.o = o;
    a.gate = gate;
    a.gate_stride = gs;
    a.weight = weight;
    a.eps = eps;
    a.blocks = gated_blocks(rows, H, d);
    r[0] = {o, rows * static_cast<size_t>(width) * elem(o_dtype)};
    r[1] = {gate, rows > 0 ? ((rows - 1) * static_cast<size_t>(gs) + width) * elem(dtype) : 0};
    r[2] = {weight, static_cast<size_t>(d) * 4};
    return DL_OK;
}

} // namespace

extern "C" {

size_t dl_scan_workspace_bytes(const dl_scan_desc *d)
{
    return check_sizes(d) == DL_OK ? ScanSizes(d).forward() : 0;
}

size_t dl_scan_saved_bytes(const dl_scan_desc *d)
{
    return check_sizes(d) == DL_OK ? ScanSizes(d).saved() : 0;
}

size_t dl_scan_backward_workspace_bytes(const dl_scan_desc *d)
{
    return check_sizes(d) == DL_OK ? ScanSizes(d).backward() : 0;
}

dl_status dl_scan(const dl_scan_desc *d, const float *initial, float *final_state, const int *state_rows,
                  int n_state_rows, void *o, void *saved, void *workspace, void *stream)
{
    dl::ScanArgs a;
    Span in[7];
    const dl_status st = scan_inputs(d, a, in);
    if (st != DL_OK)
        return st;
    if (!workspace || (d->tokens > 0 && !o) || (state_rows && n_state_rows < 1))
        return DL_E_INVALID;
    if (!aligned(initial, 16) || !aligned(final_state, 16) || !aligned(o, elem(d->in_dtype)) ||
        !aligned(saved, 256) || !aligned(workspace, 256) || !aligned(state_rows, 4))
        return DL_E_ALIGN;
    const ScanSizes z(d);
    const size_t rows = state_rows ? n_state_rows : d->seqs;
    const size_t states = rows * d->H * d->d_k * d->d_v * 4;
    const Span w[4] = {{o, static_cast<size_t>(d->tokens) * d->H * d->d_v * elem(d->in_dtype)},
                       {final_state, states},
                       {saved, z.saved()},
                       {workspace, z.forward()}};
    const Span r[9] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6],
                       {initial == final_state ? nullptr : initial, states},
                       {state_rows, static_cast<size_t>(d->seqs) * 4}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.init = initial;
    a.fin = final_state;
    a.rows = state_rows;
    a.nrows = n_state_rows;
    a.o = o;
    z.place(a, workspace);
    if (saved) {
        a.save_s = static_cast<float *>(saved);
        a.save_e = reinterpret_cast<float *>(static_cast<char *>(saved) + z.states);
    }
    return launch_scan(d, false, a, stream);
}

dl_status dl_scan_backward(const dl_scan_desc *d, const void *saved, const void *d_o, const float *d_final,
                           void *dq, void *dk, void *dv, float *dbeta, float *dlog_decay, float *du,
                           float *d_initial, void *workspace, void *stream)
{
    dl::ScanArgs a;
    Span in[7];
    const dl_status st = scan_inputs(d, a, in);
    if (st != DL_OK)
        return st;
    const bool delta = d->op != DL_OP_RWKV6;
    if (!workspace || !saved || (!delta && !du))
        return DL_E_INVALID;
    if (d->tokens > 0 && (!dq || !dk || !dv || !dlog_decay || (delta && !dbeta)))
        return DL_E_INVALID;
    const size_t es = elem(d->in_dtype);
    if (!aligned(saved, 256) || !aligned(workspace, 256) || !aligned(d_o, es) || !aligned(d_final, 16) ||
        !aligned(dq, es) || !aligned(dk, es) || !aligned(dv, es) || !aligned(dbeta, 4) || !aligned(dlog_decay, 4) ||
        !aligned(du, 4) || !aligned(d_initial, 16))
        return DL_E_ALIGN;
    const ScanSizes z(d);
    const size_t TH = static_cast<size_t>(d->tokens) * d->H;
    const size_t states = static_cast<size_t>(d->seqs) * d->H * d->d_k * d->d_v * 4;
    const Span w[8] = {{dq, TH * d->d_k * es},
                       {dk, TH * d->d_k * es},
                       {dv, TH * d->d_v * es},
                       {delta ? dbeta : nullptr, TH * 4},
                       {dlog_decay, in[4].bytes},
                       {delta ? nullptr : du, static_cast<size_t>(d->H) * d->d_k * 4},
                       {d_initial, states},
                       {workspace, z.backward()}};
    const Span r[10] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], {saved, z.saved()},
                        {d_o, TH * d->d_v * es}, {d_final, states}};
    if (clash(w, r))
        return DL_E_INVALID;
    a.save_s = static_cast<float *>(const_cast<void *>(saved));
    a.save_e = reinterpret_cast<float *>(static_cast<char *>(const_cast<void *>(saved)) + z.states);
    a.d_o = d_o;
    a.dfin = d_final;
    a.d_q = dq;
    a.d_k = dk;
    a.d_v = dv;
    a.d_beta = dbeta;
    a.d_ld = dlog_decay;
    a.d_u = du;
    a.dinit = d_initial;
    char *p = z.place(a, workspace);
    a.w_ds = reinterpret_cast<float *>(p);
    a.w_z = reinterpret_cast<float *>(p += z.states);
    a.w_db = reinterpret_cast<float *>(p += z.rows_dv);
    a.w_du = reinterpret_cast<float *>(p += z.db);
    return launch_scan(d, true, a, stream);
}

dl_status dl_gated_norm(int rows, int H, int d, dl_dtype o_dtype, dl_dtype dtype, const void *o,
                        const void *gate, long long gate_stride, const float *weight, float eps, void *y,
                        void *stream)
{
    dl::GatedNormArgs a;
    Span in[3];
    const dl_status st = gated_inputs(rows, H, d, o_dtype, dtype, o, gate, gate_stride, weight, eps, a, in);
    if (st != DL_OK)
        return st;
    if (rows == 0)
        return DL_OK;
    if (!y)
        return DL_E_INVALID;
    if (!aligned(y, elem(dtype)))
        return DL_E_ALIGN;
    // a lane reads its columns of o and gate before it writes them in y
    const bool over_o = y == o && o_dtype == dtype;
    const bool over_gate = y == gate && a.gate_stride == static_cast<long>(H) * d;
    const Span w[1] = {{y, static_cast<size_t>(rows) * H * d * elem(dtype)}};
    const Span r[3] = {{over_o ? nullptr : o, in[0].bytes}, {over_gate ? nullptr : gate, in[1].bytes}, in[2]};
    if (clash(w, r))
        return DL_E_INVALID;
    a.y = y;
    return dl::launch_gated_norm(o_dtype, dtype, false, a, static_cast<hipStream_t>(stream)) == hipSuccess ? DL_OK
                                                                                                        : DL_E_HIP;
}

size_t dl_gated_norm_workspace_bytes(int rows, int H, int d)
{
    if (rows < 0 || H < 1 || !dim_ok(d) || !gated_size_ok(rows, H, d))
        return 0;
    return up256(static_cast<size_t>(gated_blocks(rows, H, d)) * d * 4);
}

dl_status dl_gated_norm_backward(int rows, int H, int d, dl_dtype o_dtype, dl_dtype dtype, const void *o,
                                 const void *gate, long long gate_stride, const float *weight, float eps,
                                 const void *dy, void *d_o, void *d_gate, float *d_weight, void *workspace,
                                 void *stream)
{
    dl::GatedNormArgs a;
    Span in[3];
    const dl_status st = gated_inputs(rows, H, d, o_dtype, dtype, o, gate, gate_stride, weight, eps, a, in);
    if (st != DL_OK)
        return st;
    if ((rows > 0 && (!dy || !d_o || !d_gate)) || (d_weight && !workspace))
        return DL_E_INVALID;
    if (!aligned(dy, elem(dtype)) || !aligned(d_o, elem(o_dtype)) || !aligned(d_gate, elem(dtype)) ||
        !aligned(d_weight, 4) || !aligned(workspace, 256))
        return DL_E_ALIGN;
    const size_t n = static_cast<size_t>(rows) * H * d;
    const Span w[4] = {{d_o, n * elem(o_dtype)},
                       {d_gate, n * elem(dtype)},
                       {d_weight, static_cast<size_t>(d) * 4},
                       {d_weight ? workspace : nullptr, dl_gated_norm_workspace_bytes(rows, H, d)}};
    const Span r[4] = {in[0], in[1], in[2], {dy, n * elem(dtype)}};
    if (clash(w, r))
        return DL_E_INVALID;
    if (rows == 0 && !d_weight)
        return DL_OK;
    a.dy = dy;
    a.d_o = d_o;
    a.d_gate = d_gate;
    a.d_weight = d_weight;
    a.partial = static_cast<float *>(workspace);
    return dl::launch_gated_norm(o_dtype, dtype, true, a, static_cast<hipStream_t>(stream)) == hipSuccess ? DL_OK
                                                                                                       : DL_E_HIP;
}

dl_status dl_residual_norm(int rows, int D, dl_dtype dtype, const float *x, const void *y, const float *scale,
                           const float *weight, float eps, float *x_out, void *h, void *stream)
{
    if (rows < 0 || !dtype_ok(dtype) || !eps_ok(eps))
        return DL_E_INVALID;
    if (D < 1 || D > 16384)
        return DL_E_SHAPE;
    if (rows == 0)
        return DL_OK;
    if (!x || !h || (y && !x_out) || (!y && (x_out || scale)))
        return DL_E_INVALID;
    if (!aligned(x, 4) || !aligned(x_out, 4) || !aligned(scale, 4) || !aligned(weight, 4) ||
        !aligned(y, elem(dtype)) || !aligned(h, elem(dtype)))
        return DL_E_ALIGN;
    const size_t n = static_cast<size_t>(rows) * D;
    const Span w[2] = {{x_out, n * 4}, {h, n * elem(dtype)}};
    const Span r[4] = {{x_out == x ? nullptr : x, n * 4},
                       {y, n * elem(dtype)},
                       {scale, static_cast<size_t>(D) * 4},
                       {weight, static_cast<size_t>(D) * 4}};
    if (clash(w, r))
        return DL_E_INVALID;
    dl::ResidualNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.x = x;
    a.y = y;
    a.scale = scale;
    a.weight = weight;
    a.eps = eps;
    a.x_out = x_out;
    a.h = h;
    return dl::launch_residual_norm(dtype, false, a, static_cast<hipStream_t>(stream)) == hipSuccess ? DL_OK
                                                                                                   : DL_E_HIP;
}

size_t dl_residual_norm_workspace_bytes(int rows, int D)
{
    if (rows < 0 || D < 1 || D > 16384)
        return 0;
    return up256(static_cast<size_t>(residual_blocks(rows)) * 2 * D * 4);
}

dl_status dl_residual_norm_backward(int rows, int D, dl_dtype dtype, const float *x_out, const void *y,
                                    const float *scale, const float *weight, float eps,
                                    const float *d_x_out, const void *d_h, float *d_x, void *d_y,
                                    float *d_scale, float *d_weight, void *workspace, void *stream)
{
    if (rows < 0 || !dtype_ok(dtype) || !eps_ok(eps))
        return DL_E_INVALID;
    if (D < 1 || D > 16384)
        return DL_E_SHAPE;
    if (rows > 0 && (!x_out || !d_x || (scale && d_y && !y)))
        return DL_E_INVALID;
    if ((d_scale && (!scale || (rows > 0 && !d_y))) || ((d_scale || d_weight) && !workspace))
        return DL_E_INVALID;
    if (!aligned(x_out, 4) || !aligned(d_x_out, 4) || !aligned(d_x, 4) || !aligned(scale, 4) ||
        !aligned(weight, 4) || !aligned(d_scale, 4) || !aligned(d_weight, 4) || !aligned(y, elem(dtype)) ||
        !aligned(d_h, elem(dtype)) || !aligned(d_y, elem(dtype)) || !aligned(workspace, 256))
        return DL_E_ALIGN;
    const size_t n = static_cast<size_t>(rows) * D, row = static_cast<size_t>(D) * 4;
    const Span w[5] = {{d_x, n * 4},
                       {d_y, n * elem(dtype)},
                       {d_scale, row},
                       {d_weight, row},
                       {d_scale || d_weight ? workspace : nullptr, dl_residual_norm_workspace_bytes(rows, D)}};
    const Span r[6] = {{x_out, n * 4}, {scale && d_y ? y : nullptr, n * elem(dtype)}, {scale, row}, {weight, row},
                       {d_x_out == d_x ? nullptr : d_x_out, n * 4}, {d_h, n * elem(dtype)}};
    if (clash(w, r))
        return DL_E_INVALID;
    if (rows == 0 && !d_scale && !d_weight)
        return DL_OK;
    dl::ResidualNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.x = x_out;
    a.y = y;
    a.scale = scale;
    a.weight = weight;
    a.eps = eps;
    a.d_x_out = d_x_out;
    a.d_h = d_h;
    a.d_x = d_x;
    a.d_y = d_y;
    a.d_scale = d_scale;
    a.d_weight = d_weight;
    a.partial = static_cast<float *>(workspace);
    a.blocks = residual_blocks(rows);
    return dl::launch_residual_norm(dtype, true, a, static_cast<hipStream_t>(stream)) == hipSuccess ? DL_OK
                                                                                                  : DL_E_HIP;
}

} // extern "C"
