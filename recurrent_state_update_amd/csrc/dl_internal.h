// dl_internal.h -- declarations shared by the host API and the kernel files of
// libdeltalog.  Not installed; the public interface is include/deltalog.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace dl {

enum Op : int { GDN = 0, KDA = 1, RWKV6 = 2 };
enum DType : int { F32 = 0, BF16 = 1 };

// What one launch of the step kernel does with a tile of the state.
enum Mode : int {
    APPEND = 0,  // two-stage append phase: read S-bar, outputs + b_t, no state write
    MERGE = 1,   // two-stage merge phase: as APPEND, then fold all M entries, write S-bar
    EAGER = 2,   // eager baseline: decay, delta rule, rank-1 update, write state
    FOLD = 3,    // standalone merge: fold the n pending entries, write S-bar
    FAPPEND = 4, // one-launch append phase (replay coefficients computed in place)
    FMERGE = 5,  // one-launch merge phase
    SSTEP = 6,   // one-launch step with per-slot logs: each slot appends or merges
    SFOLD = 7    // standalone merge with per-slot logs (one slot or all)
};

// Byte offsets of the log and coefficient arrays inside the workspace.
// Each segment starts on a 256-byte boundary.
struct Layout {
    size_t a_off;   // a-log      [B*H, M, d_k]  input dtype (a_j = k_j)
    size_t b_off;   // b-log      [B*H, M, d_v]  fp32 (delta rule) / input dtype (RWKV6)
    size_t L_off;   // Lambda-log [B*H, M] (GDN) or [B*H, M, d_k] fp32
    size_t c_off;   // coef       [B*H, cstride] fp32: c^q_0..M-1, c^k_0..M-1, kappa
    size_t t_off;   // slot phase [B] int32 (per-slot schedule)
    size_t total;
    int cstride;
};

Layout workspace_layout(long B, long H, int dk, int dv, int M, int op, int dtype);

// Everything a launch needs, passed by value as the kernel argument.
struct StepArgs {
    int BH;          // slot-heads
    int H;           // heads (RWKV6's bonus u is per head)
    int M;           // merge interval
    int n;           // log entries before this step
    const void *q;   // [BH, dk] (r for RWKV6)
    const void *k;   // [BH, dk]
    const void *v;   // [BH, dv]
    const float *beta; // [BH]
    const float *ld;   // [BH] (GDN) or [BH, dk]: this step's log-decay (EAGER and prep)
    const float *u;    // [H, dk] (RWKV6)
    float *base;       // [BH, dk, dv]
    float *o;          // [BH, dv]
    void *alog;
    void *blog;
    float *Llog;
    float *coef;
    int cstride;
    // per-slot schedule: slot b's log length is (tm - t0[b]) mod M
    int tm;          // the handle's step counter mod M
    const int *t0;   // [B] step (mod M) at which each slot's log was last emptied
    int slot;        // SFOLD: the one slot to fold, or -1 for all
};

// Kernel launchers, one set per operator (dl_gdn.hip, dl_kda.hip, dl_rwkv6.hip).
// They return the launch status (hipGetLastError after the launch) or
// hipErrorInvalidValue for an unsupported shape.
hipError_t launch_prep_gdn(int dtype, int dk, const StepArgs &a, hipStream_t st);
hipError_t launch_prep_kda(int dtype, int dk, const StepArgs &a, hipStream_t st);
hipError_t launch_prep_rwkv6(int dtype, int dk, const StepArgs &a, hipStream_t st);
// Set slot phases: one slot (slot >= 0), or all slots (slot < 0; with
// active_only, only those not released).  A kernel, so calls stay capturable.
hipError_t launch_slot_phase(int *t0, int B, int slot, int value, bool active_only, hipStream_t st);
// The static device scratch of dl_decode_step_staged_noalloc (dl_device.hip):
// its size in floats, and its device address on the current device (looked
// up once per device).
constexpr size_t kScratchFloats = size_t(1) << 20; // 4 MiB
hipError_t scratch_on_current_device(float **out);
hipError_t launch_step_gdn(int dtype, int dk, int dv, int mode, const StepArgs &a, hipStream_t st);
hipError_t launch_step_kda(int dtype, int dk, int dv, int mode, const StepArgs &a, hipStream_t st);
hipError_t launch_step_rwkv6(int dtype, int dk, int dv, int mode, const StepArgs &a, hipStream_t st);

// ---- sequence operators (dl_sequence_api.hip; kernels in dl_scan.h, dl_norm.hip)

constexpr int kScanChunk = 64; // tokens per chunk of the scan

// Chunk slots of a scan: every sequence has enough of them, and the rows
// behind the last one too (dl_scan.h).
constexpr long scan_slots(long tokens, long seqs) { return tokens / kScanChunk + seqs + 1; }
// Keys as the kernels take them (d_k = 16 runs as 32, the rest zero).
constexpr int scan_keys(int dk) { return dk < 32 ? 32 : dk; }
// bf16 planes of the keys' operands: GDN's are the inputs themselves, exact in
// one plane where they are bf16; the others carry fp32 decays.
constexpr int scan_planes(int op, int dtype) { return op == GDN && dtype == BF16 ? 1 : 3; }
// Chunks per segment where the carries cut their sequences (dl_scan_carry.h),
// 0 where they do not.  Uncut, a sequence's chunks are one chain, of 1.8 us each
// (GDN, d = 128); cut, it is two chains of a segment's length and a join per
// segment, and about three times the work: worth it where a quarter of the CUs or
// fewer have a tile and the chain is long.  us, uncut -> cut, of a forward scan:
//   tokens, heads   1100, 1   1100, 8   1600, 1   1600, 8   1900, 1   1900, 8
//   GDN             46 -> 43  46 -> 51  58 -> 48  59 -> 59  67 -> 49  68 -> 62
//   KDA             72 -> 59  71 -> 71  92 -> 64  92 -> 83  105 -> 68 106 -> 90
//   RWKV6           47 -> 43  47 -> 48  61 -> 48  59 -> 55  69 -> 49  69 -> 58
// (d = 64, 2000 tokens, 8 heads: 52 -> 42, 74 -> 51, 40 -> 35.  The host takes
// 10 us more for the two launches more in either direction, which is all that
// a training step of these shows.)  As many segments as give every CU a tile, and
// no more than balance the joins (twice as many: GDN, 8192 tokens, 1 head
// 88 -> 124 us).
constexpr long kCus = 256;
constexpr long scan_segment(long tokens, long seqs, long H, int dv)
{
    const long tiles = seqs * H * (dv / 16), chunks = tokens / kScanChunk / seqs;
    if (tiles > kCus / 4 || chunks < 30)
        return 0;
    long n = 4;
    while (n < kCus / tiles && (n + 1) * (n + 1) <= 2 * chunks)
        ++n;
    return (chunks + n - 1) / n;
}
constexpr long scan_segments(long tokens, long seqs, long segment) { return tokens / (kScanChunk * segment) + seqs + 1; }

// Bytes of one chunk and head's operands: three chunk x keys matrices (bf16
// where one plane holds them, else fp32), two chunk x chunk ones, twenty
// 16 x 16 blocks, a decay per key, and three numbers per row.
constexpr size_t scan_op_bytes(int planes, int keys)
{
    return size_t(3) * kScanChunk * keys * (planes == 1 ? 2 : 4) + size_t(2) * kScanChunk * kScanChunk * 4 +
           20 * 16 * 16 * 4 + 4 * (keys + 3 * kScanChunk);
}

// One scan, forward or backward.  Token strides in elements.
struct ScanArgs {
    int T, N, H, dk, dv; // tokens in all, sequences, heads
    int slots;           // scan_slots(T, N)
    const int *cu;       // [N + 1] token offsets, or NULL: N equal lengths
    const void *q, *k, *v;
    long qs, ks, vs;
    const float *beta, *ld, *u;
    const float *init; // state rows, or NULL (zero)
    float *fin;        // state rows, or NULL
    const int *rows;   // [N] state row of each sequence, or NULL: row n
    int nrows;         // state rows there are
    void *o;
    char *ops;     // [slots][H] operands
    int seg;       // chunks per segment, or 0: sequences uncut
    int segments;  // scan_segments(T, N, seg)
    // [segments][H][dk][dv] a segment's start state (until joined, what its
    // predecessor adds) and [segments][H][dk][dk] its predecessor's transition;
    // backward: its end state's gradient, and what its successor adds and does
    float *seg_s, *seg_m;
    float *save_s; // [slots][H][dk][dv] start state of every chunk, or NULL
    float *save_e; // [slots][H][chunk][dv] E (delta rule)
    // backward
    const void *d_o;   // [T][H][dv], or NULL (zero)
    const float *dfin; // [N][H][dk][dv], or NULL (zero)
    void *d_q, *d_k, *d_v;
    float *d_beta, *d_ld, *d_u, *dinit;
    float *w_ds; // [slots][H][dk][dv] gradient of every chunk's end state
    float *w_z;  // [slots][H][chunk][dv] (delta rule)
    float *w_db; // [slots][H][dv / 16][chunk] partial sums of dbeta
    float *w_du; // [slots][H][dk] partial sums of du
};
hipError_t launch_scan_gdn(int dtype, bool backward, const ScanArgs &a, hipStream_t st);
hipError_t launch_scan_kda(int dtype, bool backward, const ScanArgs &a, hipStream_t st);
hipError_t launch_scan_rwkv6(int dtype, bool backward, const ScanArgs &a, hipStream_t st);

struct GatedNormArgs {
    long units; // rows x H
    int H, d;
    const void *o, *gate, *dy;
    long gate_stride; // elements between rows
    const float *weight;
    float eps;
    void *y, *d_o, *d_gate;
    float *d_weight, *partial; // [blocks][d]
    int blocks;
};
hipError_t launch_gated_norm(int o_dtype, int dtype, bool backward, const GatedNormArgs &a, hipStream_t st);

struct ResidualNormArgs {
    long rows;
    int D;
    const float *x; // forward: the stream; backward: its new value
    const void *y;
    const float *scale, *weight;
    float eps;
    float *x_out;
    void *h;
    const float *d_x_out;
    const void *d_h;
    float *d_x;
    void *d_y;
    float *d_scale, *d_weight, *partial; // [blocks][D] each
    int blocks;
};
hipError_t launch_residual_norm(int dtype, bool backward, const ResidualNormArgs &a, hipStream_t st);

} // namespace dl
