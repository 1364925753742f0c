// Host-only build of the sequence operators' C ABI (dl_sequence_api.hip, plain
// host code) for the sanitizer test: compiled with g++ under AddressSanitizer
// and UndefinedBehaviorSanitizer, every kernel launcher replaced by a stub that
// records its arguments.  Checks that good calls reach the launcher with the
// workspace laid out as sized (segments in order, apart, inside the buffer),
// and sweeps sizes and bad arguments.  Exit status 0 when every check holds.
#include "dl_sequence_api.hip"

#include <climits>
#include <cstdio>
#include <cmath>

namespace dl {
static int g_scans, g_gated, g_residual;
static ScanArgs g_scan;
static bool g_backward;
static hipError_t rec(bool backward, const ScanArgs &a)
{
    ++g_scans;
    g_scan = a;
    g_backward = backward;
    return hipSuccess;
}
hipError_t launch_scan_gdn(int, bool b, const ScanArgs &a, hipStream_t) { return rec(b, a); }
hipError_t launch_scan_kda(int, bool b, const ScanArgs &a, hipStream_t) { return rec(b, a); }
hipError_t launch_scan_rwkv6(int, bool b, const ScanArgs &a, hipStream_t) { return rec(b, a); }
hipError_t launch_gated_norm(int, int, bool, const GatedNormArgs &a, hipStream_t)
{
    ++g_gated;
    return a.blocks >= 1 ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_residual_norm(int, bool, const ResidualNormArgs &, hipStream_t)
{
    ++g_residual;
    return hipSuccess;
}
} // namespace dl

static int g_fail = 0;
#define CHECK(c)                                                                 \
    do {                                                                         \
        if (!(c)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

// fake device addresses, 2^36 bytes apart, never dereferenced
static char *fake(int i) { return reinterpret_cast<char *>(uintptr_t(0x100000000000) + (uintptr_t(i) << 40)); }

int main()
{
    const int dims[] = {16, 32, 64, 128}, tokens[] = {0, 1, 63, 64, 65, 4096, 1 << 20}, seqs[] = {1, 3, 100};
    for (int op = 0; op < 3; ++op)
        for (int dt = 0; dt < 2; ++dt)
            for (int dk : dims)
                for (int dv : dims)
                    for (int T : tokens)
                        for (int N : seqs) {
                            dl_scan_desc d{};
                            d.op = op;
                            d.in_dtype = dt;
                            d.tokens = T;
                            d.seqs = N;
                            d.H = 2;
                            d.d_k = dk;
                            d.d_v = dv;
                            d.cu_seqlens = reinterpret_cast<int *>(fake(1));
                            d.q = fake(2);
                            d.k = fake(3);
                            d.v = fake(4);
                            d.beta = reinterpret_cast<float *>(fake(5));
                            d.log_decay = reinterpret_cast<float *>(fake(6));
                            d.u = op == DL_OP_RWKV6 ? reinterpret_cast<float *>(fake(7)) : nullptr;
                            const size_t ws = dl_scan_workspace_bytes(&d), sv = dl_scan_saved_bytes(&d),
                                         wb = dl_scan_backward_workspace_bytes(&d);
                            CHECK(ws > 0 && sv > 0 && wb > ws);
                            const int before = dl::g_scans;
                            float *s0 = reinterpret_cast<float *>(fake(8));
                            CHECK(dl_scan(&d, s0, s0, nullptr, 0, fake(9), fake(10), fake(11), nullptr) == DL_OK);
                            CHECK(dl::g_scans == before + 1 && !dl::g_backward);
                            const dl::ScanArgs f = dl::g_scan;
                            const size_t sh = size_t(f.slots) * 2;
                            CHECK(f.slots == T / 64 + N + 1 && f.qs == 2 * dk && f.vs == 2 * dv);
                            CHECK(sh * dl::scan_op_bytes(dl::scan_planes(op, dt), dk < 32 ? 32 : dk) <= ws);
                            CHECK((char *)f.save_e - (char *)f.save_s >= (long)(sh * dk * dv * 4));
                            if (op != DL_OP_RWKV6)
                                CHECK((char *)f.save_e + sh * 64 * dv * 4 <= fake(10) + sv);
                            float *g = reinterpret_cast<float *>(fake(12));
                            CHECK(dl_scan_backward(&d, fake(10), fake(13), nullptr, fake(14), fake(15), fake(16),
                                                   op == DL_OP_RWKV6 ? nullptr : g, reinterpret_cast<float *>(fake(17)),
                                                   op == DL_OP_RWKV6 ? g : nullptr, nullptr, fake(18), nullptr) == DL_OK);
                            const dl::ScanArgs b = dl::g_scan;
                            CHECK(dl::g_backward && b.ops == fake(18));
                            CHECK((char *)b.w_ds - b.ops >= (long)(sh * dl::scan_op_bytes(dl::scan_planes(op, dt), dk < 32 ? 32 : dk)));
                            CHECK((char *)b.w_z - (char *)b.w_ds >= (long)(sh * dk * dv * 4));
                            const size_t z = op == DL_OP_RWKV6 ? 0 : sh * 64 * dv * 4, db = op == DL_OP_RWKV6 ? 0 : sh * (dv / 16) * 64 * 4;
                            CHECK((size_t)((char *)b.w_db - (char *)b.w_z) >= z);
                            CHECK((size_t)((char *)b.w_du - (char *)b.w_db) >= db);
                            CHECK((char *)b.w_du + (op == DL_OP_RWKV6 ? sh * dk * 4 : 0) <= fake(18) + wb);
                            for (const void *p : {(void *)b.w_ds, (void *)b.w_z, (void *)b.w_db, (void *)b.w_du})
                                CHECK((uintptr_t)p % 256 == 0);
                        }
    // long sequences with few heads: segments, behind the operands, in both passes
    for (int op : {DL_OP_GDN, DL_OP_KDA, DL_OP_RWKV6})
        for (int dk : dims)
            for (int dv : dims)
                for (int N : {1, 3})
                    for (int T : {1919 * N, 1920 * N, 100000 * N, 4194304 * N}) {
                        dl_scan_desc d{};
                        d.op = op;
                        d.in_dtype = DL_BF16;
                        d.tokens = T;
                        d.seqs = N;
                        d.H = 2;
                        d.d_k = dk;
                        d.d_v = dv;
                        d.cu_seqlens = reinterpret_cast<int *>(16);
                        d.q = d.k = d.v = reinterpret_cast<void *>(16);
                        d.beta = d.log_decay = d.u = reinterpret_cast<float *>(16);
                        const size_t ws = dl_scan_workspace_bytes(&d);
                        char *const at = reinterpret_cast<char *>(size_t(1) << 44), *const o = reinterpret_cast<char *>(size_t(1) << 45);
                        float *const st = reinterpret_cast<float *>(size_t(1) << 46);
                        CHECK(dl_scan(&d, nullptr, st, nullptr, 0, o, nullptr, at, nullptr) == DL_OK);
                        const dl::ScanArgs f = dl::g_scan;
                        CHECK((f.seg > 0) == (T >= 1920 * N && N * 2 * (dv / 16) <= 64));
                        if (f.seg == 0)
                            continue;
                        // a sequence has four segments or more, and every one a slot
                        CHECK(f.seg * 64L * 3 < T / N && f.segments >= T / (64L * f.seg) + N + 1);
                        const size_t sh = size_t(f.segments) * 2;
                        CHECK((char *)f.seg_s >= f.ops + size_t(f.slots) * 2 * dl::scan_op_bytes(dl::scan_planes(op, DL_BF16), dk < 32 ? 32 : dk));
                        CHECK((char *)f.seg_m >= (char *)f.seg_s + sh * dk * dv * 4 && (char *)f.seg_m + sh * dk * dk * 4 <= at + ws);
                        CHECK((uintptr_t)f.seg_s % 256 == 0 && (uintptr_t)f.seg_m % 256 == 0);
                    }
    const int bad[] = {INT_MIN, -1, 0, 17, 24, 129, INT_MAX};
    int launched = dl::g_scans;
    for (int x : bad)
        for (int field = 0; field < 6; ++field) {
            dl_scan_desc d{};
            d.in_dtype = DL_BF16;
            d.tokens = 64;
            d.seqs = 1;
            d.H = 1;
            d.d_k = d.d_v = 64;
            if (field == 0) d.d_k = x;
            if (field == 1) d.d_v = x;
            if (field == 2) d.H = x > 0 ? INT_MAX : x;
            if (field == 3) d.seqs = x > 0 ? INT_MAX : x;
            if (field == 4) d.op = x == 0 ? 3 : x;
            if (field == 5) d.tokens = x < 0 ? x : INT_MIN;
            CHECK(dl_scan_workspace_bytes(&d) == 0 && dl_scan_saved_bytes(&d) == 0);
            CHECK(dl_scan(&d, nullptr, nullptr, nullptr, 0, fake(9), nullptr, fake(11), nullptr) != DL_OK);
        }
    CHECK(dl_scan_workspace_bytes(nullptr) == 0);
    CHECK(dl_scan(nullptr, nullptr, nullptr, nullptr, 0, nullptr, nullptr, nullptr, nullptr) == DL_E_INVALID);
    CHECK(dl::g_scans == launched);
    for (int rows : {0, 1, 77, 1 << 20})
        for (int d : dims) {
            const size_t n = dl_gated_norm_workspace_bytes(rows, 3, d);
            CHECK(n >= size_t(d) * 4 && n <= size_t(1024) * d * 4);
            CHECK(dl_gated_norm(rows, 3, d, DL_F32, DL_BF16, fake(1), fake(2), 0, nullptr, 1e-6f, fake(3), nullptr) == DL_OK);
            CHECK(dl_gated_norm(rows, 3, d, DL_F32, DL_BF16, fake(1), fake(2), 0, nullptr, NAN, fake(3), nullptr) == DL_E_INVALID);
        }
    for (int rows : {0, 1, 77, 1 << 20})
        for (int D : {1, 7, 2048, 16384}) {
            CHECK(dl_residual_norm_workspace_bytes(rows, D) >= size_t(2) * D * 4);
            CHECK(dl_residual_norm(rows, D, DL_BF16, reinterpret_cast<float *>(fake(1)), nullptr, nullptr, nullptr, 1e-6f,
                                   nullptr, fake(3), nullptr) == DL_OK);
        }
    CHECK(dl::g_gated == 3 * 4 && dl::g_residual == 3 * 4);
    if (!g_fail)
        std::printf("sequence host API checks passed\n");
    return g_fail ? 1 : 0;
}
