// Host-only build of the state space layer's C ABI (dl_layer_api.hip, plain host
// code) for the sanitizer test: compiled with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer, every kernel launcher replaced by a stub that records
// its arguments.  Checks that good calls reach the launcher with the workspaces laid
// out as sized and with launches that fit, and sweeps sizes and bad arguments.  Exit
// status 0 when every check holds.
#include "dl_layer_api.hip"

#include <climits>
#include <cmath>
#include <cstdio>

namespace dl {
static int g_launched;
static ConvArgs g_conv;
static SsmArgs g_ssm, g_ahead;
static NormFp8Args g_norm;
hipError_t launch_short_conv(int, const ConvArgs &a, hipStream_t) { ++g_launched; g_conv = a; return hipSuccess; }
hipError_t launch_short_conv_backward(int, const ConvArgs &a, hipStream_t) { ++g_launched; g_conv = a; return hipSuccess; }
hipError_t launch_short_conv_step(int, const ConvArgs &a, hipStream_t) { ++g_launched; g_conv = a; return hipSuccess; }
hipError_t launch_ssm_scan(int, const SsmArgs &a, hipStream_t) { ++g_launched; g_ssm = a; return hipSuccess; }
hipError_t launch_ssm_backward(int, const SsmArgs &ahead, const SsmArgs &a, hipStream_t)
{
    ++g_launched;
    g_ssm = a;
    g_ahead = ahead;
    return hipSuccess;
}
hipError_t launch_ssm_step(int, const SsmArgs &a, hipStream_t) { ++g_launched; g_ssm = a; return hipSuccess; }
hipError_t launch_residual_norm_fp8(int, const NormFp8Args &a, hipStream_t) { ++g_launched; g_norm = a; return hipSuccess; }
} // namespace dl

static int g_fail = 0;
#define CHECK(c)                                                                 \
    do {                                                                         \
        if (!(c)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

// fake device addresses, 2^44 bytes apart, never dereferenced
template <typename T = void> static T *fake(int i) { return reinterpret_cast<T *>(uintptr_t(i + 1) << 44); }

int main()
{
    const int tokens[] = {0, 1, 63, 64, 65, 255, 256, 4096, 100000, 1 << 20}, seqs[] = {1, 3, 100};
    for (int dt = 0; dt < 2; ++dt)
        for (int T : tokens)
            for (int N : seqs)
                for (int C : {1, 7, 64, 4096, 12288})
                    for (int W : {2, 3, 4}) {
                        dl_conv_desc d{};
                        d.dtype = dt;
                        d.tokens = T;
                        d.seqs = N;
                        d.channels = C;
                        d.taps = W;
                        d.cu_seqlens = fake<int>(1);
                        d.x = fake(2);
                        d.weight = fake<float>(3);
                        const size_t ws = dl_short_conv_workspace_bytes(&d);
                        CHECK(ws > 0 && ws % 256 == 0);
                        CHECK(dl_short_conv(&d, fake(4), fake(5), fake(6), nullptr) == DL_OK);
                        const dl::ConvArgs f = dl::g_conv;
                        CHECK(f.xs == C && long(f.runs) * f.run >= T && long(f.runs - 1) * f.run < (T ? T : 1) && f.run <= 64);
                        CHECK(f.vec == (C % 4 == 0));
                        CHECK(dl_short_conv_backward(&d, fake(4), fake(6), nullptr, fake(7), fake<float>(8), fake<float>(9),
                                                     nullptr, fake(10), nullptr) == DL_OK);
                        const dl::ConvArgs b = dl::g_conv;
                        CHECK(long(b.runs) * b.run >= T && b.run <= 128);
                        const size_t rows = size_t(b.runs) * C * 4;
                        CHECK((char *)b.part_w == fake<char>(10) && (char *)b.part_b >= (char *)b.part_w + rows * W);
                        CHECK((char *)b.part_b + rows <= fake<char>(10) + ws);
                        // an offset within a run fits 32 bits, at the longest stride too
                        CHECK((b.run + W) * (1LL << 22) < (1LL << 32));
                    }
    for (int T : tokens)
        for (int N : seqs)
            for (int G : {1, 3})
                for (int C : {3, 15, 48, 2048 * 3, 12288})
                    for (int S : {1, 8, 16, 17, 64})
                        for (int gate = 0; gate < 2; ++gate) {
                            dl_ssm_desc d{};
                            d.dtype = DL_BF16;
                            d.tokens = T;
                            d.seqs = N;
                            d.channels = C;
                            d.states = S;
                            d.groups = G;
                            d.cu_seqlens = fake<int>(1);
                            d.x = fake(2);
                            d.dt = fake(3);
                            d.z = gate ? fake(4) : nullptr;
                            d.b = fake(5);
                            d.c = fake(6);
                            d.a = fake<float>(7);
                            d.d = fake<float>(8);
                            d.dt_bias = fake<float>(9);
                            const size_t ws = dl_ssm_workspace_bytes(&d), sv = dl_ssm_saved_bytes(&d),
                                         wb = dl_ssm_backward_workspace_bytes(&d);
                            CHECK(ws > 0 && sv > 0 && wb > 0 && ws % 256 == 0 && sv % 256 == 0 && wb % 256 == 0);
                            CHECK(dl_ssm_scan(&d, nullptr, fake<float>(10), fake(11), fake(12), fake(13), nullptr) == DL_OK);
                            const dl::SsmArgs f = dl::g_ssm;
                            const size_t state = size_t(C) * S * 4;
                            for (const dl::SsmArgs *a : {&f}) {
                                CHECK(a->slots >= N && a->slots * ((a->tiles + 7L) / 8 * 8) * 2 < (1L << 24));
                                CHECK(a->seg % 64 == 0);
                                if (a->seg) // every sequence has its slots, of tokens that an int counts
                                    CHECK(a->slots >= T / a->seg + N && long(a->slots) * a->seg < INT_MAX);
                                CHECK(a->tiles * 16L >= C && (a->tiles - G) * 16L < C);
                            }
                            if (f.seg) {
                                CHECK((char *)f.seg_h == fake<char>(13) && (char *)f.seg_d >= (char *)f.seg_h + f.slots * state);
                                CHECK((char *)f.seg_d + size_t(f.slots) * C * 4 <= fake<char>(13) + ws);
                            }
                            CHECK((char *)f.saved == fake<char>(12));
                            CHECK((char *)f.plain >= (char *)f.saved + (T / 16 + size_t(N)) * state);
                            if (gate)
                                CHECK((char *)f.plain + size_t(T) * C * 4 <= fake<char>(12) + sv);
                            CHECK(dl_ssm_scan_backward(&d, fake(12), fake(14), nullptr, fake(15), fake(16), gate ? fake(17) : nullptr,
                                                       fake(18), fake(19), fake<float>(20), fake<float>(21), fake<float>(22),
                                                       nullptr, fake(23), nullptr) == DL_OK);
                            const dl::SsmArgs b = dl::g_ssm, h = dl::g_ahead;
                            CHECK(b.saved == f.saved && b.plain == f.plain && h.seg == b.seg && h.slots == b.slots && h.tiles == f.tiles);
                            CHECK(b.tiles * 64L >= C && b.seg % 16 == 0 && b.slots * ((b.tiles + 7L) / 8 * 8) < (1L << 24));
                            CHECK(b.slots * ((h.tiles + 7L) / 8 * 8) < (1L << 24));
                            if (b.seg)
                                CHECK(b.slots >= T / b.seg + N && long(b.slots) * b.seg < INT_MAX);
                            char *const w = fake<char>(23);
                            CHECK((char *)b.part_bc == w);
                            CHECK((char *)b.part_a >= w + size_t(b.tiles / G) * T * G * 2 * S * 4);
                            CHECK((char *)b.part_a + b.slots * (state + size_t(C) * 8) <= w + wb);
                            if (b.seg) {
                                CHECK((char *)b.seg_h >= (char *)b.part_a + b.slots * (state + size_t(C) * 8));
                                CHECK((char *)b.seg_d >= (char *)b.seg_h + b.slots * state);
                                CHECK((char *)b.seg_d + size_t(b.slots) * C * 4 <= w + wb);
                            }
                            for (const void *p : {(void *)b.part_a, (void *)b.seg_h, (void *)b.seg_d, (void *)b.plain})
                                CHECK((uintptr_t)p % 256 == 0);
                        }
    const int launched = dl::g_launched, bad[] = {INT_MIN, -1, INT_MAX};
    for (int x : bad)
        for (int field = 0; field < 6; ++field) {
            dl_ssm_desc d{};
            d.dtype = field == 0 ? x : DL_BF16;
            d.tokens = field == 1 ? x : 64;
            d.seqs = field == 2 ? x : 1;
            d.channels = field == 3 ? x : 64;
            d.states = field == 4 ? x : 16;
            d.groups = field == 5 ? x : 1;
            CHECK(dl_ssm_workspace_bytes(&d) == 0 && dl_ssm_saved_bytes(&d) == 0 && dl_ssm_backward_workspace_bytes(&d) == 0);
            CHECK(dl_ssm_scan(&d, nullptr, nullptr, fake(9), nullptr, fake(11), nullptr) != DL_OK);
            CHECK(dl_ssm_step(&d, fake<float>(1), nullptr, 1, fake(9), nullptr) != DL_OK);
            dl_conv_desc c{};
            c.dtype = field == 0 ? x : DL_BF16;
            c.tokens = field == 1 ? x : 64;
            c.seqs = field == 2 ? x : 1;
            c.channels = field == 3 ? x : 64;
            c.taps = field >= 4 ? x : 4;
            CHECK(dl_short_conv_workspace_bytes(&c) == 0 && dl_short_conv(&c, nullptr, nullptr, fake(9), nullptr) != DL_OK);
        }
    CHECK(dl_ssm_workspace_bytes(nullptr) == 0 && dl_short_conv_workspace_bytes(nullptr) == 0);
    CHECK(dl_ssm_scan(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr) == DL_E_INVALID);
    CHECK(dl_short_conv(nullptr, nullptr, nullptr, nullptr, nullptr) == DL_E_INVALID);
    CHECK(dl::g_launched == launched);
    for (int rows : {0, 1, 1 << 20})
        for (int D : {1, 127, 128, 2048, 16384})
            for (int group : {0, 128}) {
                const int before = dl::g_launched;
                const dl_status st = dl_residual_norm_quant(rows, D, DL_BF16, fake<float>(1), fake(2), nullptr, nullptr, 1e-6f,
                                                            fake<float>(3), group, fake(4), fake<float>(5), nullptr);
                CHECK(st == (group && D % 128 ? DL_E_SHAPE : DL_OK));
                CHECK(dl::g_launched == before + (st == DL_OK && rows > 0));
                if (st == DL_OK && rows > 0)
                    CHECK(dl::g_norm.group == (group ? 128 : D));
            }
    if (!g_fail)
        std::printf("layer host API checks passed\n");
    return g_fail ? 1 : 0;
}
