// Host-only build of the state space layer's C ABI (dl_layer_api.hip, plain host code)
// for the sanitizer test, with every kernel launcher replaced by a stub that counts:
// what the calls check for overlaps at the largest sizes that they take.  Exit status
// 0 when every check holds.
#include "dl_layer_api.hip"

#include <climits>
#include <cstdio>

namespace dl {
static int g_launched;
hipError_t launch_short_conv(int, const ConvArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_short_conv_backward(int, const ConvArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_short_conv_step(int, const ConvArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_ssm_scan(int, const SsmArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_ssm_backward(int, const SsmArgs &, const SsmArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_ssm_step(int, const SsmArgs &, hipStream_t) { ++g_launched; return hipSuccess; }
hipError_t launch_residual_norm_fp8(int, const NormFp8Args &, hipStream_t) { ++g_launched; return hipSuccess; }
} // namespace dl

static int g_fail = 0;
#define CHECK(c)                                                                 \
    do {                                                                         \
        if (!(c)) {                                                              \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
            ++g_fail;                                                            \
        }                                                                        \
    } while (0)

// fake device addresses, 2^56 bytes apart, never dereferenced
template <typename T = void> static T *fake(int i, size_t bytes = 0)
{
    return reinterpret_cast<T *>((uintptr_t(i + 1) << 56) + bytes);
}

int main()
{
    // A cache's last row counts, however many there are.
    for (int rows : {1 << 20, (1 << 30) - 1, 1 << 30, INT_MAX})
        for (int W : {2, 3, 4})
            for (int C : {8, 1 << 20}) {
                dl_conv_desc d{};
                d.dtype = DL_BF16;
                d.tokens = 4;
                d.seqs = 1;
                d.channels = C;
                d.taps = W;
                d.x = fake(1);
                d.weight = fake<float>(2);
                const size_t row = size_t(W - 1) * C * 2, all = rows * row;
                CHECK(dl_short_conv_step(&d, fake(3), fake<int>(4), rows, fake(3, all), nullptr) == DL_OK);
                CHECK(dl_short_conv_step(&d, fake(3), fake<int>(4), rows, fake(3, all - 16), nullptr) == DL_E_INVALID);
                CHECK(dl_short_conv_step(&d, fake(3), fake<int>(3, all - 4), rows, fake(5), nullptr) == DL_E_INVALID);
            }
    for (int rows : {1 << 20, 1 << 30, INT_MAX})
        for (int S : {1, 64})
            for (int C : {8, 1 << 16}) {
                dl_ssm_desc d{};
                d.dtype = DL_F32;
                d.tokens = 4;
                d.seqs = d.groups = 1;
                d.channels = C;
                d.states = S;
                d.x = fake(1);
                d.dt = fake(2);
                d.b = fake(4);
                d.c = fake(5);
                d.a = fake<float>(6);
                const size_t all = size_t(rows) * C * S * 4;
                CHECK(dl_ssm_step(&d, fake<float>(7), fake<int>(10), rows, fake(7, all), nullptr) == DL_OK);
                CHECK(dl_ssm_step(&d, fake<float>(7), fake<int>(10), rows, fake(7, all - 4), nullptr) == DL_E_INVALID);
            }
    // The longest inputs and strides.
    for (int N : {1, 1 << 20}) {
        dl_conv_desc d{};
        d.dtype = DL_F32;
        d.tokens = (1 << 24) - (1 << 20) - 1;
        d.seqs = N;
        d.channels = 1024;
        d.taps = 4;
        d.x_stride = 1 << 22;
        d.cu_seqlens = fake<int>(1);
        d.x = fake(2);
        d.weight = fake<float>(3);
        const size_t x = (size_t(d.tokens - 1) * d.x_stride + 1024) * 4, out = size_t(d.tokens) * 4096;
        CHECK(dl_short_conv(&d, nullptr, fake(4), fake(2, x), nullptr) == DL_OK);
        CHECK(dl_short_conv(&d, nullptr, fake(4), fake(2, x - 4), nullptr) == DL_E_INVALID);
        CHECK(dl_short_conv(&d, nullptr, fake(4, out), fake(4), nullptr) == DL_OK);
        CHECK(dl_short_conv(&d, nullptr, fake(4, out - 4), fake(4), nullptr) == DL_E_INVALID);
        const size_t ws = dl_short_conv_workspace_bytes(&d);
        CHECK(dl_short_conv_backward(&d, nullptr, fake(5), nullptr, fake(6, ws), fake<float>(7), fake<float>(8), nullptr,
                                     fake(6), nullptr) == DL_OK);
        CHECK(dl_short_conv_backward(&d, nullptr, fake(5), nullptr, fake(6, ws - 4), fake<float>(7), fake<float>(8), nullptr,
                                     fake(6), nullptr) == DL_E_INVALID);
    }
    for (int D : {1, 16384}) {
        const size_t n = size_t(INT_MAX) * D;
        CHECK(dl_residual_norm_quant(INT_MAX, D, DL_BF16, fake<float>(1), nullptr, nullptr, nullptr, 1e-6f, nullptr, 0,
                                     fake(2), fake<float>(2, (n + 3) / 4 * 4), nullptr) == DL_OK);
        CHECK(dl_residual_norm_quant(INT_MAX, D, DL_BF16, fake<float>(1), nullptr, nullptr, nullptr, 1e-6f, nullptr, 0,
                                     fake(2), fake<float>(2, (n - 1) / 4 * 4), nullptr) == DL_E_INVALID);
    }
    if (!g_fail)
        std::printf("layer span checks passed\n");
    return g_fail ? 1 : 0;
}
