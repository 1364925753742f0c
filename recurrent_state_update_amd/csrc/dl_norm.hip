// dl_norm.hip -- the norms around a recurrent block, forward and backward:
//   gated norm     y = rms(o) w silu(g) per head (behind the recurrence)
//   residual norm  x' = x + s y,  h = rms(x') w  (before the next block)
// with rms(a) = a / sqrt(mean(a^2) + eps).  Both are a few operations per
// byte and bound by HBM: one pass over the data, each row held in registers
// between its sum and its use, sums in fp32.  The gradients of the per-column
// weights are summed over rows in registers, per workgroup, then over the
// workgroups in their order: the result does not depend on timing.
#include <hip/hip_runtime.h>

#include "dl_internal.h"
#include "dl_vec.h"

namespace dl {

namespace {

constexpr long kForwardBlocks = 2048; // eight per CU: every wave slot, several turns each

// --------------------------------------------------------------- gated norm --

// A unit is one head of one row; G = d / 8 lanes hold it, eight columns each.
// A workgroup takes every gridDim.x-th group of units (the weight is loaded
// once), and loads a turn ahead of the sum that the stores wait for.
template <typename TO, typename T, int D, bool ALIGNED>
__global__ __launch_bounds__(256) void gated_norm_kernel(GatedNormArgs a)
{
    constexpr int G = D / 8;
    const int c = threadIdx.x % G * 8;
    const long step = static_cast<long>(gridDim.x) * (256 / G);
    long u = (static_cast<long>(blockIdx.x) * 256 + threadIdx.x) / G;
    if (u >= a.units) // whole groups
        return;
    float w[8], o[8], g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = a.weight ? a.weight[c + i] : 1.f;
    const auto read = [&](long v) {
        load<8, ALIGNED>(o, static_cast<const TO *>(a.o) + v * D + c);
        load<8, ALIGNED>(g, static_cast<const T *>(a.gate) + v / a.H * a.gate_stride + v % a.H * D + c);
    };
    read(u);
    for (;;) {
        float y[8], z[8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = o[i];
            z[i] = g[i];
            ss = fmaf(y[i], y[i], ss);
        }
        const long next = u + step;
        if (next < a.units)
            read(next);
        const float r = 1.f / sqrtf(group_sum<G>(ss) / D + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = y[i] * r * w[i] * (z[i] / (1.f + expf(-z[i])));
        store<8, ALIGNED>(static_cast<T *>(a.y) + u * D + c, y);
        if (next >= a.units)
            return;
        u = next;
    }
}

// With n = rms(o), sig = sigmoid(g): dn = dy w g sig,
// do = r (dn - n mean(dn n)), dgate = dy n w sig (1 + g (1 - sig)),
// dw = sum dy n g sig.
template <typename TO, typename T, int D, bool ALIGNED>
__global__ __launch_bounds__(256) void gated_norm_bwd_kernel(GatedNormArgs a)
{
    constexpr int G = D / 8;
    __shared__ float part[256 * 8];
    const int c = threadIdx.x % G * 8;
    float w[8], dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = a.weight ? a.weight[c + i] : 1.f;
        dw[i] = 0.f;
    }
    float on[8], gn[8], yn[8]; // the next turn's
    const auto read = [&](long v) {
        load<8, ALIGNED>(on, static_cast<const TO *>(a.o) + v * D + c);
        load<8, ALIGNED>(gn, static_cast<const T *>(a.gate) + v / a.H * a.gate_stride + v % a.H * D + c);
        load<8, ALIGNED>(yn, static_cast<const T *>(a.dy) + v * D + c);
    };
    const long first = (static_cast<long>(blockIdx.x) * 256 + threadIdx.x) / G, step = static_cast<long>(a.blocks) * (256 / G);
    if (first < a.units)
        read(first);
    for (long u = first; u < a.units; u += step) {
        float o[8], g[8], dy[8], dn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = on[i];
            g[i] = gn[i];
            dy[i] = yn[i];
        }
        if (u + step < a.units)
            read(u + step);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(o[i], o[i], ss);
        const float r = 1.f / sqrtf(group_sum<G>(ss) / D + a.eps);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = o[i] * r, sig = 1.f / (1.f + expf(-g[i]));
            const float t = dy[i] * sig;
            o[i] = n;
            dn[i] = t * g[i];
            dw[i] = fmaf(dn[i], n, dw[i]);
            dn[i] *= w[i];
            dot = fmaf(dn[i], n, dot);
            g[i] = t * n * w[i] * (1.f + g[i] * (1.f - sig));
        }
        dot = group_sum<G>(dot) / D;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = r * (dn[i] - o[i] * dot);
        store<8, ALIGNED>(static_cast<TO *>(a.d_o) + u * D + c, o);
        store<8, ALIGNED>(static_cast<T *>(a.d_gate) + u * D + c, g);
    }
    if (!a.d_weight)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        part[threadIdx.x * 8 + i] = dw[i];
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += 256) {
        float x = 0.f;
        for (int t = 0; t < 256 / G; ++t)
            x += part[t * D + j];
        a.partial[static_cast<long>(blockIdx.x) * D + j] = x;
    }
}

// out[j] = the sum over the blocks' rows of partial [blocks][n] (blockIdx.y:
// the second array, of n1 columns).  A workgroup takes 16 columns; 16 threads per column
// take every 16th row, eight loads at a time.  In 64 bits: the norms have up to 1024
// rows, the convolution one for every run of tokens, and the time is the loads', of few
// columns and many rows their latency (128 rows x 20480 columns 4.4 us, 16384 x 80 48).
__global__ __launch_bounds__(256) void column_sum_kernel(const float *partial, int blocks, int n, float *out0,
                                                         int n1, float *out1)
{
    __shared__ double part[16][17];
    const int c = threadIdx.x % 16, s = threadIdx.x / 16, j = blockIdx.x * 16 + c;
    float *out = out0;
    if (blockIdx.y) {
        partial += static_cast<long>(blocks) * n;
        n = n1;
        out = out1;
    }
    double x = 0.;
    if (j < n) {
        int b = s;
        for (; b + 7 * 16 < blocks; b += 8 * 16) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = partial[static_cast<long>(b + 16 * i) * n + j];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x += v[i];
        }
        for (; b < blocks; b += 16)
            x += partial[static_cast<long>(b) * n + j];
    }
    part[s][c] = x;
    __syncthreads();
    if (s == 0 && j < n) {
        for (int t = 1; t < 16; ++t)
            x += part[t][c];
        out[j] = static_cast<float>(x);
    }
}

} // namespace

hipError_t column_sum(const float *partial, int blocks, int n, float *out0, int n1, float *out1, hipStream_t st)
{
    const int most = out1 && n1 > n ? n1 : n;
    hipLaunchKernelGGL(column_sum_kernel, dim3((most + 15) / 16, out1 ? 2 : 1), dim3(256), 0, st, partial, blocks, n,
                       out0, n1, out1);
    return hipGetLastError();
}

namespace {

template <typename TO, typename T, int D>
hipError_t gated_norm_t(bool aligned, bool backward, const GatedNormArgs &a, hipStream_t st)
{
    if (!backward) {
        const long groups = (a.units * (D / 8) + 255) / 256;
        if (groups == 0)
            return hipSuccess;
        const long blocks = groups < kForwardBlocks ? groups : kForwardBlocks;
        if (aligned)
            hipLaunchKernelGGL((gated_norm_kernel<TO, T, D, true>), dim3(blocks), dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((gated_norm_kernel<TO, T, D, false>), dim3(blocks), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    if (aligned)
        hipLaunchKernelGGL((gated_norm_bwd_kernel<TO, T, D, true>), dim3(a.blocks), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((gated_norm_bwd_kernel<TO, T, D, false>), dim3(a.blocks), dim3(256), 0, st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.d_weight)
        return e;
    return column_sum(a.partial, a.blocks, D, a.d_weight, 0, nullptr, st);
}

template <typename TO, typename T>
hipError_t gated_norm_d(bool aligned, bool backward, const GatedNormArgs &a, hipStream_t st)
{
    switch (a.d) {
    case 16: return gated_norm_t<TO, T, 16>(aligned, backward, a, st);
    case 32: return gated_norm_t<TO, T, 32>(aligned, backward, a, st);
    case 64: return gated_norm_t<TO, T, 64>(aligned, backward, a, st);
    default: return gated_norm_t<TO, T, 128>(aligned, backward, a, st);
    }
}

bool at16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// ------------------------------------------------------------ residual norm --

// NT threads per row, E x 8 columns each: VEC = 4 consecutive ones at a time
// (a wave's fp32 load is then one contiguous KiB) where every row starts on a
// boundary of four elements, else single ones.
template <int NT, int VEC, int E> struct Cols {
    static constexpr int K = E * 8 / VEC;
    static __device__ __forceinline__ int col(int k) { return (k * NT + static_cast<int>(threadIdx.x)) * VEC; }
};

template <int NT> __device__ __forceinline__ float row_sum(float x, float *part)
{
    x = group_sum<64>(x);
    if constexpr (NT > 64) {
        __syncthreads(); // part's last use
        if (threadIdx.x % 64 == 0)
            part[threadIdx.x / 64] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w)
            x += part[w];
    }
    return x;
}

// A workgroup takes every gridDim.x-th row; loads run a row ahead.
template <typename T, int NT, int VEC, int E, bool ONCE>
__global__ __launch_bounds__(NT) void residual_norm_kernel(ResidualNormArgs a)
{
    using L = Cols<NT, VEC, E>;
    __shared__ float part[NT / 64];
    float xn[L::K][VEC], yn[L::K][VEC];
    const auto read = [&](long row) {
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
            load<VEC, true, ONCE>(xn[k], a.x + row * a.D + c);
            if (a.y)
                load<VEC, true, ONCE>(yn[k], static_cast<const T *>(a.y) + row * a.D + c);
        }
    };
    constexpr bool AHEAD = E <= 2; // else the registers do not hold two rows
    if (AHEAD)
        read(blockIdx.x);
    for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!AHEAD)
            read(row);
        const long at = row * a.D;
        float x[L::K][VEC], ss = 0.f;
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[k][i] = xn[k][i];
                if (a.y)
                    x[k][i] += a.scale ? yn[k][i] * a.scale[c + i] : yn[k][i];
                ss = fmaf(x[k][i], x[k][i], ss);
            }
            if (a.y)
                store<VEC, true>(a.x_out + at + c, x[k]);
        }
        if (AHEAD && row + gridDim.x < a.rows)
            read(row + gridDim.x);
        const float r = 1.f / sqrtf(row_sum<NT>(ss, part) / a.D + a.eps);
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                x[k][i] *= a.weight ? r * a.weight[c + i] : r;
            store<VEC, true>(static_cast<T *>(a.h) + at + c, x[k]);
        }
    }
}

// With n = x' r: dn = dh w, d = dx' + r (dn - n mean(dn n)), dx = d,
// dy = d s, ds = sum d y, dw = sum dh n.  A workgroup takes every
// gridDim.x-th row and keeps its sums of ds and dw in registers.
template <typename T, int NT, int VEC, int E, bool ONCE>
__global__ __launch_bounds__(NT) void residual_norm_bwd_kernel(ResidualNormArgs a)
{
    using L = Cols<NT, VEC, E>;
    __shared__ float part[NT / 64];
    float ds[L::K][VEC], dw[L::K][VEC];
#pragma unroll
    for (int k = 0; k < L::K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            ds[k][i] = dw[k][i] = 0.f;
    // x', dh, dx' (and y) of the next row
    float nx[L::K][VEC], nh[L::K][VEC], nd[L::K][VEC], ny[L::K][VEC];
    const bool scaled = a.scale && a.d_y;
#pragma unroll
    for (int k = 0; k < L::K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            nh[k][i] = nd[k][i] = ny[k][i] = 0.f;
    const auto read = [&](long row) {
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
            const long at = row * a.D + c;
            load<VEC, true, ONCE>(nx[k], a.x + at);
            if (a.d_h)
                load<VEC, true, ONCE>(nh[k], static_cast<const T *>(a.d_h) + at);
            if (a.d_x_out)
                load<VEC, true, ONCE>(nd[k], a.d_x_out + at);
            if (scaled)
                load<VEC, true, ONCE>(ny[k], static_cast<const T *>(a.y) + at);
        }
    };
    constexpr bool AHEAD = E <= 2;
    if (AHEAD && blockIdx.x < a.rows)
        read(blockIdx.x);
    for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!AHEAD)
            read(row);
        const long at = row * a.D;
        float x[L::K][VEC], dn[L::K][VEC], dx[L::K][VEC], y[L::K][VEC], ss = 0.f, dot = 0.f;
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const bool in = L::col(k) < a.D;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[k][i] = nx[k][i];
                dn[k][i] = nh[k][i];
                dx[k][i] = nd[k][i];
                y[k][i] = ny[k][i];
                ss = in ? fmaf(x[k][i], x[k][i], ss) : ss;
            }
        }
        if (AHEAD && row + gridDim.x < a.rows)
            read(row + gridDim.x);
        const float r = 1.f / sqrtf(row_sum<NT>(ss, part) / a.D + a.eps);
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[k][i] *= r;
                dw[k][i] = fmaf(dn[k][i], x[k][i], dw[k][i]);
                if (a.weight)
                    dn[k][i] *= a.weight[c + i];
                dot = fmaf(dn[k][i], x[k][i], dot);
            }
        }
        dot = row_sum<NT>(dot, part) / a.D;
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                d[i] = dx[k][i] + r * (dn[k][i] - x[k][i] * dot);
            store<VEC, true>(a.d_x + at + c, d);
            if (a.d_y) {
                if (scaled) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        ds[k][i] = fmaf(d[i], y[k][i], ds[k][i]);
                        d[i] *= a.scale[c + i];
                    }
                }
                store<VEC, true>(static_cast<T *>(a.d_y) + at + c, d);
            }
        }
    }
    const long at = static_cast<long>(blockIdx.x) * a.D;
    float *pw = a.partial + (a.d_scale ? static_cast<long>(a.blocks) * a.D : 0);
#pragma unroll
    for (int k = 0; k < L::K; ++k) {
        const int c = L::col(k);
        if (c >= a.D)
            continue;
        if (a.d_scale)
            store<VEC, true>(a.partial + at + c, ds[k]);
        if (a.d_weight)
            store<VEC, true>(pw + at + c, dw[k]);
    }
}

template <typename T, int NT, int VEC, int E, bool ONCE>
hipError_t residual_norm_k(bool backward, const ResidualNormArgs &a, hipStream_t st)
{
    if (!backward) {
        if (a.rows == 0)
            return hipSuccess;
        hipLaunchKernelGGL((residual_norm_kernel<T, NT, VEC, E, ONCE>), dim3(a.rows < kForwardBlocks ? a.rows : kForwardBlocks),
                           dim3(NT), 0, st, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((residual_norm_bwd_kernel<T, NT, VEC, E, ONCE>), dim3(a.blocks), dim3(NT), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && (a.d_scale || a.d_weight))
        e = column_sum(a.partial, a.blocks, a.D, a.d_scale ? a.d_scale : a.d_weight, a.D, a.d_scale ? a.d_weight : nullptr,
                       st);
    return e;
}

// Loads past the caches where a pass moves more than the last-level cache's 256
// MiB: nothing that it reads is still there, and it reads nothing twice.  us
// (plain, past the caches) of D = 2048, bf16, with the data's last use just
// before: 16384 rows forward 87.1, 81.7, backward 122.7, 107.0 (402 and 604 MB);
// 4096 rows 21.6, 21.8 and 27.0, 31.5.  The gated norm gains nothing so.
template <typename T, int NT, int VEC, int E>
hipError_t residual_norm_t(bool backward, const ResidualNormArgs &a, hipStream_t st)
{
    const long per = backward ? 4 * (a.d_x_out ? 3 : 2) + sizeof(T) * ((a.d_h ? 1 : 0) + (a.d_y ? 1 : 0) + (a.scale && a.d_y ? 1 : 0))
                              : 4 * (a.y ? 2 : 1) + sizeof(T) * (a.y ? 2 : 1);
    if constexpr (VEC > 1)
        if (a.rows * static_cast<long>(a.D) * per > (256L << 20))
            return residual_norm_k<T, NT, VEC, E, true>(backward, a, st);
    return residual_norm_k<T, NT, VEC, E, false>(backward, a, st);
}

template <typename T, int VEC> hipError_t residual_norm_e(bool backward, const ResidualNormArgs &a, hipStream_t st)
{
    // one wave per row up to 512 columns, else four, with up to 64 columns
    // per thread in registers
    if (a.D <= 512)
        return residual_norm_t<T, 64, VEC, 1>(backward, a, st);
    if (a.D <= 2048)
        return residual_norm_t<T, 256, VEC, 1>(backward, a, st);
    if (a.D <= 4096)
        return residual_norm_t<T, 256, VEC, 2>(backward, a, st);
    if (a.D <= 8192)
        return residual_norm_t<T, 256, VEC, 4>(backward, a, st);
    return residual_norm_t<T, 256, VEC, 8>(backward, a, st);
}

// ------------------------------------------- residual norm, output in 8 bits --

// The maximum over G = 32 or 64 consecutive lanes.
template <int G> __device__ __forceinline__ float group_max(float x)
{
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xF, 0xF, false)));
    x = fmaxf(x, __shfl_xor(x, 16));
    if constexpr (G == 64)
        x = fmaxf(x, __shfl_xor(x, 32));
    return x;
}

constexpr float kE4m3Most = 448.f;
constexpr float kSmallest = 0x1p-126f; // normal number

// As residual_norm_kernel, with h = rms(x') w as e4m3 values times a scale, of a
// row or (GROUPS) of 128 columns.  With m = max |x' w| and r the row's 1 / rms, the
// scale is r m / 448 and the value x' w (448 / m): one pass, since r cancels, and
// the largest is 448 whatever the rounding.  m is 1e-30 at the least, and the scale of
// what is all zeros the smallest normal number at the least: it has one, too, that can be
// divided by.  A row that holds a NaN has scales of NaN, one with an infinity where that is.
//
// Bound by HBM.  A thread keeps its columns' scale and weight in registers for all of
// its workgroup's rows: read again for every row they come from the caches, but behind
// the next row's loads, for which a wave then waits (16384 x 2048, bf16, 370 MB: 103 ->
// 66 us).
template <typename T, int NT, int VEC, int E, bool GROUPS, bool ONCE>
__global__ __launch_bounds__(NT) void residual_norm_fp8_kernel(NormFp8Args a)
{
    using L = Cols<NT, VEC, E>;
    using Raw = T __attribute__((ext_vector_type(VEC)));
    __shared__ float part[2 * (NT / 64)];
    float xn[L::K][VEC], s[L::K][VEC], w[L::K][VEC];
    Raw yn[L::K];
    const auto read = [&](long row) {
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if (c >= a.D)
                continue;
            load<VEC, true, ONCE>(xn[k], a.x + row * a.D + c);
            if (a.y) {
                const Raw *const y = reinterpret_cast<const Raw *>(static_cast<const T *>(a.y) + row * a.D + c);
                yn[k] = ONCE ? __builtin_nontemporal_load(y) : *y;
            }
        }
    };
    read(blockIdx.x);
#pragma unroll
    for (int k = 0; k < L::K; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = L::col(k) < a.D ? L::col(k) + i : 0;
            s[k][i] = a.scale ? a.scale[c] : 1.f;
            w[k][i] = a.weight ? a.weight[c] : 1.f;
        }
    for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long at = row * a.D;
        float x[L::K][VEC], m[GROUPS ? L::K : 1], ss = 0.f;
        m[0] = 0.f;
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            const int c = L::col(k);
            if constexpr (GROUPS)
                m[k] = 0.f;
            if (c >= a.D)
                continue;
            float &most = m[GROUPS ? k : 0];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma clang fp contract(off) // x' bit for bit residual_norm's
                x[k][i] = xn[k][i];
                if (a.y)
                    x[k][i] += to_f(yn[k][i]) * s[k][i];
                ss = fmaf(x[k][i], x[k][i], ss);
            }
            if (a.y)
                store<VEC, true>(a.x_out + at + c, x[k]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[k][i] *= w[k][i];
                most = fmaxf(most, fabsf(x[k][i]));
            }
        }
        if (row + gridDim.x < a.rows)
            read(row + gridDim.x);
        ss = group_sum<64>(ss);
        if constexpr (!GROUPS)
            m[0] = group_max<64>(m[0]);
        if constexpr (NT > 64) {
            __syncthreads(); // part's last use
            if (threadIdx.x % 64 == 0) {
                part[threadIdx.x / 64] = ss;
                if constexpr (!GROUPS)
                    part[NT / 64 + threadIdx.x / 64] = m[0];
            }
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int w = 0; w < NT / 64; ++w) {
                ss += part[w];
                if constexpr (!GROUPS)
                    m[0] = fmaxf(m[0], part[NT / 64 + w]);
            }
        }
        const float r = 1.f / sqrtf(ss / a.D + a.eps);
#pragma unroll
        for (int k = 0; k < L::K; ++k) {
            if constexpr (GROUPS)
                m[k] = group_max<32>(m[k]); // whole groups are there or none of their lanes
            const int c = L::col(k);
            if (c >= a.D)
                continue;
            const float most = fmaxf(m[GROUPS ? k : 0], 1e-30f);
            float scale = r * (most / kE4m3Most);
            // where all are zero r can take it to zero (a row's rms beyond 3e12)
            if (m[GROUPS ? k : 0] == 0.f && scale < kSmallest)
                scale = kSmallest;
            // 0 r: NaN where the row's norm is none
            const float by = kE4m3Most / most + 0.f * r;
            if constexpr (VEC == 4) {
                unsigned v = __builtin_amdgcn_cvt_pk_fp8_f32(x[k][0] * by, x[k][1] * by, 0, false);
                v = __builtin_amdgcn_cvt_pk_fp8_f32(x[k][2] * by, x[k][3] * by, v, true);
                *reinterpret_cast<unsigned *>(a.h + at + c) = v;
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    a.h[at + c + i] = __builtin_amdgcn_cvt_pk_fp8_f32(x[k][i] * by, 0.f, 0, false) & 0xFF;
            }
            if constexpr (GROUPS) {
                if (c % 128 == 0)
                    a.h_scale[row * (a.D / 128) + c / 128] = scale;
            } else if (c == 0) {
                a.h_scale[row] = scale;
            }
        }
    }
}

template <typename T, int NT, int VEC, int E, bool GROUPS, bool ONCE> hipError_t norm_fp8_o(const NormFp8Args &a, hipStream_t st)
{
    constexpr long blocks = kForwardBlocks * 256 / NT; // every wave slot
    hipLaunchKernelGGL((residual_norm_fp8_kernel<T, NT, VEC, E, GROUPS, ONCE>),
                       dim3(static_cast<unsigned>(a.rows < blocks ? a.rows : blocks)), dim3(NT), 0, st, a);
    return hipGetLastError();
}
template <typename T, int NT, int VEC, int E> hipError_t norm_fp8_k(const NormFp8Args &a, hipStream_t st)
{
    if constexpr (VEC > 1) {
        // past the caches where a pass moves more than the last-level one holds, as
        // residual_norm_t.  us (plain, past the caches) of D = 2048, bf16: 16384 rows 75.5,
        // 65.8; 12000 49.5, 49.2; 8192 31.6, 35.8; 4096 18.7, 22.4.
        const bool once = a.rows * a.D * static_cast<long>(a.y ? 9 + sizeof(T) : 5) > (256L << 20);
        if (a.group != a.D)
            return once ? norm_fp8_o<T, NT, VEC, E, true, true>(a, st) : norm_fp8_o<T, NT, VEC, E, true, false>(a, st);
        if (once)
            return norm_fp8_o<T, NT, VEC, E, false, true>(a, st);
    }
    return norm_fp8_o<T, NT, VEC, E, false, false>(a, st);
}

template <typename T, int VEC> hipError_t norm_fp8_e(const NormFp8Args &a, hipStream_t st)
{
    // eight columns per thread, sixteen in the widest rows (the registers hold their scale
    // and weight); few threads in short rows, whose waves then have rows of their own
    if (a.D <= 512)
        return norm_fp8_k<T, 64, VEC, 1>(a, st);
    if (a.D <= 2048)
        return norm_fp8_k<T, 256, VEC, 1>(a, st);
    if (a.D <= 4096)
        return norm_fp8_k<T, 512, VEC, 1>(a, st);
    if (a.D <= 8192)
        return norm_fp8_k<T, 1024, VEC, 1>(a, st);
    return norm_fp8_k<T, 1024, VEC, 2>(a, st);
}

} // namespace

hipError_t launch_gated_norm(int o_dtype, int dtype, bool backward, const GatedNormArgs &a, hipStream_t st)
{
    // sixteen-byte accesses where every row allows them
    const bool aligned = at16(a.o) && at16(a.gate) && a.gate_stride % 8 == 0 &&
                         (backward ? at16(a.dy) && at16(a.d_o) && at16(a.d_gate) : at16(a.y));
    if (o_dtype == F32)
        return dtype == F32 ? gated_norm_d<float, float>(aligned, backward, a, st)
                            : gated_norm_d<float, __bf16>(aligned, backward, a, st);
    return dtype == F32 ? gated_norm_d<__bf16, float>(aligned, backward, a, st)
                        : gated_norm_d<__bf16, __bf16>(aligned, backward, a, st);
}

hipError_t launch_residual_norm(int dtype, bool backward, const ResidualNormArgs &a, hipStream_t st)
{
    const bool aligned = a.D % 4 == 0 && at16(a.x) && at16(a.y) && at16(a.x_out) && at16(a.h) && at16(a.d_x_out) &&
                         at16(a.d_h) && at16(a.d_x) && at16(a.d_y) && at16(a.partial); // NULL is aligned
    if (dtype == F32)
        return aligned ? residual_norm_e<float, 4>(backward, a, st) : residual_norm_e<float, 1>(backward, a, st);
    return aligned ? residual_norm_e<__bf16, 4>(backward, a, st) : residual_norm_e<__bf16, 1>(backward, a, st);
}

hipError_t launch_residual_norm_fp8(int dtype, const NormFp8Args &a, hipStream_t st)
{
    const bool aligned = a.D % 4 == 0 && at16(a.x) && at16(a.y) && at16(a.x_out) && at16(a.h); // NULL is aligned
    if (!aligned && a.group != a.D)
        return hipErrorInvalidValue;
    if (dtype == F32)
        return aligned ? norm_fp8_e<float, 4>(a, st) : norm_fp8_e<float, 1>(a, st);
    return aligned ? norm_fp8_e<__bf16, 4>(a, st) : norm_fp8_e<__bf16, 1>(a, st);
}

} // namespace dl
