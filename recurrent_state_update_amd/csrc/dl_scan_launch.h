// dl_scan_launch.h -- launches of the scan, templated on the operator.
#pragma once

#include <atomic>

#include "dl_scan_carry.h"
#include "dl_scan_grads.h"
#include "dl_scan_prep.h"

namespace dl {

// Allow a kernel its dynamic LDS, once per kernel and device (the pointer is
// the template's argument: one flag each).
template <auto *KERNEL> hipError_t set_lds(int bytes)
{
    static std::atomic<bool> done[64];
    int dev = 0;
    if (hipError_t e = hipGetDevice(&dev); e != hipSuccess)
        return e;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed))
        return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(KERNEL),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && dev >= 0 && dev < 64)
        done[dev].store(true, std::memory_order_relaxed);
    return e;
}

inline bool at16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int OP, typename TIn, int DKP, bool BWD> hipError_t launch_prep(const ScanArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return hipSuccess;
    const dim3 grid(a.slots * a.H);
    if constexpr (OP == GDN) {
        const bool vec = at16(a.q) && at16(a.k) && a.qs % 8 == 0 && a.ks % 8 == 0;
        constexpr auto *prep = scan_prep_gdn_kernel<TIn, DKP, BWD>;
        if (hipError_t e = set_lds<prep>(sizeof(PrepGdnLds<TIn, DKP>)); e != hipSuccess)
            return e;
        hipLaunchKernelGGL(prep, grid, dim3(256), sizeof(PrepGdnLds<TIn, DKP>), st, a, vec);
    } else {
        const bool vec = at16(a.q) && at16(a.k) && at16(a.ld) && a.qs % 8 == 0 && a.ks % 8 == 0;
        constexpr auto *prep = scan_prep_kernel<OP, TIn, DKP, BWD>;
        if (hipError_t e = set_lds<prep>(sizeof(PrepLds<OP, DKP>)); e != hipSuccess)
            return e;
        hipLaunchKernelGGL(prep, grid, dim3(prep_threads<DKP>()), sizeof(PrepLds<OP, DKP>), st, a, vec);
    }
    return hipGetLastError();
}

// Workgroups of a carry: a grid in which the value tiles of one sequence and
// head run on one XCD (carry_work), which then reads their operands once.
inline dim3 carry_grid(long groups, int tiles) { return dim3((groups + kXcds - 1) / kXcds * kXcds * tiles); }

// Value tiles of 32 columns instead of 16 where those of 16 are more than the
// CUs: a workgroup is bound by its own chunk's chain, so while each has a CU to
// itself more of them are faster, and beyond that the operands, read half as
// often, count.  Forward carry, 1024 tokens, bf16, d = 128, us (16 columns, 32):
//   heads            32 (256 tiles)   48 (384)        64 (512)
//   GDN              36.2, 48.9       64.3, 49.8      63.9, 51.6
//   KDA              58.5, 70.5       98.4, 70.6      97.1, 70.0
//   RWKV6            35.2, 42.2       62.3, 42.3      62.2, 42.8
// (backward, 36 heads: 82.2, 61.2; 107, 76.3; 49.6, 44.2; d = 64, 96 heads: 72.5,
// 62.8; 83.2, 63.8; 38.3, 33.7).  Packed sequences count half: where their
// lengths, not known here, differ, the short ones' tiles end early, and the
// long ones are left alone with the GPU.  A whole forward scan of 288 to 480 tiles:
//   tokens of each   3 x 1024 (16 heads)  82, 1605, 1312 (16)  3000, 40 (20)
//   GDN              82.7, 67.2           73.0, 92.9           110, 148
//   tokens of each   3 x 1024 (16)        1950, 876, 172 (16)  3000, 40 (20)
//   KDA              138, 110             137, 167             183, 232
// (of 45 packings, those of equal lengths gain up to 23 %, uneven ones lose up to
// 35 %; with the backward pass 26 and 24 %.  Equal lengths can come as a batch,
// which does not count half.)
inline bool wide_tiles(const ScanArgs &a)
{
    const long tiles = static_cast<long>(a.N) * a.H * (a.dv / 16);
    return a.dv % 32 == 0 && tiles >= (a.cu && a.N > 1 ? 2 * kCus : kCus + 1);
}

template <int OP, typename TIn, int DKP> hipError_t scan_forward_t(const ScanArgs &a, hipStream_t st)
{
    if (hipError_t e = launch_prep<OP, TIn, DKP, false>(a, st); e != hipSuccess)
        return e;
    if (a.seg) {
        const long groups = static_cast<long>(a.segments) * a.H;
        hipLaunchKernelGGL((scan_carry_kernel<OP, TIn, DKP, 1, LOCAL>), carry_grid(groups, (a.dv + a.dk) / 16), dim3(512), 0,
                           st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        hipLaunchKernelGGL((scan_join_kernel<DKP, false>), dim3(a.N * a.H * (a.dv / 16)), dim3(DKP * 4), 0, st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        auto *carry = a.save_s ? scan_carry_kernel<OP, TIn, DKP, 1, SAVE> : scan_carry_kernel<OP, TIn, DKP, 1, PLAIN>;
        hipLaunchKernelGGL(carry, carry_grid(groups, a.dv / 16), dim3(512), 0, st, a);
        return hipGetLastError();
    }
    const bool wide = wide_tiles(a);
    auto *carry = a.save_s ? (wide ? scan_carry_kernel<OP, TIn, DKP, 2, SAVE> : scan_carry_kernel<OP, TIn, DKP, 1, SAVE>)
                           : (wide ? scan_carry_kernel<OP, TIn, DKP, 2, PLAIN> : scan_carry_kernel<OP, TIn, DKP, 1, PLAIN>);
    hipLaunchKernelGGL(carry, carry_grid(static_cast<long>(a.N) * a.H, a.dv / (wide ? 32 : 16)), dim3(512), 0, st, a);
    return hipGetLastError();
}

template <int OP, typename TIn, int DKP> hipError_t scan_backward_t(const ScanArgs &a, hipStream_t st)
{
    if (hipError_t e = launch_prep<OP, TIn, DKP, true>(a, st); e != hipSuccess)
        return e;
    const long groups = static_cast<long>(a.seg ? a.segments : a.N) * a.H;
    if (a.seg) {
        hipLaunchKernelGGL((scan_carry_bwd_kernel<OP, TIn, DKP, 1, LOCAL>), carry_grid(groups, (a.dv + a.dk) / 16), dim3(512),
                           0, st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
        hipLaunchKernelGGL((scan_join_kernel<DKP, true>), dim3(a.N * a.H * (a.dv / 16)), dim3(DKP * 4), 0, st, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    const bool wide = !a.seg && wide_tiles(a);
    auto *carry = wide ? scan_carry_bwd_kernel<OP, TIn, DKP, 2, PLAIN> : scan_carry_bwd_kernel<OP, TIn, DKP, 1, PLAIN>;
    hipLaunchKernelGGL(carry, carry_grid(groups, a.dv / (wide ? 32 : 16)), dim3(512), 0, st, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    const bool vec = at16(a.q) && at16(a.k) && at16(a.v) && at16(a.d_o) && a.qs % 8 == 0 && a.ks % 8 == 0 &&
                     a.vs % 8 == 0;
    using Lds = GradLds<OP, TIn, DKP>;
    static_assert(sizeof(Lds) <= 160 * 1024, "a CU's LDS");
    constexpr auto *grads = scan_grads_kernel<OP, TIn, DKP>;
    if (hipError_t e = set_lds<grads>(sizeof(Lds)); e != hipSuccess)
        return e;
    hipLaunchKernelGGL(grads, dim3(a.slots * a.H), dim3(DKP * 4), sizeof(Lds), st, a, vec,
                       a.dv / (wide ? 32 : 16));
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (OP == RWKV6) {
        hipLaunchKernelGGL(scan_du_kernel, dim3((a.H * a.dk + 15) / 16), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    return hipSuccess;
}

template <int OP> hipError_t scan_launch(int dtype, bool backward, const ScanArgs &a, hipStream_t st)
{
#define DL_SCAN_CASE(TIN, DKP)                                                                                        \
    return backward ? scan_backward_t<OP, TIN, DKP>(a, st) : scan_forward_t<OP, TIN, DKP>(a, st)
    const int dkp = a.dk < 32 ? 32 : a.dk;
    if (dtype == BF16) {
        if (dkp == 128)
            DL_SCAN_CASE(__bf16, 128);
        if (dkp == 64)
            DL_SCAN_CASE(__bf16, 64);
        DL_SCAN_CASE(__bf16, 32);
    }
    if (dkp == 128)
        DL_SCAN_CASE(float, 128);
    if (dkp == 64)
        DL_SCAN_CASE(float, 64);
    DL_SCAN_CASE(float, 32);
#undef DL_SCAN_CASE
}

} // namespace dl
