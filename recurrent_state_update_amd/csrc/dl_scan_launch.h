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
// often, count.  Forward, 1024 tokens, bf16, d = 128, us (16 columns, 32):
//   heads            32 (256 tiles)   48 (384)        64 (512)
//   GDN              32.8, 45.0       61.8, 47.1      64.8, 49.2
//   KDA              46.3, 59.6       86.1, 62.5      91.0, 65.7
//   RWKV6            29.6, 36.0                       45.3, 40.0
// (backward, 36 heads: GDN 77.5, 56.8, KDA 106.6, 76.6; d = 64, 96 heads: GDN
// 68.4, 60.4, RWKV6 43.3, 36.4).  Packed sequences count half: their lengths,
// not known here, differ, and the long ones are left with the GPU (a KDA
// training step over 1000, 17 and 911 tokens, 16 heads: 259 us, and 273 wide).
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
