// Launchers of the linear attention kernels, one translation unit per type.
#pragma once
#include <hip/hip_runtime.h>

#include "linear_attn.hpp"

namespace b2b {

struct LinLaunch {
    // segs: the grid's segments (all sequences'); state: only the segments' own states
    hipError_t (*run)(const b2bk::LinArgs&, int dim, bool state, int64_t segs, hipStream_t);
    hipError_t (*scan)(const b2bk::LinArgs&, int dim, hipStream_t);
    hipError_t (*step)(const b2bk::LinArgs&, int dim, hipStream_t);
};

const LinLaunch& lin_f16();
const LinLaunch& lin_bf16();

template <int DT>
struct LinLaunchers {
    static hipError_t run(const b2bk::LinArgs& a, int dim, bool state, int64_t segs, hipStream_t s) {
        auto go = [&](auto c) {
            using C = decltype(c);
            hipLaunchKernelGGL(b2bk::lin_kernel<C>, dim3((unsigned)(segs * a.heads)), dim3(C::THREADS), 0, s, a);
        };
        if (dim == 64) {
            if (state) go(b2bk::LinCfg<DT, 64, true>{});
            else go(b2bk::LinCfg<DT, 64, false>{});
        } else {
            if (state) go(b2bk::LinCfg<DT, 128, true>{});
            else go(b2bk::LinCfg<DT, 128, false>{});
        }
        return hipGetLastError();
    }
    static hipError_t scan(const b2bk::LinArgs& a, int dim, hipStream_t s) {
        const unsigned grid = (unsigned)((int64_t)a.seqs * a.heads * (dim * dim / 1024));
        if (dim == 64) hipLaunchKernelGGL(b2bk::lin_scan_kernel<64>, dim3(grid), dim3(256), 0, s, a);
        else hipLaunchKernelGGL(b2bk::lin_scan_kernel<128>, dim3(grid), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    static hipError_t step(const b2bk::LinArgs& a, int dim, hipStream_t s) {
        const dim3 grid((unsigned)(a.rows * a.heads));
        if (dim == 64) hipLaunchKernelGGL((b2bk::lin_step_kernel<DT, 64>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((b2bk::lin_step_kernel<DT, 128>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
    static const LinLaunch& table() {
        static const LinLaunch t = {&run, &scan, &step};
        return t;
    }
};

}  // namespace b2b
