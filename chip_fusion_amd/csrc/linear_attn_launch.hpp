// Launchers of the linear attention kernels, one translation unit per type.
#pragma once
#include <hip/hip_runtime.h>

#include "attn_launch.hpp"
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
            return launch(b2bk::lin_kernel<C>, (unsigned)(segs * a.heads), C::THREADS, s, a);
        };
        if (dim == 64) return state ? go(b2bk::LinCfg<DT, 64, true>{}) : go(b2bk::LinCfg<DT, 64, false>{});
        return state ? go(b2bk::LinCfg<DT, 128, true>{}) : go(b2bk::LinCfg<DT, 128, false>{});
    }
    static hipError_t scan(const b2bk::LinArgs& a, int dim, hipStream_t s) {
        const unsigned grid = (unsigned)((int64_t)a.seqs * a.heads * (dim * dim / 1024));
        return dim == 64 ? launch(b2bk::lin_scan_kernel<64>, grid, 256, s, a) : launch(b2bk::lin_scan_kernel<128>, grid, 256, s, a);
    }
    static hipError_t step(const b2bk::LinArgs& a, int dim, hipStream_t s) {
        const unsigned grid = (unsigned)(a.rows * a.heads);
        return dim == 64 ? launch(b2bk::lin_step_kernel<DT, 64>, grid, 256, s, a)
                         : launch(b2bk::lin_step_kernel<DT, 128>, grid, 256, s, a);
    }
    static const LinLaunch& table() {
        static const LinLaunch t = {&run, &scan, &step};
        return t;
    }
};

}  // namespace b2b
