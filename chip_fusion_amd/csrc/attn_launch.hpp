// Launchers of the attention kernels, one translation unit per type.
#pragma once
#include <hip/hip_runtime.h>

#include "attn.hpp"

namespace b2b {

constexpr int kAttnRows = b2bk::AttnCfg<b2bk::DT_F16, 2, false>::BM;   // row tile of the many-rows kernel

struct AttnLaunch {
    // grid workgroups of the many-rows kernel (part: partial results)
    hipError_t (*tile)(const b2bk::AttnArgs&, bool part, unsigned grid, hipStream_t);
    // prefix_grid workgroups of the prefix's keys and own_grid of the requests' own
    hipError_t (*prefix)(const b2bk::AttnArgs& p, const b2bk::AttnArgs& own, unsigned prefix_grid, unsigned own_grid,
                         hipStream_t);
    hipError_t (*join)(const b2bk::AttnArgs&, int slots, hipStream_t);
};

const AttnLaunch& attn_f16();
const AttnLaunch& attn_bf16();

template <int DT>
struct AttnLaunchers {
    template <int DB>
    static hipError_t tile_db(const b2bk::AttnArgs& a, bool part, unsigned grid, hipStream_t s) {
        auto go = [&](auto c) {
            using C = decltype(c);
            hipLaunchKernelGGL(b2bk::attn_tile_kernel<C>, dim3(grid), dim3(C::THREADS), 0, s, a);
        };
        if (part) go(b2bk::AttnCfg<DT, DB, true>{});
        else go(b2bk::AttnCfg<DT, DB, false>{});
        return hipGetLastError();
    }
    static hipError_t tile(const b2bk::AttnArgs& a, bool part, unsigned grid, hipStream_t s) {
        if (a.dim <= 64) return tile_db<2>(a, part, grid, s);
        if (a.dim <= 96) return tile_db<3>(a, part, grid, s);
        return tile_db<4>(a, part, grid, s);
    }
    static hipError_t prefix(const b2bk::AttnArgs& p, const b2bk::AttnArgs& own, unsigned prefix_grid, unsigned own_grid,
                             hipStream_t s) {
        auto go = [&](auto db) {
            hipLaunchKernelGGL((b2bk::attn_prefix_kernel<DT, decltype(db)::value>), dim3(prefix_grid + own_grid), dim3(256), 0,
                               s, p, own, (int)prefix_grid);
        };
        if (p.dim <= 64) go(std::integral_constant<int, 2>{});
        else if (p.dim <= 96) go(std::integral_constant<int, 3>{});
        else go(std::integral_constant<int, 4>{});
        return hipGetLastError();
    }
    static hipError_t join(const b2bk::AttnArgs& a, int slots, hipStream_t s) {
        const int64_t n = a.rows * a.heads;
        if (slots >= 4)
            hipLaunchKernelGGL((b2bk::attn_join_kernel<DT, 4>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, s, a, slots);
        else
            hipLaunchKernelGGL((b2bk::attn_join_kernel<DT, 1>), dim3((unsigned)((n + 15) / 16)), dim3(256), 0, s, a, slots);
        return hipGetLastError();
    }
    static const AttnLaunch& table() {
        static const AttnLaunch t = {&tile, &prefix, &join};
        return t;
    }
};

}  // namespace b2b
