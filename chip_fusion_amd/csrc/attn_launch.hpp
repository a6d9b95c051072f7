// Launchers of the attention kernels, one translation unit per type.
#pragma once
#include <hip/hip_runtime.h>

#include <tuple>

#include "attn.hpp"

namespace b2b {

constexpr int kAttnRows = b2bk::AttnCfg<b2bk::DT_F16, 2, false>::BM;   // row tile of the many-rows kernel

// Launches a kernel; the status is this launch's own (hipGetLastError would also
// report what an earlier, unrelated call of the thread has left).
template <class... P>
hipError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, hipStream_t s, P... args) {
    return std::apply(
        [&](auto&... a) {
            void* at[] = {&a...};
            return hipLaunchKernel((const void*)kernel, dim3(grid), dim3(threads), at, 0, s);
        },
        std::tie(args...));
}

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
            return launch(b2bk::attn_tile_kernel<C>, grid, C::THREADS, s, a);
        };
        return part ? go(b2bk::AttnCfg<DT, DB, true>{}) : go(b2bk::AttnCfg<DT, DB, false>{});
    }
    static hipError_t tile(const b2bk::AttnArgs& a, bool part, unsigned grid, hipStream_t s) {
        if (a.dim <= 64) return tile_db<2>(a, part, grid, s);
        if (a.dim <= 96) return tile_db<3>(a, part, grid, s);
        return tile_db<4>(a, part, grid, s);
    }
    static hipError_t prefix(const b2bk::AttnArgs& p, const b2bk::AttnArgs& own, unsigned prefix_grid, unsigned own_grid,
                             hipStream_t s) {
        auto go = [&](auto db) {
            return launch(b2bk::attn_prefix_kernel<DT, decltype(db)::value>, prefix_grid + own_grid, 256, s, p, own,
                          (int)prefix_grid);
        };
        if (p.dim <= 64) return go(std::integral_constant<int, 2>{});
        if (p.dim <= 96) return go(std::integral_constant<int, 3>{});
        return go(std::integral_constant<int, 4>{});
    }
    static hipError_t join(const b2bk::AttnArgs& a, int slots, hipStream_t s) {
        const int64_t n = a.rows * a.heads;
        if (slots >= 4) return launch(b2bk::attn_join_kernel<DT, 4>, (unsigned)((n + 3) / 4), 256, s, a, slots);
        return launch(b2bk::attn_join_kernel<DT, 1>, (unsigned)((n + 15) / 16), 256, s, a, slots);
    }
    static const AttnLaunch& table() {
        static const AttnLaunch t = {&tile, &prefix, &join};
        return t;
    }
};

}  // namespace b2b
