// Launchers of the paged and windowed attention kernels, one translation unit per type.
#pragma once
#include "attn_launch.hpp"
#include "paged_attn.hpp"

namespace b2b {

struct KeyLaunch {
    hipError_t (*run)(const b2bk::KeyArgs&, int where, unsigned grid, hipStream_t);
    hipError_t (*join)(const b2bk::KeyArgs&, int where, unsigned grid, hipStream_t);
};

const KeyLaunch& key_attn_f16();
const KeyLaunch& key_attn_bf16();

template <int DT>
struct KeyLaunchers {
    template <int DB>
    static hipError_t run_db(const b2bk::KeyArgs& a, int where, unsigned grid, hipStream_t s) {
        auto go = [&](auto c) {
            using C = decltype(c);
            return launch(b2bk::key_attn_kernel<C>, grid, C::THREADS, s, a);
        };
        using namespace b2bk;
        if (where == KEYS_PACKED) return go(KeyCfg<DT, DB, KEYS_PACKED, true>{});       // (without a window: attn.hpp)
        auto flag = [](bool on, auto f) { return on ? f(std::true_type{}) : f(std::false_type{}); };
        return flag(a.window != 0, [&](auto WIN) {
            return flag(a.spread != 0, [&](auto FEW) {
                // (few rows: their kernel takes pages of any size alike)
                if (where == KEYS_PAGES16 && !FEW.value)
                    return go(KeyCfg<DT, DB, KEYS_PAGES16, decltype(WIN)::value, false>{});
                return go(KeyCfg<DT, DB, KEYS_PAGES, decltype(WIN)::value, decltype(FEW)::value>{});
            });
        });
    }
    static hipError_t run(const b2bk::KeyArgs& a, int where, unsigned grid, hipStream_t s) {
        if (a.dim <= 64) return run_db<2>(a, where, grid, s);
        if (a.dim <= 96) return run_db<3>(a, where, grid, s);
        return run_db<4>(a, where, grid, s);
    }
    static hipError_t join(const b2bk::KeyArgs& a, int where, unsigned grid, hipStream_t s) {
        using namespace b2bk;
        auto go = [&](auto kernel) { return launch(kernel, grid, 256, s, a); };
        if (where == KEYS_PACKED) return go(key_join_kernel<DT, 2, false, true>);
        if (a.subs == 1) return a.window ? go(key_join_kernel<DT, 4, true, true>) : go(key_join_kernel<DT, 4, true, false>);
        return a.window ? go(key_join_kernel<DT, 2, true, true>) : go(key_join_kernel<DT, 2, true, false>);
    }
    static const KeyLaunch& table() {
        static const KeyLaunch t = {&run, &join};
        return t;
    }
};

}  // namespace b2b
