// Launchers of the paged and windowed attention kernels, one translation unit per type.
#pragma once
#include "attn_launch.hpp"
#include "paged_attn.hpp"

namespace b2b {

enum { KEYS_WINDOW = 0, KEYS_PAGED = 1, KEYS_PAGED_WINDOW = 2 };

struct KeyLaunch {
    hipError_t (*run)(const b2bk::KeyArgs&, int keys, unsigned grid, hipStream_t);
    hipError_t (*join)(const b2bk::KeyArgs&, int keys, unsigned grid, hipStream_t);
};

const KeyLaunch& key_attn_f16();
const KeyLaunch& key_attn_bf16();

template <int DT>
struct KeyLaunchers {
    template <int DB>
    static hipError_t run_db(const b2bk::KeyArgs& a, int keys, unsigned grid, hipStream_t s) {
        auto go = [&](auto c) {
            using C = decltype(c);
            return launch(b2bk::key_attn_kernel<C>, grid, C::THREADS, s, a);
        };
        if (keys == KEYS_WINDOW) return go(b2bk::KeyCfg<DT, DB, false, true>{});
        if (keys == KEYS_PAGED) return go(b2bk::KeyCfg<DT, DB, true, false>{});
        return go(b2bk::KeyCfg<DT, DB, true, true>{});
    }
    static hipError_t run(const b2bk::KeyArgs& a, int keys, unsigned grid, hipStream_t s) {
        if (a.dim <= 64) return run_db<2>(a, keys, grid, s);
        if (a.dim <= 96) return run_db<3>(a, keys, grid, s);
        return run_db<4>(a, keys, grid, s);
    }
    static hipError_t join(const b2bk::KeyArgs& a, int keys, unsigned grid, hipStream_t s) {
        if (keys == KEYS_WINDOW) return launch(b2bk::key_join_kernel<DT, false, true>, grid, 256, s, a);
        if (keys == KEYS_PAGED) return launch(b2bk::key_join_kernel<DT, true, false>, grid, 256, s, a);
        return launch(b2bk::key_join_kernel<DT, true, true>, grid, 256, s, a);
    }
    static const KeyLaunch& table() {
        static const KeyLaunch t = {&run, &join};
        return t;
    }
};

}  // namespace b2b
