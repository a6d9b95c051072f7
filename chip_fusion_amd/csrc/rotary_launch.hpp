// Launcher of the norm and rotation kernels, one translation unit per type.
#pragma once
#include "attn_launch.hpp"
#include "norm_rotary.hpp"

namespace b2b {

struct RotaryKind {
    bool append, norm, interleaved;
};
using RotaryLaunch = hipError_t (*)(const b2bk::RotaryArgs&, RotaryKind, unsigned grid, hipStream_t);

RotaryLaunch rotary_f16();
RotaryLaunch rotary_bf16();

template <int DT>
hipError_t launch_rotary(const b2bk::RotaryArgs& a, RotaryKind k, unsigned grid, hipStream_t s) {
    auto flag = [](bool on, auto go) { return on ? go(std::true_type{}) : go(std::false_type{}); };
    return flag(a.dim > 64, [&](auto WIDE) {
        return flag(k.append, [&](auto APPEND) {
            return flag(k.norm, [&](auto NORM) {
                return flag(k.interleaved, [&](auto INTER) {
                    return launch(b2bk::rotary_kernel<DT, decltype(WIDE)::value ? 16 : 8, decltype(APPEND)::value,
                                                      decltype(NORM)::value, decltype(INTER)::value>,
                                  grid, 256, s, a);
                });
            });
        });
    });
}

}  // namespace b2b
