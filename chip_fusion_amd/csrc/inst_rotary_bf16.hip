// Norm and rotation kernels, bf16.
#include "rotary_launch.hpp"
b2b::RotaryLaunch b2b::rotary_bf16() { return &launch_rotary<b2bk::DT_BF16>; }
