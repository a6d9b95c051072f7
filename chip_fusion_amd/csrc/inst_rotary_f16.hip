// Norm and rotation kernels, f16.
#include "rotary_launch.hpp"
b2b::RotaryLaunch b2b::rotary_f16() { return &launch_rotary<b2bk::DT_F16>; }
