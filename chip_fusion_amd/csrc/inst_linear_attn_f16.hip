// Linear attention kernels, f16.
#include "linear_attn_launch.hpp"
const b2b::LinLaunch& b2b::lin_f16() { return LinLaunchers<b2bk::DT_F16>::table(); }
