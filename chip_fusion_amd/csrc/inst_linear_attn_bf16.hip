// Linear attention kernels, bf16.
#include "linear_attn_launch.hpp"
const b2b::LinLaunch& b2b::lin_bf16() { return LinLaunchers<b2bk::DT_BF16>::table(); }
