// Attention kernels, f16.
#include "attn_launch.hpp"
const b2b::AttnLaunch& b2b::attn_f16() { return AttnLaunchers<b2bk::DT_F16>::table(); }
