// Attention kernels, bf16.
#include "attn_launch.hpp"
const b2b::AttnLaunch& b2b::attn_bf16() { return AttnLaunchers<b2bk::DT_BF16>::table(); }
