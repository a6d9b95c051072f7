// Paged and windowed attention kernels, f16.
#include "paged_attn_launch.hpp"
const b2b::KeyLaunch& b2b::key_attn_f16() { return KeyLaunchers<b2bk::DT_F16>::table(); }
