// Paged and windowed attention kernels, bf16.
#include "paged_attn_launch.hpp"
const b2b::KeyLaunch& b2b::key_attn_bf16() { return KeyLaunchers<b2bk::DT_BF16>::table(); }
