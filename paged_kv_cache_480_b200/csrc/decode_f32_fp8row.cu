// Decode kernels for fp32 q and out over an 8-bit row cache (E4M3 codes, one scale a row).
#include "decode_launch.cuh"

PKV_DEFINE_TYPES(f32_fp8row, float, fp8row)
