// Decode kernels for f16 q and out over an 8-bit row cache (E4M3 codes, one scale a row).
#include "decode_launch.cuh"

PKV_DEFINE_TYPES(f16_fp8row, __half, fp8row)
