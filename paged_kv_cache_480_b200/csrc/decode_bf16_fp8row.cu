// Decode kernels for bf16 q and out over an 8-bit row cache (E4M3 codes, one scale a row).
#include "decode_launch.cuh"

PKV_DEFINE_TYPES(bf16_fp8row, __nv_bfloat16, fp8row)
