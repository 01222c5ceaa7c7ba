// Parameter blocks and launchers of the row kernels: rotary positions, the
// cache writes that rotate or quantise, and the read-back of sequences.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

// Where the rows of k (and v) go.
enum class RowSink { kRows, kCache, kCacheFp8Row };

struct RotaryParams {
    const void* q;
    const void* k;
    const void* v;             // kCache and kCacheFp8Row
    void* q_out;
    void* k_out;               // kRows
    unsigned char* k_cache;
    unsigned char* v_cache;
    const int64_t* positions;
    const int64_t* slot_mapping;
    const float* inv_freq;     // [rot / 2]
    unsigned int* errors;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements between tokens
    int64_t pool_slots;
    float mscale;              // multiplies cos and sin
    int num_tokens, num_heads, num_kv_heads, head_size, rot;
    int block_shift;           // log2(block size)
    // filled by the launcher
    int units_row;             // threads a row takes
    int units_token;           // threads a token takes
    int tokens_cta, units_cta; // tokens a CTA takes; units of its tokens it takes (grid.y parts)
    uint32_t row_inverse, token_inverse;   // divide by units_row and units_token
};

cudaError_t launch_rotary(RotaryParams p, RowSink sink, bool interleaved, int dtype, int num_sms, cudaStream_t stream);

// Cache element kinds of the read-back.
enum class CacheKind { kSame, kFp8, kFp8Row };

struct GatherParams {
    void* k_out;
    void* v_out;               // [N][Hkv][D]
    const unsigned char* k_cache;
    const unsigned char* v_cache;
    const int32_t* block_tables;
    const int32_t* start_loc;  // [S + 1]
    unsigned int* errors;
    float k_scale, v_scale;
    int num_tokens, num_seqs, num_kv_heads, head_size, block_shift, num_blocks, max_blocks_per_seq;
    int tokens_cta;            // filled by the launcher, as
    uint32_t token_inverse;    // the inverse of a token's units
};

cudaError_t launch_gather(GatherParams p, CacheKind kind, int dtype, int num_sms, cudaStream_t stream);

}  // namespace pkv
