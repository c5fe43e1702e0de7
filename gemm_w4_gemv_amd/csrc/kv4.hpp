// The 4-bit key/value cache on the device, and the launchers of the step's
// operators (arguments already validated by step_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w4_step.h"

namespace w4 {

// The cache's arrays as the kernels take them.
struct Kv4 {
    uint32_t* kc;  // [blocks][heads][block][D/8]
    uint32_t* vc;  // [blocks][heads][block/4][D/8][4]
    uint32_t* km;  // [blocks][heads][D/G][block], (s, m) as an fp16 pair
    uint32_t* vm;
    int blocks;
    int shift;  // log2 of the block size
    int heads;
};

inline Kv4 kv4_of(const w4_kv4_cache& c) {
    return {static_cast<uint32_t*>(c.k_codes), static_cast<uint32_t*>(c.v_codes), static_cast<uint32_t*>(c.k_meta),
            static_cast<uint32_t*>(c.v_meta), c.num_blocks, __builtin_ctz((unsigned)c.block_size), c.kv_heads};
}

struct PlanArgs {
    const int32_t *cached, *fresh;
    int32_t* table;
    const int32_t *free_blocks, *free_count;
    int B, width, capacity, shift, rows;
    int32_t *q_start, *kv_lens, *positions, *slots, *counts;
};
hipError_t launch_kv4_plan(const PlanArgs& a, hipStream_t stream);

// Workgroups of 256 threads that these two launch (T and n at least 1).
int64_t qk_norm_rope_groups(const w4_qk_args& a, bool cached);
int64_t kv4_read_groups(const w4_kv4_cache& c, int n);
hipError_t launch_qk_norm_rope(const w4_qk_args& a, const w4_kv4_cache* cache, hipStream_t stream);
hipError_t launch_kv4_read(const w4_kv4_cache& c, const int32_t* slots, int n, void* k_out, void* v_out,
                           hipStream_t stream);

size_t kv4_attn_workspace_bytes(const w4_attn_args& a, const w4_kv4_cache& c);
hipError_t launch_kv4_attn(const w4_attn_args& a, const w4_kv4_cache& c, void* workspace, hipStream_t stream);

size_t sample_workspace_bytes(int rows, int vocab);
struct SampleArgs {
    const uint16_t* logits;
    int64_t stride;
    const double* uniform;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p;
    int32_t* tokens;
    int rows, vocab;
};
hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream);

}  // namespace w4
