// Launchers of the operators around a block's products (arguments already
// validated by block_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w4_block.h"

namespace w4 {

hipError_t launch_block_norm(const w4_norm_args& a, hipStream_t stream);
size_t block_norm_grad_workspace_bytes(int T, int D);
hipError_t launch_block_norm_grad(const w4_norm_args& a, const w4_norm_grad_args& g, void* workspace, hipStream_t stream);

size_t moe_sort_workspace_bytes(int T, int top, int num_experts);
hipError_t launch_moe_sort(const w4_moe_sort_args& a, void* workspace, hipStream_t stream);
// Values of all choices' rows from which on they go past the caches.  6 choices, rows
// of 4096, sorted and combined again: 64 tokens 10.2 us kept and 10.3 so, 256 15.3 and 14.3,
// 1024 32.5 and 29.2; 8191 tokens sorted 103 and 75.
constexpr int64_t kRowsApart = 1 << 22;
hipError_t launch_moe_combine(const w4_moe_combine_args& a, hipStream_t stream);
hipError_t launch_moe_combine_grad(const w4_moe_combine_grad_args& a, hipStream_t stream);

}  // namespace w4
