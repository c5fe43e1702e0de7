// The experts' rows back to their tokens, and the gradient of that.
//
//   out[t] = add[t] + sum_j w[t][j] y[row[t][j]],   dy[row] = w dout,   dw = <dout, y[row]>
//
// Memory bounds both: every row is read (and in the gradient written) once,
// 16 bytes a lane, and all of a token's rows are asked for before the first
// is used.  The sum goes over j in order, in FP32.
#include "block.hpp"
#include "block_device.hpp"

namespace w4 {
namespace {

constexpr int kAtOnce = 8;  // rows of a token asked for together

__device__ __forceinline__ u32x4_t load8(const void* p, int64_t at) {
    return *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
}

// The row and weight of choice j of token t; row -1 where there is none.
template <typename A>
__device__ __forceinline__ int row_at(const A& a, int64_t i) {
    const int row = a.row_of ? a.row_of[i] : (int)i;
    return (unsigned)row < (unsigned)a.R ? row : -1;
}

template <int kThreads>
__global__ __launch_bounds__(kThreads) void moe_combine_kernel(w4_moe_combine_args a) {
    const int64_t t = blockIdx.x;
    for (int d = (blockIdx.y * kThreads + threadIdx.x) * 8; d < a.N; d += gridDim.y * kThreads * 8) {
        f32x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.add) v = widen(load8(a.add, t * a.add_stride + d));
        for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
            u32x4_t y[kAtOnce];
            float w[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int row = j0 + j < a.top ? row_at(a, t * a.top + j0 + j) : -1;
                y[j] = u32x4_t{0, 0, 0, 0};
                w[j] = 0;
                if (row >= 0) {
                    y[j] = load8(a.y, row * a.y_stride + d);
                    w[j] = a.weights ? a.weights[t * a.top + j0 + j] : 1.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const f32x8_t x = widen(y[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(w[j], x[e], v[e]);
            }
        }
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + t * a.out_stride + d) = narrow(v);
    }
}

// A workgroup a token; each choice's product over the row is summed over lanes
// and waves in a fixed order.
template <int kWaves>
__global__ __launch_bounds__(kWaves* kWave) void moe_combine_grad_kernel(w4_moe_combine_grad_args a) {
    constexpr int kThreads = kWaves * kWave;
    __shared__ float box[kWaves][kAtOnce];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
        int row[kAtOnce];
        float w[kAtOnce], dot[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t i = t * a.top + j0 + j;
            row[j] = j0 + j < a.top ? row_at(a, i) : -1;
            w[j] = row[j] >= 0 && a.weights ? a.weights[i] : 1.0f;
            dot[j] = 0;
        }
        for (int d = threadIdx.x * 8; d < a.N; d += kThreads * 8) {
            const f32x8_t g = widen(load8(a.dout, t * a.dout_stride + d));
            u32x4_t y[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (a.dweights && row[j] >= 0) y[j] = load8(a.y, row[j] * a.y_stride + d);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (row[j] < 0) continue;
                if (a.dweights) {
                    const f32x8_t x = widen(y[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(g[e], x[e], dot[j]);
                }
                if (a.dy)
                    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.dy) + row[j] * a.dy_stride + d) = narrow(g * w[j]);
            }
        }
        if (!a.dweights) continue;
        // lane / 8 is the choice whose sum a lane holds after this
        const float sum = reduce_rows<kAtOnce>(dot, lane);
        if (lane % 8 == 0) box[wave][lane / 8] = sum;
        __syncthreads();
        if (threadIdx.x < kAtOnce && j0 + (int)threadIdx.x < a.top) {
            float s = box[0][threadIdx.x];
            for (int v = 1; v < kWaves; ++v) s += box[v][threadIdx.x];
            a.dweights[t * a.top + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_moe_combine(const w4_moe_combine_args& a, hipStream_t stream) {
    constexpr int kThreads = 64;
    const int pieces = (a.N / 8 + kThreads - 1) / kThreads;
    moe_combine_kernel<kThreads><<<dim3((unsigned)a.T, (unsigned)(pieces < 65535 ? pieces : 65535)), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const w4_moe_combine_grad_args& a, hipStream_t stream) {
    moe_combine_grad_kernel<4><<<dim3((unsigned)a.T), dim3(4 * kWave), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4
