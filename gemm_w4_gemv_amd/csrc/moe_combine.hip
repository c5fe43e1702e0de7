// The experts' rows back to their tokens, and the gradient of that.
//
//   out[t] = add[t] + sum_j w[t][j] y[row[t][j]],   dy[row] = w dout,   dw = <dout, y[row]>
//
// Memory bounds both: every row is read (and in the gradient written) once,
// 16 bytes a lane, and all of a token's rows are asked for before the first
// is used.  The sum goes over j in order, in FP32.
// Measured with 6 choices and rows of 4096: 8191 tokens onto another output 74 us,
// 6.2 TB/s (84 with rows that the caches keep, 103 in workgroups of one wave); the gradient
// of 4096 tokens 79 us, 5.2 TB/s (88 so).
#include <type_traits>

#include "block.hpp"
#include "block_device.hpp"

namespace w4 {
namespace {

constexpr int kAtOnce = 8;  // rows of a token asked for together

template <bool kApart = false>
__device__ __forceinline__ u32x4_t load8(const void* p, int64_t at) {
    return take<kApart>(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at));
}
template <bool kApart>
__device__ __forceinline__ void store8(void* p, int64_t at, const f32x8_t& v) {
    put<kApart>(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at), narrow(v));
}

// The row and weight of choice j of token t; row -1 where there is none.
template <typename A>
__device__ __forceinline__ int row_at(const A& a, int64_t i) {
    const int row = a.row_of ? a.row_of[i] : (int)i;
    return (unsigned)row < (unsigned)a.R ? row : -1;
}

template <int kThreads, bool kApart>
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
                    y[j] = load8<kApart>(a.y, row * a.y_stride + d);
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
        store8<kApart>(a.out, t * a.out_stride + d, v);
    }
}

// A workgroup a token; each choice's product over the row is summed over lanes
// and waves in a fixed order.
template <int kWaves, bool kApart>
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
                if (a.dweights && row[j] >= 0) y[j] = load8<kApart>(a.y, row[j] * a.y_stride + d);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (row[j] < 0) continue;
                if (a.dweights) {
                    const f32x8_t x = widen(y[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(g[e], x[e], dot[j]);
                }
                if (a.dy) store8<kApart>(a.dy, row[j] * a.dy_stride + d, g * w[j]);
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

// f(apart): whether the choices' rows, of N values, go past the caches.
template <typename F>
hipError_t with_apart(int64_t choices, int N, F f) {
    return choices * N >= kRowsApart ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace

hipError_t launch_moe_combine(const w4_moe_combine_args& a, hipStream_t stream) {
    return with_apart((int64_t)a.T * a.top, a.N, [&](auto apart) {
        const auto launch = [&](auto threads) {
            constexpr int kThreads = decltype(threads)::value;
            const int pieces = (a.N / 8 + kThreads - 1) / kThreads;
            moe_combine_kernel<kThreads, decltype(apart)::value>
                <<<dim3((unsigned)a.T, (unsigned)pieces), dim3(kThreads), 0, stream>>>(a);
            return hipGetLastError();
        };
        return a.N <= 512 ? launch(std::integral_constant<int, 64>{}) : launch(std::integral_constant<int, 256>{});
    });
}

hipError_t launch_moe_combine_grad(const w4_moe_combine_grad_args& a, hipStream_t stream) {
    return with_apart((int64_t)a.T * a.top, a.N, [&](auto apart) {
        // as many waves as a row has work for
        const auto launch = [&](auto waves) {
            constexpr int kWaves = decltype(waves)::value;
            moe_combine_grad_kernel<kWaves, decltype(apart)::value>
                <<<dim3((unsigned)a.T), dim3(kWaves * kWave), 0, stream>>>(a);
            return hipGetLastError();
        };
        if (a.N <= 512) return launch(std::integral_constant<int, 1>{});
        if (a.N <= 1024) return launch(std::integral_constant<int, 2>{});
        // (a launch counts its work-items in 32 bits)
        if (a.N <= 2048 || a.T > 1 << 22) return launch(std::integral_constant<int, 4>{});
        return launch(std::integral_constant<int, 8>{});
    });
}

}  // namespace w4
