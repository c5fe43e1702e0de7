// The norms before and after a block with its gate and residual sum, and their
// gradients.
//
//   u = y r1 (w1 + add),  h' = a h + b g u,  z = h' r2 (w2 + add),  r = 1 / sqrt(mean(x^2) + eps)
//
// Memory bounds both (a row is read and written once, a few operations a
// value), so a team of waves holds a row in registers, 16 bytes a load, and
// the two sums of squares are all that it exchanges.  Those are FP64: the
// squares of BF16's largest and smallest values leave FP32, and the few FP64
// instructions hide behind the loads.
#include <math.h>

#include <type_traits>

#include "block.hpp"
#include "block_device.hpp"

namespace w4 {
namespace {

// ------------------------------------------------------------ sums of a team
__device__ __forceinline__ double of_words(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int kOff>
__device__ __forceinline__ double pair_sum64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
    if constexpr (kOff >= 16) {
        uint32_t l0, l1, h0, h1;
        if constexpr (kOff == 32) {
            const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
            const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
            l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
        } else {
            const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
            const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
            l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
        }
        return of_words(l0, h0) + of_words(l1, h1);
    } else {
        const float l = dpp_partner<kOff>(__builtin_bit_cast(float, lo)), h = dpp_partner<kOff>(__builtin_bit_cast(float, hi));
        return v + of_words(__builtin_bit_cast(uint32_t, l), __builtin_bit_cast(uint32_t, h));
    }
}
__device__ __forceinline__ double wave_sum(double v) {
    v = pair_sum64<32>(v);
    v = pair_sum64<16>(v);
    v = pair_sum64<8>(v);
    v = pair_sum64<4>(v);
    v = pair_sum64<2>(v);
    return pair_sum64<1>(v);
}

// Sum over the kWaves waves of a team, in wave order; ``box`` is LDS of the
// team's own for this one sum (a second sum before the next barrier needs
// another).  All teams of a workgroup must come here together.
template <int kWaves>
__device__ __forceinline__ double team_sum(double v, double* box, int wave) {
    v = wave_sum(v);
    if constexpr (kWaves == 1) return v;
    box[wave] = v;  // every lane holds the sum; one address, one value
    __syncthreads();
    v = box[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += box[w];
    return v;
}

// 1 / sqrt(m) as two factors: neither the squares of large values nor those of
// small ones leave what FP32 holds.  x / sqrt(m) = x * power * rest.
struct Inverse {
    float power, rest;
    __device__ __forceinline__ float of(float x) const { return x * power * rest; }
};
__device__ __forceinline__ Inverse inverse_root(double m) {
    const int e = __builtin_amdgcn_frexp_exp(m) & ~1;              // 0 for 0, infinity and NaN
    const float f = (float)__builtin_amdgcn_ldexp(m, -e);          // in [0.5, 2)
    float r = __builtin_amdgcn_rsqf(f);
    // one step of Newton's: the instruction is off by one unit in the last place
    const float better = fmaf(0.5f * r, fmaf(-f * r, r, 1.0f), r);
    if (f > 0 && f < INFINITY) r = better;
    const int k = -e / 2, c = min(max(k, -126), 126);
    return {__builtin_amdgcn_ldexpf(1.0f, c), __builtin_amdgcn_ldexpf(r, k - c)};
}

// ------------------------------------------------------------- eight values
// Eight values as they lie in memory: BF16, or FP32 with kF32.
template <bool kF32>
struct Raw {
    u32x4_t w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (kF32) {
            const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p) + at);
            w[0] = q[0];
            w[1] = q[1];
        } else {
            w[0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
        }
    }
    __device__ __forceinline__ f32x8_t values() const {
        if constexpr (kF32) {
            f32x8_t v;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = w[i / 4][i % 4];  // a bit_cast of the element itself would read element 0
                v[i] = __builtin_bit_cast(float, b);
            }
            return v;
        } else {
            return widen(w[0]);
        }
    }
};
template <bool kF32>
__device__ __forceinline__ void store(void* p, int64_t at, const f32x8_t& v) {
    if constexpr (kF32) {
        f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at);
        q[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        q[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at) = narrow(v);
    }
}

__device__ __forceinline__ double squares(const f32x8_t& v, double s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma((double)v[i], (double)v[i], s);
    return s;
}

// A team of kWaves waves holds a row, kChunks times 8 values a lane; small
// teams share a workgroup of four waves.
template <int kWaves>
constexpr int teams() {
    return kWaves < 4 ? 4 / kWaves : 1;
}

// ------------------------------------------------------------------ forward
template <int kWaves, int kChunks, bool kF32>
__global__ __launch_bounds__(kWaves* teams<kWaves>() * kWave) void block_norm_kernel(w4_norm_args a) {
    constexpr int kTeams = teams<kWaves>(), kLanes = kWaves * kWave;
    __shared__ double box[2][kTeams][kWaves];
    const int team = kTeams == 1 ? 0 : (int)sgpr(threadIdx.x / kLanes);
    const int tid = threadIdx.x % kLanes, wave = tid / kWave;
    const int64_t t = (int64_t)blockIdx.x * kTeams + team;
    // a team of one wave meets no other; larger ones have the workgroup to themselves
    if (t >= a.T) return;

    const int64_t last = a.D;
    Raw<kF32> h[kChunks];
    Raw<false> y[kChunks], wy[kChunks], wz[kChunks], g[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (d >= last) continue;
        if (a.y) y[c].load(a.y, t * a.y_stride + d);
        h[c].load(a.h, t * a.h_stride + d);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (d >= last) continue;
        if (a.y_weight) wy[c].load(a.y_weight, d);
        if (a.gate) g[c].load(a.gate, t * a.gate_stride + d);
        if (a.z_weight) wz[c].load(a.z_weight, d);
    }

    f32x8_t x[kChunks];  // h'
    Inverse r1 = {1.0f, 1.0f};
    if (a.y && a.y_weight) {
        double s = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if ((c * kLanes + tid) * 8 < last) s = squares(y[c].values(), s);
        r1 = inverse_root(team_sum<kWaves>(s, box[0][team], wave) / a.D + (double)a.eps);
    }
    double s = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (d >= last) continue;
        x[c] = h[c].values();
        if (a.y) {
            f32x8_t u = y[c].values();
            if (a.y_weight) {
                const f32x8_t w = wy[c].values();
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = r1.of(u[i]) * (w[i] + a.weight_add);
            }
            if (a.gate) u *= g[c].values();
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = fmaf(a.residual_scale, x[c][i], a.branch_scale * u[i]);
            if (a.h_out) store<kF32>(a.h_out, t * a.h_out_stride + d, x[c]);
        }
        if (a.z && a.z_weight) s = squares(x[c], s);
    }
    if (!a.z) return;
    Inverse r2 = {1.0f, 1.0f};
    if (a.z_weight) r2 = inverse_root(team_sum<kWaves>(s, box[1][team], wave) / a.D + (double)a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (d >= last) continue;
        f32x8_t v = x[c];
        if (a.z_weight) {
            const f32x8_t w = wz[c].values();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r2.of(v[i]) * (w[i] + a.weight_add);
        }
        store<false>(a.z, t * a.z_stride + d, v);
    }
}

// ----------------------------------------------------------------- gradient
// Sums over the rows are taken in two steps: a workgroup adds its run of rows
// in registers, row by row, and a second kernel adds the workgroups' sums, so
// that no atomic decides their order.
constexpr int kRuns = 512;

struct GradArgs {
    w4_norm_args a;
    w4_norm_grad_args g;
    float* part;  // [3][runs][D]: y_weight, z_weight, gate
    int runs;
};

template <int kWaves, int kChunks, bool kF32>
__global__ __launch_bounds__(kWaves* kWave) void block_norm_grad_kernel(GradArgs k) {
    constexpr int kLanes = kWaves * kWave;
    __shared__ double box[4][kWaves];
    const w4_norm_args& a = k.a;
    const w4_norm_grad_args& g = k.g;
    const int tid = threadIdx.x, wave = tid / kWave, run = blockIdx.x;
    const int64_t first = (int64_t)run * a.T / k.runs, end = (int64_t)(run + 1) * a.T / k.runs;
    const int64_t last = a.D;
    const bool shared_gate = a.gate && a.gate_stride == 0;

    f32x8_t sum_y[kChunks], sum_z[kChunks], sum_g[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) sum_y[c] = sum_z[c] = sum_g[c] = f32x8_t{0, 0, 0, 0, 0, 0, 0, 0};

    for (int64_t t = first; t < end; ++t) {
        Raw<kF32> h[kChunks], dho[kChunks];
        Raw<false> y[kChunks], dz[kChunks], gate[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t d = (c * kLanes + tid) * 8;
            if (d >= last) continue;
            if (a.y) y[c].load(a.y, t * a.y_stride + d);
            h[c].load(a.h, t * a.h_stride + d);
            if (g.dz) dz[c].load(g.dz, t * g.dz_stride + d);
            if (g.dh_out) dho[c].load(g.dh_out, t * g.dh_out_stride + d);
            if (a.gate) gate[c].load(a.gate, t * a.gate_stride + d);
        }
        Inverse r1 = {1.0f, 1.0f}, r2 = {1.0f, 1.0f};
        if (a.y && a.y_weight) {
            double s = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if ((c * kLanes + tid) * 8 < last) s = squares(y[c].values(), s);
            r1 = inverse_root(team_sum<kWaves>(s, box[0], wave) / a.D + (double)a.eps);
        }
        // h', and with dz the norm behind it
        f32x8_t x[kChunks], dx[kChunks];
        double s = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t d = (c * kLanes + tid) * 8;
            if (d >= last) continue;
            x[c] = h[c].values();
            if (a.y) {
                f32x8_t u = y[c].values();
                if (a.y_weight) {
                    Raw<false> raw;
                    raw.load(a.y_weight, d);
                    const f32x8_t w = raw.values();
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = r1.of(u[i]) * (w[i] + a.weight_add);
                }
                if (a.gate) u *= gate[c].values();
#pragma unroll
                for (int i = 0; i < 8; ++i) x[c][i] = fmaf(a.residual_scale, x[c][i], a.branch_scale * u[i]);
            }
            s = squares(x[c], s);
        }
        if (g.dz && a.z_weight) {
            r2 = inverse_root(team_sum<kWaves>(s, box[1], wave) / a.D + (double)a.eps);
            double m = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t d = (c * kLanes + tid) * 8;
                if (d >= last) continue;
                Raw<false> raw;
                raw.load(a.z_weight, d);
                const f32x8_t w = raw.values(), v = dz[c].values();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[c][i] = r2.of(x[c][i]);  // n2
                    sum_z[c][i] = fmaf(v[i], x[c][i], sum_z[c][i]);
                    dx[c][i] = v[i] * (w[i] + a.weight_add);
                    m = fma((double)dx[c][i], (double)x[c][i], m);
                }
            }
            const float mean = (float)(team_sum<kWaves>(m, box[2], wave) / a.D);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[c][i] = r2.of(fmaf(-mean, x[c][i], dx[c][i]));
        } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) dx[c] = g.dz ? dz[c].values() : f32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
        }
        double m = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t d = (c * kLanes + tid) * 8;
            if (d >= last) continue;
            if (g.dh_out) dx[c] += dho[c].values();
            if (g.dh) {
                f32x8_t v = dx[c];
                if (a.y) v *= a.residual_scale;
                store<kF32>(g.dh, t * g.dh_stride + d, v);
            }
            if (!a.y) continue;
            f32x8_t n = y[c].values(), w, b = dx[c] * a.branch_scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
            if (a.y_weight) {
                Raw<false> raw;
                raw.load(a.y_weight, d);
                w = raw.values();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[i] += a.weight_add;
                    n[i] = r1.of(n[i]);
                }
            }
            if (a.gate) {
                f32x8_t dg;
#pragma unroll
                for (int i = 0; i < 8; ++i) dg[i] = b[i] * (n[i] * w[i]);
                if (shared_gate) {
                    sum_g[c] += dg;
                } else if (g.d_gate) {
                    store<false>(g.d_gate, t * g.d_gate_stride + d, dg);
                }
                b *= gate[c].values();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum_y[c][i] = fmaf(b[i], n[i], sum_y[c][i]);
                dx[c][i] = b[i] * w[i];
                x[c][i] = n[i];
                m = fma((double)dx[c][i], (double)n[i], m);
            }
        }
        if (a.y && g.dy) {
            float mean = 0;
            if (a.y_weight) mean = (float)(team_sum<kWaves>(m, box[3], wave) / a.D);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t d = (c * kLanes + tid) * 8;
                if (d >= last) continue;
                if (a.y_weight) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dx[c][i] = r1.of(fmaf(-mean, x[c][i], dx[c][i]));
                }
                store<false>(g.dy, t * g.dy_stride + d, dx[c]);
            }
        }
        // the next row's first sum must not reach a box that another wave still reads
        if constexpr (kWaves > 1) __syncthreads();
    }
    const auto put = [&](int which, const f32x8_t* v) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t d = (c * kLanes + tid) * 8;
            if (d < last) store<true>(k.part, ((int64_t)which * k.runs + run) * a.D + d, v[c]);
        }
    };
    if (g.d_y_weight) put(0, sum_y);
    if (g.d_z_weight) put(1, sum_z);
    if (g.d_gate && shared_gate) put(2, sum_g);
}

// Adds the runs of one column of one of the three sums, four lanes a column.
__global__ __launch_bounds__(256) void block_norm_runs_kernel(GradArgs k) {
    __shared__ double box[4][kWave];
    float* out[3] = {k.g.d_y_weight, k.g.d_z_weight,
                     k.a.gate && k.a.gate_stride == 0 ? static_cast<float*>(k.g.d_gate) : nullptr};
    float* to = out[blockIdx.y];
    if (!to) return;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int d = blockIdx.x * kWave + lane;
    double s = 0;
    if (d < k.a.D)
        for (int r = wave; r < k.runs; r += 4) s += (double)k.part[((int64_t)blockIdx.y * k.runs + r) * k.a.D + d];
    box[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && d < k.a.D) to[d] = (float)(box[0][lane] + box[1][lane] + box[2][lane] + box[3][lane]);
}

int runs_of(int T) { return T < kRuns ? T : kRuns; }

// f(waves, chunks) with the team that holds a row of D values.
template <typename F>
hipError_t with_team(int D, F f) {
    using std::integral_constant;
    if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (D <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    if (D <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (D <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (D <= 8192) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_block_norm(const w4_norm_args& a, hipStream_t stream) {
    return with_team(a.D, [&](auto waves, auto chunks) {
        constexpr int kW = decltype(waves)::value, kC = decltype(chunks)::value, kT = teams<kW>();
        const dim3 grid((unsigned)((a.T + kT - 1) / kT)), block(kW * kT * kWave);
        if (a.h_f32) {
            block_norm_kernel<kW, kC, true><<<grid, block, 0, stream>>>(a);
        } else {
            block_norm_kernel<kW, kC, false><<<grid, block, 0, stream>>>(a);
        }
        return hipGetLastError();
    });
}

size_t block_norm_grad_workspace_bytes(int T, int D) { return (size_t)3 * runs_of(T) * D * sizeof(float); }

hipError_t launch_block_norm_grad(const w4_norm_args& a, const w4_norm_grad_args& g, void* workspace, hipStream_t stream) {
    GradArgs k = {a, g, static_cast<float*>(workspace), runs_of(a.T)};
    if (a.T > 0) {
        const hipError_t err = with_team(a.D, [&](auto waves, auto chunks) {
            constexpr int kW = decltype(waves)::value, kC = decltype(chunks)::value;
            const dim3 grid((unsigned)k.runs), block(kW * kWave);
            if (a.h_f32) {
                block_norm_grad_kernel<kW, kC, true><<<grid, block, 0, stream>>>(k);
            } else {
                block_norm_grad_kernel<kW, kC, false><<<grid, block, 0, stream>>>(k);
            }
            return hipGetLastError();
        });
        if (err != hipSuccess) return err;
    }
    if (!g.d_y_weight && !g.d_z_weight && !(g.d_gate && a.gate_stride == 0)) return hipSuccess;
    block_norm_runs_kernel<<<dim3((unsigned)((a.D + kWave - 1) / kWave), 3), dim3(256), 0, stream>>>(k);
    return hipGetLastError();
}

}  // namespace w4
