// The norms before and after a block with its gate and residual sum, and their
// gradients.
//
//   u = y r1 (w1 + add),  h' = a h + b g u,  z = h' r2 (w2 + add),  r = 1 / sqrt(mean(x^2) + eps)
//
// Memory bounds both (a row is read and written once, a few operations a
// value), so a team of waves holds a row in registers, 16 bytes a load, and
// the two sums of squares are all that it exchanges, in FP64; a lane's own share
// is FP32 where that holds it, since the squares of BF16's largest and smallest
// values do not fit.
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
// As swap_pair_sum: a's sum over the lane pair in lanes whose bit kOff is clear, b's in the others.
template <int kOff>
__device__ __forceinline__ double swap_pair_sum64(double a, double b) {
    const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
    uint32_t l0, l1, h0, h1;
    if constexpr (kOff == 32) {
        const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)y, false, false);
        const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(x >> 32), (uint32_t)(y >> 32), false, false);
        l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
    } else {
        const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)y, false, false);
        const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(x >> 32), (uint32_t)(y >> 32), false, false);
        l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
    }
    return of_words(l0, h0) + of_words(l1, h1);
}
// Sum over the lanes that differ in bits kFrom, kFrom / 2, .. 1 (kFrom at most 16).
template <int kFrom>
__device__ __forceinline__ double low_sum64(double v) {
    if constexpr (kFrom == 16) {
        return low_sum64<8>(swap_pair_sum64<16>(v, v));
    } else if constexpr (kFrom >= 1) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
        const float l = dpp_partner<kFrom>(__builtin_bit_cast(float, lo)), h = dpp_partner<kFrom>(__builtin_bit_cast(float, hi));
        return low_sum64<kFrom / 2>(v + of_words(__builtin_bit_cast(uint32_t, l), __builtin_bit_cast(uint32_t, h)));
    } else {
        return v;
    }
}
template <int kLane>
__device__ __forceinline__ double lane_of(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return of_words(__builtin_amdgcn_readlane((uint32_t)b, kLane), __builtin_amdgcn_readlane((uint32_t)(b >> 32), kLane));
}

// Two sums over the kWaves waves of a team at once: lanes 0 .. 31 take a's, the
// others b's.  ``box`` is LDS of the team's own for these; its next use must be
// behind another barrier than this one.  All teams of a workgroup must come here
// together.
template <int kWaves>
__device__ __forceinline__ void team_sums(double& a, double& b, double (*box)[2], int wave, int lane) {
    double v = low_sum64<16>(swap_pair_sum64<32>(a, b));
    if constexpr (kWaves > 1) {
        box[wave][lane >> 5] = v;  // 32 lanes hold a sum; one address, one value
        __syncthreads();
        v = low_sum64<kWaves / 2>(box[lane & (kWaves - 1)][lane >> 5]);
    }
    a = lane_of<0>(v);
    b = lane_of<32>(v);
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
template <bool kF32, bool kApart = false>
__device__ __forceinline__ void store(void* p, int64_t at, const f32x8_t& v) {
    if constexpr (kF32) {
        f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at);
        put<kApart>(q, f32x4_t{v[0], v[1], v[2], v[3]});
        put<kApart>(q + 1, f32x4_t{v[4], v[5], v[6], v[7]});
    } else {
        put<kApart>(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at), narrow(v));
    }
}

// A lane's sums of x^2 and x y over its values, of a row (there(c): the lane has a
// chunk c).  In FP32, if the squares of no lane of the wave come near to what FP32
// holds, which is all but always so, and a third of the time of FP64.
template <int kChunks, typename X, typename Y, typename F>
__device__ __forceinline__ void products(double& xx, double& xy, X x, Y y, F there) {
    float s = 0, m = 0;
    bool any = false;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (!there(c)) continue;
        any = true;
        const f32x8_t v = x(c), w = y(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s = fmaf(v[i], v[i], s);
            m = fmaf(v[i], w[i], m);
        }
    }
    xx = s;
    xy = m;
    const bool plain = s > 0x1p-40f && s < 0x1p100f && m < INFINITY && m > -INFINITY;
    if (!__any(any && !plain)) return;
    xx = xy = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (!there(c)) continue;
        const f32x8_t v = x(c), w = y(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            xx = fma((double)v[i], (double)v[i], xx);
            xy = fma((double)v[i], (double)w[i], xy);
        }
    }
}
template <int kChunks, typename X, typename F>
__device__ __forceinline__ double squares(X x, F there) {
    double xx, unused;
    products<kChunks>(xx, unused, x, x, there);
    return xx;
}

// A team of kWaves waves holds a row, kChunks times 8 values a lane; teams of one
// wave share a workgroup of four.
template <int kWaves>
constexpr int teams() {
    return kWaves < 2 ? 4 : 1;
}

// ------------------------------------------------------------------ forward
// Measured: 4099 rows of 3840, a BF16 stream 21 us, 6.1 TB/s; one row 5.5 us, which is the
// call's.
// kApart: results go past the caches' ways of keeping them.  4099 rows of 3840: 28
// us without, 21 with; a row later read by another norm, 256 rows 9.1 and 8.3, 64
// rows 7.3 and 7.5.
template <int kWaves, int kChunks, bool kF32, bool kApart>
__global__ __launch_bounds__(kWaves* teams<kWaves>() * kWave) void block_norm_kernel(w4_norm_args a) {
    constexpr int kTeams = teams<kWaves>(), kLanes = kWaves * kWave;
    __shared__ double box[2][kTeams][kWaves][2];
    const int team = kTeams == 1 ? 0 : (int)sgpr(threadIdx.x / kLanes);
    const int tid = threadIdx.x % kLanes, wave = tid / kWave, lane = tid % kWave;
    const int64_t t = (int64_t)blockIdx.x * kTeams + team;
    // a team of one wave meets no other; larger ones have the workgroup to themselves
    if (t >= a.T) return;

    const auto there = [&](int c) { return (c * kLanes + tid) * 8 < a.D; };
    Raw<kF32> h[kChunks];
    Raw<false> y[kChunks], wy[kChunks], wz[kChunks], g[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (!there(c)) continue;
        if (a.y) y[c].load(a.y, t * a.y_stride + d);
        h[c].load(a.h, t * a.h_stride + d);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (!there(c)) continue;
        if (a.y_weight) wy[c].load(a.y_weight, d);
        if (a.gate) g[c].load(a.gate, t * a.gate_stride + d);
        if (a.z_weight) wz[c].load(a.z_weight, d);
    }

    f32x8_t x[kChunks];  // h'
    Inverse r1 = {1.0f, 1.0f};
    if (a.y && a.y_weight) {
        double s = squares<kChunks>([&](int c) { return y[c].values(); }, there), unused = 0;
        team_sums<kWaves>(s, unused, box[0][team], wave, lane);
        r1 = inverse_root(s / a.D + (double)a.eps);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (!there(c)) continue;
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
            if (a.h_out) store<kF32, kApart>(a.h_out, t * a.h_out_stride + (c * kLanes + tid) * 8, x[c]);
        }
    }
    if (!a.z) return;
    Inverse r2 = {1.0f, 1.0f};
    if (a.z_weight) {
        double s = squares<kChunks>([&](int c) { return x[c]; }, there), unused = 0;
        team_sums<kWaves>(s, unused, box[1][team], wave, lane);
        r2 = inverse_root(s / a.D + (double)a.eps);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (!there(c)) continue;
        f32x8_t v = x[c];
        if (a.z_weight) {
            const f32x8_t w = wz[c].values();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r2.of(v[i]) * (w[i] + a.weight_add);
        }
        store<false, kApart>(a.z, t * a.z_stride + (c * kLanes + tid) * 8, v);
    }
}

// ----------------------------------------------------------------- gradient
// A workgroup of eight waves (four: see two_groups), in teams of as many as a row takes, goes over a run
// of rows.  The next row is on its way while one is worked on: a row is four
// sums over it, two of which can wait for the others, so a row costs two
// barriers; the sum of the next row's y^2 goes with the second.
//
//   first   sum h'^2 and sum g2 h'   (g2 = dz w2: mean(g2 n2) = r2 mean(g2 h'))
//   second  sum g1 n1 of this row, sum y^2 of the next
//
// Measured, all gradients, an FP32 stream: 8192 rows of 4096 138 us, 4.4 TB/s, and no
// less with a tenth of the instructions taken out or with two workgroups a compute
// unit: memory bounds it, four arrays read and two written at once.
// Rows past 8192 (kLong) would fill the registers: their sums over the rows lie in
// LDS, weights are read row by row and no row is ahead (4 chunks of eight
// waves, some 100 of whose registers the compiler moves to memory: 2048 rows of 16384 270 us,
// 2 chunks of sixteen 328, with all in registers, most of which it then moves, 1250; 2730 of
// 12288, none moved, 184, 329 and 1217).
// Few rows are two launches' latency: 512 rows of 2048, 16 us, 9 of them this kernel's (first
// loads, two rows and their barriers, the teams' sums) and 7 the runs'.
//
// Sums over the rows are taken in three steps, none of whose order is left to
// chance: a lane adds its columns row by row, the teams join in LDS, and a second
// kernel adds the workgroups' sums in FP64.
constexpr int kMaxRuns = 512;
constexpr int kRunWaves = 16;  // of block_norm_runs_kernel

struct GradArgs {
    w4_norm_args a;
    w4_norm_grad_args g;
    float* part;  // [3][runs][D]: y_weight, z_weight, gate
    int runs;
};

template <int kWaves, int kChunks, bool kF32, int kGroup>
__global__ __launch_bounds__(kGroup* kWave, 2) void block_norm_grad_kernel(GradArgs k) {
    constexpr int kLanes = kWaves * kWave, kTeams = kGroup / kWaves;
    constexpr bool kLong = kChunks > 2;
    constexpr f32x8_t kZero = {0, 0, 0, 0, 0, 0, 0, 0};
    __shared__ double box[kLong ? 3 : 2][kTeams][kWaves][2];
    __shared__ f32x4_t far_sums[kLong ? 2 : 1][kLong ? 2 * kChunks : 1][kLong ? kLanes : 1];
    __shared__ f32x8_t join[kTeams == 1 ? 1 : kGroup / 2 * kWave][kChunks];
    const w4_norm_args& a = k.a;
    const w4_norm_grad_args& g = k.g;
    const int team = kTeams == 1 ? 0 : (int)sgpr(threadIdx.x / kLanes);
    const int tid = threadIdx.x % kLanes, wave = tid / kWave, lane = tid % kWave, run = blockIdx.x;
    const int64_t first = (int64_t)run * a.T / k.runs, end = (int64_t)(run + 1) * a.T / k.runs;
    const bool shared_gate = a.gate && a.gate_stride == 0, normed_z = g.dz && a.z_weight;

    struct Row {
        Raw<kF32> h[kChunks], dho[kChunks];
        Raw<false> y[kChunks], dz[kChunks];
    };
    const auto here = [&](int c) { return (c * kLanes + tid) * 8 < a.D; };
    const auto fetch = [&](Row& r, int64_t t) {
        if (t >= end) return;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int64_t d = (c * kLanes + tid) * 8;
            if (!here(c)) continue;
            if (a.y) r.y[c].load(a.y, t * a.y_stride + d);
            r.h[c].load(a.h, t * a.h_stride + d);
            if (g.dz) r.dz[c].load(g.dz, t * g.dz_stride + d);
            if (g.dh_out) r.dho[c].load(g.dh_out, t * g.dh_out_stride + d);
        }
    };
    const auto squares_of_y = [&](const Row& r, int64_t t) {
        if (t >= end || !a.y || !a.y_weight) return 0.0;
        return squares<kChunks>([&](int c) { return r.y[c].values(); }, here);
    };

    f32x8_t sum_y[kChunks], sum_z[kChunks], sum_g[kChunks];
    Raw<false> wy[kChunks], wz[kChunks], gate[kChunks];
    const auto weights = [&](int c) {
        const int64_t d = (c * kLanes + tid) * 8;
        if (a.y_weight) wy[c].load(a.y_weight, d);
        if (a.z_weight) wz[c].load(a.z_weight, d);
        if (shared_gate) gate[c].load(a.gate, d);
    };
    // sum += x * y in the lane's columns
    const auto grow = [&](int which, int c, f32x8_t* sum, const f32x8_t& x, const f32x8_t& y) {
        if constexpr (kLong) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f32x4_t& far = far_sums[which][2 * c + half][tid];
                f32x4_t v = far;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(x[4 * half + i], y[4 * half + i], v[i]);
                far = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[c][i] = fmaf(x[i], y[i], sum[c][i]);
        }
    };
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        sum_y[c] = sum_z[c] = sum_g[c] = kZero;
        if constexpr (kLong) {
#pragma unroll
            for (int i = 0; i < 4; ++i) far_sums[i / 2][2 * c + i % 2][tid] = f32x4_t{0, 0, 0, 0};
        } else if (here(c)) {
            weights(c);
        }
    }

    Row row;
    double sy = 0, unused = 0;
    if constexpr (!kLong) {
        fetch(row, first + team);
        sy = squares_of_y(row, first + team);
        team_sums<kWaves>(sy, unused, box[1][team], wave, lane);
    }
    const double per = 1.0 / a.D;
    for (int64_t t0 = first; t0 < end; t0 += kTeams) {  // every team as often: the barriers are the workgroup's
        const int64_t t = t0 + team;
        const bool live = t < end;
        Row next;
        if constexpr (kLong) {
            fetch(row, t);
            sy = squares_of_y(row, t);
            team_sums<kWaves>(sy, unused, box[kLong ? 2 : 0][team], wave, lane);
        } else {
            fetch(next, t + kTeams);
        }
        const Inverse r1 = a.y && a.y_weight ? inverse_root(sy * per + (double)a.eps) : Inverse{1.0f, 1.0f};
        f32x8_t normed[kChunks], x[kChunks], dx[kChunks];  // y's norm before its weight; h'; dz w2
        const auto n1_of = [&](int c) {
            f32x8_t v = row.y[c].values();
            if (a.y_weight) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r1.of(v[i]);
            }
            return v;
        };
        const auto n1 = [&](int c) { return kLong ? n1_of(c) : normed[c]; };
        double s = 0, m = 0;
        if (live) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (!here(c)) continue;
                if constexpr (kLong) weights(c);
                x[c] = row.h[c].values();
                if (a.gate && !shared_gate) gate[c].load(a.gate, t * a.gate_stride + (c * kLanes + tid) * 8);
                if (a.y) {
                    f32x8_t u = n1_of(c);
                    if constexpr (!kLong) normed[c] = u;
                    if (a.y_weight) u *= wy[c].values() + a.weight_add;
                    if (a.gate) u *= gate[c].values();
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[c][i] = fmaf(a.residual_scale, x[c][i], a.branch_scale * u[i]);
                }
                dx[c] = g.dz ? row.dz[c].values() : kZero;
                if (normed_z) dx[c] *= wz[c].values() + a.weight_add;
            }
            if (normed_z) products<kChunks>(s, m, [&](int c) { return x[c]; }, [&](int c) { return dx[c]; }, here);
        }
        team_sums<kWaves>(s, m, box[0][team], wave, lane);
        const Inverse r2 = normed_z ? inverse_root(s * per + (double)a.eps) : Inverse{1.0f, 1.0f};
        // mean(g2 n2): the sum may leave FP32 where its product with 1 / rms does not
        const float mean2 = normed_z ? (float)(m * per * r2.power * r2.rest) : 0.0f;
        float m1 = 0;
        if (live) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t d = (c * kLanes + tid) * 8;
                if (!here(c)) continue;
                if (kLong && a.y) {
                    weights(c);
                    if (a.gate && !shared_gate) gate[c].load(a.gate, t * a.gate_stride + d);
                }
                if (normed_z) {
                    f32x8_t n2;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        n2[i] = r2.of(x[c][i]);
                        dx[c][i] = r2.of(fmaf(-mean2, n2[i], dx[c][i]));
                    }
                    grow(1, c, sum_z, row.dz[c].values(), n2);
                }
                if (g.dh_out) dx[c] += row.dho[c].values();
                if (g.dh) store<kF32, !kF32>(g.dh, t * g.dh_stride + d, a.y ? dx[c] * a.residual_scale : dx[c]);
                if (!a.y) continue;
                f32x8_t b = dx[c] * a.branch_scale;
                if (a.gate) {
                    f32x8_t u = n1(c);
                    if (a.y_weight) u *= wy[c].values() + a.weight_add;
                    u *= b;
                    if (shared_gate) {
                        sum_g[c] += u;
                    } else if (g.d_gate) {
                        store<false, !kF32>(g.d_gate, t * g.d_gate_stride + d, u);
                    }
                    b *= gate[c].values();
                }
                grow(0, c, sum_y, b, n1(c));
                if (a.y_weight) b *= wy[c].values() + a.weight_add;
                dx[c] = b;
                const f32x8_t n = n1(c);
#pragma unroll
                for (int i = 0; i < 8; ++i) m1 = fmaf(b[i], n[i], m1);
            }
        }
        m = m1;
        // in FP64, as in products, where the lane's sum leaves FP32
        if (live && a.y && a.y_weight && __any(!(m1 < INFINITY && m1 > -INFINITY))) {
            m = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (!here(c)) continue;
                const f32x8_t n = n1(c);
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fma((double)dx[c][i], (double)n[i], m);
            }
        }
        if constexpr (!kLong) sy = squares_of_y(next, t + kTeams);
        team_sums<kWaves>(m, sy, box[1][team], wave, lane);
        if (live && a.y && g.dy) {
            const float mean1 = (float)(m * per);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (!here(c)) continue;
                if (a.y_weight) {
                    const f32x8_t n = n1(c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dx[c][i] = r1.of(fmaf(-mean1, n[i], dx[c][i]));
                }
                store<false, !kF32>(g.dy, t * g.dy_stride + (c * kLanes + tid) * 8, dx[c]);
            }
        }
        if constexpr (!kLong) row = next;
    }
    if constexpr (kLong) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum_y[c][i] = far_sums[0][2 * c + i / 4][tid][i % 4];
                sum_z[c][i] = far_sums[1][2 * c + i / 4][tid][i % 4];
            }
    }

    const auto put = [&](int which, f32x8_t* v) {
        // the teams' sums, halving their number
        if constexpr (kTeams > 1) {
#pragma unroll
            for (int half = kTeams / 2; half >= 1; half /= 2) {
                __syncthreads();
                if (team >= half && team < 2 * half) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) join[(team - half) * kLanes + tid][c] = v[c];
                }
                __syncthreads();
                if (team < half) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) v[c] += join[team * kLanes + tid][c];
                }
            }
            if (team != 0) return;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if (here(c)) store<true>(k.part, ((int64_t)which * k.runs + run) * a.D + (c * kLanes + tid) * 8, v[c]);
    };
    if (g.d_y_weight) put(0, sum_y);
    if (g.d_z_weight) put(1, sum_z);
    if (g.d_gate && shared_gate) put(2, sum_g);
}

// Adds the runs (kMost at most) of one column of one of the three sums: sixteen lanes a
// column, all their loads at once.
template <int kMost>
__global__ __launch_bounds__(kRunWaves * kWave) void block_norm_runs_kernel(GradArgs k) {
    __shared__ double box[kRunWaves][kWave];
    float* out[3] = {k.g.d_y_weight, k.g.d_z_weight,
                     k.a.gate && k.a.gate_stride == 0 ? static_cast<float*>(k.g.d_gate) : nullptr};
    float* to = out[blockIdx.y];
    if (!to) return;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int d = blockIdx.x * kWave + lane;
    const float* from = k.part + (int64_t)blockIdx.y * k.runs * k.a.D + d;
    float v[kMost / kRunWaves];
#pragma unroll
    for (int i = 0; i < kMost / kRunWaves; ++i) {
        const int r = wave + kRunWaves * i;
        v[i] = r < k.runs && d < k.a.D ? from[(int64_t)r * k.a.D] : 0.0f;
    }
    double s = 0;
#pragma unroll
    for (int i = 0; i < kMost / kRunWaves; ++i) s += (double)v[i];
    box[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && d < k.a.D) {
#pragma unroll
        for (int w = 1; w < kRunWaves; ++w) s += box[w][lane];
        to[d] = (float)s;
    }
}

// Whether four waves take a row of 2049 to 4096 values and two workgroups share a compute
// unit, each at its own row, in place of eight waves a row and one workgroup: a barrier
// then stops half of the unit.  Twice the runs are twice the sums to join.  All
// gradients, a BF16 stream, us with two workgroups and with one: rows of 4096, 2048 of
// them 39 and 36, 4096 54 and 54, 6000 70 and 73, 8192 97 and 110; rows of 2056, 2048 33 and
// 31, 4096 45 and 48, 8192 69 and 82.  Rows of up to 2048 have teams of four waves in a
// workgroup of eight: of 2048, 4096 40 and 35, 16384 113 and 112.  An FP32 stream, more
// of it memory, 8192 rows of 4096 139 and 138.
bool two_groups(int T, int D, bool f32) { return !f32 && T >= 4096 && D > 2048 && D <= 4096; }
// Each team has a row at least, a sum more to join costs more than a second row: 256 rows
// of 1024, four teams a workgroup, 64 runs 10.7 us, 128 11.4, 256 14.4; 512 rows 12.6, 12.0, 14.3.
// Then as many as workgroups are on the chip: 128, 256 and 512 runs of 2048 rows of 4096 48,
// 36 and 44 us, of 32768 of 1024 175, 107 and 117, of 8192 of 512 27, 22 and 30, of 2048 of
// 16384 316, 221 and 256; with two workgroups a unit 256 and 512 of 8192 rows of 4096 131 and 98.
int runs_of(int T, int D, bool f32) {
    const int most = two_groups(T, D, f32) ? kMaxRuns : kMaxRuns / 2;
    const int teams = D <= 512 ? 8 : D <= 1024 ? 4 : D <= 2048 ? 2 : 1;
    const int runs = (T + teams - 1) / teams;
    return runs < most ? runs : most;
}

// f(waves, chunks) with the team that holds a row of D values: waves as few as keep
// registers for many, for a row's barriers are theirs.  us of 2^25 values, a BF16 stream
// then an FP32 one: 1152 (2, 2) 45 and 63, (4, 1) 60 and 64; 2048 40 and 65, 41 and 63; 4096
// (4, 2) 39 and 65, (8, 1) 42 and 65; 8192 (8, 2) 41 and 66, (16, 1) 46 and 65; 12288 (8, 3) 42 and 66,
// (16, 2) 58 and 73; 16384 (8, 4) 47 and 70, (16, 2) 54 and 71.
template <typename F>
hipError_t with_team(int D, F f) {
    using std::integral_constant;
    if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (D <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    if (D <= 2048) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    if (D <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (D <= 8192) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    if (D <= 12288) return f(integral_constant<int, 8>{}, integral_constant<int, 3>{});
    return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_block_norm(const w4_norm_args& a, hipStream_t stream) {
    return with_team(a.D, [&](auto waves, auto chunks) {
        constexpr int kW = decltype(waves)::value, kC = decltype(chunks)::value, kT = teams<kW>();
        const dim3 grid((unsigned)((a.T + kT - 1) / kT)), block(kW * kT * kWave);
        const auto launch = [&](auto apart) {
            if (a.h_f32) {
                block_norm_kernel<kW, kC, true, decltype(apart)::value><<<grid, block, 0, stream>>>(a);
            } else {
                block_norm_kernel<kW, kC, false, decltype(apart)::value><<<grid, block, 0, stream>>>(a);
            }
            return hipGetLastError();
        };
        return (int64_t)a.T * a.D >= 1 << 19 ? launch(std::true_type{}) : launch(std::false_type{});
    });
}

size_t block_norm_grad_workspace_bytes(int T, int D) { return (size_t)3 * runs_of(T, D, false) * D * sizeof(float); }

hipError_t launch_block_norm_grad(const w4_norm_args& a, const w4_norm_grad_args& g, void* workspace, hipStream_t stream) {
    GradArgs k = {a, g, static_cast<float*>(workspace), runs_of(a.T, a.D, a.h_f32)};
    if (a.T > 0) {
        const auto launch = [&](auto waves, auto chunks, auto group) {
            constexpr int kW = decltype(waves)::value, kC = decltype(chunks)::value, kG = decltype(group)::value;
            const dim3 grid((unsigned)k.runs), block(kG * kWave);
            if (!a.h_f32) {
                block_norm_grad_kernel<kW, kC, false, kG><<<grid, block, 0, stream>>>(k);
            } else if constexpr (kG == 8) {
                block_norm_grad_kernel<kW, kC, true, kG><<<grid, block, 0, stream>>>(k);
            }
            return hipGetLastError();
        };
        using std::integral_constant;
        constexpr integral_constant<int, 1> one{};
        constexpr integral_constant<int, 2> two{};
        constexpr integral_constant<int, 4> four{};
        constexpr integral_constant<int, 8> eight{};
        const hipError_t err = a.D <= 512     ? launch(one, one, eight)
                               : a.D <= 1024  ? launch(two, one, eight)
                               : a.D <= 2048  ? launch(four, one, eight)
                               : two_groups(a.T, a.D, a.h_f32) ? launch(four, two, four)
                               : a.D <= 4096  ? launch(eight, one, eight)
                               : a.D <= 8192  ? launch(eight, two, eight)
                               : a.D <= 12288 ? launch(eight, integral_constant<int, 3>{}, eight)
                                              : launch(eight, four, eight);
        if (err != hipSuccess) return err;
    }
    if (!g.d_y_weight && !g.d_z_weight && !(g.d_gate && a.gate_stride == 0)) return hipSuccess;
    const dim3 grid((unsigned)((a.D + kWave - 1) / kWave), 3), block(kRunWaves * kWave);
    if (k.runs <= kMaxRuns / 2) {
        block_norm_runs_kernel<kMaxRuns / 2><<<grid, block, 0, stream>>>(k);
    } else {
        block_norm_runs_kernel<kMaxRuns><<<grid, block, 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace w4
