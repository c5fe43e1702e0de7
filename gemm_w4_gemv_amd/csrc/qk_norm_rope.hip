// RMS norm of query and key heads, rotation by position, and keys and values
// quantised into the 4-bit cache, in one pass; and the cache read back.
//
// Eight values a lane: a head is a run of D / 8 lanes, so a wave holds
// 64 / (D / 8) heads of one token and walks over the token's heads with the
// row of cosines and sines in registers (it is as large as two heads).  A
// lane's eight 4-bit codes are one word of the cache.  The partner of a
// rotated pair is either in the lane or in one lane of the same head, taken
// as raw BF16 before its norm is applied (four exchanges instead of eight).
// Memory bounds it for prompts; launch and latency for a decode step, where
// the token's heads are spread over waves instead.
#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const u32x4_t& w, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
}

// Reductions over the kLanes (8, 16 or 32) lanes of one head, in every lane.
template <int kLanes, typename T>
__device__ __forceinline__ T head_sum(T v) {
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// One group's min, max and "holds a NaN or infinity" over its lanes.
template <int kLanes>
__device__ __forceinline__ void group_range(float& lo, float& hi, uint32_t& bad) {
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m));
        hi = fmaxf(hi, __shfl_xor(hi, m));
        bad |= __shfl_xor(bad, m);
    }
}

__device__ __forceinline__ uint32_t f16_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// Quantises a lane's eight BF16 values with its group; returns the word of
// codes and sets the (s, m) pair.  All lanes of the group take part.
template <int D>
__device__ __forceinline__ uint32_t quantise8(const u32x4_t& w, uint32_t& meta) {
    constexpr int kGroupLanes = (D < W4_KV4_GROUP ? D : W4_KV4_GROUP) / 8;
    float x[8];
    unpack8(w, x);
    float lo = 3.0e38f, hi = -3.0e38f;
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bad |= !(fabsf(x[i]) <= 3.4e38f);
        x[i] = fminf(fmaxf(x[i], -65504.0f), 65504.0f);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    group_range<kGroupLanes>(lo, hi, bad);
    const float s = (float)(_Float16)((hi - lo) * (1.0f / 15.0f)), m = (float)(_Float16)lo;
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fminf(fmaxf(rintf((x[i] - m) * inv), 0.0f), 15.0f);
        word |= (uint32_t)t << (4 * i);
    }
    meta = bad ? 0x00007E00u : f16_bits(s) | (f16_bits(m) << 16);
    return bad ? 0u : word;
}

struct Turn {
    float c[8], s[8];  // of the lane's eight values (interleaved: four pairs)
};

// Norm and rotation of a lane's eight values, in T.
template <typename T, int kLanes>
__device__ __forceinline__ u32x4_t turned(const u32x4_t& w, const u32x4_t& gain, const u32x4_t& gain_partner,
                                          bool norm, float weight_add, float eps, const Turn& turn, int role,
                                          int partner, bool nan) {
    // role: 0 not rotated, 1 first of a distant pair, 2 second of one, 3 neighbouring pairs
    float x[8];
    unpack8(w, x);
    T y[8], inv = 1;
    if (norm) {
        T sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (T)x[i] * (T)x[i];
        sum = head_sum<kLanes>(sum);
        inv = (T)1 / sqrt(sum / (T)(8 * kLanes) + (T)eps);
        float g[8];
        unpack8(gain, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (T)x[i] * inv * ((T)g[i] + (T)weight_add);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
    }
    T r[8];
    u32x4_t other;
#pragma unroll
    for (int i = 0; i < 4; ++i) other[i] = __shfl(w[i], partner);
    if (role == 1 || role == 2) {
        float z[8], g[8];
        unpack8(other, z);
        if (norm) unpack8(gain_partner, g);
        const T sign = role == 1 ? (T)-1 : (T)1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T p = norm ? (T)z[i] * inv * ((T)g[i] + (T)weight_add) : (T)z[i];
            r[i] = y[i] * (T)turn.c[i] + sign * p * (T)turn.s[i];
        }
    } else if (role == 3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = y[2 * i] * (T)turn.c[i] - y[2 * i + 1] * (T)turn.s[i];
            r[2 * i + 1] = y[2 * i + 1] * (T)turn.c[i] + y[2 * i] * (T)turn.s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = y[i];
    }
    u32x4_t out;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = nan ? 0x7FC07FC0u : pack_bf16x2((float)r[2 * i], (float)r[2 * i + 1]);
    return out;
}

// The token's heads in runs of kHeads (the wave's width): q's, then k's, then
// v's.  A wave takes runs ``part``, part + parts, ... of its token.
template <int D, bool kCached>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(w4_qk_args a, Kv4 cache, int parts) {
    constexpr int kLanes = D / 8, kHeads = kWave / kLanes;
    constexpr int kGroups = D < W4_KV4_GROUP ? 1 : D / W4_KV4_GROUP;
    const int lane = threadIdx.x & (kWave - 1);
    const int li = lane % kLanes, hi = lane / kLanes;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / kWave) + sgpr(threadIdx.x / kWave);
    const int t = (int)(unit / parts), part = (int)(unit % parts);
    if (t >= a.T) return;

    bool nan = false;
    int role = 0, partner = lane;
    Turn turn = {};
    if (a.rot_dim) {
        const int pos = a.positions[t];
        if (pos < 0) return;  // padding
        nan = pos >= a.max_pos;
        const float* row = a.cos_sin + (size_t)(nan ? 0 : pos) * a.rot_dim;
        const int half = a.rot_dim / 2, e = 8 * li;
        if (e < a.rot_dim) {
            if (a.interleaved) {
                role = 3;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    turn.c[i] = row[e / 2 + i];
                    turn.s[i] = row[half + e / 2 + i];
                }
            } else {
                role = e < half ? 1 : 2;
                const int at = e < half ? e : e - half;
                partner = role == 1 ? lane + half / 8 : lane - half / 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    turn.c[i] = row[at + i];
                    turn.s[i] = row[half + at + i];
                }
            }
        }
    } else if (a.positions && a.positions[t] < 0) {
        return;
    }
    int64_t page = -1;
    int off = 0;
    if constexpr (kCached) {
        const int slot = a.slots[t];
        if (slot >= 0 && (slot >> cache.shift) < cache.blocks) {
            page = slot >> cache.shift;
            off = slot & ((1 << cache.shift) - 1);
        }
    }

    const int q_runs = (a.q_heads + kHeads - 1) / kHeads, k_runs = (a.kv_heads + kHeads - 1) / kHeads;
    const int runs = q_runs + (kCached ? 2 : 1) * k_runs;
    const int pli = (partner % kLanes);
    const auto vec = [&](const void* p, int i) {
        return reinterpret_cast<const u32x4_t*>(p)[i];
    };
    const u32x4_t zero = {0, 0, 0, 0};
    const bool qn = a.q_weight != nullptr, kn = a.k_weight != nullptr;
    u32x4_t gq = zero, gqp = zero, gk = zero, gkp = zero;
    if (qn) gq = vec(a.q_weight, li), gqp = vec(a.q_weight, pli);
    if (kn) gk = vec(a.k_weight, li), gkp = vec(a.k_weight, pli);

    for (int run = part; run < runs; run += parts) {
        // wave-uniform: which input the run is of
        const int kind = run < q_runs ? 0 : run < q_runs + k_runs ? 1 : 2;
        const int heads = kind == 0 ? a.q_heads : a.kv_heads;
        const int h = (run - (kind == 0 ? 0 : kind == 1 ? q_runs : q_runs + k_runs)) * kHeads + hi;
        const bool live = h < heads;
        const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
        const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
        u32x4_t w = zero;
        if (live) w = *reinterpret_cast<const u32x4_t*>(src + t * stride + (size_t)h * D + 8 * li);
        if (kind == 0) {
            const u32x4_t y = turned<float, kLanes>(w, gq, gqp, qn, a.weight_add, a.eps, turn, role, partner, nan);
            if (live)
                *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride + (size_t)h * D +
                                            8 * li) = y;
            continue;
        }
        if (kind == 1) {
            w = turned<double, kLanes>(w, gk, gkp, kn, a.weight_add, a.eps, turn, role, partner, nan);
            if (live && a.k_out)
                *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.k_out) + t * a.k_out_stride + (size_t)h * D +
                                            8 * li) = w;
        }
        if constexpr (kCached) {
            uint32_t meta;
            const uint32_t word = quantise8<D>(w, meta);
            if (live && page >= 0) {
                const size_t ph = (size_t)page * cache.heads + h;
                const size_t bs = (size_t)1 << cache.shift;
                if (kind == 1) {
                    cache.kc[(ph * bs + off) * kLanes + li] = word;
                } else {
                    cache.vc[((ph * (bs / 4) + off / 4) * kLanes + li) * 4 + off % 4] = word;
                }
                if (li % (kLanes / kGroups) == 0)
                    (kind == 1 ? cache.km : cache.vm)[(ph * kGroups + li / (kLanes / kGroups)) * bs + off] = meta;
            }
        }
    }
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4 cache, const int32_t* __restrict__ slots, int n,
                                                            uint16_t* k_out, uint16_t* v_out) {
    constexpr int kLanes = D / 8;
    constexpr int kGroups = D < W4_KV4_GROUP ? 1 : D / W4_KV4_GROUP;
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int li = (int)(at % kLanes);
    const int64_t row = at / kLanes;  // (token, head)
    const int h = (int)(row % cache.heads);
    const int64_t i = row / cache.heads;
    if (i >= n) return;
    const int slot = slots[i];
    if (slot < 0 || (slot >> cache.shift) >= cache.blocks) return;
    const size_t ph = (size_t)(slot >> cache.shift) * cache.heads + h;
    const size_t bs = (size_t)1 << cache.shift, off = slot & (bs - 1);
    const size_t mi = (ph * kGroups + li / (kLanes / kGroups)) * bs + off;
    const auto put = [&](uint16_t* out, uint32_t word, uint32_t meta) {
        const float s = f16_to_f32((uint16_t)meta), m = f16_to_f32((uint16_t)(meta >> 16));
        u32x4_t w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = pack_bf16x2(fmaf((float)((word >> (8 * j)) & 15u), s, m), fmaf((float)((word >> (8 * j + 4)) & 15u), s, m));
        *reinterpret_cast<u32x4_t*>(out + (size_t)row * D + 8 * li) = w;
    };
    if (k_out) put(k_out, cache.kc[(ph * bs + off) * kLanes + li], cache.km[mi]);
    if (v_out) put(v_out, cache.vc[((ph * (bs / 4) + off / 4) * kLanes + li) * 4 + off % 4], cache.vm[mi]);
}

template <int D>
hipError_t launch_d(const w4_qk_args& a, const w4_kv4_cache* c, hipStream_t stream) {
    constexpr int kHeads = kWave / (D / 8);
    const int runs = (a.q_heads + kHeads - 1) / kHeads + (c ? 2 : 1) * ((a.kv_heads + kHeads - 1) / kHeads);
    // Few tokens: one run a wave, all in flight at once; many: a token's runs
    // in one wave, which then loads its cosines and sines once.
    int parts = (8192 + a.T - 1) / a.T;
    parts = parts < 1 ? 1 : parts > runs ? runs : parts;
    const int64_t waves = (int64_t)a.T * parts, per = kThreads / kWave;
    const dim3 grid((unsigned)((waves + per - 1) / per)), block(kThreads);
    if (c) {
        qk_norm_rope_kernel<D, true><<<grid, block, 0, stream>>>(a, kv4_of(*c), parts);
    } else {
        qk_norm_rope_kernel<D, false><<<grid, block, 0, stream>>>(a, Kv4{}, parts);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const w4_qk_args& a, const w4_kv4_cache* c, hipStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_d<64>(a, c, stream);
        case 128: return launch_d<128>(a, c, stream);
        default: return launch_d<256>(a, c, stream);
    }
}

hipError_t launch_kv4_read(const w4_kv4_cache& c, const int32_t* slots, int n, void* k_out, void* v_out,
                           hipStream_t stream) {
    const Kv4 cache = kv4_of(c);
    const int64_t lanes = (int64_t)n * c.kv_heads * (c.head_dim / 8);
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads)), block(kThreads);
    uint16_t *k = static_cast<uint16_t*>(k_out), *v = static_cast<uint16_t*>(v_out);
    switch (c.head_dim) {
        case 64: kv4_read_kernel<64><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
        case 128: kv4_read_kernel<128><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
        default: kv4_read_kernel<256><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
    }
    return hipGetLastError();
}

}  // namespace w4
