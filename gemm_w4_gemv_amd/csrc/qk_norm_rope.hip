// RMS norm of query and key heads, rotation by position, and keys and values
// quantised into the 4-bit cache, in one pass; and the cache read back.
//
// Eight values a lane: a head is a run of D / 8 lanes, so a wave holds
// 64 / (D / 8) heads of one token and walks over the token's heads.  With
// weights w, the rotated value is
//   inv * (x_i (w_i c_i) -+ x_j (w_j s_i)),  inv = 1 / sqrt(mean(x^2) + eps),
// and what stands in brackets is the token's, made once: two multiply-adds
// and a product a value are left for each head.  The partner x_j is in the
// lane or in one lane of the same head, taken as raw BF16 (four exchanges).  A
// lane's eight 4-bit codes are one word of the cache.
// Memory bounds it for prompts, as long as enough of it is asked for at once
// (four heads' loads ahead): 8192 tokens of 40 heads of 128 without a cache 39 us,
// 4.3 TB/s.  4099 tokens of 32 heads of 256 into the cache take 38 us, half of the
// waves' cycles waits: 72 MB are read as they must be, but 58 MB written where 43
// are due, for the cache is written four bytes at a time (values' words at a stride
// of 16).  Launch and latency bound a decode step, where the token's heads are
// spread over waves instead.
#include <type_traits>

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

// Exchanges inside a head's kLanes (8, 16 or 32) lanes, without LDS: across
// lane bit 4 by a row swap, below it by DPP, from the highest bit down.
template <int kOff, typename F>
__device__ __forceinline__ float folded(float v, F f) {
    if constexpr (kOff == 16) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t r0 = r[0], r1 = r[1];
        return f(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
    } else {
        return f(v, dpp_partner<kOff>(v));
    }
}
template <int kOff, typename F>
__device__ __forceinline__ double folded(double v, F f) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
    const auto join = [](uint32_t l, uint32_t h) { return __builtin_bit_cast(double, (uint64_t)h << 32 | l); };
    if constexpr (kOff == 16) {
        const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        const uint32_t a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1];
        return f(join(a0, b0), join(a1, b1));
    } else {
        return f(v, join(__builtin_bit_cast(uint32_t, dpp_partner<kOff>(__builtin_bit_cast(float, lo))),
                         __builtin_bit_cast(uint32_t, dpp_partner<kOff>(__builtin_bit_cast(float, hi)))));
    }
}
template <int kLanes, typename T, typename F>
__device__ __forceinline__ T head_fold(T v, F f) {
    if constexpr (kLanes > 1) return head_fold<kLanes / 2>(folded<kLanes / 2>(v, f), f);
    return v;
}
template <int kLanes, typename T>
__device__ __forceinline__ T head_sum(T v) {
    return head_fold<kLanes>(v, [](T a, T b) { return a + b; });
}

// A value in FP32, where it is rounded: out of the compiler's sight, which joins
// two conversions that follow each other (FP64 to FP32 to BF16), and a product
// with its conversion to FP16, into one rounding.
__device__ __forceinline__ float in_f32(float v) {
    asm("" : "+v"(v));
    return v;
}

__device__ __forceinline__ uint32_t f16_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// Quantises a lane's eight BF16 values with its group; returns the word of
// codes and sets the (s, m) pair.  All lanes of the group take part.
template <int D>
__device__ __forceinline__ uint32_t quantise8(const u32x4_t& w, uint32_t& meta) {
    constexpr int kGroupLanes = (D < W4_KV4_GROUP ? D : W4_KV4_GROUP) / 8;
    float x[8];
    unpack8(w, x);
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = x[i] == x[i] ? x[i] : INFINITY;  // min and max pass a NaN over
        lo = fminf(lo, y);
        hi = fmaxf(hi, y);
    }
    lo = head_fold<kGroupLanes>(lo, [](float a, float b) { return fminf(a, b); });
    hi = head_fold<kGroupLanes>(hi, [](float a, float b) { return fmaxf(a, b); });
    const bool bad = !(lo > -INFINITY && hi < INFINITY);
    lo = fminf(fmaxf(lo, -65504.0f), 65504.0f);
    hi = fminf(fmaxf(hi, -65504.0f), 65504.0f);
    const float s = (float)(_Float16)in_f32((hi - lo) * (1.0f / 15.0f)), m = (float)(_Float16)lo;
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // a value past +-65504 ends at 0 or 15 like that one
        const float t = __builtin_amdgcn_fmed3f(rintf((x[i] - m) * inv), 0.0f, 15.0f);
        word |= (uint32_t)t << (4 * i);
    }
    meta = bad ? 0x00007E00u : f16_bits(s) | (f16_bits(m) << 16);
    return bad ? 0u : word;
}

__device__ __forceinline__ double half_of(uint32_t pair, int k) { return bf16_to_f32(k ? pair >> 16 : pair & 0xFFFFu); }

template <int kLanes, typename T>
__device__ __forceinline__ T mean_square(const u32x4_t& w) {
    float x[8];
    unpack8(w, x);
    T sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (T)x[i] * (T)x[i];
    return head_sum<kLanes>(sum) * (T)(1.0 / (8 * kLanes));
}

// What a token's position and the weights make of a lane's eight values:
// y = inv * (x * own + partner * other).
template <typename T>
struct Turn {
    T own[8], other[8];
};

// The eight values of a lane after norm and rotation.  ``partner`` is the lane
// that holds the other values of its pairs, unless they are neighbours.  far: in
// FP32, whether the head's mean square lies where its squares or the factor
// 1 / sqrt(mean square) come near the ends of FP32's range (a NaN does).
template <int kLanes, bool kNeighbours, typename T>
__device__ __forceinline__ u32x4_t turned(const u32x4_t& w, const Turn<T>& turn, bool norm, float eps, bool rotated,
                                          int partner, bool nan, bool& far) {
    float x[8], z[8];
    unpack8(w, x);
    if constexpr (kNeighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = x[i ^ 1];
    } else {
        u32x4_t other;
#pragma unroll
        for (int i = 0; i < 4; ++i) other[i] = __shfl(w[i], partner);
        unpack8(other, z);
    }
    T inv = 1;
    if (norm) {
        const T square = mean_square<kLanes, T>(w) + (T)eps;
        far = !(square > (T)0x1p-40 && square < (T)0x1p40);
        inv = (T)1 / sqrt(square);
    }
    u32x4_t out;
    T r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // an unrotated value takes no part of another, which may be an infinity
        r[i] = ((T)x[i] * turn.own[i] + (T)(rotated ? z[i] : 0.0f) * turn.other[i]) * inv;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = (float)r[i];
        if constexpr (sizeof(T) == 8) x[i] = in_f32(x[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = nan ? 0x7FC07FC0u : pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return out;
}

// The token's heads in runs of kHeads (the wave's width): q's, then k's, then
// v's.  A wave takes runs ``part``, part + parts, ... of its token, four loads
// at a time.
template <int D, bool kCached, bool kNeighbours>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(w4_qk_args a, Kv4 cache, int parts) {
    constexpr int kLanes = D / 8, kHeads = kWave / kLanes;
    constexpr int kGroups = D < W4_KV4_GROUP ? 1 : D / W4_KV4_GROUP;
    const int lane = threadIdx.x & (kWave - 1);
    const int li = lane % kLanes, hi = lane / kLanes, e = 8 * li;
    const uint32_t unit = blockIdx.x * (kThreads / kWave) + sgpr(threadIdx.x / kWave);
    const int t = (int)(unit / (uint32_t)parts), part = (int)(unit % (uint32_t)parts);
    if (t >= a.T) return;
    const int pos = a.positions ? (int)sgpr((uint32_t)a.positions[t]) : 0;
    if (pos < 0) return;  // padding

    const bool nan = a.rot_dim && pos >= a.max_pos;
    const int half = a.rot_dim / 2;
    const bool rotated = e < a.rot_dim, first = e < half;
    const int partner = kNeighbours || !rotated ? lane : first ? lane + half / 8 : lane - half / 8;
    float c[8] = {1, 1, 1, 1, 1, 1, 1, 1}, s[8] = {};
    if (rotated) {
        const float* row = a.cos_sin + (size_t)(nan ? 0 : pos) * a.rot_dim;
        const auto four = [](const float* p) { return *reinterpret_cast<const f32x4_t*>(p); };
        // y_i = x_i c - x_j s for the first of a pair, x_j c + x_i s for the second
        if constexpr (kNeighbours) {
            const f32x4_t vc = four(row + e / 2), vs = four(row + half + e / 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = vc[i / 2];
                s[i] = i % 2 ? vs[i / 2] : -vs[i / 2];
            }
        } else {
            const float* at = row + (first ? e : e - half);
            const f32x4_t vc[2] = {four(at), four(at + 4)}, vs[2] = {four(at + half), four(at + half + 4)};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = vc[i / 4][i % 4];
                s[i] = first ? -vs[i / 4][i % 4] : vs[i / 4][i % 4];
            }
        }
    }
    const auto turn_of = [&](const void* weight, auto& turn) {
        typedef std::remove_reference_t<decltype(turn.own[0])> T;
        const u32x4_t one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(weight);
        const T add = weight ? (T)a.weight_add : (T)0;
        float g[8], gp[8];
        unpack8(weight ? p[li] : one, g);
        unpack8(weight ? p[partner % kLanes] : one, gp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            turn.own[i] = ((T)g[i] + add) * (T)c[i];
            turn.other[i] = ((T)gp[kNeighbours ? i ^ 1 : i] + add) * (T)s[i];
        }
    };

    int64_t page = -1;
    int off = 0;
    if constexpr (kCached) {
        const int slot = (int)sgpr((uint32_t)a.slots[t]);
        if (slot >= 0 && (slot >> cache.shift) < cache.blocks) {
            page = slot >> cache.shift;
            off = slot & ((1 << cache.shift) - 1);
        }
    }
    // Quantises a lane's values of head h into the cache.
    const auto store = [&](const u32x4_t& y, int h, uint32_t* codes, uint32_t* metas, bool values) {
        uint32_t meta;
        const uint32_t word = quantise8<D>(y, meta);
        if (h >= a.kv_heads || page < 0) return;
        const size_t ph = (size_t)page * cache.heads + h, bs = (size_t)1 << cache.shift;
        codes[values ? ((ph * (bs / 4) + off / 4) * kLanes + li) * 4 + off % 4 : (ph * bs + off) * kLanes + li] = word;
        if (li % (kLanes / kGroups) == 0) metas[(ph * kGroups + li / (kLanes / kGroups)) * bs + off] = meta;
    };
    // Calls f(values, head) for this wave's runs of one input, from its run on.
    // f may ask for a call of g instead, with the same, by giving true; it has
    // then written nothing, so the values are read again (an output may be its
    // input), in a loop of its own: inside the other it would hold a third of the registers.
    const auto each = [&](const void* in, int64_t stride, int heads, int from, auto f, auto g) {
        constexpr int kAhead = 4;
        const uint16_t* src = static_cast<const uint16_t*>(in) + t * stride + e;
        const int runs = (heads + kHeads - 1) / kHeads;
        const auto values = [&](int run) {
            const int h = min(run * kHeads + hi, heads - 1);  // behind the last head: that one again
            return *reinterpret_cast<const u32x4_t*>(src + (size_t)h * D);
        };
        for (int r = from; r < runs; r += kAhead * parts) {
            u32x4_t w[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (r + u * parts < runs) w[u] = values(r + u * parts);
            uint32_t again = 0;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (r + u * parts < runs) again |= (uint32_t)f(w[u], (r + u * parts) * kHeads + hi) << u;
            if (__any(again != 0)) {
#pragma unroll 1
                for (int u = 0; u < kAhead; ++u) {
                    const bool mine = again >> u & 1;
                    if (!__any(mine)) continue;
                    const u32x4_t x = values(r + u * parts);
                    g(x, (r + u * parts) * kHeads + hi, mine);
                }
            }
        }
        // where the next input's runs go on
        return from < runs ? (parts - (runs - from) % parts) % parts : from - runs;
    };
    const auto never = [](const u32x4_t&, int, bool) {};

    int at = part;
    if (a.q_heads > 0) {
        Turn<float> turn;
        turn_of(a.q_weight, turn);
        // Weights whose products with a query could pass FP32's range: the token's, so the same for all its heads.
        float most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fmaxf(fabsf(turn.own[i]), fabsf(turn.other[i])));
        const bool wild = a.q_weight && __any(!(most < 0x1p60f));
        uint16_t* out = static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride + e;
        const auto put = [&](const u32x4_t& y, int h) { *reinterpret_cast<u32x4_t*>(out + (size_t)h * D) = y; };
        at = each(a.q, a.q_stride, a.q_heads, at, [&](const u32x4_t& w, int h) {
            bool far = false;
            const u32x4_t y = turned<kLanes, kNeighbours>(w, turn, a.q_weight != nullptr, a.eps, rotated, partner, nan, far);
            if (h < a.q_heads && !(far | wild)) put(y, h);
            return far | wild;
        }, [&](const u32x4_t& w, int h, bool mine) {
            // Such a head in FP64, whose range holds all of it; the others have
            // what they have, whatever stands beside them.  Two values at a time
            // and with their factors made here: in advance they would hold registers.
            const u32x4_t* p = reinterpret_cast<const u32x4_t*>(a.q_weight);
            const u32x4_t g = p[li], gp = p[partner % kLanes];
            u32x4_t y, z = w;
            if constexpr (!kNeighbours) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = __shfl(w[i], partner);
            }
            const double inv = 1.0 / sqrt(mean_square<kLanes, double>(w) + (double)a.eps), add = a.weight_add;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                asm volatile("" : "+v"(c[2 * i]), "+v"(c[2 * i + 1]), "+v"(s[2 * i]), "+v"(s[2 * i + 1]));
                float r[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int pair = kNeighbours ? 1 - k : k;
                    const double own = (half_of(g[i], k) + add) * c[2 * i + k];
                    const double other = (half_of(gp[i], pair) + add) * s[2 * i + k];
                    r[k] = (float)((half_of(w[i], k) * own + (rotated ? half_of(z[i], pair) : 0.0) * other) * inv);
                }
                y[i] = nan ? 0x7FC07FC0u : pack_bf16x2(in_f32(r[0]), in_f32(r[1]));
                __builtin_amdgcn_sched_barrier(0);
            }
            if (h < a.q_heads && mine) put(y, h);
        });
    }
    if (at < (a.kv_heads + kHeads - 1) / kHeads) {
        Turn<double> turn;
        turn_of(a.k_weight, turn);
        at = each(a.k, a.k_stride, a.kv_heads, at, [&](const u32x4_t& w, int h) {
            bool any;
            const u32x4_t y = turned<kLanes, kNeighbours>(w, turn, a.k_weight != nullptr, a.eps, rotated, partner, nan, any);
            if (h < a.kv_heads && a.k_out)
                *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.k_out) + t * a.k_out_stride + e + (size_t)h * D) = y;
            if constexpr (kCached) store(y, h, cache.kc, cache.km, false);
            return false;
        }, never);
    } else {
        at -= (a.kv_heads + kHeads - 1) / kHeads;
    }
    if constexpr (kCached)
        each(a.v, a.v_stride, a.kv_heads, at, [&](const u32x4_t& w, int h) {
            store(w, h, cache.vc, cache.vm, true);
            return false;
        }, never);
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

// Waves that share a token: few tokens, one run of heads each, all in flight at
// once; many, one wave, which then loads its cosines and sines once.
int64_t parts_of(const w4_qk_args& a, bool cached) {
    const int64_t heads = kWave / (a.head_dim / 8);
    const int64_t runs = (a.q_heads + heads - 1) / heads + (cached ? 2 : 1) * ((a.kv_heads + heads - 1) / heads);
    const int64_t parts = (8192 + (int64_t)a.T - 1) / a.T;
    return parts > runs ? runs : parts;
}

template <int D>
hipError_t launch_d(const w4_qk_args& a, const w4_kv4_cache* c, hipStream_t stream) {
    const int parts = (int)parts_of(a, c != nullptr);
    const dim3 grid((unsigned)qk_norm_rope_groups(a, c != nullptr)), block(kThreads);
    const Kv4 cache = c ? kv4_of(*c) : Kv4{};
    if (c) {
        if (a.interleaved) {
            qk_norm_rope_kernel<D, true, true><<<grid, block, 0, stream>>>(a, cache, parts);
        } else {
            qk_norm_rope_kernel<D, true, false><<<grid, block, 0, stream>>>(a, cache, parts);
        }
    } else if (a.interleaved) {
        qk_norm_rope_kernel<D, false, true><<<grid, block, 0, stream>>>(a, cache, parts);
    } else {
        qk_norm_rope_kernel<D, false, false><<<grid, block, 0, stream>>>(a, cache, parts);
    }
    return hipGetLastError();
}

}  // namespace

int64_t qk_norm_rope_groups(const w4_qk_args& a, bool cached) {
    const int64_t per = kThreads / kWave;
    return ((int64_t)a.T * parts_of(a, cached) + per - 1) / per;
}
int64_t kv4_read_groups(const w4_kv4_cache& c, int n) {
    return ((int64_t)n * c.kv_heads * (c.head_dim / 8) + kThreads - 1) / kThreads;
}

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
    const dim3 grid((unsigned)kv4_read_groups(c, n)), block(kThreads);
    uint16_t *k = static_cast<uint16_t*>(k_out), *v = static_cast<uint16_t*>(v_out);
    switch (c.head_dim) {
        case 64: kv4_read_kernel<64><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
        case 128: kv4_read_kernel<128><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
        default: kv4_read_kernel<256><<<grid, block, 0, stream>>>(cache, slots, n, k, v); break;
    }
    return hipGetLastError();
}

}  // namespace w4
