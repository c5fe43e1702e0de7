// Attention over the 4-bit cache, for one row a request or many.
//
// The unit of work is a wave with 16 * kNB rows (a row: one query head of one
// token, all of one key/value head) against tiles of 32 tokens.  Both products
// run on v_mfma_f32_16x16x32_bf16 with the codes as they are, never scaled:
//
//   scores   S[t][r] = s_t (A - 128 X) + m_t X,  A = sum (128 + q_td) x_rd,  X = sum x_rd
//            (per group of 128 d; -128 X is the accumulator's start)
//   outputs  O[d][r] = sum_t p s_t (q_td - 8) + sum_t p (m_t + 8 s_t)
//
// 128 + q is exact in BF16 and is one shift and one and-or per two codes.
// In the outputs the 136 = 128 + 8 is taken off again by a second product
// with a constant operand for each tile: left in until the end, the sums of
// a long context would be 136 / 8 times larger than what they cancel to and
// FP32 would lose it.  Those extra products are free: the vector unit, which
// unpacks codes and makes the softmax, is the busier one.
//
// Layout.  S = K Q^T puts a row's scores of tokens 4 g .. 4 g + 3 (g = lane / 16)
// and 16 + 4 g .. in one lane (row = lane % 16), which is just the operand
// that O^T = V^T P^T wants from it: no exchange between lanes and no LDS in
// the loop.  The order of a product's inner index is free, so a lane loads
// its K words as 16 bytes of one token, and the values' layout (four tokens'
// words of one place together) gives it its V words as 16 bytes too.
//
// A workgroup's four waves take a request's tiles in turn and join their
// sums in LDS; a launch with few rows splits the tiles over workgroups too,
// and a second kernel joins those.
#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;  // tokens

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride;
    const int32_t *table, *kv_lens, *q_start;
    Kv4 c;
    int T, B, g, width;  // g: query heads of a key/value head
    int max_q, row_tiles, splits;
    int window, sinks;
    float scale2;  // scale * log2(e)
    float* part_o;   // [T * q_heads][splits][D]
    float* part_ml;  // [T * q_heads][splits][2]
};

__device__ __forceinline__ f32x4_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Over the four lanes of one row (lane bits 4 and 5).
__device__ __forceinline__ float row_sum(float v) { return pair_sum<32>(pair_sum<16>(v)); }
__device__ __forceinline__ float row_max(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a0 = a[0], a1 = a[1];
    const float m = fmaxf(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
    const uint32_t w = __builtin_bit_cast(uint32_t, m);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const uint32_t b0 = b[0], b1 = b[1];
    return fmaxf(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
}

__device__ __forceinline__ float lo16(uint32_t v) { return f16_to_f32((uint16_t)v); }
__device__ __forceinline__ float hi16(uint32_t v) { return f16_to_f32((uint16_t)(v >> 16)); }

// The eight codes of a word as the biased operand, pairs (j, j + 4).
__device__ __forceinline__ u32x4_t key_operand(uint32_t w, uint32_t bias) {
    uint32_t p[4];
    int4_word_biased_pairs(w, bias, p);
    return u32x4_t{p[0], p[1], p[2], p[3]};
}

// A request's rows and tokens, as this workgroup sees them.
struct Request {
    int first, rows, kv;
};
__device__ __forceinline__ Request request_of(const AttnArgs& a, int b) {
    int q0 = b, q1 = b + 1;
    if (a.q_start) {
        q0 = min(max(a.q_start[b], 0), a.T);
        q1 = min(max(a.q_start[b + 1], 0), a.T);
    }
    return {q0, max(min(q1 - q0, 0x7FFFFFFF), 0), max(a.kv_lens[b], 0)};
}

// The tiles that some of a run of rows (positions low .. high) see: those of
// the first tokens, then those of the window.
struct Tiles {
    int head, from, count;  // tile v of 0 .. count - 1 is v < head ? v : v - head + from
    __device__ __forceinline__ int at(int v) const { return v < head ? v : v - head + from; }
};
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, int low, int high) {
    if (high < 0) return {0, 0, 0};
    const int end = high / kTile + 1;
    if (a.window == 0) return {0, 0, end};
    const int from = max(max(low, 0) - a.window + 1, 0) / kTile;
    const int head = min((min(a.sinks, high + 1) + kTile - 1) / kTile, from);
    return {head, from, head + end - from};
}

template <int D>
struct Frag {  // one tile's share of a lane
    static constexpr int kG = D < W4_KV4_GROUP ? 1 : D / W4_KV4_GROUP;
    static constexpr int kW = D == 64 ? 2 : 4;  // K words per group
    uint32_t k[2][kG][kW];
    u32x4_t v[2][kG];
    u32x4_t km[2][kG], vm[2][kG];
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs& a, Frag<D>& f, int t0, int head, const int page[2], int lane) {
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW, kWords = D / 8;
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int bs = 1 << a.c.shift, off = (t0 + 16 * h) & (bs - 1);
        const size_t ph = (size_t)page[h] * a.c.heads + head;
        const uint32_t* kc = a.c.kc + (ph * bs + off) * kWords;
        const uint32_t* vc = a.c.vc + (ph * bs + off) * kWords;  // (off / 4) * kWords * 4
        const uint32_t* km = a.c.km + ph * kG * bs + off;
        const uint32_t* vm = a.c.vm + ph * kG * bs + off;
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            if constexpr (kW == 4) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(kc + c * kWords + q * 16 + 4 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) f.k[h][q][i] = w[i];
            } else {
                const u32x2_t w = *reinterpret_cast<const u32x2_t*>(kc + c * kWords + 2 * g);
                f.k[h][q][0] = w.x;
                f.k[h][q][1] = w.y;
            }
            const int vw = D == 64 ? c >> 1 : q * 16 + c;
            f.v[h][q] = *reinterpret_cast<const u32x4_t*>(vc + (g * kWords + vw) * 4);
            f.km[h][q] = *reinterpret_cast<const u32x4_t*>(km + q * bs + 4 * g);
            f.vm[h][q] = *reinterpret_cast<const u32x4_t*>(vm + q * bs + 4 * g);
        }
    }
}

// Pages of a tile's halves; -1 where the table has none for tokens that are seen.
__device__ __forceinline__ void pages_of(const AttnArgs& a, const int32_t* table, int t0, int high, int page[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = t0 + 16 * h, p = t >> a.c.shift;
        int id = 0;
        if (t <= high) {
            id = p < a.width ? table[p] : -1;
            if (id >= a.c.blocks) id = -1;
        }
        page[h] = (int)sgpr((uint32_t)max(id, -1));
    }
}

template <int D, int kNB>
__global__ __launch_bounds__(kThreads) void kv4_attn_kernel(AttnArgs a) {
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW;
    constexpr int kJ = D == 64 ? 4 : 8;  // blocks of 16 d per group
    constexpr int kCols = 16 * kNB;
    __shared__ float so[2][kCols][D + 4];
    __shared__ float sm[kWaves][kCols], sl[kWaves][kCols];

    const int lane = threadIdx.x & (kWave - 1), wave = (int)sgpr(threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    // key/value heads innermost: workgroups that share a head's pages meet on one XCD
    int id = blockIdx.x;
    const int head = id % a.c.heads;
    id /= a.c.heads;
    const int split = id % a.splits;
    id /= a.splits;
    const int row_tile = a.row_tiles - 1 - id % a.row_tiles;  // the longest first
    const int b = id / a.row_tiles;

    const Request req = request_of(a, b);
    const int rows = min(req.rows, a.max_q) * a.g;  // < 2^31: checked on the host
    const int r0 = row_tile * kCols;
    if (r0 >= rows) return;
    const int first_pos = req.kv - req.rows;
    const int low = first_pos + r0 / a.g, high = first_pos + (min(r0 + kCols, rows) - 1) / a.g;
    const Tiles tiles = tiles_of(a, low, high);
    const int32_t* table = a.table + (size_t)b * a.width;

    // this lane's rows, their queries as the score product's operand and sums
    int pos[kNB];
    u32x4_t xq[kNB][kG][kW];
    float xs[kNB][kG];
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        const int r = r0 + 16 * n + c;
        const bool live = r < rows;
        pos[n] = live ? max(first_pos + r / a.g, -1) : -1;
        const uint16_t* src = a.q + (int64_t)(req.first + r / a.g) * a.q_stride + (size_t)(head * a.g + r % a.g) * D;
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            float sum = 0;
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                u32x4_t w = {0, 0, 0, 0};
                if (live) w = *reinterpret_cast<const u32x4_t*>(src + q * W4_KV4_GROUP + (kW * g + i) * 8);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += bf16_to_f32(w[e] & 0xFFFFu) + __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
                uint32_t in[4] = {w.x, w.y, w.z, w.w}, pr[4];
                x_pairs_for_biased(in, pr);
                xq[n][q][i] = u32x4_t{pr[0], pr[1], pr[2], pr[3]};
            }
            xs[n][q] = row_sum(sum);
        }
    }

    f32x4_t o[kNB][kG][kJ];
    float extra[kNB][kG], m[kNB], l[kNB];
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        m[n] = -INFINITY;
        l[n] = 0;
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            extra[n][q] = 0;
#pragma unroll
            for (int j = 0; j < kJ; ++j) o[n][q][j] = f32x4_t{0, 0, 0, 0};
        }
    }

    const uint32_t bias = vgpr_const(kInt4BiasPair);
    const uint32_t c136 = 0xC308C308u;  // bf16 pair (-136, -136)
    const u32x4_t minus = {c136, c136, c136, c136};
    const uint32_t half_sel = (D == 64 && (c & 1)) ? 0x07060302u : 0x05040100u;

    // this split's tiles, in turn over the waves
    const int per = (tiles.count + a.splits - 1) / a.splits;
    const int v1 = min(tiles.count, (split + 1) * per);
    for (int v = split * per + wave; v < v1; v += kWaves) {
        const int t0 = tiles.at(v) * kTile;
        int page[2];
        pages_of(a, table, t0, high, page);
        Frag<D> f;
        {
            const int at[2] = {max(page[0], 0), max(page[1], 0)};
            load_tile<D>(a, f, t0, head, at, lane);
        }
        // Whether every row sees every token of the tile.
        const bool whole = t0 + kTile - 1 <= low && (a.window == 0 || t0 > high - a.window || t0 + kTile <= a.sinks) &&
                           page[0] >= 0 && page[1] >= 0 && r0 + kCols <= rows;

        // scores
        float s[kNB][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                u32x4_t kop[kW];
#pragma unroll
                for (int i = 0; i < kW; ++i) kop[i] = key_operand(f.k[h][q][i], bias);
#pragma unroll
                for (int n = 0; n < kNB; ++n) {
                    const float x0 = -128.0f * xs[n][q];
                    f32x4_t acc = {x0, x0, x0, x0};
#pragma unroll
                    for (int i = 0; i < kW; ++i) acc = mfma(kop[i], xq[n][q][i], acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float base = q == 0 ? 0.0f : s[n][h][r];
                        s[n][h][r] = fmaf(lo16(f.km[h][q][r]), acc[r], fmaf(hi16(f.km[h][q][r]), xs[n][q], base));
                    }
                }
            }
        }
        uint32_t seen[kNB];  // bit 4 h + r
#pragma unroll
        for (int n = 0; n < kNB; ++n) seen[n] = 0xFFu;
        if (!whole) {
#pragma unroll
            for (int n = 0; n < kNB; ++n) {
                seen[n] = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = t0 + 16 * h + 4 * g + r;
                        const bool see = t <= pos[n] && (a.window == 0 || t > pos[n] - a.window || t < a.sinks);
                        if (see) seen[n] |= 1u << (4 * h + r);
                        s[n][h][r] = !see ? -INFINITY : page[h] < 0 ? NAN : s[n][h][r];
                    }
            }
        }

        // softmax and the second product's operand, per row block
        u32x4_t pop[kNB][kG];
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                              fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
            top = row_max(top);
            if (__any(top > m[n])) {
                const float now = fmaxf(m[n], top);
                const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[n] - now) * a.scale2);
                m[n] = now;
                l[n] *= keep;
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    extra[n][q] *= keep;
#pragma unroll
                    for (int j = 0; j < kJ; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[n][q][j][r] *= keep;
                }
            }
            const float base = m[n] == -INFINITY ? 0.0f : m[n] * a.scale2;
            float p[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[h][r] = __builtin_amdgcn_exp2f(fmaf(s[n][h][r], a.scale2, -base));
                    l[n] += p[h][r];
                }
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                float ps[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t meta = f.vm[h][q][r];
                        float sv = lo16(meta), mv = hi16(meta);
                        // what a row does not see may hold anything, an infinity or a NaN too
                        if (!whole && !(seen[n] >> (4 * h + r) & 1)) sv = mv = 0.0f;
                        ps[h][r] = p[h][r] * sv;
                        extra[n][q] = fmaf(p[h][r], fmaf(8.0f, sv, mv), extra[n][q]);
                    }
                pop[n][q] = u32x4_t{pack_bf16x2(ps[0][0], ps[0][1]), pack_bf16x2(ps[0][2], ps[0][3]),
                                    pack_bf16x2(ps[1][0], ps[1][1]), pack_bf16x2(ps[1][2], ps[1][3])};
            }
        }

        // outputs
#pragma unroll
        for (int q = 0; q < kG; ++q) {
#pragma unroll
            for (int z = 0; z < (D == 64 ? 1 : 2); ++z) {
                // codes 4 z .. 4 z + 3 of each token pair, one token in each half
                uint32_t pr[4];
                const uint32_t sel = D == 64 ? half_sel : z ? 0x07060302u : 0x05040100u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4_t w = f.v[i >> 1][q];
                    pr[i] = __builtin_amdgcn_perm(w[2 * (i & 1) + 1], w[2 * (i & 1)], sel);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32x4_t vop;
#pragma unroll
                    for (int i = 0; i < 4; ++i) vop[i] = ((pr[i] >> (4 * j)) & 0x000F000Fu) | bias;
#pragma unroll
                    for (int n = 0; n < kNB; ++n)
                        o[n][q][4 * z + j] = mfma(minus, pop[n][q], mfma(vop, pop[n][q], o[n][q][4 * z + j]));
                }
            }
        }
    }

    // each wave's own part, whole over its tokens
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        l[n] = row_sum(l[n]);
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            const float e = row_sum(extra[n][q]);
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[n][q][j][r] += e;
        }
    }
    // join the four waves: common maximum, then two rounds through LDS
    if (lane < 16) {
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            sm[wave][16 * n + c] = m[n];
            sl[wave][16 * n + c] = l[n];
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        const int col = 16 * n + c;
        const float now = fmaxf(fmaxf(sm[0][col], sm[1][col]), fmaxf(sm[2][col], sm[3][col]));
        const auto weight = [&](float x) { return x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((x - now) * a.scale2); };
        float sum = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            // a wave that saw nothing has l = 0; a NaN stays one
            const float lw = sl[w][col];
            sum += lw == 0.0f ? 0.0f : lw * weight(sm[w][col]);
        }
        const float mine = l[n] == 0.0f ? 0.0f : weight(m[n]);
        l[n] = sum;
        m[n] = now;
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[n][q][j][r] *= mine;
    }
    // d of (q, j, r): 128 q + 8 (4 g + r) + j, or 4 (4 g + r) + j for heads of 64
    const auto place = [&](int q, int r) { return D == 64 ? 4 * (4 * g + r) : q * W4_KV4_GROUP + 8 * (4 * g + r); };
    const auto put = [&](int slot) {
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kJ; ++j) so[slot][16 * n + c][place(q, r) + j] = o[n][q][j][r];
    };
    const auto take = [&](int slot) {
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kJ; ++j) o[n][q][j][r] += so[slot][16 * n + c][place(q, r) + j];
    };
    if (wave & 1) put(wave >> 1);
    __syncthreads();
    if (!(wave & 1)) take(wave >> 1);
    __syncthreads();
    if (wave == 2) put(0);
    __syncthreads();
    if (wave != 0) return;
    take(0);

#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        const int row = r0 + 16 * n + c;
        if (row >= rows) continue;
        const int t = req.first + row / a.g, h = head * a.g + row % a.g;
        if (a.splits == 1) {
            const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
            uint16_t* dst = a.out + (int64_t)t * a.out_stride + (size_t)h * D;
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    uint32_t w[kJ / 2];
#pragma unroll
                    for (int j = 0; j < kJ; j += 2) w[j / 2] = pack_bf16x2(o[n][q][j][r] * inv, o[n][q][j + 1][r] * inv);
                    if constexpr (kJ == 8) {
                        *reinterpret_cast<u32x4_t*>(dst + place(q, r)) = u32x4_t{w[0], w[1], w[2], w[3]};
                    } else {
                        *reinterpret_cast<u32x2_t*>(dst + place(q, r)) = u32x2_t{w[0], w[1]};
                    }
                }
        } else {
            const size_t at = ((size_t)t * a.g * a.c.heads + h) * a.splits + split;
            if (g == 0) {
                a.part_ml[2 * at] = m[n];
                a.part_ml[2 * at + 1] = l[n];
            }
            float* dst = a.part_o + at * D;
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kJ; j += 4)
                        *reinterpret_cast<f32x4_t*>(dst + place(q, r) + j) =
                            f32x4_t{o[n][q][j][r], o[n][q][j + 1][r], o[n][q][j + 2][r], o[n][q][j + 3][r]};
        }
    }
}

// Joins the splits of one row; a lane owns D / 64 values.
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_attn_join_kernel(AttnArgs a) {
    constexpr int kPer = D / kWave;
    const int lane = threadIdx.x & (kWave - 1);
    const int heads = a.g * a.c.heads;
    const int64_t unit = (int64_t)blockIdx.x * kWaves + sgpr(threadIdx.x / kWave);
    const int h = (int)(unit % heads);
    const int i = (int)((unit / heads) % a.max_q), b = (int)(unit / heads / a.max_q);
    if (b >= a.B) return;
    const Request req = request_of(a, b);
    if (i >= req.rows) return;
    const int t = req.first + i;
    const size_t at = ((size_t)t * heads + h) * a.splits;
    float now = -INFINITY;
    for (int s = 0; s < a.splits; ++s) now = fmaxf(now, a.part_ml[2 * (at + s)]);
    float sum = 0, v[kPer] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float ms = a.part_ml[2 * (at + s)], ls = a.part_ml[2 * (at + s) + 1];
        if (ls == 0.0f) continue;
        const float w = ms == -INFINITY ? NAN : __builtin_amdgcn_exp2f((ms - now) * a.scale2);
        sum += w * ls;
        const float* src = a.part_o + (at + s) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = fmaf(w, src[e], v[e]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* dst = a.out + (int64_t)t * a.out_stride + (size_t)h * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) dst[e] = f32_to_bf16(v[e] * inv);
}

constexpr int kNBDefault = 1;

int row_tiles_of(const w4_attn_args& a, const w4_kv4_cache& c) {
    const int64_t rows = (int64_t)a.max_q * (a.q_heads / c.kv_heads);
    return (int)((rows + 16 * kNBDefault - 1) / (16 * kNBDefault));
}

// How many workgroups share one row tile's tokens: enough to fill the chip
// twice, at least two tiles for each of a workgroup's waves.
int splits_of(const w4_attn_args& a, const w4_kv4_cache& c) {
    const int64_t groups = (int64_t)a.B * c.kv_heads * row_tiles_of(a, c);
    int64_t tokens = a.max_kv;
    if (a.window > 0) tokens = tokens < (int64_t)a.window + a.sinks + a.max_q ? tokens : (int64_t)a.window + a.sinks + a.max_q;
    const int64_t tiles = (tokens + kTile - 1) / kTile;
    int64_t want = (512 + groups - 1) / (groups > 0 ? groups : 1);
    const int64_t most = tiles / (2 * kWaves);
    want = want < most ? want : most;
    return (int)(want < 1 ? 1 : want > 128 ? 128 : want);
}

template <int D>
hipError_t launch_d(AttnArgs& k, int64_t groups, hipStream_t stream) {
    kv4_attn_kernel<D, kNBDefault><<<dim3((unsigned)groups), dim3(kThreads), 0, stream>>>(k);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || k.splits == 1) return err;
    const int64_t units = (int64_t)k.B * k.max_q * k.g * k.c.heads;
    kv4_attn_join_kernel<D><<<dim3((unsigned)((units + kWaves - 1) / kWaves)), dim3(kThreads), 0, stream>>>(k);
    return hipGetLastError();
}

}  // namespace

size_t kv4_attn_workspace_bytes(const w4_attn_args& a, const w4_kv4_cache& c) {
    const int splits = splits_of(a, c);
    if (splits == 1) return 0;
    return (size_t)a.T * a.q_heads * splits * (c.head_dim + 2) * sizeof(float);
}

hipError_t launch_kv4_attn(const w4_attn_args& a, const w4_kv4_cache& c, void* workspace, hipStream_t stream) {
    AttnArgs k = {};
    k.q = static_cast<const uint16_t*>(a.q);
    k.out = static_cast<uint16_t*>(a.out);
    k.q_stride = a.q_stride;
    k.out_stride = a.out_stride;
    k.table = a.block_table;
    k.kv_lens = a.kv_lens;
    k.q_start = a.q_start;
    k.c = kv4_of(c);
    k.T = a.T;
    k.B = a.B;
    k.g = a.q_heads / c.kv_heads;
    k.width = a.max_blocks;
    k.max_q = a.max_q;
    k.row_tiles = row_tiles_of(a, c);
    k.splits = splits_of(a, c);
    k.window = a.window;
    k.sinks = a.sinks;
    k.scale2 = a.scale * 1.4426950408889634f;
    if (k.splits > 1) {
        k.part_o = static_cast<float*>(workspace);
        k.part_ml = k.part_o + (size_t)a.T * a.q_heads * k.splits * c.head_dim;
    }
    const int64_t groups = (int64_t)a.B * c.kv_heads * k.row_tiles * k.splits;
    switch (c.head_dim) {
        case 64: return launch_d<64>(k, groups, stream);
        case 128: return launch_d<128>(k, groups, stream);
        default: return launch_d<256>(k, groups, stream);
    }
}

}  // namespace w4
