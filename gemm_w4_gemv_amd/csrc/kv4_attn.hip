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
// In the outputs the 136 = 128 + 8 comes off as 136 times the sum of the
// rounded weights, which one more product per group (with ones) keeps, every
// few tiles: left in until the end, the sums of a long context would be
// 136 / 8 times larger than what they cancel to and FP32 would lose it.
//
// Layout.  S = K Q^T puts a row's scores of tokens 4 g .. 4 g + 3 (g = lane / 16)
// and 16 + 4 g .. in one lane (row = lane % 16), which is just the operand
// that O^T = V^T P^T wants from it: no exchange between lanes and no LDS in
// the loop.  The order of a product's inner index is free, so a lane loads
// its K words as 16 bytes of one token, and the values' layout (four tokens'
// words of one place together) gives it its V words as 16 bytes too.
//
// A workgroup's waves take a request's tiles in turn and join their sums in
// LDS; a launch with few rows splits the tiles over workgroups too,
// and a second kernel joins those.
#include <type_traits>

#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

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

// The tables are constant while a kernel runs: read through the constant
// address space a uniform load is a scalar one.  As a vector load it would
// queue behind the tiles in flight, and waiting for it would wait for them.
typedef const __attribute__((address_space(4))) int32_t* table_ptr;
__device__ __forceinline__ table_ptr as_table(const int32_t* p) {
    return (table_ptr)(reinterpret_cast<uintptr_t>(p));
}

// A request's rows and tokens, as this workgroup sees them.
struct Request {
    int first, rows, kv;
};
__device__ __forceinline__ Request request_of(const AttnArgs& a, int b) {
    int q0 = b, q1 = b + 1;
    if (a.q_start) {
        q0 = min(max(as_table(a.q_start)[b], 0), a.T);
        q1 = min(max(as_table(a.q_start)[b + 1], 0), a.T);
    }
    return {q0, max(q1 - q0, 0), max(as_table(a.kv_lens)[b], 0)};
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

// Where a tile lies: byte addresses, the same for all lanes (a lane adds a
// 32-bit offset of its own).  With pages of 32 tokens or more (kWide) a tile
// is in one page and its second half follows the first.
template <bool kWide>
struct Place {
    static constexpr int kN = kWide ? 1 : 2;
    uint64_t code[kN], meta[kN];
};
template <int D, bool kWide>
__device__ __forceinline__ Place<kWide> place_of(const AttnArgs& a, int t0, int head, const int page[2]) {
    Place<kWide> p;
#pragma unroll
    for (int h = 0; h < Place<kWide>::kN; ++h) {
        const uint32_t off = (uint32_t)(t0 + 16 * h) & ((1u << a.c.shift) - 1);
        const uint64_t ph = (uint64_t)(uint32_t)max(page[h], 0) * (uint32_t)a.c.heads + (uint32_t)head;
        const uint64_t slot = (ph << a.c.shift) + off;
        p.code[h] = slot * (D / 2);
        p.meta[h] = (ph << a.c.shift) * (Frag<D>::kG * 4) + off * 4;
    }
    return p;
}

// One of a lane's loads: uniform base, the lane's offset, a constant.
template <typename T>
__device__ __forceinline__ T fetch(const uint32_t* base, uint64_t uniform, uint32_t lane_off) {
    return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + uniform + lane_off);
}

// A lane's offsets within a tile.
struct Offsets {
    uint32_t k, v, meta;
};
template <int D>
__device__ __forceinline__ Offsets offsets_of(int lane) {
    const uint32_t c = lane & 15, g = lane >> 4;
    return {c * (D / 2) + (D == 64 ? 8 : 16) * g, g * (D * 2) + 16 * (D == 64 ? c >> 1 : c), 16 * g};
}

template <int D, bool kWide>
__device__ __forceinline__ void load_keys(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t code = kWide ? p.code[0] + h * 16 * (D / 2) : p.code[h % Place<kWide>::kN];
        const uint64_t meta = kWide ? p.meta[0] + h * 64 : p.meta[h % Place<kWide>::kN];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            if constexpr (kW == 4) {
                const u32x4_t w = fetch<u32x4_t>(a.c.kc, code + q * 64, l.k);
#pragma unroll
                for (int i = 0; i < 4; ++i) f.k[h][q][i] = w[i];
            } else {
                const u32x2_t w = fetch<u32x2_t>(a.c.kc, code, l.k);
                f.k[h][q][0] = w.x;
                f.k[h][q][1] = w.y;
            }
            f.km[h][q] = fetch<u32x4_t>(a.c.km, meta + (q ? (uint64_t)(4u * q << a.c.shift) : 0), l.meta);
        }
    }
}

template <int D, bool kWide>
__device__ __forceinline__ void load_values(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
    constexpr int kG = Frag<D>::kG;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t code = kWide ? p.code[0] + h * 16 * (D / 2) : p.code[h % Place<kWide>::kN];
        const uint64_t meta = kWide ? p.meta[0] + h * 64 : p.meta[h % Place<kWide>::kN];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            f.v[h][q] = fetch<u32x4_t>(a.c.vc, code + q * 256, l.v);
            f.vm[h][q] = fetch<u32x4_t>(a.c.vm, meta + (q ? (uint64_t)(4u * q << a.c.shift) : 0), l.meta);
        }
    }
}

// The table's entries for a tile's halves, as they are (0 for none): nothing
// waits for them here.
struct Entries {
    int e[2];
};
template <bool kWide>
__device__ __forceinline__ Entries entries_of(const AttnArgs& a, table_ptr table, int t0) {
    Entries x;
#pragma unroll
    for (int h = 0; h < 2; ++h) x.e[h] = kWide && h ? x.e[0] : table[min((t0 + 16 * h) >> a.c.shift, a.width - 1)];
    return x;
}
// Pages from entries; -1 where there is none for tokens that are seen.
template <bool kWide>
__device__ __forceinline__ void pages_of(const AttnArgs& a, const Entries& x, int t0, int high, int page[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (kWide && h) {
            page[1] = page[0];
            break;
        }
        const int t = t0 + 16 * h;
        const bool sound = (t >> a.c.shift) < a.width && (unsigned)x.e[h] < (unsigned)a.c.blocks;
        page[h] = t > high ? 0 : sound ? x.e[h] : -1;
    }
}

template <int D, int kNB, int kWaves, bool kWide>
__global__ __launch_bounds__(kWaves * kWave) void kv4_attn_kernel(AttnArgs a) {
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW;
    constexpr int kJ = D == 64 ? 4 : 8;  // blocks of 16 d per group
    constexpr int kCols = 16 * kNB;
    __shared__ float so[kWaves / 2][kCols][D + 4];
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
    const table_ptr table = as_table(a.table + (size_t)b * a.width);

    // this split's tiles, in turn over the waves
    const int per = (tiles.count + a.splits - 1) / a.splits;
    const int v1 = min(tiles.count, (split + 1) * per);
    int v = split * per + wave;
    const bool any = v < v1 && a.width > 0;
    const auto clamped = [&](int x) { return x < v1 ? x : v1 - 1; };

    // this lane's rows (past the last one: that one again, unseen) and their
    // queries, on their way before the first tile
    int pos[kNB];
    u32x4_t xq[kNB][kG][kW];
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        const int mine = r0 + 16 * n + c, r = min(mine, rows - 1);
        pos[n] = mine < rows ? max(first_pos + r / a.g, -1) : -1;
        const uint16_t* src = a.q + (int64_t)(req.first + r / a.g) * a.q_stride + (size_t)(head * a.g + r % a.g) * D;
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int i = 0; i < kW; ++i)
                xq[n][q][i] = *reinterpret_cast<const u32x4_t*>(src + q * W4_KV4_GROUP + (kW * g + i) * 8);
    }
    const Offsets offs = offsets_of<D>(lane);
    Frag<D> f;
    int page[2] = {-1, -1};
    Entries next = {};
    if (any) {
        const Entries now = entries_of<kWide>(a, table, tiles.at(v) * kTile);
        next = entries_of<kWide>(a, table, tiles.at(clamped(v + kWaves)) * kTile);
        pages_of<kWide>(a, now, tiles.at(v) * kTile, high, page);
        const Place<kWide> p = place_of<D, kWide>(a, tiles.at(v) * kTile, head, page);
        load_keys<D, kWide>(a, f, p, offs);
        load_values<D, kWide>(a, f, p, offs);
    }
    // the queries as the score product's operand, and their sums
    f32x4_t xstart[kNB][kG];
    float xs[kNB][kG];
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            float sum = 0;
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const u32x4_t w = xq[n][q][i];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += bf16_to_f32(w[e] & 0xFFFFu) + __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
                uint32_t in[4] = {w.x, w.y, w.z, w.w}, pr[4];
                x_pairs_for_biased(in, pr);
                xq[n][q][i] = u32x4_t{pr[0], pr[1], pr[2], pr[3]};
            }
            xs[n][q] = row_sum(sum);
            const float x0 = -128.0f * xs[n][q];
            xstart[n][q] = f32x4_t{x0, x0, x0, x0};
        }
    }

    f32x4_t o[kNB][kG][kJ], ones_sum[kNB][kG];  // of ones_sum only element 0 counts
    float extra[kNB][kG], m[kNB], l[kNB];
    float means[kNB][kG], scales[kNB][kG];  // sums of p m and p s since the last settling
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
        m[n] = -INFINITY;
        l[n] = 0;
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            extra[n][q] = means[n][q] = scales[n][q] = 0;
            ones_sum[n][q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < kJ; ++j) o[n][q][j] = f32x4_t{0, 0, 0, 0};
        }
    }

    // The running maximum moves only when a score passes it by 2^8: weights up
    // to 256 lose nothing, and a move costs a pass over the outputs.
    const float slack = 8.0f / a.scale2;
    const uint32_t bias = vgpr_const(kInt4BiasPair);
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    // takes 136 times the weights' sum off the outputs; p (m + 8 s) so far
    const auto settle = [&]() {
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                const float off = -136.0f * ones_sum[n][q][0];
                ones_sum[n][q] = f32x4_t{0, 0, 0, 0};
                extra[n][q] += fmaf(8.0f, scales[n][q], means[n][q]);
                means[n][q] = scales[n][q] = 0;
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[n][q][j][r] += off;
            }
    };
    const uint32_t half_sel = (D == 64 && (c & 1)) ? 0x07060302u : 0x05040100u;

    // The next tile's keys are fetched when the scores are done with this
    // one's, its values behind the outputs; page numbers a tile earlier.  The
    // last tile fetches itself again: under a condition the compiler would
    // load into other registers and wait for them to copy them over.
    int t0 = tiles.at(clamped(v)) * kTile, t1 = tiles.at(clamped(v + kWaves)) * kTile;
    if (!any) v = v1;
    for (int done = 1; v < v1; v += kWaves, ++done) {
        int coming[2];
        pages_of<kWide>(a, next, t1, high, coming);
        const Place<kWide> ahead = place_of<D, kWide>(a, t1, head, coming);
        const int t2 = tiles.at(clamped(v + 2 * kWaves)) * kTile;
        next = entries_of<kWide>(a, table, t2);
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
                    f32x4_t acc = xstart[n][q];
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
        __builtin_amdgcn_sched_barrier(0);  // else loads above the last use of these registers land in others
        load_keys<D, kWide>(a, f, ahead, offs);
        __builtin_amdgcn_sched_barrier(0);
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
                        // no short cuts: branches would cost more than the comparisons
                        const bool see = (t <= pos[n]) & ((a.window == 0) | (t > pos[n] - a.window) | (t < a.sinks));
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
            if (__any(top > m[n] + slack)) {
                const float now = fmaxf(m[n], top);
                const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[n] - now) * a.scale2);
                m[n] = now;
                l[n] *= keep;
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    extra[n][q] *= keep;
                    means[n][q] *= keep;
                    scales[n][q] *= keep;
                    ones_sum[n][q][0] *= keep;
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
            // what a row does not see may hold anything, an infinity or a NaN too
            const auto weigh = [&](auto masked) {
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    float ps[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            uint32_t meta = f.vm[h][q][r];
                            if constexpr (masked.value) meta = seen[n] >> (4 * h + r) & 1 ? meta : 0;
                            ps[h][r] = p[h][r] * lo16(meta);
                            means[n][q] = fmaf(p[h][r], hi16(meta), means[n][q]);
                            scales[n][q] += ps[h][r];
                        }
                    // here, not put off behind the loads that reuse f.vm's registers
                    asm volatile("" : "+v"(means[n][q]), "+v"(scales[n][q]));
                    pop[n][q] = u32x4_t{pack_bf16x2(ps[0][0], ps[0][1]), pack_bf16x2(ps[0][2], ps[0][3]),
                                        pack_bf16x2(ps[1][0], ps[1][1]), pack_bf16x2(ps[1][2], ps[1][3])};
                }
            };
            if (whole) {
                weigh(std::false_type{});
            } else {
                weigh(std::true_type{});
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
                        o[n][q][4 * z + j] = mfma(vop, pop[n][q], o[n][q][4 * z + j]);
                }
            }
#pragma unroll
            for (int n = 0; n < kNB; ++n) ones_sum[n][q] = mfma(ones, pop[n][q], ones_sum[n][q]);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_values<D, kWide>(a, f, ahead, offs);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            page[h] = coming[h];
        }
        t0 = t1;
        t1 = t2;
        if (done % 8 == 0) settle();
    }
    settle();

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
    // join the waves: common maximum, then pairwise through LDS
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
        float now = sm[0][col];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) now = fmaxf(now, sm[w][col]);
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
#pragma unroll
    for (int step = 1; step < kWaves; step *= 2) {
        const int pair = wave / (2 * step);
        if (wave % (2 * step) == step) put(pair);
        __syncthreads();
        if (wave % (2 * step) == 0) take(pair);
        if (2 * step < kWaves) __syncthreads();
    }
    if (wave != 0) return;

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

// Joins the splits of one row, a workgroup a row: D / 4 lanes hold its values,
// so 1024 / D splits are read at once.
constexpr int kMaxSplits = 128;
constexpr int kThreads = 256;
template <int D>
__global__ __launch_bounds__(kThreads) void kv4_attn_join_kernel(AttnArgs a) {
    constexpr int kLanes = D / 4, kAtOnce = kThreads / kLanes;
    __shared__ float weight[kMaxSplits];
    __shared__ f32x4_t part[kThreads];
    __shared__ float inv_sum;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int heads = a.g * a.c.heads;
    const int h = (int)(blockIdx.x % heads);
    const int i = (int)((blockIdx.x / heads) % a.max_q), b = (int)(blockIdx.x / heads / a.max_q);
    const Request req = request_of(a, b);
    if (i >= req.rows) return;
    const int t = req.first + i;
    const size_t at = ((size_t)t * heads + h) * a.splits;
    if (tid < kWave) {
        float ms[kMaxSplits / kWave], ls[kMaxSplits / kWave], now = -INFINITY, sum = 0;
#pragma unroll
        for (int u = 0; u < kMaxSplits / kWave; ++u) {
            const int s = u * kWave + lane;
            ms[u] = s < a.splits ? a.part_ml[2 * (at + s)] : -INFINITY;
            ls[u] = s < a.splits ? a.part_ml[2 * (at + s) + 1] : 0.0f;
            now = fmaxf(now, ms[u]);
        }
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1) now = fmaxf(now, __shfl_xor(now, x));
#pragma unroll
        for (int u = 0; u < kMaxSplits / kWave; ++u) {
            // a split that saw nothing has l = 0 and counts for nothing; a NaN stays one
            const float w = ls[u] == 0.0f ? 0.0f : ms[u] == -INFINITY ? NAN : __builtin_amdgcn_exp2f((ms[u] - now) * a.scale2);
            weight[u * kWave + lane] = w;
            sum += ls[u] == 0.0f ? 0.0f : w * ls[u];
        }
#pragma unroll
        for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x);
        if (lane == 0) inv_sum = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    __syncthreads();
    const int li = tid % kLanes;
    f32x4_t v = {0, 0, 0, 0};
#pragma unroll 8
    for (int s = tid / kLanes; s < a.splits; s += kAtOnce) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(a.part_o + (at + s) * D + 4 * li);
        const float w = weight[s];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(w, x[e], v[e]);
    }
    part[tid] = v;
    __syncthreads();
    if (tid >= kLanes) return;
#pragma unroll
    for (int s = 1; s < kAtOnce; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += part[s * kLanes + li][e];
    const float inv = inv_sum;
    *reinterpret_cast<u32x2_t*>(a.out + (int64_t)t * a.out_stride + (size_t)h * D + 4 * li) =
        u32x2_t{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
}

#ifndef W4_ATTN_GROUPS
#define W4_ATTN_GROUPS 512
#endif
#ifndef W4_ATTN_WAVES
#define W4_ATTN_WAVES 4
#endif
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
    int64_t want = (W4_ATTN_GROUPS + groups - 1) / (groups > 0 ? groups : 1);
    const int64_t most = tiles / (2 * W4_ATTN_WAVES);
    want = want < most ? want : most;
    return (int)(want < 1 ? 1 : want > kMaxSplits ? kMaxSplits : want);
}

template <int D, bool kWide>
hipError_t launch_d(AttnArgs& k, int64_t groups, hipStream_t stream) {
    constexpr int kWaves = W4_ATTN_WAVES;
    kv4_attn_kernel<D, kNBDefault, kWaves, kWide><<<dim3((unsigned)groups), dim3(kWaves * kWave), 0, stream>>>(k);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || k.splits == 1) return err;
    const int64_t units = (int64_t)k.B * k.max_q * k.g * k.c.heads;
    kv4_attn_join_kernel<D><<<dim3((unsigned)units), dim3(kThreads), 0, stream>>>(k);
    return hipGetLastError();
}

template <int D>
hipError_t launch_w(AttnArgs& k, int64_t groups, hipStream_t stream) {
    return k.c.shift >= 5 ? launch_d<D, true>(k, groups, stream) : launch_d<D, false>(k, groups, stream);
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
        case 64: return launch_w<64>(k, groups, stream);
        case 128: return launch_w<128>(k, groups, stream);
        default: return launch_w<256>(k, groups, stream);
    }
}

}  // namespace w4
