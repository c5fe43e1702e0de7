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
// (p s is rounded to BF16, in two parts: see two_parts.)
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
//
// Measured: 32 requests of up to 8192 tokens, 16 query and 8 key/value heads of
// 256: 77 us, 4.7 TB/s of codes and pairs (requests of equal length with as many
// tokens 69, the longest first 70); one of 131071 tokens, 32 and 8 heads of 128: 31
// us, 4.6 TB/s; a prompt's 2048 tokens after 2048 others, 16 and 8 heads of 256: 204
// us, 505 TFLOP/s.
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
    bool in_turn;
    int window, sinks;
    float scale2;  // scale * log2(e)
    float* part_o;   // [T * q_heads][splits][D]
    float* part_ml;  // [T * q_heads][splits][2]
};

__device__ __forceinline__ f32x4_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// A pair of weights in two parts, each of BF16.  As one part a weight is off by
// up to 2^-8 of itself, which moves an output by about as much as its own
// rounding to BF16 (error against 64 bits 2.3e-3 instead of 1.7e-3); the second
// part costs one more product a block of values.  Memory bounds the decode
// kernels (32 requests up to 8192 tokens: 77 us either way); long prompts, bound by
// instructions, pay a seventh (2048 tokens after 2048, heads of 256: 179 us with
// one part, 204 with two; eight prompts of 1000, heads of 64: 92 and 106), so that a
// request's answer does not depend on the kernel that its company picks.
struct Pair {
    uint32_t high, low;
};
__device__ __forceinline__ Pair two_parts(float x, float y) {
    const uint32_t high = pack_bf16x2(x, y);
    return {high, pack_bf16x2(x - __builtin_bit_cast(float, high << 16), y - __builtin_bit_cast(float, high & 0xFFFF0000u))};
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
// the first tokens, then those of the window.  A row that sees any token past
// the table is NaN, so of those only as far as every such row sees one: a
// length of no sense takes no longer than the table is.
struct Tiles {
    int head, from, count;  // tile v of 0 .. count - 1 is v < head ? v : v - head + from
    __device__ __forceinline__ int at(int v) const { return v < head ? v : v - head + from; }
};
__device__ __forceinline__ Tiles tiles_of(const AttnArgs& a, int low, int high) {
    if (high < 0) return {0, 0, 0};
    const int past = (int)min((int64_t)a.width << a.c.shift, (int64_t)0x7FFFFFFF);
    if (a.window == 0) return {0, 0, min(high, past) / kTile + 1};
    const int end = min(high, max(past, high - a.window + 1)) / kTile + 1;
    const int from = max(max(low, 0) - a.window + 1, 0) / kTile;
    // tokens 0 .. last of the first ones (a.sinks = 0: none)
    const int last = min(min(a.sinks - 1, high), past);
    const int head = min(last < 0 ? 0 : last / kTile + 1, from);
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

// One of a lane's loads: uniform base, the lane's offset, a constant.  With
// kOnce nobody reads it again, and it need not stay in the caches.
template <typename T, bool kOnce = false>
__device__ __forceinline__ T fetch(const uint32_t* base, uint64_t uniform, uint32_t lane_off) {
    const T* p = reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + uniform + lane_off);
    if constexpr (kOnce) return __builtin_nontemporal_load(p);
    return *p;
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

template <int D, bool kWide, bool kOnce = false>
__device__ __forceinline__ void load_key_codes(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t code = kWide ? p.code[0] + h * 16 * (D / 2) : p.code[h % Place<kWide>::kN];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            if constexpr (kW == 4) {
                const u32x4_t w = fetch<u32x4_t, kOnce>(a.c.kc, code + q * 64, l.k);
#pragma unroll
                for (int i = 0; i < 4; ++i) f.k[h][q][i] = w[i];
            } else {
                const u32x2_t w = fetch<u32x2_t, kOnce>(a.c.kc, code, l.k);
                f.k[h][q][0] = w.x;
                f.k[h][q][1] = w.y;
            }
        }
    }
}
template <int D, bool kWide, bool kOnce = false>
__device__ __forceinline__ void load_value_codes(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t code = kWide ? p.code[0] + h * 16 * (D / 2) : p.code[h % Place<kWide>::kN];
#pragma unroll
        for (int q = 0; q < Frag<D>::kG; ++q) f.v[h][q] = fetch<u32x4_t, kOnce>(a.c.vc, code + q * 256, l.v);
    }
}
// The (s, m) pairs of a tile, four tokens a lane.
template <int D, bool kWide>
__device__ __forceinline__ void load_meta(const AttnArgs& a, const uint32_t* from, u32x4_t to[2][Frag<D>::kG],
                                          const Place<kWide>& p, const Offsets& l) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t meta = kWide ? p.meta[0] + h * 64 : p.meta[h % Place<kWide>::kN];
#pragma unroll
        for (int q = 0; q < Frag<D>::kG; ++q)
            to[h][q] = fetch<u32x4_t>(from, meta + (q ? (uint64_t)(4u * q << a.c.shift) : 0), l.meta);
    }
}
template <int D, bool kWide>
__device__ __forceinline__ void load_keys(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
    load_key_codes<D, kWide>(a, f, p, l);
    load_meta<D, kWide>(a, a.c.km, f.km, p, l);
}
template <int D, bool kWide>
__device__ __forceinline__ void load_values(const AttnArgs& a, Frag<D>& f, const Place<kWide>& p, const Offsets& l) {
    load_value_codes<D, kWide>(a, f, p, l);
    load_meta<D, kWide>(a, a.c.vm, f.vm, p, l);
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

// What a wave holds of its 16 * kNB rows: queries, running softmax and outputs.
// A lane's rows are those of its column (lane % 16) of each block of 16; of
// the tokens and of the outputs it has the share of its lane / 16.
template <int D, int kNB>
struct Rows {
    static constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW;
    static constexpr int kJ = D == 64 ? 4 : 8;  // blocks of 16 d per group

    int pos[kNB];  // -1: sees nothing
    u32x4_t xq[kNB][kG][kW];
    f32x4_t xstart[kNB][kG];  // -128 X
    float xs[kNB][kG];        // X
    f32x4_t o[kNB][kG][kJ], ones_sum[kNB][kG];  // of ones_sum only element 0 counts
    float extra[kNB][kG], m[kNB], l[kNB];
    float means[kNB][kG], scales[kNB][kG];  // sums of p m and p s since the last settling
    u32x4_t pop[2][kNB][kG];  // p s of the tile and what its rounding left, the second product's operands

    // Sends for the queries of rows r0 ..; past the last row that one again, unseen.
    __device__ __forceinline__ void fetch(const AttnArgs& a, const Request& req, int head, int r0, int rows, int lane) {
        const int c = lane & 15, g = lane >> 4, first_pos = req.kv - req.rows;
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
    }

    // The queries as the score product's operand, their sums; empty outputs.
    __device__ __forceinline__ void start() {
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            m[n] = -INFINITY;
            l[n] = 0;
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
                extra[n][q] = means[n][q] = scales[n][q] = 0;
                ones_sum[n][q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kJ; ++j) o[n][q][j] = f32x4_t{0, 0, 0, 0};
            }
        }
    }

    // Scores of a tile, from key(h, q, i): the operand of half h's word i of group q.
    // Word by word over halves and groups, so that products that follow each
    // other do not wait for each other.
    template <int kAhead, typename F>
    __device__ __forceinline__ void scores(float s[kNB][2][4], F key, const u32x4_t km[2][kG]) {
        f32x4_t acc[kNB][2][kG];
#pragma unroll
        for (int i = 0; i < kW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    const u32x4_t kop = key(h, q, i);
#pragma unroll
                    for (int n = 0; n < kNB; ++n)
                        acc[n][h][q] = mfma(kop, xq[n][q][i], i == 0 ? xstart[n][q] : acc[n][h][q]);
                }
        if constexpr (kAhead > 0) in_order<2 * kG * kW, kAhead, kNB>();
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < kG; ++q)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float base = q == 0 ? 0.0f : s[n][h][r];
                        s[n][h][r] = fmaf(lo16(km[h][q][r]), acc[n][h][q][r], fmaf(hi16(km[h][q][r]), xs[n][q], base));
                    }
    }

    // Takes scores a row does not see out (and makes those of a bad page NaN);
    // seen: bit 4 h + r.
    __device__ __forceinline__ void mask(const AttnArgs& a, float s[kNB][2][4], uint32_t seen[kNB], int t0,
                                         const int page[2], int g) {
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

    // Softmax weights of the tile, and with the values' scales the operand pop.
    __device__ __forceinline__ void weigh(const float s[kNB][2][4], const u32x4_t vm[2][kG], bool whole,
                                          const uint32_t seen[kNB], float scale2, float slack) {
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                              fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
            top = row_max(top);
            if (__any(top > m[n] + slack)) {
                const float now = fmaxf(m[n], top);
                const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[n] - now) * scale2);
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
            const float base = m[n] == -INFINITY ? 0.0f : m[n] * scale2;
            float p[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[h][r] = __builtin_amdgcn_exp2f(fmaf(s[n][h][r], scale2, -base));
                    l[n] += p[h][r];
                }
            // what a row does not see may hold anything, an infinity or a NaN too
            const auto by_scale = [&](auto masked) {
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    float ps[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            uint32_t meta = vm[h][q][r];
                            if constexpr (masked.value) meta = seen[n] >> (4 * h + r) & 1 ? meta : 0;
                            ps[h][r] = fmaf(p[h][r], lo16(meta), 0.0f);  // one mixed instruction, conversion and all
                            means[n][q] = fmaf(p[h][r], hi16(meta), means[n][q]);
                            scales[n][q] += ps[h][r];
                        }
                    // here, not put off behind the loads that reuse vm's registers
                    asm volatile("" : "+v"(means[n][q]), "+v"(scales[n][q]));
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; r += 2) {
                            const Pair w = two_parts(ps[h][r], ps[h][r + 1]);
                            pop[0][n][q][2 * h + r / 2] = w.high;
                            pop[1][n][q][2 * h + r / 2] = w.low;
                        }
                }
            };
            if (whole) {
                by_scale(std::false_type{});
            } else {
                by_scale(std::true_type{});
            }
        }
    }

    // Adds the tile's values, from value(q, j): the operand of block j of group q.
    // kAhead: how many operands are read from LDS ahead of their products (0:
    // none are).
    template <int kAhead, typename F>
    __device__ __forceinline__ void outputs(F value, const u32x4_t& ones) {
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            // a block's second product a block later: it waits for the first one's sums
            u32x4_t last;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const u32x4_t vop = value(q, j);
#pragma unroll
                for (int n = 0; n < kNB; ++n) {
                    o[n][q][j] = mfma(vop, pop[0][n][q], o[n][q][j]);
                    if (j > 0) o[n][q][j - 1] = mfma(last, pop[1][n][q], o[n][q][j - 1]);
                }
                last = vop;
            }
#pragma unroll
            for (int n = 0; n < kNB; ++n) {
                ones_sum[n][q] = mfma(ones, pop[0][n][q], ones_sum[n][q]);
                o[n][q][kJ - 1] = mfma(last, pop[1][n][q], o[n][q][kJ - 1]);
                ones_sum[n][q] = mfma(ones, pop[1][n][q], ones_sum[n][q]);
            }
        }
        if constexpr (kAhead > 0) in_order<kG * kJ, kAhead, 2 * kNB>();
    }

    // Asks the scheduler for kAhead reads from LDS, then a read after each
    // kEach products: left alone it reads an operand just before its use.
    template <int kReads, int kAhead, int kEach>
    static __device__ __forceinline__ void in_order() {
        constexpr int kRead = 0x100, kProduct = 0x008;
        __builtin_amdgcn_sched_group_barrier(kRead, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kReads - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(kProduct, kEach, 0);
            __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kProduct, kAhead * kEach, 0);
    }

    // Takes 136 times the weights' sum off the outputs; p (m + 8 s) so far.
    __device__ __forceinline__ void settle() {
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
    }

    // Sums over a row's four lanes: its outputs and weights are whole after that.
    __device__ __forceinline__ void finish(const AttnArgs& a) {
        settle();
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            l[n] = row_sum(l[n]);
            if (a.width <= 0 && pos[n] >= 0) l[n] = NAN;  // no table: what the row sees lies past it
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                const float e = row_sum(extra[n][q]);
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[n][q][j][r] += e;
            }
        }
    }

    // d of (q, j, r) is this + j: 128 q + 8 (4 g + r), or 4 (4 g + r) for heads of 64
    static __device__ __forceinline__ int place(int q, int r, int g) {
        return D == 64 ? 4 * (4 * g + r) : q * W4_KV4_GROUP + 8 * (4 * g + r);
    }

    // The rows' results, or with splits their part.
    __device__ __forceinline__ void store(const AttnArgs& a, const Request& req, int head, int split, int r0, int rows,
                                          int lane) const {
        const int c = lane & 15, g = lane >> 4;
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
                        for (int j = 0; j < kJ; j += 2)
                            w[j / 2] = pack_bf16x2(o[n][q][j][r] * inv, o[n][q][j + 1][r] * inv);
                        if constexpr (kJ == 8) {
                            *reinterpret_cast<u32x4_t*>(dst + place(q, r, g)) = u32x4_t{w[0], w[1], w[2], w[3]};
                        } else {
                            *reinterpret_cast<u32x2_t*>(dst + place(q, r, g)) = u32x2_t{w[0], w[1]};
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
                            *reinterpret_cast<f32x4_t*>(dst + place(q, r, g) + j) =
                                f32x4_t{o[n][q][j][r], o[n][q][j + 1][r], o[n][q][j + 2][r], o[n][q][j + 3][r]};
            }
        }
    }
};

// The operand of block j of a group's values, from the words of a lane's eight
// tokens: codes j % 4 + 4 z of each, a token in each half of a register.
template <int D>
__device__ __forceinline__ u32x4_t value_operand(const u32x4_t& first, const u32x4_t& second, int j, int c, uint32_t bias) {
    const uint32_t sel = D == 64 ? ((c & 1) ? 0x07060302u : 0x05040100u) : j >= 4 ? 0x07060302u : 0x05040100u;
    u32x4_t op;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const u32x4_t& w = i < 2 ? first : second;
        const uint32_t pair = __builtin_amdgcn_perm(w[2 * (i & 1) + 1], w[2 * (i & 1)], sel);
        op[i] = ((pair >> (4 * (j % 4))) & 0x000F000Fu) | bias;
    }
    return op;
}

// Where a workgroup's work lies.
struct Share {
    int head, split, row_tile, b;
};
__device__ __forceinline__ Share share_of(const AttnArgs& a) {
    // key/value heads innermost: workgroups that share a head's pages meet on one XCD
    int id = blockIdx.x;
    Share s;
    s.head = id % a.c.heads;
    id /= a.c.heads;
    s.split = id % a.splits;
    id /= a.splits;
    // Late rows see most tokens.  Where all workgroups are on the chip at once
    // (two a compute unit, the second 256 after the first) the second half
    // goes the other way, so that a long one shares its unit with a short
    // one; else the longest come first.
    s.b = id % a.B;
    const int t = id / a.B;
    s.row_tile = a.in_turn && 2 * t >= a.row_tiles ? t - (a.row_tiles + 1) / 2 : a.row_tiles - 1 - t;
    return s;
}

// Few rows: the waves take a row tile's token tiles in turn.
template <int D, int kNB, int kWaves, bool kWide>
__global__ __launch_bounds__(kWaves * kWave) void kv4_attn_kernel(AttnArgs a) {
    typedef Rows<D, kNB> R;
    constexpr int kG = R::kG, kJ = R::kJ, kCols = 16 * kNB;
    __shared__ float so[kWaves / 2][kCols][D + 4];
    __shared__ float sm[kWaves][kCols], sl[kWaves][kCols];

    const int lane = threadIdx.x & (kWave - 1), wave = (int)sgpr(threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    const Share mine = share_of(a);
    const int head = mine.head;
    const Request req = request_of(a, mine.b);
    const int rows = min(req.rows, a.max_q) * a.g;  // < 2^31: checked on the host
    const int r0 = mine.row_tile * kCols;
    if (r0 >= rows) return;
    const int first_pos = req.kv - req.rows;
    const int low = first_pos + r0 / a.g, high = first_pos + (min(r0 + kCols, rows) - 1) / a.g;
    const Tiles tiles = tiles_of(a, low, high);
    const table_ptr table = as_table(a.table + (size_t)mine.b * a.width);

    // this split's tiles, in turn over the waves
    const int per = (tiles.count + a.splits - 1) / a.splits;
    const int v1 = min(tiles.count, (mine.split + 1) * per);
    int v = mine.split * per + wave;
    const bool any = v < v1 && a.width > 0;
    const auto clamped = [&](int x) { return x < v1 ? x : v1 - 1; };

    R rw;
    rw.fetch(a, req, head, r0, rows, lane);
    const Offsets offs = offsets_of<D>(lane);
    Frag<D> f;
    int page[2] = {-1, -1};
    Entries next = {};
    int t0 = 0, t1 = 0;
    if (any) {
        t0 = tiles.at(v) * kTile;
        t1 = tiles.at(clamped(v + kWaves)) * kTile;
        const Entries now = entries_of<kWide>(a, table, t0);
        next = entries_of<kWide>(a, table, t1);
        pages_of<kWide>(a, now, t0, high, page);
        const Place<kWide> p = place_of<D, kWide>(a, t0, head, page);
        load_keys<D, kWide>(a, f, p, offs);
        load_values<D, kWide>(a, f, p, offs);
    } else {
        v = v1;
    }
    rw.start();

    // The running maximum moves only when a score passes it by 2^8: weights up
    // to 256 lose nothing, and a move costs a pass over the outputs.
    const float slack = fminf(8.0f / a.scale2, 3e38f);
    const uint32_t bias = vgpr_const(kInt4BiasPair);
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    // The next tile's keys are fetched when the scores are done with this
    // one's, its values behind the outputs; page numbers a tile earlier.  The
    // last tile fetches itself again: under a condition the compiler would
    // load into other registers and wait for them to copy them over.
    for (int done = 1; v < v1; v += kWaves, ++done) {
        int coming[2];
        pages_of<kWide>(a, next, t1, high, coming);
        const Place<kWide> ahead = place_of<D, kWide>(a, t1, head, coming);
        const int t2 = tiles.at(clamped(v + 2 * kWaves)) * kTile;
        next = entries_of<kWide>(a, table, t2);
        // Whether every row sees every token of the tile.
        const bool whole = t0 + kTile - 1 <= low && (a.window == 0 || t0 > high - a.window || t0 + kTile <= a.sinks) &&
                           page[0] >= 0 && page[1] >= 0 && r0 + kCols <= rows;

        float s[kNB][2][4];
        rw.template scores<0>(s, [&](int h, int q, int i) { return key_operand(f.k[h][q][i], bias); }, f.km);
        __builtin_amdgcn_sched_barrier(0);  // else loads above the last use of these registers land in others
        load_keys<D, kWide>(a, f, ahead, offs);
        __builtin_amdgcn_sched_barrier(0);
        uint32_t seen[kNB];
#pragma unroll
        for (int n = 0; n < kNB; ++n) seen[n] = 0xFFu;
        if (!whole) rw.mask(a, s, seen, t0, page, g);
        rw.weigh(s, f.vm, whole, seen, a.scale2, slack);
        rw.template outputs<0>([&](int q, int j) { return value_operand<D>(f.v[0][q], f.v[1][q], j, c, bias); }, ones);
        __builtin_amdgcn_sched_barrier(0);
        load_values<D, kWide>(a, f, ahead, offs);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) page[h] = coming[h];
        t0 = t1;
        t1 = t2;
        if (done % 8 == 0) rw.settle();
    }
    rw.finish(a);

    // join the waves: common maximum, then pairwise through LDS
    if (lane < 16) {
#pragma unroll
        for (int n = 0; n < kNB; ++n) {
            sm[wave][16 * n + c] = rw.m[n];
            sl[wave][16 * n + c] = rw.l[n];
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
        const float scale = rw.l[n] == 0.0f ? 0.0f : weight(rw.m[n]);
        rw.l[n] = sum;
        rw.m[n] = now;
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) rw.o[n][q][j][r] *= scale;
    }
    const auto exchange = [&](int slot, auto put) {
#pragma unroll
        for (int n = 0; n < kNB; ++n)
#pragma unroll
            for (int q = 0; q < kG; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        float& x = so[slot][16 * n + c][R::place(q, r, g) + j];
                        if constexpr (put.value) {
                            x = rw.o[n][q][j][r];
                        } else {
                            rw.o[n][q][j][r] += x;
                        }
                    }
    };
#pragma unroll
    for (int step = 1; step < kWaves; step *= 2) {
        const int pair = wave / (2 * step);
        if (wave % (2 * step) == step) exchange(pair, std::true_type{});
        __syncthreads();
        if (wave % (2 * step) == 0) exchange(pair, std::false_type{});
        if (2 * step < kWaves) __syncthreads();
    }
    if (wave == 0) rw.store(a, req, head, mine.split, r0, rows, lane);
}

// Value of lane l ^ kOff within a row of 16, for any set of other lane bits.
template <int kOff>
__device__ __forceinline__ float lane_xor(float v) {
    if constexpr (kOff == 4) {  // half mirror (^ 7), then the quad reversed (^ 3)
        const int b = __builtin_bit_cast(int, v);
        const int m = __builtin_amdgcn_update_dpp(b, b, 0x141, 0xF, 0xF, false);
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(m, m, 0x1B, 0xF, 0xF, false));
    } else {
        return dpp_partner<kOff>(v);
    }
}

// Sums n values over the lanes whose column differs in bits kOff, kOff / 2,
// ... kLast, each step leaving a lane half of the values: on return it holds
// v[0 .. n / steps) of the part that its bits (the highest first) select.
template <int kOff, int kLast, int kN>
__device__ __forceinline__ void halving_sum(float* v, int c) {
    if constexpr (kOff >= kLast) {
        const bool upper = (c & kOff) != 0;
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const float keep = upper ? v[i + kN / 2] : v[i], send = upper ? v[i] : v[i + kN / 2];
            v[i] = keep + lane_xor<kOff>(send);
        }
        halving_sum<kOff / 2, kLast, kN / 2>(v, c);
    }
}
template <int kOff, int kLast, typename F>
__device__ __forceinline__ float over_sets(float v, F f) {
    if constexpr (kOff >= kLast) return over_sets<kOff / 2, kLast>(f(v, lane_xor<kOff>(v)), f);
    return v;
}

// Very few rows (a decode step: the query heads of one key/value head, 8 at
// most).  Of the 16 columns of a product only those rows' would be of use, and
// softmax and scaling would be done 16 / rows times over.  So the columns are
// cut into kSets sets of 16 / kSets rows, all holding the same queries: set s
// keeps the scores of the s-th run of 16 tokens, a lane then has four scores
// of kSets * 16 tokens, and its own maximum and sum; in the second product a
// set's weights are 0 against the other sets' tokens.  The sets are joined at
// the end as the waves are.
// Per 32 tokens of D = 128 and 4 rows that is some 160 vector instructions
// instead of 260.
template <int D, int kSets, int kWaves, bool kWide>
__global__ __launch_bounds__(kWaves * kWave, 2) void kv4_attn_sets_kernel(AttnArgs a) {
    constexpr int kT = kSets / 2, kCols = 16 / kSets;  // tiles at a time; rows
    constexpr int kG = Frag<D>::kG, kW = Frag<D>::kW, kJ = D == 64 ? 4 : 8;
    constexpr int kAll = kG * 4 * kJ, kMine = kAll / kSets;  // a lane's outputs, before and after the sets are joined
    __shared__ float so[kWaves][kMine][kWave];
    __shared__ float sm[kWaves][kCols], sl[kWaves][kCols];

    const int lane = threadIdx.x & (kWave - 1), wave = (int)sgpr(threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4, set = c / kCols;
    const Share mine = share_of(a);
    const int head = mine.head;
    const Request req = request_of(a, mine.b);
    const int rows = min(min(req.rows, a.max_q) * a.g, kCols);
    if (rows <= 0) return;
    const int first_pos = req.kv - req.rows;
    const int low = first_pos, high = first_pos + (rows - 1) / a.g;
    const Tiles tiles = tiles_of(a, low, high);
    const table_ptr table = as_table(a.table + (size_t)mine.b * a.width);

    // this split's tiles, kT at a time in turn over the waves
    const int per = ((tiles.count + a.splits - 1) / a.splits + kT - 1) / kT * kT;
    const int v1 = min(tiles.count, (mine.split + 1) * per);
    int v = mine.split * per + wave * kT;
    if (a.width <= 0) v = max(v, v1);
    const auto tile_at = [&](int x) { return tiles.at(max(min(x, v1 - 1), 0)) * kTile; };

    // the lane's row (past the last one: that one again, unseen)
    const int row = c % kCols, r = min(row, rows - 1);
    const int pos = row < rows ? max(first_pos + r / a.g, -1) : -1;
    u32x4_t xq[kG][kW];
    {
        const uint16_t* src = a.q + (int64_t)(req.first + r / a.g) * a.q_stride + (size_t)(head * a.g + r % a.g) * D;
#pragma unroll
        for (int q = 0; q < kG; ++q)
#pragma unroll
            for (int i = 0; i < kW; ++i)
                xq[q][i] = *reinterpret_cast<const u32x4_t*>(src + q * W4_KV4_GROUP + (kW * g + i) * 8);
    }

    // Tiles v .. v + kT - 1: where they begin, their pages and places; a lane's
    // own run of 16 tokens among them.
    struct Group {
        int t0[kT], page[kT][2];
        Place<kWide> place[kT];
    };
    const Offsets offs = offsets_of<D>(lane);
    Entries entries[kT];
    const auto send_entries = [&](int at) {
#pragma unroll
        for (int t = 0; t < kT; ++t) entries[t] = entries_of<kWide>(a, table, tile_at(at + t));
    };
    const auto group_at = [&](int at) {
        Group x;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            x.t0[t] = tile_at(at + t);
            pages_of<kWide>(a, entries[t], x.t0[t], high, x.page[t]);
            x.place[t] = place_of<D, kWide>(a, x.t0[t], head, x.page[t]);
        }
        return x;
    };
    const auto of_set = [&](auto f) {  // f(tile, half) of the lane's set
        auto x = f(0, 0);
#pragma unroll
        for (int k = 1; k < kSets; ++k) {
            const auto y = f(k / 2, k % 2);  // before the choice: a choice of addresses would put all in memory
            x = set == k ? y : x;
        }
        return x;
    };
    Frag<D> f[kT];  // codes; the pairs below are the lane's set's alone
    u32x4_t km[kG], vm[kG];
    const auto fetch_meta = [&](const Group& x, const uint32_t* from, u32x4_t to[kG]) {
        const uint64_t at = of_set([&](int t, int h) { return kWide ? x.place[t].meta[0] + h * 64 : x.place[t].meta[h % Place<kWide>::kN]; });
#pragma unroll
        for (int q = 0; q < kG; ++q)
            to[q] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(from) + at + ((uint64_t)(4u * q) << a.c.shift) + offs.meta);
    };
    Group now = {};
    if (v < v1) {
        send_entries(v);
        now = group_at(v);
        send_entries(v + kWaves * kT);
#pragma unroll
        for (int t = 0; t < kT; ++t) load_key_codes<D, kWide, true>(a, f[t], now.place[t], offs);
        fetch_meta(now, a.c.km, km);
        fetch_meta(now, a.c.vm, vm);
#pragma unroll
        for (int t = 0; t < kT; ++t) load_value_codes<D, kWide, true>(a, f[t], now.place[t], offs);
    }

    f32x4_t xstart[kG];
    float xs[kG];
#pragma unroll
    for (int q = 0; q < kG; ++q) {
        float sum = 0;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const u32x4_t w = xq[q][i];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += bf16_to_f32(w[e] & 0xFFFFu) + __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
            uint32_t in[4] = {w.x, w.y, w.z, w.w}, pr[4];
            x_pairs_for_biased(in, pr);
            xq[q][i] = u32x4_t{pr[0], pr[1], pr[2], pr[3]};
        }
        xs[q] = row_sum(sum);
        const float x0 = -128.0f * xs[q];
        xstart[q] = f32x4_t{x0, x0, x0, x0};
    }
    f32x4_t o[kG][kJ], ones_sum[kG];
    float extra[kG], means[kG], scales[kG], m = -INFINITY, l = 0;
#pragma unroll
    for (int q = 0; q < kG; ++q) {
        extra[q] = means[q] = scales[q] = 0;
        ones_sum[q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kJ; ++j) o[q][j] = f32x4_t{0, 0, 0, 0};
    }
    const auto settle = [&]() {
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            const float off = -136.0f * ones_sum[q][0];
            ones_sum[q] = f32x4_t{0, 0, 0, 0};
            extra[q] += fmaf(8.0f, scales[q], means[q]);
            means[q] = scales[q] = 0;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[q][j][e] += off;
        }
    };

    const float slack = fminf(8.0f / a.scale2, 3e38f);
    const uint32_t bias = vgpr_const(kInt4BiasPair);
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (int done = 1; v < v1; v += kWaves * kT, ++done) {
        const Group next = group_at(v + kWaves * kT);
        send_entries(v + 2 * kWaves * kT);
        bool whole = v + kT <= v1 && rows == kCols;
#pragma unroll
        for (int t = 0; t < kT; ++t)
            whole = whole && now.t0[t] + kTile - 1 <= low &&
                    (a.window == 0 || now.t0[t] > high - a.window || now.t0[t] + kTile <= a.sinks) &&
                    now.page[t][0] >= 0 && now.page[t][1] >= 0;

        // scores: each run's products, of which its set keeps its columns
        f32x4_t acc[kG];
#pragma unroll
        for (int q = 0; q < kG; ++q) acc[q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if (v + t < v1) {
                f32x4_t x[2][kG];
#pragma unroll
                for (int i = 0; i < kW; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < kG; ++q)
                            x[h][q] = mfma(key_operand(f[t].k[h][q][i], bias), xq[q][i], i == 0 ? xstart[q] : x[h][q]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < kG; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[q][e] = set == 2 * t + h ? x[h][q][e] : acc[q][e];
            }
            __builtin_amdgcn_sched_barrier(0);  // else loads above the last use of these registers land in others
            load_key_codes<D, kWide, true>(a, f[t], next.place[t], offs);
            __builtin_amdgcn_sched_barrier(0);
        }
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] = 0;
#pragma unroll
            for (int q = 0; q < kG; ++q) s[e] = fmaf(lo16(km[q][e]), acc[q][e], fmaf(hi16(km[q][e]), xs[q], s[e]));
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch_meta(next, a.c.km, km);
        __builtin_amdgcn_sched_barrier(0);
        if (!whole) {
            const int t0 = of_set([&](int t, int h) { return now.t0[t] + 16 * h; }) + 4 * g;
            const bool bad = of_set([&](int t, int h) { return now.page[t][h] < 0; });
            const bool run = of_set([&](int t, int) { return v + t < v1; });
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t0 + e;
                const bool see = run & (t <= pos) & ((a.window == 0) | (t > pos - a.window) | (t < a.sinks));
                s[e] = !see ? -INFINITY : bad ? NAN : s[e];
                // what a row does not see may hold anything, an infinity or a NaN too
#pragma unroll
                for (int q = 0; q < kG; ++q) vm[q][e] = see ? vm[q][e] : 0;
            }
        }

        // softmax of the lane's four scores
        const float top = row_max(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])));
        if (__any(top > m + slack)) {
            const float top_now = fmaxf(m, top);
            const float keep = top_now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - top_now) * a.scale2);
            m = top_now;
            l *= keep;
#pragma unroll
            for (int q = 0; q < kG; ++q) {
                extra[q] *= keep;
                means[q] *= keep;
                scales[q] *= keep;
                ones_sum[q][0] *= keep;
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[q][j][e] *= keep;
            }
        }
        const float base = m == -INFINITY ? 0.0f : m * a.scale2;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], a.scale2, -base));
            l += p[e];
        }
        Pair weights[kG][2];
#pragma unroll
        for (int q = 0; q < kG; ++q) {
            float ps[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ps[e] = fmaf(p[e], lo16(vm[q][e]), 0.0f);  // one mixed instruction, conversion and all
                means[q] = fmaf(p[e], hi16(vm[q][e]), means[q]);
                scales[q] += ps[e];
            }
            // here, not put off behind the loads that reuse vm's registers
            asm volatile("" : "+v"(means[q]), "+v"(scales[q]));
            weights[q][0] = two_parts(ps[0], ps[1]);
            weights[q][1] = two_parts(ps[2], ps[3]);
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch_meta(next, a.c.vm, vm);
        __builtin_amdgcn_sched_barrier(0);

        // outputs: a tile's tokens against its two sets' weights
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if (v + t < v1) {
#pragma unroll
                for (int q = 0; q < kG; ++q) {
                    const bool first = set == 2 * t, second = set == 2 * t + 1;
                    const auto part = [&](uint32_t w0, uint32_t w1) {
                        return u32x4_t{first ? w0 : 0, first ? w1 : 0, second ? w0 : 0, second ? w1 : 0};
                    };
                    const u32x4_t high = part(weights[q][0].high, weights[q][1].high);
                    const u32x4_t low = part(weights[q][0].low, weights[q][1].low);
                    // a block's second product a block later: it waits for the first one's sums
                    u32x4_t last;
#pragma unroll
                    for (int j = 0; j < kJ; ++j) {
                        const u32x4_t vop = value_operand<D>(f[t].v[0][q], f[t].v[1][q], j, c, bias);
                        o[q][j] = mfma(vop, high, o[q][j]);
                        if (j > 0) o[q][j - 1] = mfma(last, low, o[q][j - 1]);
                        last = vop;
                    }
                    ones_sum[q] = mfma(ones, high, ones_sum[q]);
                    o[q][kJ - 1] = mfma(last, low, o[q][kJ - 1]);
                    ones_sum[q] = mfma(ones, low, ones_sum[q]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            load_value_codes<D, kWide, true>(a, f[t], next.place[t], offs);
            __builtin_amdgcn_sched_barrier(0);
        }
        now = next;
        if (done % 8 == 0) settle();
    }
    settle();

    // The sets of a wave: common maximum, sums, a part of the outputs for each lane.
    constexpr int kBit = 8;
    l = row_sum(l);
    if (a.width <= 0 && pos >= 0) l = NAN;  // no table: what the row sees lies past it
    const float top = over_sets<kBit, kCols>(m, [](float x, float y) { return fmaxf(x, y); });
    const float scale = l == 0.0f ? 0.0f : m == -INFINITY ? NAN : __builtin_amdgcn_exp2f((m - top) * a.scale2);
    l = over_sets<kBit, kCols>(l == 0.0f ? 0.0f : l * scale, [](float x, float y) { return x + y; });
    float out[kAll];  // (q, r, j)
#pragma unroll
    for (int q = 0; q < kG; ++q) {
        const float e = row_sum(extra[q]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < kJ; ++j) out[(q * 4 + x) * kJ + j] = l == 0.0f ? 0.0f : (o[q][j][x] + e) * scale;
    }
    halving_sum<kBit, kCols, kAll>(out, c);

    // The waves.
#pragma unroll
    for (int i = 0; i < kMine; ++i) so[wave][i][lane] = out[i];
    if (lane < kCols) {
        sm[wave][lane] = top;
        sl[wave][lane] = l;
    }
    __syncthreads();
    float now_top = sm[0][row];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) now_top = fmaxf(now_top, sm[w][row]);
    float by[kWaves], sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        // a wave that saw nothing has l = 0; a NaN stays one
        const float lw = sl[w][row], mw = sm[w][row];
        by[w] = lw == 0.0f ? 0.0f : mw == -INFINITY ? NAN : __builtin_amdgcn_exp2f((mw - now_top) * a.scale2);
        sum += lw == 0.0f ? 0.0f : lw * by[w];
    }
    if (row >= rows) return;
    // Each wave finishes a share of the lane's values, neighbours in d.
    constexpr int kEnd = kMine >= kWaves ? kMine / kWaves : 1;
    if (wave * kEnd >= kMine) return;
    float end[kEnd];
#pragma unroll
    for (int i = 0; i < kEnd; ++i) {
        end[i] = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) end[i] = fmaf(by[w], so[w][wave * kEnd + i][lane], end[i]);
    }
    const int at = set * kMine + wave * kEnd;  // (q, r, j) as one number
    const int d = Rows<D, 1>::place(at / kJ / 4, at / kJ % 4, g) + at % kJ;
    const int t = req.first + row / a.g, h = head * a.g + row % a.g;
    if (a.splits == 1) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* dst = a.out + (int64_t)t * a.out_stride + (size_t)h * D + d;
        if constexpr (kEnd % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kEnd; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(end[i] * inv, end[i + 1] * inv);
        } else {
            dst[0] = f32_to_bf16(end[0] * inv);
        }
    } else {
        const size_t part = ((size_t)t * a.g * a.c.heads + h) * a.splits + mine.split;
        if (g == 0 && wave == 0 && set == 0) {
            a.part_ml[2 * part] = now_top;
            a.part_ml[2 * part + 1] = sum;
        }
#pragma unroll
        for (int i = 0; i < kEnd; ++i) a.part_o[part * D + d + i] = end[i];
    }
}

// Waits for a workgroup's LDS accesses and meets the others; loads from
// memory stay on their way.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Many rows (prompts): four waves with rows of their own against the same
// tiles.  Unpacking a tile costs the vector unit as much as 16 rows' softmax
// does, so each wave unpacks a quarter of it, and the operands go through LDS,
// a register's 64 lanes together (16 bytes a lane, no conflicts either way).
// Two buffers: while a tile is worked on, the next one is unpacked and the
// one after is on its way from memory.
// Heads of 64 fit three waves a SIMD, with two operands of the values read ahead
// in place of four where a tile is one page (eight prompts of 1000 tokens, 32 query
// and 8 key/value heads: 106 us, 124 with 173 registers and two waves).
template <int D, int kNB, bool kWide>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void kv4_attn_many_kernel(AttnArgs a) {
    typedef Rows<D, kNB> R;
    constexpr int kWaves = 4, kG = R::kG, kW = R::kW, kJ = R::kJ, kCols = 16 * kNB;
    constexpr int kKeys = 2 * kG * kW, kValues = kG * kJ;  // operands of a tile
    constexpr int kMyKeys = kKeys / kWaves, kMyValues = kValues / kWaves;
    constexpr int kAheadKeys = kKeys < 6 ? kKeys : 6, kAheadValues = D == 64 ? (kWide ? 2 : 4) : 8;
    __shared__ u32x4_t ops[2][kKeys + kValues][kWave];

    const int lane = threadIdx.x & (kWave - 1), wave = (int)sgpr(threadIdx.x / kWave);
    const int c = lane & 15, g = lane >> 4;
    const Share mine = share_of(a);
    const int head = mine.head;
    const Request req = request_of(a, mine.b);
    const int rows = min(req.rows, a.max_q) * a.g;
    const int base = mine.row_tile * kWaves * kCols;
    if (base >= rows) return;
    const int first_pos = req.kv - req.rows;
    const int high = first_pos + (min(base + kWaves * kCols, rows) - 1) / a.g;
    const Tiles tiles = tiles_of(a, first_pos + base / a.g, high);
    const table_ptr table = as_table(a.table + (size_t)mine.b * a.width);
    // this wave's rows; past the last there may be none
    const int r0 = min(base + wave * kCols, rows);
    const int my_low = first_pos + min(r0, rows - 1) / a.g, my_high = first_pos + (min(r0 + kCols, rows) - 1) / a.g;

    int v = 0;
    const int v1 = a.width <= 0 ? 0 : tiles.count;
    const auto tile_at = [&](int x) { return tiles.at(max(min(x, v1 - 1), 0)) * kTile; };

    R rw;
    rw.fetch(a, req, head, r0, rows, lane);
    const Offsets offs = offsets_of<D>(lane);
    const uint32_t bias = vgpr_const(kInt4BiasPair);

    // A wave's part: kMyKeys words of one half and group, and kMyValues blocks
    // of one group (for which it needs the words of all 32 tokens).
    const int kh = wave * kMyKeys / (kG * kW), kq = wave * kMyKeys / kW % kG, kw = wave * kMyKeys % kW;
    const int vq = wave * kMyValues / kJ, vj = wave * kMyValues % kJ;
    uint32_t raw_k[kMyKeys];
    u32x4_t raw_v[2];
    const auto fetch_codes = [&](const Place<kWide>& p) {
        const uint64_t key = kWide ? p.code[0] + kh * 16 * (D / 2) : p.code[kh % Place<kWide>::kN];
        if constexpr (kMyKeys == 4) {
            const u32x4_t w = fetch<u32x4_t>(a.c.kc, key + kq * 64, offs.k);
#pragma unroll
            for (int i = 0; i < 4; ++i) raw_k[i] = w[i];
        } else if constexpr (kMyKeys == 2) {
            const u32x2_t w = fetch<u32x2_t>(a.c.kc, key + kq * 64 + 4 * kw, offs.k);
            raw_k[0] = w.x;
            raw_k[1] = w.y;
        } else {
            raw_k[0] = fetch<uint32_t>(a.c.kc, key + 4 * kw, offs.k);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            raw_v[h] = fetch<u32x4_t>(a.c.vc, (kWide ? p.code[0] + h * 16 * (D / 2) : p.code[h % Place<kWide>::kN]) + vq * 256, offs.v);
    };
    const auto unpack = [&](int buffer) {
#pragma unroll
        for (int i = 0; i < kMyKeys; ++i) ops[buffer][wave * kMyKeys + i][lane] = key_operand(raw_k[i], bias);
        // the shift by 4 (j % 4) is uniform, but not known here for kMyValues < 4
#pragma unroll
        for (int i = 0; i < kMyValues; ++i) {
            const int j = vj + i;
            const uint32_t sel = D == 64 ? ((c & 1) ? 0x07060302u : 0x05040100u) : j >= 4 ? 0x07060302u : 0x05040100u;
            u32x4_t op;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const u32x4_t& w = raw_v[e >> 1];
                const uint32_t pair = __builtin_amdgcn_perm(w[2 * (e & 1) + 1], w[2 * (e & 1)], sel);
                op[e] = ((pair >> (4 * (j % 4))) & 0x000F000Fu) | bias;
            }
            ops[buffer][kKeys + wave * kMyValues + i][lane] = op;
        }
    };
    u32x4_t km[2][kG], vm[2][kG];
    const auto fetch_meta = [&](const Place<kWide>& p, const uint32_t* from, u32x4_t to[2][kG]) {
        load_meta<D, kWide>(a, from, to, p, offs);
    };

    int t0 = 0, t1 = 0, page[2] = {-1, -1}, coming[2] = {-1, -1};
    Entries next = {};
    Place<kWide> ahead = {};
    if (v < v1) {
        t0 = tile_at(v);
        t1 = tile_at(v + 1);
        const Entries now = entries_of<kWide>(a, table, t0), then = entries_of<kWide>(a, table, t1);
        pages_of<kWide>(a, now, t0, high, page);
        const Place<kWide> p = place_of<D, kWide>(a, t0, head, page);
        fetch_codes(p);
        fetch_meta(p, a.c.km, km);
        fetch_meta(p, a.c.vm, vm);
        unpack(0);
        pages_of<kWide>(a, then, t1, high, coming);
        ahead = place_of<D, kWide>(a, t1, head, coming);
        fetch_codes(ahead);
        next = entries_of<kWide>(a, table, tile_at(v + 2));
    }
    rw.start();
    lds_barrier();

    const float slack = fminf(8.0f / a.scale2, 3e38f);
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (int done = 1; v < v1; ++v, ++done) {
        const int buffer = (done - 1) & 1;
        // the next tile's codes into the other buffer, the one after's sent for
        // (at the end the last tile again: loads under a condition would be
        // waited for and copied)
        unpack(buffer ^ 1);
        const int t2 = tile_at(v + 2);
        int after[2];
        pages_of<kWide>(a, next, t2, high, after);
        const Place<kWide> place = ahead;
        ahead = place_of<D, kWide>(a, t2, head, after);
        next = entries_of<kWide>(a, table, tile_at(v + 3));
        __builtin_amdgcn_sched_barrier(0);
        fetch_codes(ahead);
        __builtin_amdgcn_sched_barrier(0);

        // Rows of a wave that lie before the tile, or before whose window it ends, pass
        // it over.  (Positions below 0 see nothing; less a window they could pass 32 bits.)
        const bool sees = r0 < rows && t0 <= my_high &&
                          (a.window == 0 || t0 + kTile - 1 > max(my_low, 0) - a.window || t0 < a.sinks);
        if (sees) {
            const bool whole = t0 + kTile - 1 <= my_low && (a.window == 0 || t0 > my_high - a.window || t0 + kTile <= a.sinks) &&
                               page[0] >= 0 && page[1] >= 0 && r0 + kCols <= rows;
            float s[kNB][2][4];
            rw.template scores<kAheadKeys>(s, [&](int h, int q, int i) { return ops[buffer][(h * kG + q) * kW + i][lane]; }, km);
            uint32_t seen[kNB];
#pragma unroll
            for (int n = 0; n < kNB; ++n) seen[n] = 0xFFu;
            if (!whole) rw.mask(a, s, seen, t0, page, g);
            rw.weigh(s, vm, whole, seen, a.scale2, slack);
            rw.template outputs<kAheadValues>([&](int q, int j) { return ops[buffer][kKeys + q * kJ + j][lane]; }, ones);
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch_meta(place, a.c.km, km);
        fetch_meta(place, a.c.vm, vm);
        __builtin_amdgcn_sched_barrier(0);
        if (done % 8 == 0) rw.settle();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            page[h] = coming[h];
            coming[h] = after[h];
        }
        t0 = t1;
        t1 = t2;
        lds_barrier();
    }
    rw.finish(a);
    if (r0 < rows) rw.store(a, req, head, 0, r0, rows, lane);
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

// How a call is cut into workgroups.
struct Cut {
    bool many;      // kv4_attn_many_kernel
    int sets;       // kv4_attn_sets_kernel if over 1
    bool two;       // 32 rows a wave of kv4_attn_kernel
    int row_tiles;  // of a request, each a workgroup's rows
    int splits;     // workgroups that share a row tile's tokens
    int waves;      // of a workgroup
};
constexpr int kFewWaves = 4;
// 16-row blocks of a wave: as many as leave two waves a SIMD.
constexpr int many_blocks(int d) { return d == 256 ? 1 : 2; }

Cut cut_of(const w4_attn_args& a, const w4_kv4_cache& c) {
    Cut k;
    const int64_t rows = (int64_t)a.max_q * (a.q_heads / c.kv_heads);
    // Shared tiles take the fewest instructions, but a workgroup passes over all
    // of its rows' tokens a tile at a time, where kv4_attn_kernel's four waves
    // share them: it pays where nearly every compute unit has two workgroups (heads
    // of 64, whose tiles are the least work, four), for then the shortest can go with
    // the longest.  us of both kernels, shared tiles first, prompts with nothing
    // before them unless said: heads of 256, 256 workgroups 104 and 78 (1024 tokens
    // after 1024), 448 198 and 198 (1792 after 2048), 512 204 and 225 (2048 after
    // 2048) and 22 and 42 (eight prompts of 250), 1024 155 and 185 (two of 2048); heads
    // of 128, 384 196 and 152 (1536 after 2048), 464 53 and 55 (two of 912), 576 26
    // and 47 (nine of 250), 1008 156 and 171 (two of 2000); heads of 64, 512 49 and
    // 40 (1024 tokens), 1024 59 and 77 (four of 1000), 2048 106 and 142 (eight).
    // One prompt of heads of 128, whose workgroups differ most: 456 96 and 78 (1824),
    // 576 303 and 248 (2304 after 2048), 1024 302 and 295 (4096), 531 and 538 (4096
    // after 2048).  A few workgroups past 512 run on their own when the first end,
    // which counts where each has far to go: 576 180 and 164 (two of 1152 after 1000,
    // heads of 256), 323 and 260 (2304 after 2048), 128 and 108 at 640 (16 of 144 after
    // 1000, heads of 128), but 72 and 85 (two of 1152), and 768 155 and 176 (four of
    // 768 after 1000).
    const int64_t many_rows = 64 * many_blocks(c.head_dim);
    const int64_t shared = (int64_t)a.B * c.kv_heads * ((rows + many_rows - 1) / many_rows);
    const bool few_left = shared > 512 && shared < 704 && (int64_t)a.max_kv >= (int64_t)a.max_q + 800;
    k.many = rows >= many_rows && !few_left &&
             shared >= (c.head_dim == 64 || (c.head_dim == 128 && a.B == 1) ? 1024 : 448);
    // Sets: four with up to 4 rows, but two with heads of 256, for the registers
    // of a group's codes (32 requests of 4096 tokens, 8 key/value heads: heads
    // of 128 32 us with four and 35 with two, heads of 256 with pages of 64 58
    // and 57, with pages of 16 79 and 60; without sets 38, 63 and 66; eight sets
    // take 37 us where four take 32).
    k.sets = rows > 8 ? 1 : rows > 4 || c.head_dim == 256 ? 2 : 4;
    // Heads of 128: 32 rows a wave unpack half as often, where that still makes
    // enough workgroups (2000 tokens after 3000, 16 query and 4 key/value heads, 1000
    // workgroups of 32 rows: 139 us, 168 with 16; half as many 88 and 87; 768, 1536
    // after 2000, 82 and 94; 600, 1200 after 2000, 76 and 80, which says that fewer
    // would do; heads of 64, with half the work in a tile, 106 either way).
    k.two = !k.many && c.head_dim == 128 && rows > 16 && (int64_t)a.B * c.kv_heads * ((rows + 31) / 32) >= 768;
    const int64_t tile = k.many ? many_rows : k.two ? 32 : 16;
    k.row_tiles = (int)((rows + tile - 1) / tile);
    // As many workgroups as are on the chip at once, two a compute unit: with a
    // few more, the rest would run after them.  Twice that number where requests
    // differ in length (a window makes them alike) and a wave keeps four tiles: 32
    // requests of up to 8192 tokens take 80 us then, 86 without; one of 131071
    // tokens 33 instead of 32.  Two tiles at least for each of the waves, eight
    // where there is a workgroup a compute unit without splits: 56 requests of
    // 1000 tokens, 16 query and 8 key/value heads of 256, 27 us instead of 41 (of
    // 8000 tokens 178 either way).
    const int64_t groups = (int64_t)a.B * c.kv_heads * k.row_tiles;
    int64_t tokens = a.max_kv;
    if (a.window > 0) tokens = tokens < (int64_t)a.window + a.sinks + a.max_q ? tokens : (int64_t)a.window + a.sinks + a.max_q;
    const int64_t tiles = (tokens + kTile - 1) / kTile;
    const int64_t fill = a.B > 1 && a.window == 0 && tiles * groups >= 1024 * 4 * kFewWaves ? 1024 : 512;
    int64_t want = k.many ? 1 : fill / (groups > 0 ? groups : 1);
    const int64_t most = tiles / ((groups > 256 ? 8 : 2) * kFewWaves);
    want = want < most ? want : most;
    k.splits = (int)(want < 1 ? 1 : want > kMaxSplits ? kMaxSplits : want);
    // Up to 256 workgroups (512 with heads of 64, of half the registers) can have
    // eight waves, each with half the tiles: unsplit they save the join's launch.
    // Worth it for short contexts, by what a tile takes (heads of 128, 8 requests
    // of 1000 tokens: 10.2 us, split 11.5; of 2000 14.3, split 13.1; heads of 64,
    // of 2500 tokens 12.5, split 10.5) and where splits would share a
    // compute unit anyway (32 of 1000 tokens 11.0, split 14.8; of 4000 24, split
    // 27; heads of 256, 32 of 1000 tokens 16.7, split 24.3; but 16, 128
    // workgroups, of 4000 tokens 44, split 36).  With more than 8 rows only in
    // place of splits (200 tokens after 500, 16 query and 8 key/value heads of 128:
    // 11.2 us, split 17.8; joining eight waves there costs 1 to 2 us, which
    // 30 tokens after 200 do not win back: 8.5, four waves 7.7).
    // On both sides of the bounds, eight waves first, 16 query and 8 key/value heads:
    // heads of 256, 8 requests of 640 tokens 12.4 and 13.8 us, of 800 14.5 and 13.9;
    // heads of 128, one of 1050 10.5 and 11.7, of 1300 11.7 and 11.8; heads of 64, one
    // of 1600 10.1 and 10.5, of 1900 11.3 and 10.8; ten rows a request, heads of
    // 128, 800 tokens 11.5 and 12.9, 1000 12.8 and 11.6; heads of 64, 1100 11.0 and
    // 11.9, 1250 11.9 and 10.5.  144 workgroups of heads of 256, 2000 tokens 26.4 and
    // 25.5, 160 25.5 and 25.1, 192 26.2 and 30.5; 256 with 4300 tokens 53 and 62.
    k.waves = 4;
    if (!k.many && !k.two && (k.sets > 1 || k.splits > 1) && groups <= (c.head_dim == 64 ? 512 : 256) &&
        (tiles * (c.head_dim + 64) <= (k.sets > 1 ? 6800 : 5120) || (groups >= 160 && tiles <= 128))) {
        k.waves = 8;
        k.splits = 1;
    }
    return k;
}

template <int D, bool kWide>
hipError_t launch_d(const AttnArgs& k, const Cut& cut, int64_t groups, hipStream_t stream) {
    const dim3 grid((unsigned)groups), block((unsigned)cut.waves * kWave);
    if (cut.sets == 2 && cut.waves == 8) {
        kv4_attn_sets_kernel<D, 2, 8, kWide><<<grid, block, 0, stream>>>(k);
    } else if (cut.sets == 2) {
        kv4_attn_sets_kernel<D, 2, 4, kWide><<<grid, block, 0, stream>>>(k);
    } else if (cut.sets == 4) {
        if constexpr (D < 256) {
            if (cut.waves == 8) {
                kv4_attn_sets_kernel<D, 4, 8, kWide><<<grid, block, 0, stream>>>(k);
            } else {
                kv4_attn_sets_kernel<D, 4, 4, kWide><<<grid, block, 0, stream>>>(k);
            }
        }
    } else if (cut.many) {
        kv4_attn_many_kernel<D, many_blocks(D), kWide><<<grid, block, 0, stream>>>(k);
    } else if (cut.two) {
        if constexpr (D == 128) kv4_attn_kernel<D, 2, kFewWaves, kWide><<<grid, block, 0, stream>>>(k);
    } else if (cut.waves == 8) {
        kv4_attn_kernel<D, 1, 8, kWide><<<grid, block, 0, stream>>>(k);
    } else {
        kv4_attn_kernel<D, 1, 4, kWide><<<grid, block, 0, stream>>>(k);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || k.splits == 1) return err;
    const int64_t units = (int64_t)k.B * k.max_q * k.g * k.c.heads;
    kv4_attn_join_kernel<D><<<dim3((unsigned)units), dim3(kThreads), 0, stream>>>(k);
    return hipGetLastError();
}

template <int D>
hipError_t launch_w(const AttnArgs& k, const Cut& cut, int64_t groups, hipStream_t stream) {
    return k.c.shift >= 5 ? launch_d<D, true>(k, cut, groups, stream) : launch_d<D, false>(k, cut, groups, stream);
}

}  // namespace

size_t kv4_attn_workspace_bytes(const w4_attn_args& a, const w4_kv4_cache& c) {
    const int splits = cut_of(a, c).splits;
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
    const Cut cut = cut_of(a, c);
    k.row_tiles = cut.row_tiles;
    k.splits = cut.splits;
    k.in_turn = cut.many && (int64_t)a.B * c.kv_heads * k.row_tiles * k.splits <= 512;
    k.window = a.window;
    k.sinks = a.sinks;
    k.scale2 = a.scale * 1.4426950408889634f;
    if (k.splits > 1) {
        k.part_o = static_cast<float*>(workspace);
        k.part_ml = k.part_o + (size_t)a.T * a.q_heads * k.splits * c.head_dim;
    }
    const int64_t groups = (int64_t)a.B * c.kv_heads * k.row_tiles * k.splits;
    switch (c.head_dim) {
        case 64: return launch_w<64>(k, cut, groups, stream);
        case 128: return launch_w<128>(k, cut, groups, stream);
        default: return launch_w<256>(k, cut, groups, stream);
    }
}

}  // namespace w4
