// Sampling: temperature, top-k, top-p and min-p over BF16 logits.
//
// A BF16 has 65536 values, so the counts of a row's values are the whole of
// its sorted order: no sort.  Everything asked is a beginning of that order
// (the first k, the shortest that reaches a mass, the ones above a weight,
// the draw), found from running counts and masses over the values; equal
// logits are told apart by index only at the very end.
//   1. count, a workgroup a chunk of at most 32768 logits: counts in LDS (16
//      bits, 128 KB), written out as a sorted list of (value, count).  A list
//      is a tenth of its chunk, and lists need no clearing and no atomics in
//      memory (adding the counts there instead measured 21 us for one row of
//      262144 and 35 us for 64, all of it contention);
//   2. pick, a workgroup a row: the lists joined in LDS (with a top-k, the
//      first k entries of each: no chunk can have more of the first k),
//      running counts over 1024 segments of 64 values, masses (count *
//      exp(z), FP64) of those up to the k-th, the cuts and the draw; then the
//      chunk, and in it the index, of the drawn value's j-th place.
// Rows of up to 32768 logits are one chunk: the pick counts them itself, in
// one launch and without lists (one row of 32000: 15 us instead of 21, 300 rows
// 30 instead of 44).
// What bounds it: the count by the turns that LDS atomics take (64 rows of
// 262144: 16.5 us, 2 TB/s of logits; bank conflicts are 40 % of the LDS cycles), the pick by the length of its chain of
// dependent steps (14 us for one row, 21 for 64, a compute unit each).
// Counts are whole numbers and masses are summed in a fixed order, so a
// result depends on no order in which anything finishes.
#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

constexpr int kBins = 65536;
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxChunk = 32768;  // four 16-byte loads a thread, and counts that fit 16 bits
constexpr int kMinChunk = 8192;
constexpr int kBlocks = kBins / 2 / kWave;  // of 128 bins, a word a lane
constexpr int kRun = 256;  // entries of a list that a wave joins at a time
constexpr int kMaxChunks = W4_SAMPLE_MAX_VOCAB / kMinChunk;

// A value's bin is its rank among the 65536, the largest first: the bits of a
// negative number, the complement of the lower fifteen of a positive one.
// NaN and -infinity fall on bins that are left out of the lists (no weight,
// behind everything); -0 lies next to +0 and is counted there.
constexpr uint32_t kFirstBin = 0x007F;  // +infinity
constexpr uint32_t kEndBin = 0xFF80;    // -infinity
constexpr uint32_t kPlusZero = 0x7FFF, kMinusZero = 0x8000;
__device__ __forceinline__ uint32_t bits_of_bin(uint32_t bin) { return bin & 0x8000u ? bin : bin ^ 0x7FFFu; }
__device__ __forceinline__ uint32_t bins_of_pair(uint32_t w) {  // two logits -> two bins
    typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
    const uint32_t negative = __builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2, w) >> (i16x2)15);
    return w ^ (~negative & 0x7FFF7FFFu);
}

// 2^y for y <= 0: the power of the nearest whole number, and the Taylor
// series of 2^f to the 13th term for the rest (|f| <= 1/2, so the next term is
// under 2^-53).  A weight costs 15 operations instead of some 60 with a
// division and the library's exp.  The series is off by a few 2^-53; its argument
// has the roundings of a difference times a rate, so a weight 2^y is off by some
// |y| 2^-53 besides.
__device__ __forceinline__ double exp2_series(double y) {
    y = fmax(y, -2000.0);  // 0 far above that
    const double n = rint(y), f = y - n;
    constexpr double kLn2 = 0.69314718055994530942;
    double term[14] = {1.0};
    for (int k = 1; k < 14; ++k) term[k] = term[k - 1] * kLn2 / k;
    double r = term[13];
#pragma unroll
    for (int k = 12; k >= 0; --k) r = fma(r, f, term[k]);
    return ldexp(r, (int)n);
}

// What the first kernel leaves of a chunk: its list's length and its largest
// count; the list itself holds (bin << 16 | count), bins rising.
struct ChunkInfo {
    uint32_t entries, largest;
};
// The workspace: lists [rows][chunks][chunk], infos [rows][chunks], and for
// vocabularies past 65535 32-bit counts [rows][65536].
struct Space {
    uint32_t* lists;
    ChunkInfo* infos;
    uint32_t* counts;
    int chunk, chunks;
};

// Running sums over a wave in six DPP steps (row_shr 1, 2, 4, 8, then the last
// lane of a row of 16, and of the lower half, to the rows above).
template <int kCtrl, int kRows>
__device__ __forceinline__ int moved(int v) {
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xF, false);  // 0 where nothing comes
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)moved<kCtrl, kRows>((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)moved<kCtrl, kRows>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {  // inclusive
    v += moved<0x111, 0xF>(v);
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    v += moved<0x143, 0xC>(v);
    return v;
}
// Values that all lanes share are kept in scalar registers: a branch on one is
// then a jump, and a loop over one no loop over lanes.
__device__ __forceinline__ int last_of(int v) { return __builtin_amdgcn_readlane(v, kWave - 1); }
__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)lane_of((int)(uint32_t)u, lane), hi = (uint32_t)lane_of((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <typename T>
__device__ __forceinline__ T shared_by_all(T v) {
    if constexpr (sizeof(T) == 8) {
        return __builtin_bit_cast(T, lane_of(__builtin_bit_cast(double, v), 0));
    } else {
        return __builtin_bit_cast(T, sgpr(__builtin_bit_cast(uint32_t, v)));
    }
}

// Counts logits i0 .. i1 - 1 of a row into LDS, two 16-bit counts a word, and
// takes out what is in no list.  On return all counts are there for all.
__device__ __forceinline__ void count_into(uint32_t* bins, const uint16_t* row, int i0, int i1) {
    const int tid = threadIdx.x;
    // 16-byte loads from the first aligned logit on, on their way while LDS is cleared
    const int skew = (int)((reinterpret_cast<uintptr_t>(row + i0) >> 1) & 7);
    const int first = min(i0 + ((8 - skew) & 7), i1), wide = (i1 - first) / 8, tail = first + 8 * wide;
    constexpr int kLoads = kMaxChunk / 8 / kThreads;
    u32x4_t w[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
        if (tid + u * kThreads < wide) w[u] = *reinterpret_cast<const u32x4_t*>(row + first + 8 * (tid + u * kThreads));
    uint32_t edge = 0;
    const bool has_edge = tid < first - i0 || (tid >= 8 && tid - 8 < i1 - tail);
    if (has_edge) edge = row[tid < 8 ? i0 + tid : tail + tid - 8];
    u32x4_t* clear = reinterpret_cast<u32x4_t*>(bins);
#pragma unroll
    for (int i = 0; i < kBins / 8 / kThreads; ++i) clear[i * kThreads + tid] = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    const auto count = [&](uint32_t bin) { atomicAdd(&bins[bin >> 1], bin & 1 ? 0x10000u : 1u); };
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
        if (tid + u * kThreads < wide) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t pair = bins_of_pair(w[u][e]);
                count(pair & 0xFFFFu);
                count(pair >> 16);
            }
        }
    if (has_edge) count(bins_of_pair(edge) & 0xFFFFu);
    __syncthreads();
    constexpr int kBefore = kFirstBin >> 1, kAfter = (kBins - kEndBin) >> 1;
    static_assert(kBefore <= kThreads / 2 && kAfter <= kThreads / 2 && kFirstBin % 2 == 1 && kEndBin % 2 == 0, "a thread a word");
    if (tid < kBefore) bins[tid] = 0;
    if (tid >= kThreads / 2 && tid < kThreads / 2 + kAfter) bins[kEndBin / 2 + tid - kThreads / 2] = 0;
    if (tid == kBefore) {
        bins[kPlusZero >> 1] += bins[kMinusZero >> 1] << 16;
        bins[kMinusZero >> 1] &= 0xFFFF0000u;
        bins[kBefore] &= 0xFFFF0000u;  // +infinity is the upper half of its word
    }
    __syncthreads();
}

__global__ __launch_bounds__(kThreads) void sample_count_kernel(SampleArgs a, Space sp) {
    __shared__ uint32_t bins[kBins / 2];  // two 16-bit counts a word
    __shared__ uint32_t block_entries[kBlocks], wave_largest[kWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = (int)sgpr(tid / kWave);
    const int i0 = blockIdx.x * sp.chunk, i1 = min(i0 + sp.chunk, a.vocab);
    const uint16_t* row = a.logits + (int64_t)blockIdx.y * a.stride;

    if (tid < kBlocks) block_entries[tid] = 0;
    count_into(bins, row, i0, i1);

    // Blocks of 128 bins in turn over the waves, since those in use lie
    // together (a wave with 4096 bins of its own made a workgroup 1.5 us
    // longer): which are in use at all, how many entries each has, the
    // entries before each, then the list.
    constexpr int kRounds = kBlocks / kWaves;
    const auto word_of = [&](int i) { return (i * kWaves + wave) * kWave + lane; };
    uint32_t used = 0;
#pragma unroll 8
    for (int i = 0; i < kRounds; ++i) {
        used |= (uint32_t)(__any(bins[word_of(i)] != 0) != 0) << i;
    }
    uint32_t largest = 0;
    used = sgpr(used);
#pragma unroll 1
    for (uint32_t rest = used; rest; rest &= rest - 1) {
        const int i = __ffs(rest) - 1;
        const uint32_t c = bins[word_of(i)];
        const int n = __popcll(__ballot(c & 0xFFFFu)) + __popcll(__ballot(c >> 16));
        if (lane == 0) block_entries[i * kWaves + wave] = n;
        largest = max(largest, max(c & 0xFFFFu, c >> 16));
    }
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) largest = max(largest, (uint32_t)__shfl_xor((int)largest, m));
    if (lane == 0) wave_largest[wave] = largest;
    __syncthreads();
    // a lane's eight blocks: the wave's block of round i is one of lane 2 i + wave / 8
    constexpr int kEach = kBlocks / kWave;
    static_assert(kEach == 8 && kWaves == 16, "a lane's blocks and the waves' turns");
    int all = 0, before = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int n = (int)block_entries[lane * kEach + k];
        if (k < wave % kEach) before += n;
        all += n;
    }
    const int upto = wave_scan(all);
    before += upto - all;
    const int sum = last_of(upto);
#pragma unroll 4
    for (int u = 0; u < kWaves; ++u) largest = max(largest, wave_largest[u]);
    const size_t mine = (size_t)blockIdx.y * sp.chunks + blockIdx.x;
    if (tid == 0) sp.infos[mine] = {(uint32_t)sum, largest};
    uint32_t* list = sp.lists + mine * sp.chunk;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll 1
    for (uint32_t rest = used; rest; rest &= rest - 1) {
        const int i = __ffs(rest) - 1;
        const uint32_t word = word_of(i), c = bins[word];
        const uint64_t lo = __ballot(c & 0xFFFFu), hi = __ballot(c >> 16);
        uint32_t to = lane_of(before, 2 * i + wave / kEach) + __popcll(lo & below) + __popcll(hi & below);
        if (c & 0xFFFFu) list[to++] = 2 * word << 16 | (c & 0xFFFFu);
        if (c >> 16) list[to] = (2 * word + 1) << 16 | c >> 16;
    }
}

// kWhole: rows of one chunk, counted here; there are no lists.
template <bool kWhole>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a, Space sp) {
    __shared__ uint32_t bins[kBins / 2];
    __shared__ int cnt[kThreads + 1];      // tokens before a segment of 64 bins
    __shared__ double mass[kThreads + 1];  // their weight
    __shared__ int own_cnt[kThreads];
    __shared__ double own_mass[kThreads];
    __shared__ double wave_mass[kWaves];
    __shared__ int wave_cnt[kWaves];
    __shared__ int drawn[2];  // the bin, and the place among its tokens
    __shared__ int strong;  // tokens with w >= min_p
    constexpr int kLists = kWhole ? 1 : kMaxChunks;
    __shared__ int at_chunk[kLists], entries[kLists], runs[kLists + 1];
    __shared__ int first_bin;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = (int)sgpr(tid / kWave);
    const int row = blockIdx.x;
    const ChunkInfo* infos = sp.infos + (size_t)row * sp.chunks;
    const uint32_t* lists = sp.lists + (size_t)row * sp.chunks * sp.chunk;
    uint32_t* far = sp.counts + (size_t)row * kBins;

    // the row's settings and the first 64 chunks' infos, on their way while LDS is cleared
    const float own_heat = a.temperature ? a.temperature[row] : 1.0f, own_floor = a.min_p ? a.min_p[row] : 0.0f;
    const float own_p = a.top_p ? a.top_p[row] : 1.0f;
    const int own_k = a.top_k ? a.top_k[row] : 0;
    const double own_uniform = a.uniform[row];
    ChunkInfo first_info = {0, 0};
    uint32_t first_entry = 0;
    if constexpr (!kWhole) {
        if (lane < sp.chunks) {
            first_info = infos[lane];
            first_entry = lists[(size_t)lane * sp.chunk];
        }
        u32x4_t* clear = reinterpret_cast<u32x4_t*>(bins);
#pragma unroll
        for (int i = 0; i < kBins / 8 / kThreads; ++i) clear[i * kThreads + tid] = u32x4_t{0, 0, 0, 0};
    }
    own_cnt[tid] = 0;
    own_mass[tid] = 0;
    if (tid == 0) {
        strong = 0;
        first_bin = kBins;
    }
    const float heat = shared_by_all(own_heat), floor_p = shared_by_all(own_floor), p = shared_by_all(own_p);
    const int top_k = shared_by_all(own_k);
    const double uniform = shared_by_all(own_uniform);
    const bool greedy = !(heat > 0.0f);
    int keep = a.vocab;
    if (top_k > 0) keep = min(keep, top_k);
    if (greedy) keep = 1;

    int top = kBins;
    bool near = true;  // the counts are in LDS, in 16 bits
    bool held = false;
    uint32_t x[4][kRun / kWave] = {};  // entries of four runs; 0: none, adds nothing
    int chunk_of_run[4] = {};
    if constexpr (kWhole) {
        count_into(bins, a.logits + (int64_t)row * a.stride, 0, a.vocab);
    } else {
        // The largest value, whether the joined counts fit 16 bits, and the runs
        // of entries up to each chunk.
        uint32_t most = 0;
        int run_base = 0;
        for (int c0 = 0; c0 < sp.chunks; c0 += kWave) {
            const int c = c0 + lane;
            ChunkInfo info = first_info;
            uint32_t first = first_entry;  // of no meaning in an empty list
            if (c0 > 0) {
                info = {0, 0};
                if (c < sp.chunks) {
                    info = infos[c];
                    first = lists[(size_t)c * sp.chunk];
                }
            }
            if (info.entries) top = min(top, (int)(first >> 16));
            most += info.largest;
            const int joined = min((int)info.entries, keep);
            const int upto = run_base + wave_scan((joined + kRun - 1) / kRun);
            if (wave == 0 && c < sp.chunks) {
                at_chunk[c] = 0;
                entries[c] = (int)info.entries;
                runs[c + 1] = upto;
            }
            run_base = last_of(upto);
        }
        if (tid == 0) runs[0] = 0;
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) {
            top = min(top, __shfl_xor(top, m));
            most += __shfl_xor((int)most, m);
        }
        top = shared_by_all(top);
        near = shared_by_all(most) < 65536u;  // else the counts are kept in memory
        if (top == kBins) {
            if (tid == 0) a.tokens[row] = -1;
            return;
        }
        if (!near) {
            for (int i = tid; i < kBins; i += kThreads) __hip_atomic_store(&far[i], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __threadfence();
        }
        __syncthreads();
        // A wave takes every 16th run, four of them in flight.  Where that is all
        // of them, they are kept for the search at the end.
        held = run_base <= 4 * kWaves;
#pragma unroll 1
        for (int r0 = wave, c = 0; r0 < run_base; r0 += 4 * kWaves) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * kWaves;
#pragma unroll
                for (int u = 0; u < kRun / kWave; ++u) x[k][u] = 0;
                if (r >= run_base) continue;
                while (r >= runs[c + 1]) ++c;
                chunk_of_run[k] = c;
                const int i = (r - runs[c]) * kRun + lane, n = min(entries[c], keep);
                const uint32_t* list = lists + (size_t)c * sp.chunk;
#pragma unroll
                for (int u = 0; u < kRun / kWave; ++u)
                    if (i + u * kWave < n) x[k][u] = list[i + u * kWave];
            }
            if (near) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int u = 0; u < kRun / kWave; ++u)
                        if (x[k][u])  // adding 0 to one place from many lanes costs a turn each
                            atomicAdd(&bins[x[k][u] >> 17], (x[k][u] & 0xFFFFu) << (x[k][u] >> 12 & 16));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int u = 0; u < kRun / kWave; ++u)
                        if (x[k][u])
                            __hip_atomic_fetch_add(&far[x[k][u] >> 16], x[k][u] & 0xFFFFu, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (!near) __threadfence();
        __syncthreads();
    }
    const auto count = [&](int bin) -> int {
        if (kWhole || near) return (int)(bins[bin >> 1] >> (16 * (bin & 1)) & 0xFFFFu);
        return (int)__hip_atomic_load(&far[bin], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };

    // Running sums over the segments, a thread each.
    const auto run_over = [&](auto own, auto* part) {
        auto sum = wave_scan(own);
        if (lane == kWave - 1) part[wave] = sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) sum += part[w];
        return sum;
    };
    // Tokens of each segment, pairs of them in turn over the waves (those in
    // use lie together): first which of a wave's 32 pairs are in use.
    const auto pair_of = [&](int i) { return i * kWaves + wave; };
    uint32_t used = 0;
    if (kWhole || near) {
#pragma unroll
        for (int i = 0; i < kThreads / kWaves / 2; ++i)  // a pair's 128 counts are 64 words
            if (__any(bins[pair_of(i) * kWave + lane] != 0)) used |= 1u << i;
    } else {
        for (int i = 0; i < kThreads / kWaves / 2; ++i)
            if (__any((count(2 * pair_of(i) * kWave + lane) | count((2 * pair_of(i) + 1) * kWave + lane)) != 0)) used |= 1u << i;
    }
    if constexpr (kWhole) {
        if (used) {  // this wave's first value, of which the first of all is the largest logit
            const int word = pair_of(__ffs(used) - 1) * kWave + lane;
            const uint64_t some = __ballot(bins[word] != 0);
            if (lane == __ffsll((unsigned long long)some) - 1) atomicMin(&first_bin, 2 * word + ((bins[word] & 0xFFFFu) == 0));
        }
    }
#pragma unroll 1
    for (uint32_t rest = used; rest; rest &= rest - 1) {
        const int e = 2 * pair_of(__ffs(rest) - 1);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const int c = wave_scan(count((e + h) * kWave + lane));
            if (lane == kWave - 1) own_cnt[e + h] = c;
        }
    }
    __syncthreads();
    if constexpr (kWhole) {
        top = shared_by_all(first_bin);
        if (top == kBins) {
            if (tid == 0) a.tokens[row] = -1;
            return;
        }
    }
    const double largest = bf16_to_f32(bits_of_bin(top));
    const double rate = greedy ? 1.0 : 1.4426950408889634074 / (double)heat;
    const auto weight = [&](int bin) {
        if (bin == top) return 1.0;  // also where the largest is an infinity
        return exp2_series(((double)bf16_to_f32(bits_of_bin(bin)) - largest) * rate);
    };

    const int own_c = own_cnt[tid];
    const int sc = run_over(own_c, wave_cnt);
    cnt[tid + 1] = sc;
    if (tid == 0) cnt[0] = 0, mass[0] = 0;
    __syncthreads();
    keep = min(keep, shared_by_all(cnt[kThreads]));  // NaN and -infinity are in no list
    // Their weight, up to the last that can be kept.
    int above = 0;
#pragma unroll 1
    for (uint32_t rest = used; rest; rest &= rest - 1) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const int e = 2 * pair_of(__ffs(rest) - 1) + h;
            if (shared_by_all(cnt[e]) >= keep) continue;
            const int n = count(e * kWave + lane);
            const double w = n ? weight(e * kWave + lane) : 0.0;
            if (n && !(w < (double)floor_p)) above += n;
            const double sum = wave_scan(w * (double)n);
            if (lane == kWave - 1) own_mass[e] = sum;
        }
    }
    above = last_of(wave_scan(above));
    if (lane == 0 && above) atomicAdd(&strong, above);
    __syncthreads();
    const double sm = run_over(own_mass[tid], wave_mass);
    mass[tid + 1] = sm;
    __syncthreads();

    // Five looks into the order, one after the other: what the first ``keep``
    // weigh, where top-p of that is reached, what those weigh that are then
    // kept, where the draw falls, and the value of that rank.  One wave does
    // them, with one body for all.  The third and the last are answered as a
    // rule by the one before, in the place that it found.
    if (wave == 0) {
        const bool cut = p < 1.0f && keep > 1;
        double goal = 0, kept_mass = 0;
        int rank = 0, kept = -1;  // what the first ``kept`` weigh is known
        // a draw stays below the whole weight by more than the sums' rounding
        const double part = fmin(fmax(uniform, 0.0), 1.0 - 0x1p-40);
#pragma unroll 1
        for (int look = cut ? 0 : 2; look < 5; ++look) {
            if (look == 2) {
                if (floor_p > 0.0f) keep = min(keep, max(shared_by_all(strong), 1));
                rank = keep - 1;
                if (keep == kept) {
                    goal = part * kept_mass;
                    continue;
                }
            }
            // looks 0, 2: the token of rank keep - 1; 1: at least goal; 3: past goal; 4: the token of rank
            const bool by_rank = look % 2 == 0;
            const int k = look == 4 ? rank : keep - 1;
            const auto ends = [&](int tokens, double weighs) {
                return by_rank ? tokens > k : look == 1 ? weighs >= goal : weighs > goal;
            };
            // The first segment at whose end it holds (so one in use): among
            // the ends of 16 runs of 64, then in that run.
            const int end = (lane < kWaves ? lane + 1 : kWaves) * kWave;
            const uint64_t runs_past = __ballot(ends(cnt[end], mass[end]));
            if (!runs_past && !by_rank) continue;  // top-p: all of it, by rounding
            const int from = min(__ffsll((unsigned long long)runs_past) - 1 + (runs_past == 0) * kWaves, kWaves - 1) * kWave;
            const uint64_t past = __ballot(ends(cnt[from + lane + 1], mass[from + lane + 1]));
            const int e = from + (past ? __ffsll((unsigned long long)past) - 1 : kWave - 1);
            // its values, one a lane: tokens, those before, their weights
            const int n = count(e * kWave + lane);
            const double w = n ? weight(e * kWave + lane) : 0.0;
            const double own = w * (double)n, m = mass[e] + (wave_scan(own) - own);
            const int c = cnt[e] + wave_scan(n) - n;
            const int l = __ffsll((unsigned long long)__ballot(n > 0 && ends(c + n, m + own))) - 1;
            const int last = shared_by_all(cnt[e + 1]);
            if (by_rank) {
                const int at = max(l, 0);
                const double weighs = m + w * (double)(k + 1 - c);
                if (look == 4) {
                    const int among = lane_of(rank - c, at);
                    if (lane == 0) drawn[0] = e * kWave + at, drawn[1] = among;
                } else {
                    const double all = lane_of(weighs, at);
                    goal = (look == 0 ? (double)p : part) * all;
                }
            } else {
                // tokens of this value before the goal: with less than it before them (look 1), or not past it (3)
                const double steps = (goal - m) / w, whole = look == 1 ? ceil(steps) : floor(steps);
                const int most = look == 1 ? n : n - 1;
                const int more = whole > 0.0 ? (int)fmin(whole, (double)most) : 0;
                const int at = l >= 0 ? lane_of(c + more, l) : look == 1 ? last : last - 1;
                const int among = lane_of(more, max(l, 0));
                if (look == 1) {
                    keep = min(keep, max(at, 1));
                    if (l >= 0 && among > 0 && keep == at) {
                        kept = keep;
                        kept_mass = lane_of(m + w * (double)more, l);
                    }
                } else {
                    rank = min(rank, at);
                    if (l >= 0 && rank == at) {
                        if (lane == 0) drawn[0] = e * kWave + l, drawn[1] = among;
                        break;
                    }
                }
            }
        }
    }
    __syncthreads();
    const uint32_t want = (uint32_t)shared_by_all(drawn[0]);
    const int among = shared_by_all(drawn[1]);

    int before = 0, chunk = 0;  // the chunk with the among-th, and those before it
    if constexpr (!kWhole) {
        // How many of them each chunk holds: from the entries joined (with a
        // top-k those that are not cannot have any), if they are still there; else
        // its list is sorted, so 64 places of it at a time narrow it down.
        if (held) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int u = 0; u < kRun / kWave; ++u)
                    if (x[k][u] && x[k][u] >> 16 == want) at_chunk[chunk_of_run[k]] = (int)(x[k][u] & 0xFFFFu);
        }
        for (int c = wave; !held && c < sp.chunks; c += kWaves) {
            const uint32_t* list = lists + (size_t)c * sp.chunk;
            int lo = 0, n = shared_by_all(entries[c]);  // entries lo .. lo + n - 1 may be the one
            while (n > kWave) {
                const int step = (n + kWave - 1) / kWave, i = lane * step;
                // places at or below the value: a beginning of the lanes
                const int below = __popcll(__ballot(i < n && list[lo + (i < n ? i : 0)] >> 16 <= want));
                const int from = max(below - 1, 0) * step;
                lo += from;
                n = min(step, n - from);
            }
            const uint32_t y = lane < n ? list[lo + lane] : 0;
            const uint64_t found = __ballot(lane < n && y >> 16 == want);
            if (found >> lane & 1) at_chunk[c] = (int)(y & 0xFFFFu);
        }
        __syncthreads();
        for (int c0 = 0; c0 < sp.chunks; c0 += kWave) {
            const int h = c0 + lane < sp.chunks ? at_chunk[c0 + lane] : 0, sum = before + wave_scan(h);
            const uint64_t past = __ballot(sum > among);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                chunk = c0 + l;
                before = lane_of(sum - h, l);
                break;
            }
            before = last_of(sum);
        }
        __syncthreads();
    }

    // Matches in pieces of 512 of its logits (eight a lane, 16-byte aligned),
    // their running sum, then that one piece again.
    const int i0 = chunk * sp.chunk, size = min(sp.chunk, a.vocab - i0);
    const uint16_t* logits = a.logits + (int64_t)row * a.stride + i0;
    const int skew = (int)((reinterpret_cast<uintptr_t>(logits) >> 1) & 7);
    const int pieces = (size + skew + 511) / 512;  // at most 65
    int* matches = cnt;
    // The value's bits, in both halves of a word; zeros of either sign are one.
    const uint32_t bits = bits_of_bin(want), pattern = bits << 16 | bits, care = bits ? 0xFFFFFFFFu : 0x7FFF7FFFu;
    const auto first_of = [&](int piece) { return piece * 512 + 8 * lane - skew; };
    const auto inside = [&](int first) { return first >= 0 && first + 8 <= size; };
    const auto wide_at = [&](int first) {
        return inside(first) ? *reinterpret_cast<const u32x4_t*>(logits + first) : u32x4_t{0, 0, 0, 0};
    };
    // bit i: logit first + i of a lane's eight holds the value
    const auto hits_of = [&](int first, const u32x4_t& w) {
        uint32_t hits = 0;
        if (inside(first)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = (w[e] ^ pattern) & care;
                hits |= (uint32_t)((x & 0xFFFFu) == 0) << (2 * e) | (uint32_t)(x >> 16 == 0) << (2 * e + 1);
            }
        } else {
#pragma unroll 1
            for (int e = max(0, -first); e < 8 && first + e < size; ++e)
                hits |= (uint32_t)((((uint32_t)logits[first + e] ^ bits) & care & 0xFFFFu) == 0) << e;
        }
        return hits;
    };
    constexpr int kPieces = kMaxChunk / 512 / kWaves + 1;
    u32x4_t w[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) w[u] = wide_at(first_of(wave + u * kWaves));
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
        const int piece = wave + u * kWaves;
        if (piece >= pieces) break;
        const uint32_t hits = hits_of(first_of(piece), w[u]);
        int sum = 0;
        if (__any(hits != 0)) sum = last_of(wave_scan((int)__popc(hits)));
        if (lane == 0) matches[piece] = sum;
    }
    __syncthreads();
    if (wave != 0) return;
    for (int i = 0; i < pieces; i += kWave) {
        const int h = i + lane < pieces ? matches[i + lane] : 0;
        const int s = before + wave_scan(h);
        const uint64_t past = __ballot(s > among);
        if (past) {
            const int piece = __ffsll((unsigned long long)past) - 1;
            before = lane_of(s - h, piece);
            const int at = first_of(i + piece);
            const uint32_t hits = hits_of(at, wide_at(at));
            const int mine = (int)__popc(hits), first = before + wave_scan(mine) - mine;
            if (among >= first && among < first + mine) {
                uint32_t rest = hits;
                for (int k = first; k < among; ++k) rest &= rest - 1;
                a.tokens[row] = i0 + at + __ffs(rest) - 1;
            }
            return;
        }
        before = last_of(s);
    }
}

// Chunks that give the chip a workgroup a compute unit, within what one can
// count; all chunks of a call are alike.
int chunk_of(int rows, int vocab) {
    const int64_t c = (((int64_t)rows * vocab / 256) + 8191) / 8192 * 8192;
    return (int)(c < kMinChunk ? kMinChunk : c > kMaxChunk ? kMaxChunk : c);
}

}  // namespace

size_t sample_workspace_bytes(int rows, int vocab) {
    if (vocab <= kMaxChunk) return 0;
    const int chunk = chunk_of(rows, vocab);
    const size_t chunks = (size_t)rows * ((vocab + chunk - 1) / chunk);
    return chunks * chunk * 4 + chunks * sizeof(ChunkInfo) + (vocab > 65535 ? (size_t)rows * kBins * 4 : 0);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
    Space sp = {};
    if (a.vocab <= kMaxChunk) {
        sp.chunk = kMaxChunk;
        sp.chunks = 1;
        sample_pick_kernel<true><<<dim3((unsigned)a.rows), dim3(kThreads), 0, stream>>>(a, sp);
        return hipGetLastError();
    }
    sp.chunk = chunk_of(a.rows, a.vocab);
    sp.chunks = (a.vocab + sp.chunk - 1) / sp.chunk;
    const size_t chunks = (size_t)a.rows * sp.chunks;
    sp.lists = static_cast<uint32_t*>(workspace);
    sp.infos = reinterpret_cast<ChunkInfo*>(sp.lists + chunks * sp.chunk);
    sp.counts = reinterpret_cast<uint32_t*>(sp.infos + chunks);
    sample_count_kernel<<<dim3((unsigned)sp.chunks, (unsigned)a.rows), dim3(kThreads), 0, stream>>>(a, sp);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    sample_pick_kernel<false><<<dim3((unsigned)a.rows), dim3(kThreads), 0, stream>>>(a, sp);
    return hipGetLastError();
}

}  // namespace w4
