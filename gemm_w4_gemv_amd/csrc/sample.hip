// Sampling: temperature, top-k, top-p and min-p over BF16 logits.
//
// A BF16 has 65536 values, so a row's histogram over them is the whole of
// its sorted order: no sort.  Everything asked is a beginning of that order
// (the first k, the shortest that reaches a mass, the ones above a weight,
// the draw), found from running counts and masses over the bins; equal
// logits are told apart by index only at the very end.
//   1. clear the rows' histograms;
//   2. histogram: a workgroup counts a chunk of a row in LDS (16-bit counts,
//      128 KB) and adds what is not zero to the row's counts in memory;
//   3. pick, a workgroup a row: masses of the bins in use (count * exp(z),
//      FP64), running sums over 1024 segments of 64 bins, the cuts and the
//      draw, then the j-th index that holds the drawn value.
// Counts are whole numbers and masses are summed in a fixed order, so the
// result does not depend on the order in which workgroups finish.
#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

constexpr int kBins = 65536;
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxChunk = 32768;  // a chunk's counts fit 16 bits
constexpr int kSlabs = kBins / kThreads;
constexpr uint32_t kNegInf = 0xFF80u;

// BF16 bits with -0 and NaN folded away: -0 is +0, NaN is -infinity.
__device__ __forceinline__ uint32_t plain_bits(uint32_t b) {
    if ((b & 0x7FFFu) > 0x7F80u) return kNegInf;
    return b == 0x8000u ? 0u : b;
}
// Rank of a value among the 65536, the largest first.
__device__ __forceinline__ uint32_t bin_of(uint32_t b) {
    b = plain_bits(b);
    return b & 0x8000u ? b : 0x7FFFu - b;
}
__device__ __forceinline__ uint32_t bits_of_bin(uint32_t bin) { return bin & 0x8000u ? bin : 0x7FFFu - bin; }

__global__ __launch_bounds__(256) void sample_clear_kernel(u32x4_t* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = u32x4_t{0, 0, 0, 0};
}

// Calls f(element index, bits) for the calling thread's share of [i0, i1) of
// a row; 16-byte loads where the row's address allows.
template <typename F>
__device__ __forceinline__ void for_logits(const uint16_t* row, int i0, int i1, int tid, F f) {
    const int skew = (int)((reinterpret_cast<uintptr_t>(row + i0) >> 1) & 7);
    const int first = min(i0 + ((8 - skew) & 7), i1);  // 16-byte aligned from here
    const int wide = (i1 - first) / 8;
    if (tid < first - i0) f(i0 + tid, (uint32_t)row[i0 + tid]);
    for (int c = tid; c < wide; c += kThreads) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + first + 8 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f(first + 8 * c + 2 * e, w[e] & 0xFFFFu);
            f(first + 8 * c + 2 * e + 1, w[e] >> 16);
        }
    }
    const int tail = first + 8 * wide;
    if (tid < i1 - tail) f(tail + tid, (uint32_t)row[tail + tid]);
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, uint32_t* hist, int chunk) {
    __shared__ uint32_t bins[kBins / 2];  // two 16-bit counts a word
    const int tid = threadIdx.x;
    u32x4_t* wide = reinterpret_cast<u32x4_t*>(bins);
#pragma unroll
    for (int i = 0; i < kBins / 8 / kThreads; ++i) wide[i * kThreads + tid] = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    const int i0 = blockIdx.x * chunk, i1 = min(i0 + chunk, a.vocab);
    for_logits(a.logits + (int64_t)blockIdx.y * a.stride, i0, i1, tid, [&](int, uint32_t b) {
        const uint32_t bin = bin_of(b);
        atomicAdd(&bins[bin >> 1], bin & 1 ? 0x10000u : 1u);
    });
    __syncthreads();
    uint32_t* mine = hist + (size_t)blockIdx.y * kBins;
    for (int i = 0; i < kBins / 8 / kThreads; ++i) {
        const int at = i * kThreads + tid;
        const u32x4_t w = wide[at];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (w[e] & 0xFFFFu) atomicAdd(&mine[8 * at + 2 * e], w[e] & 0xFFFFu);
            if (w[e] >> 16) atomicAdd(&mine[8 * at + 2 * e + 1], w[e] >> 16);
        }
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v, int lane) {  // inclusive
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const T u = __shfl_up(v, off);
        if (lane >= off) v += u;
    }
    return v;
}

// Where a beginning of the order ends.
struct Cut {
    int64_t rank;  // tokens before it
    double mass;   // their weight
    int bin;       // of the last one counted, or the one drawn
    int among;     // how many of that bin's tokens come before
};

__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a, const uint32_t* __restrict__ hist_all) {
    // segment e = 16 * slab + wave: bins 64 e .. 64 e + 63
    __shared__ int64_t cnt[kThreads + 1];   // tokens before the segment
    __shared__ double mass[kThreads + 1];   // their weight
    __shared__ int64_t wave_cnt[kWaves];
    __shared__ double wave_mass[kWaves];
    __shared__ int top_bin;
    __shared__ int64_t strong;  // tokens with w >= min_p
    __shared__ int found[4];
    __shared__ int matches[W4_SAMPLE_MAX_VOCAB / 512 + 1];  // a row's pieces
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = (int)sgpr(tid / kWave);
    const int row = blockIdx.x;
    const uint32_t* hist = hist_all + (size_t)row * kBins;

    if (tid == 0) {
        top_bin = kBins - 1;
        strong = 0;
    }
    __syncthreads();
    // The slabs in which this wave's bins hold anything: a few dozen of the
    // 65536 bins' 1024 segments, as logits lie within a few powers of two.
    uint64_t used = 0;
#pragma unroll 8
    for (int s = 0; s < kSlabs; ++s) {
        const uint64_t any = __ballot(hist[s * kThreads + tid] != 0);
        if (any && !used && lane == 0)
            atomicMin(&top_bin, s * kThreads + wave * kWave + __ffsll((unsigned long long)any) - 1);
        if (any) used |= 1ull << s;
    }
    __syncthreads();
    const int top = top_bin;
    const uint32_t top_bits = bits_of_bin(top);
    if (top_bits == kNegInf) {
        if (tid == 0) a.tokens[row] = -1;
        return;
    }
    const double largest = bf16_to_f32(top_bits);
    const float heat = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(heat > 0.0f);
    const double t = greedy ? 1.0 : (double)heat;
    const float floor_p = a.min_p ? a.min_p[row] : 0.0f;
    const auto weight = [&](int bin) {
        if (bin == top) return 1.0;  // also where the largest is an infinity
        return exp(((double)bf16_to_f32(bits_of_bin(bin)) - largest) / t);
    };

    cnt[lane * kWaves + wave] = 0;  // a lane for each slab
    mass[lane * kWaves + wave] = 0;
    int64_t above = 0;
    for (uint64_t rest = used; rest; rest &= rest - 1) {
        const int s = __ffsll((unsigned long long)rest) - 1;
        const uint32_t n = hist[s * kThreads + tid];
        const double w = n ? weight(s * kThreads + tid) : 0.0;
        if (n && !(w < (double)floor_p)) above += n;
        const double sum = wave_sum(w * (double)n);
        int64_t c = n;
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) c += __shfl_xor(c, m);
        if (lane == 0) cnt[s * kWaves + wave] = c, mass[s * kWaves + wave] = sum;
    }
    if (above) atomicAdd(reinterpret_cast<unsigned long long*>(&strong), (unsigned long long)above);
    __syncthreads();
    // running sums over the segments
    const int64_t own_c = cnt[tid];
    const double own_m = mass[tid];
    int64_t sc = wave_scan(own_c, lane);
    double sm = wave_scan(own_m, lane);
    if (lane == kWave - 1) wave_cnt[wave] = sc, wave_mass[wave] = sm;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sc += wave_cnt[w], sm += wave_mass[w];
    __syncthreads();
    cnt[tid + 1] = sc;
    mass[tid + 1] = sm;
    if (tid == 0) cnt[0] = 0, mass[0] = 0;
    __syncthreads();

    if (wave == 0) {
        // The segment before whose end ``ends`` first holds, or the last one in use.
        const auto segment = [&](auto ends) {
            int at = kThreads;  // none
            for (int i = 0; i < kThreads; i += kWave) {
                const uint64_t hit = __ballot(cnt[i + lane + 1] > cnt[i + lane] && ends(i + lane));
                if (hit) {
                    at = i + __ffsll((unsigned long long)hit) - 1;
                    break;
                }
            }
            return at;
        };
        const auto last_used = [&]() {
            int at = 0;
            for (int i = 0; i < kThreads; i += kWave) {
                const uint64_t used = __ballot(cnt[i + lane + 1] > cnt[i + lane]);
                if (used) at = i + 63 - __clzll((long long)used);
            }
            return at;
        };
        struct Bins {
            int64_t n, c;  // a lane's bin: its tokens, those before it
            double w, m;   // a token's weight, the weight before it
        };
        const auto bins_of = [&](int e) {
            Bins b;
            b.n = hist[e * kWave + lane];
            b.w = b.n ? weight(e * kWave + lane) : 0.0;
            const double own = b.w * (double)b.n;
            b.c = cnt[e] + wave_scan(b.n, lane) - b.n;
            b.m = mass[e] + (wave_scan(own, lane) - own);
            return b;
        };
        // weight of the first k tokens
        const auto mass_of_first = [&](int64_t k) {
            const int e = min(segment([&](int i) { return cnt[i + 1] >= k; }), kThreads - 1);
            const Bins b = bins_of(e);
            const uint64_t hit = __ballot(b.n > 0 && b.c + b.n >= k);
            const int l = __ffsll((unsigned long long)hit) - 1;
            return __shfl(b.m + b.w * (double)(k - b.c), l);
        };
        const int64_t all = a.vocab;
        int64_t keep = all;
        if (a.top_k && a.top_k[row] > 0) keep = min(keep, (int64_t)a.top_k[row]);
        if (greedy) keep = 1;
        const float p = a.top_p ? a.top_p[row] : 1.0f;
        if (p < 1.0f && keep > 1) {
            // tokens with less than p of the mass before them
            const double goal = (double)p * mass_of_first(keep);
            int64_t reach = all;
            const int e = segment([&](int i) { return mass[i + 1] >= goal; });
            if (e < kThreads) {
                const Bins b = bins_of(e);
                const uint64_t hit = __ballot(b.n > 0 && b.m + b.w * (double)b.n >= goal);
                if (hit) {
                    const int l = __ffsll((unsigned long long)hit) - 1;
                    const double need = ceil((goal - b.m) / b.w);
                    const int64_t more = need > 0.0 ? (int64_t)fmin(need, (double)b.n) : 0;
                    reach = __shfl(b.c + more, l);
                } else {
                    reach = cnt[e + 1];
                }
            }
            keep = min(keep, max(reach, (int64_t)1));
        }
        if (floor_p > 0.0f) keep = min(keep, max(strong, (int64_t)1));
        // the draw
        const double goal = a.uniform[row] * mass_of_first(keep);
        int e = segment([&](int i) { return mass[i + 1] > goal; });
        int64_t rank = keep - 1;
        if (e < kThreads) {
            const Bins b = bins_of(e);
            const uint64_t hit = __ballot(b.n > 0 && b.m + b.w * (double)b.n > goal);
            if (hit) {
                const int l = __ffsll((unsigned long long)hit) - 1;
                const double past = floor((goal - b.m) / b.w);
                const int64_t more = past > 0.0 ? (int64_t)fmin(past, (double)(b.n - 1)) : 0;
                rank = min(rank, __shfl(b.c + more, l));
            } else {
                rank = min(rank, cnt[e + 1] - 1);
            }
        }
        // the bin of that rank, and the place in it
        e = segment([&](int i) { return cnt[i + 1] > rank; });
        if (e == kThreads) e = last_used();
        const Bins b = bins_of(e);
        const uint64_t hit = __ballot(b.n > 0 && b.c + b.n > rank);
        const int l = hit ? __ffsll((unsigned long long)hit) - 1 : 63;
        const int among = (int)__shfl(rank - b.c, l);
        if (lane == 0) {
            found[0] = e * kWave + l;
            found[1] = among;
        }
    }
    __syncthreads();
    const uint32_t want = (uint32_t)found[0];
    const int among = found[1];

    // The among-th index that holds the value: matches in pieces of 512
    // logits (eight a lane, 16-byte aligned), their running sum, then that one
    // piece again.
    const uint16_t* logits = a.logits + (int64_t)row * a.stride;
    const int skew = (int)((reinterpret_cast<uintptr_t>(logits) >> 1) & 7);
    const int pieces = (a.vocab + skew + 511) / 512;
    // bit i: logit first + i of a lane's eight holds the value
    const auto hits_at = [&](int piece) {
        const int first = piece * 512 + 8 * lane - skew;
        uint32_t hits = 0;
        if (first >= 0 && first + 8 <= a.vocab) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t*>(logits + first);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hits |= (uint32_t)(bin_of(w[e] & 0xFFFFu) == want) << (2 * e);
                hits |= (uint32_t)(bin_of(w[e] >> 16) == want) << (2 * e + 1);
            }
        } else {
            for (int e = max(0, -first); e < 8 && first + e < a.vocab; ++e)
                hits |= (uint32_t)(bin_of(logits[first + e]) == want) << e;
        }
        return hits;
    };
    for (int p0 = wave; p0 < pieces; p0 += 4 * kWaves) {
        uint32_t hits[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) hits[u] = p0 + u * kWaves < pieces ? hits_at(p0 + u * kWaves) : 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (p0 + u * kWaves >= pieces) break;
            int sum = 0;
            if (__any(hits[u] != 0)) sum = __shfl(wave_scan(__popc(hits[u]), lane), kWave - 1);
            if (lane == 0) matches[p0 + u * kWaves] = sum;
        }
    }
    __syncthreads();
    if (wave != 0) return;
    int before = 0;
    for (int i = 0; i < pieces; i += kWave) {
        const int h = i + lane < pieces ? matches[i + lane] : 0;
        const int s = before + wave_scan(h, lane);
        const uint64_t hit = __ballot(s > among);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            before = __shfl(s - h, l);
            const uint32_t hits = hits_at(i + l);
            const int mine = __popc(hits), first = before + wave_scan(mine, lane) - mine;
            if (among >= first && among < first + mine) {
                uint32_t rest = hits;
                for (int k = first; k < among; ++k) rest &= rest - 1;
                a.tokens[row] = (i + l) * 512 + 8 * lane - skew + __ffs(rest) - 1;
            }
            return;
        }
        before = __shfl(s, kWave - 1);
    }
}

int chunk_of(int rows, int vocab) {
    // about 512 workgroups, of 4096 to 32768 logits
    const int64_t c = (((int64_t)rows * vocab / 512) + 1023) / 1024 * 1024;
    return (int)(c < 4096 ? 4096 : c > kMaxChunk ? kMaxChunk : c);
}

}  // namespace

size_t sample_workspace_bytes(int rows, int vocab) {
    return vocab > 0 && rows > 0 ? (size_t)rows * kBins * sizeof(uint32_t) : 0;
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
    uint32_t* hist = static_cast<uint32_t*>(workspace);
    const size_t words = (size_t)a.rows * kBins / 4;
    const size_t groups = (words + 1023) / 1024;
    sample_clear_kernel<<<dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, stream>>>(
        reinterpret_cast<u32x4_t*>(hist), words);
    const int chunk = chunk_of(a.rows, a.vocab);
    sample_hist_kernel<<<dim3((unsigned)((a.vocab + chunk - 1) / chunk), (unsigned)a.rows), dim3(kThreads), 0, stream>>>(
        a, hist, chunk);
    sample_pick_kernel<<<dim3((unsigned)a.rows), dim3(kThreads), 0, stream>>>(a, hist);
    return hipGetLastError();
}

}  // namespace w4
