// Tokens sorted by expert.
//
//   row(i) = start[e] + #{i' < i : expert(i') = e},  start[e] = sum over e' < e of min(count(e'), capacity)
//
// A counting sort: nothing is compared but a workgroup's own few choices.  A
// workgroup takes a few tokens, finds the rows of their choices and copies the
// tokens there, reading each once.  What it needs of all other choices are two
// numbers an expert, how many there are and how many come before; it counts
// them itself in LDS where they are few, which takes one launch.  Else a first
// launch counts them per chunk of choices, and a workgroup sums that table, or where
// it is large a second launch has summed it over the chunks.  The counts are whole
// numbers, so LDS atomics do not decide any order.
// Measured: 8191 tokens of 6 choices, 64 experts, rows of 4096: 78 us, 5.3 TB/s; 64 tokens
// 6.1 us, one launch.
// Short rows leave lanes of a workgroup idle: 32768 tokens of 8 choices, rows of 256, 53 us,
// 42 of them the copy's launch (32 lanes of 256, two tokens a workgroup), 10 the sums' over the
// chunks, one behind the other, 5 the count's; the bytes alone take 29.
#include "block.hpp"
#include "block_device.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxE = W4_MOE_SORT_MAX_EXPERTS;
constexpr int kOwn = 64;      // choices of a workgroup, at most
constexpr int kAlone = 4096;  // choices that every workgroup counts itself
// Counts of a table that every workgroup sums, at most, its chunks of kLongChunk choices;
// larger ones are summed once, of kChunk choices or more.  us of both, the first
// first: 683 tokens of 6 choices, 64 experts, rows of 4096 (320 counts) 11.9 and 13.6; 8191
// (48 chunks) 87 either way; 4096 of 8, 256 experts, 2048 (8192) 43 and 33; 32768 of 8, 64
// experts, 256 (16384) 191 and 50.
constexpr int kTable = 4096;
constexpr int kLongChunk = 1024, kChunk = 256;
constexpr int kMaxChunks = 2048;  // of a table summed once, at most (2^21 counts)
constexpr int kScanExperts = 16;  // of a workgroup that sums over the chunks

struct SortArgs {
    w4_moe_sort_args a;
    int n;         // choices
    int per;       // tokens of a workgroup
    int chunk;     // choices of a chunk; 0: no table
    int chunks;
    bool summed;      // moe_scan_kernel runs
    int32_t* totals;  // [num_experts], if summed
    int32_t* counts;  // [chunks][num_experts]: of a chunk; if summed, of all chunks before it
};

__global__ __launch_bounds__(kThreads) void moe_count_kernel(SortArgs k) {
    __shared__ int hist[kMaxE];
    const int E = k.a.num_experts;
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * k.chunk, end = min(first + k.chunk, k.n);
    for (int i = first + threadIdx.x; i < end; i += kThreads) {
        const int e = k.a.experts[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) k.counts[blockIdx.x * E + e] = hist[e];
}

// A column of the table a lane of sixteen, its chunks in sixteen runs.
__global__ __launch_bounds__(kThreads) void moe_scan_kernel(SortArgs k) {
    constexpr int kRuns = kThreads / kScanExperts, kAtOnce = 8;
    __shared__ int sums[kRuns][kScanExperts];
    const int E = k.a.num_experts, lane = threadIdx.x % kScanExperts, run = threadIdx.x / kScanExperts;
    const int e = blockIdx.x * kScanExperts + lane, per = (k.chunks + kRuns - 1) / kRuns;
    const int first = run * per, end = e < E ? min(first + per, k.chunks) : 0;
    const auto over = [&](auto f) {
        for (int c0 = first; c0 < end; c0 += kAtOnce) {
            int x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) x[i] = c0 + i < end ? k.counts[(c0 + i) * E + e] : 0;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (c0 + i < end) f(c0 + i, x[i]);
        }
    };
    int sum = 0;
    over([&](int, int x) { sum += x; });
    sums[run][lane] = sum;
    __syncthreads();
    sum = 0;
    for (int r = 0; r < run; ++r) sum += sums[r][lane];
    if (e < E && run == kRuns - 1) k.totals[e] = sum + sums[run][lane];
    over([&](int c, int x) {
        k.counts[c * E + e] = sum;
        sum += x;
    });
}

template <bool kApart>
__global__ __launch_bounds__(kThreads) void moe_sort_kernel(SortArgs k) {
    __shared__ int total[kMaxE + 1], before[kMaxE], sums[kThreads / kWave], rows[kOwn];
    const w4_moe_sort_args& a = k.a;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, E = a.num_experts;
    const int t0 = blockIdx.x * k.per, t1 = min(t0 + k.per, a.T);
    const int i0 = t0 * a.top, i1 = t1 * a.top;
    int from = 0, to = k.n;  // the choices counted one by one
    if (k.chunk) {
        const int mine = i0 / k.chunk;
        from = mine * k.chunk;
        to = i0;
        for (int e = tid; e < E; e += kThreads) {
            total[e] = k.summed ? k.totals[e] : 0;
            before[e] = k.summed ? k.counts[mine * E + e] : 0;
        }
        if (!k.summed) {
            __syncthreads();
            for (int i = tid; i < k.chunks * E; i += kThreads) {
                const int c = k.counts[i], e = i % E;
                if (c == 0) continue;
                atomicAdd(&total[e], c);
                if (i / E < mine) atomicAdd(&before[e], c);
            }
        }
    } else {
        for (int e = tid; e < E; e += kThreads) total[e] = before[e] = 0;
    }
    __syncthreads();
    for (int i = from + tid; i < to; i += kThreads) {
        const int e = a.experts[i];
        if ((unsigned)e >= (unsigned)E) continue;
        if (!k.chunk) atomicAdd(&total[e], 1);
        if (i < i0) atomicAdd(&before[e], 1);
    }
    __syncthreads();

    // first rows: a scan over the experts, kMaxE / kThreads of them a thread
    constexpr int kPer = kMaxE / kThreads;
    int mine[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * kPer + j;
        const int c = e < E ? total[e] : 0;
        mine[j] = a.capacity > 0 ? min(c, a.capacity) : c;
        sum += mine[j];
    }
    int upto = sum;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int x = __shfl_up(upto, off);
        if (lane >= off) upto += x;
    }
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int start = upto - sum;
    for (int w = 0; w < wave; ++w) start += sums[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * kPer + j;
        if (e <= E) total[e] = start;
        start += mine[j];
    }
    if (tid == kThreads - 1 && E == kMaxE) total[E] = start;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += kThreads) a.row_start[e] = total[e];

    // the workgroup's own choices, a lane each
    if (tid < kOwn) {
        const int i = i0 + tid;
        const int e = i < i1 ? a.experts[i] : -1;
        int rank = 0;
        for (int l = 0; l < i1 - i0; ++l) rank += l < lane && __builtin_amdgcn_readlane(e, l) == e;
        int row = -1;
        if ((unsigned)e < (unsigned)E) {
            rank += before[e];
            if (a.capacity == 0 || rank < a.capacity) row = total[e] + rank;
        }
        rows[tid] = row;
        if (i < i1) {
            a.row_of[i] = row;
            if (a.source) {
                if (row >= 0) a.source[row] = i;
                if (i >= total[E]) a.source[i] = -1;  // no choice has this row
            }
        }
    }
    if (!a.x) return;
    __syncthreads();
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    uint16_t* out = static_cast<uint16_t*>(a.rows);
    const int pieces = a.D / 8;
    for (int t = t0; t < t1; ++t)
        for (int p = tid; p < pieces; p += kThreads) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + (int64_t)t * a.x_stride + 8 * p);
            for (int j = 0; j < a.top; ++j) {
                const int row = rows[(t - t0) * a.top + j];
                if ((unsigned)row < (unsigned)a.R) put<kApart>(reinterpret_cast<u32x4_t*>(out + (int64_t)row * a.rows_stride + 8 * p), v);
            }
        }
}

SortArgs cut_of(int T, int top, int E) {
    SortArgs k = {};
    k.n = T * top;
    // 16 choices a workgroup: 8191 tokens of 6 choices, rows of 4096: 74 us, of 64 80, of 6 74
    k.per = k.n <= kAlone || top > kOwn / 4 ? 1 : kOwn / 4 / top;
    if (k.n > kAlone) {
        k.summed = (int64_t)((k.n + kLongChunk - 1) / kLongChunk) * E > kTable;
        k.chunk = k.summed ? (k.n + kMaxChunks - 1) / kMaxChunks : kLongChunk;
        if (k.chunk < kChunk) k.chunk = kChunk;
        k.chunks = (k.n + k.chunk - 1) / k.chunk;
    }
    return k;
}

}  // namespace

size_t moe_sort_workspace_bytes(int T, int top, int num_experts) {
    const SortArgs k = cut_of(T, top, num_experts);
    return (size_t)(k.chunks + k.summed) * num_experts * sizeof(int32_t);
}

hipError_t launch_moe_sort(const w4_moe_sort_args& a, void* workspace, hipStream_t stream) {
    SortArgs k = cut_of(a.T, a.top, a.num_experts);
    k.a = a;
    if (k.chunk) {
        k.totals = static_cast<int32_t*>(workspace);
        k.counts = k.totals + (k.summed ? a.num_experts : 0);
        moe_count_kernel<<<dim3((unsigned)k.chunks), dim3(kThreads), 0, stream>>>(k);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        if (k.summed) {
            moe_scan_kernel<<<dim3((unsigned)((a.num_experts + kScanExperts - 1) / kScanExperts)), dim3(kThreads), 0, stream>>>(k);
            err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
        if (!a.x) k.per = kOwn / a.top;
    }
    const int groups = a.T > 0 ? (a.T + k.per - 1) / k.per : 1;
    if ((int64_t)k.n * a.D >= kRowsApart) {
        moe_sort_kernel<true><<<dim3((unsigned)groups), dim3(kThreads), 0, stream>>>(k);
    } else {
        moe_sort_kernel<false><<<dim3((unsigned)groups), dim3(kThreads), 0, stream>>>(k);
    }
    return hipGetLastError();
}

}  // namespace w4
