// Block tables, slot map, positions and row ranges of one step, in one launch.
//
// Every workgroup scans the B requests' lengths itself (at most 4096, 32 KB
// from the L2) and then fills its share of the token rows and of the newly
// needed pages; so nothing is handed between workgroups, which would cost a
// second launch.  A page that this step gives out is found from its rank by
// whoever needs it, never read back from the table: entries being written
// are read by nobody, and the result does not depend on any order.
// What bounds it is latency: a launch, the lengths' loads, a scan, then one
// binary search in LDS and one dependent load per row (4.8 us for 256 requests
// of one token, 7 for 1000 of up to 300).
#include "kv4.hpp"
#include "w4_device.hpp"

namespace w4 {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxB = W4_KV4_PLAN_MAX_BATCH;
constexpr int kPer = kMaxB / kThreads;  // requests a thread scans at most
constexpr int kRowsPer = 1024;          // rows, and page ranks, a workgroup fills

struct Lens {
    int held, pages, cached, total;
};

__device__ __forceinline__ Lens lens_of(const PlanArgs& a, int b) {
    const int64_t c = max(a.cached[b], 0), n = max(a.fresh[b], 0), lim = 0x7FFFFFFF;
    const int64_t t = min(c + n, lim), up = (1 << a.shift) - 1, w = a.width;
    return {(int)min((c + up) >> a.shift, w), (int)min((t + up) >> a.shift, w), (int)c, (int)t};
}

// The last index i in [0, n) with v[i] <= x (v rising, v[0] <= x).
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void kv4_plan_kernel(PlanArgs a) {
    __shared__ int start[kMaxB + 1];  // first row of each request
    __shared__ int rank[kMaxB + 1];   // first new page of each request
    __shared__ int64_t sums[2][kThreads / kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int per = (a.B + kThreads - 1) / kThreads;  // <= kPer, the same for every thread

    int64_t rows[kPer], need[kPer], rsum = 0, nsum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        rows[i] = need[i] = 0;
        if (i < per && b < a.B) {
            const Lens l = lens_of(a, b);
            rows[i] = max(a.fresh[b], 0);
            need[i] = l.pages - l.held;
        }
        rsum += rows[i];
        nsum += need[i];
    }
    int64_t rscan = rsum, nscan = nsum;  // inclusive over the wave
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int64_t r = __shfl_up(rscan, off), n = __shfl_up(nscan, off);
        if (lane >= off) {
            rscan += r;
            nscan += n;
        }
    }
    if (lane == kWave - 1) {
        sums[0][wave] = rscan;
        sums[1][wave] = nscan;
    }
    __syncthreads();
    int64_t rat = rscan - rsum, nat = nscan - nsum;
    for (int w = 0; w < wave; ++w) {
        rat += sums[0][w];
        nat += sums[1][w];
    }
    const int64_t lim = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        if (i < per && b < a.B) {
            start[b] = (int)min(rat, lim);
            rank[b] = (int)nat;
            rat += rows[i];
            nat += need[i];
            if (b == a.B - 1) {
                start[a.B] = (int)min(rat, lim);
                rank[a.B] = (int)nat;
            }
        }
    }
    if (a.B == 0 && tid == 0) start[0] = rank[0] = 0;
    __syncthreads();

    const int total = start[a.B], needed = rank[a.B];
    const int left = min(max(a.free_count[0], 0), a.capacity);
    const auto given = [&](int r) { return left - 1 - r >= 0 ? a.free_blocks[left - 1 - r] : -1; };

    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += kThreads) {
            a.q_start[b] = start[b];
            if (b < a.B) a.kv_lens[b] = lens_of(a, b).total;
        }
        if (tid == 0) {
            a.counts[0] = max(left - needed, 0);
            a.counts[1] = max(needed - left, 0);
        }
    }
    // rows
    for (int64_t r0 = (int64_t)blockIdx.x * kRowsPer; r0 < a.rows; r0 += (int64_t)gridDim.x * kRowsPer) {
        const int end = (int)min(r0 + kRowsPer, (int64_t)a.rows) - (int)r0;
        for (int i = tid; i < end; i += kThreads) {
            const int r = (int)r0 + i;
            int pos = -1, slot = -1;
            if (r < total) {
                const int b = last_at_most(start, a.B, r);
                const Lens l = lens_of(a, b);
                pos = (int)min((int64_t)l.cached + (r - start[b]), lim);
                const int p = pos >> a.shift;
                if (p < a.width) {
                    const int page = p < l.held ? a.table[(size_t)b * a.width + p] : given(rank[b] + p - l.held);
                    const int64_t at = ((int64_t)page << a.shift) + (pos & ((1 << a.shift) - 1));
                    if (page >= 0 && at <= lim) slot = (int)at;
                }
            }
            a.positions[r] = pos;
            a.slots[r] = slot;
        }
    }
    // new pages, by rank
    for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < needed; r += (int64_t)gridDim.x * kThreads) {
        const int b = last_at_most(rank, a.B, (int)r);
        const Lens l = lens_of(a, b);
        a.table[(size_t)b * a.width + l.held + ((int)r - rank[b])] = given((int)r);
    }
}

}  // namespace

hipError_t launch_kv4_plan(const PlanArgs& a, hipStream_t stream) {
    // Rows decide the grid; the pages' loop strides over whatever it is.
    const int groups = a.rows / kRowsPer + 1;
    kv4_plan_kernel<<<dim3(groups < 1024 ? groups : 1024), dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4
