// Sums over a CTA's threads, and the pages that requests let go of by one CTA.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {

__device__ __forceinline__ long long warp_sum_to(long long v, int lane) {  // of the lanes up to this one
    for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Sums of v over the threads before this one, and `total` over all of them.  Ends behind a barrier that leaves s_warp
// (33 of them) free once more threads pass the caller's next one.
__device__ __forceinline__ long long block_sum_before(long long v, long long* s_warp, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long sum = warp_sum_to(v, lane);
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        const long long w = lane < warps ? s_warp[lane] : 0, to = warp_sum_to(w, lane);
        s_warp[lane] = to - w;
        if (lane == 31) s_warp[32] = to;
    }
    __syncthreads();
    total = s_warp[32];
    return s_warp[warp] + sum - v;
}

// Last of the n ascending values that is at most x (the first is).
__device__ __forceinline__ int last_at_most(const long long* v, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Divide {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ int operator()(int x) const { return static_cast<int>((static_cast<uint64_t>(x) * mul) >> shift); }
};

// ----------------------------------------------------------------- release
constexpr int kEach = 4, kMostThreads = 1024;  // entries that a thread takes at a time
// Entries of a table that one CTA sees to.
constexpr int64_t kFewEntries = 16384;

// Entries that requests base .. base + n − 1 let go of: how many before each (s_first) and its first (s_want); returns
// their number.  All of a CTA's threads, of which there are at least n.
__device__ __forceinline__ long long scan_given(const KvPagesArgs& a, int base, int n, long long* s_first, int* s_want, long long* s_warp) {
    const int tid = threadIdx.x;
    const long long most = static_cast<long long>(a.width) * a.page_size;
    const Divide pages_of = {a.page_mul, a.page_shift};
    int have = 0, want = 0;
    if (tid < n) {
        const int len = a.lens[base + tid], target = a.target[base + tid];
        if (len >= 0 && target >= 0 && len <= most) {
            have = len > 0 ? pages_of(len - 1) + 1 : 0;
            want = target > 0 ? pages_of(target - 1) + 1 : 0;
        }
    }
    long long total;
    const long long first = block_sum_before(max(have - want, 0), s_warp, total);
    s_first[tid] = first;
    s_want[tid] = want;
    __syncthreads();
    return total;
}

// The entries that requests let go of, in their order, 4096 at a time: each
// counts its page's holders down; of a page that then has none, the last entry
// gives it back.  Which entry that is, the count itself tells: the entries of
// one page that find it at zero leave the largest of their numbers in it,
// below zero, and that one puts the zero back.  One CTA: a step lets go of
// few pages, and a request of 131071 tokens that ends, of 8192.
__device__ __forceinline__ void release_pages(const KvPagesArgs& a) {
    __shared__ long long s_first[kMostThreads], s_warp[33];
    __shared__ int s_want[kMostThreads];
    __shared__ int s_gone[kEach * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    const long long tail = a.range[1];
    const long long tail_at = static_cast<long long>(static_cast<uint64_t>(tail) % static_cast<uint64_t>(a.pages));
    long long given = 0;
    for (int base = 0; base < a.B; base += threads) {
        const int n = min(a.B - base, threads);
        const long long total = scan_given(a, base, n, s_first, s_want, s_warp);
        for (long long r0 = 0; r0 < total; r0 += kEach * threads) {
            int page[kEach];
            bool gone[kEach];
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const long long r = r0 + j * threads + tid;
                page[j] = -1;
                if (r < total) {
                    const int i = last_at_most(s_first, n, r);
                    page[j] = a.table[(base + i) * a.table_stride + s_want[i] + (r - s_first[i])];
                    if (page[j] < 0 || page[j] >= a.pages) {
                        record_status(a.status, kStatusInvalid);
                        page[j] = -1;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (page[j] >= 0 && atomicSub(a.holders + page[j], 1) <= 0) {
                    // Nobody holds the page: more entries than its count says.
                    record_status(a.status, kStatusInvalid);
                    atomicAdd(a.holders + page[j], 1);
                    page[j] = -1;
                }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kEach; ++j) gone[j] = page[j] >= 0 && __ldcg(a.holders + page[j]) == 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (gone[j]) atomicMin(a.holders + page[j], -1 - (j * threads + tid));
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                gone[j] = gone[j] && __ldcg(a.holders + page[j]) == -1 - (j * threads + tid);
                const unsigned votes = __ballot_sync(~0u, gone[j]);
                if (lane == 0) s_gone[j * 32 + warp] = __popc(votes);
            }
            __syncthreads();
            int before[kEach], count = 0;  // (each warp sums for itself)
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int w = lane < warps ? s_gone[j * 32 + lane] : 0;
                const int to = static_cast<int>(warp_sum_to(w, lane));
                before[j] = count + __shfl_sync(~0u, to - w, warp);
                count += __shfl_sync(~0u, to, 31);
            }
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const unsigned votes = __ballot_sync(~0u, gone[j]);
                if (gone[j]) {
                    a.holders[page[j]] = 0;
                    long long at = tail_at + (given + before[j] + __popc(votes & ((1u << lane) - 1))) % a.pages;
                    if (at >= a.pages) at -= a.pages;
                    a.ring[at] = page[j];
                }
            }
            given += count;
            __syncthreads();
        }
        __syncthreads();
    }
    if (tid == 0) a.range_out[1] = tail + given;
}

}  // namespace w4
