// Pages of the cache that several requests hold: letting go of them, requests
// that begin as another's first tokens, pages moved together, and the copies
// of pages that the two ask for.
//
// A page's holders are the table entries that it stands in.  All bookkeeping
// is whole numbers in the order of the requests, so that every result is the
// same in every run.  All but the copies are bound by latency: a chain of
// dependent loads, searches and barriers.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"
#include "w4_kv_release.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 1024;

__global__ void __launch_bounds__(kThreads) kv_release_kernel(KvPagesArgs a) {
    pdl_start();
    release_pages(a);
}

// ------------------------------------------------------- release, many pages
// Entries by all CTAs at once.  Each leaves its number in its page's word if
// that is the largest so far, and then counts the page's holders down: whoever
// finds the last of them finds the number of the last entry there as well, and
// marks that entry.  What is read and written, here, before and after, follows
// the entries that are let go of, not the table's size: the pages' kernel
// leaves their number, clears the words of their pages and a mark for each.
// 600 of 1000 requests of up to 4097 tokens that end: this kernel 9 µs, the
// pages' 11, the next 8, 22 in all, since they overlap.  A step of 1000 requests
// in which none ends: 11 µs, with tables of 260 entries and of 8192.
__global__ void __launch_bounds__(kThreads) kv_let_go_kernel(KvPagesArgs a) {
    __shared__ long long s_first[kThreads], s_warp[33];
    __shared__ int s_want[kThreads];
    pdl_start();
    const int tid = threadIdx.x;
    long long before = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int n = min(a.B - base, kThreads);
        const long long total = scan_given(a, base, n, s_first, s_want, s_warp);
        for (long long r = static_cast<long long>(blockIdx.x) * kThreads + tid; r < total; r += static_cast<long long>(gridDim.x) * kThreads) {
            const int i = last_at_most(s_first, n, r);
            const int page = a.table[(base + i) * a.table_stride + s_want[i] + (r - s_first[i])];
            if (page < 0 || page >= a.pages) {
                record_status(a.status, kStatusInvalid);
                continue;
            }
            atomicMax(a.last + page, static_cast<unsigned>(before + r) + 1);
            __threadfence();
            const int held = atomicSub(a.holders + page, 1);
            if (held <= 0) {
                record_status(a.status, kStatusInvalid);
                atomicAdd(a.holders + page, 1);
            } else if (held == 1) {
                __threadfence();
                const unsigned last = __ldcg(a.last + page) - 1;
                atomicOr(a.marks + (last >> 5), 1u << (last & 31));
            }
        }
        before += total;
        __syncthreads();
    }
}

// The marked entries' pages go to the ring, in the order of the entries.  A CTA
// has one run of the entries: it counts the marks before the run once, and
// carries the count on through the run.
__global__ void __launch_bounds__(kThreads) kv_give_back_kernel(KvPagesArgs a) {
    __shared__ long long s_first[kThreads], s_warp[33];
    __shared__ int s_want[kThreads];
    pdl_start();
    const int tid = threadIdx.x;
    const long long tail = a.range[1], entries = *a.given;
    const long long tail_at = static_cast<long long>(static_cast<uint64_t>(tail) % static_cast<uint64_t>(a.pages));
    int base = 0, m = min(a.B, kThreads);
    long long done = 0, all = scan_given(a, base, m, s_first, s_want, s_warp);  // entries of the requests before `base`, and of those from it on
    // (runs of whole blocks of entries, so that they begin with a word of marks)
    const long long run = ((entries + gridDim.x - 1) / gridDim.x + kThreads - 1) / kThreads * kThreads;
    const long long from = blockIdx.x * run, to = min(from + run, entries);
    if (from >= entries) {
        if (entries == 0 && blockIdx.x == 0 && tid == 0) a.range_out[1] = tail;
        return;
    }
    long long n = 0, given;
#pragma unroll 8
    for (long long w = tid; w < from / 32; w += kThreads) n += __popc(a.marks[w]);
    block_sum_before(n, s_warp, given);
    __syncthreads();
    while (true) {
        const long long end = min(done + all, to);
        for (long long r0 = max(done, from); r0 < end; r0 += kThreads) {
            const long long r = r0 + tid;
            const bool marked = r < end && (a.marks[r >> 5] >> (r & 31) & 1);
            long long count;
            const long long before = block_sum_before(marked, s_warp, count);
            if (marked) {
                const int i = last_at_most(s_first, m, r - done);
                long long at = tail_at + (given + before) % a.pages;
                if (at >= a.pages) at -= a.pages;
                a.ring[at] = a.table[(base + i) * a.table_stride + s_want[i] + (r - done - s_first[i])];
            }
            given += count;
            __syncthreads();
        }
        done += all;
        base += kThreads;
        if (base >= a.B || done >= to) break;
        __syncthreads();
        m = min(a.B - base, kThreads);
        all = scan_given(a, base, m, s_first, s_want, s_warp);
    }
    if (to == entries && tid == 0) a.range_out[1] = tail + given;
}

// -------------------------------------------------------------------- fork
// Every CTA scans all requests, one per thread at a time, and writes every
// gridDim.x-th block of table entries; CTA 0 writes what there is one of for
// each request.  A request that takes over tokens has none of its own, and one
// that gives some has them: the rows that are read and those that are written
// are different ones.  5 µs for eight forks of two requests, 6 for 448 of 64.
__global__ void __launch_bounds__(kThreads) kv_fork_kernel(KvForkArgs a) {
    __shared__ long long s_first[kThreads], s_warp[33], s_need[33];
    __shared__ int s_full[kThreads], s_source[kThreads], s_page[kThreads];
    pdl_start();
    const int tid = threadIdx.x;
    const long long head = a.range[0], tail = a.range[1], most = static_cast<long long>(a.width) * a.page_size;
    const long long free = min(max(tail - head, 0ll), static_cast<long long>(a.pages));
    const long long head_at = static_cast<long long>(static_cast<uint64_t>(head) % static_cast<uint64_t>(a.pages));
    const Divide pages_of = {a.page_mul, a.page_shift};
    long long asked = 0, used = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int n = min(a.B - base, kThreads), b = base + tid;
        int len = 0, source = -1, keep = 0;
        bool valid = false;
        if (tid < n) {
            len = a.lens[b];
            source = a.source[b];
            keep = a.keep[b];
            if (source != -1) {
                valid = source >= 0 && source < a.B && len == 0 && keep >= 0 && keep <= most;
                if (valid) valid = keep <= a.lens[source];
                if (!valid) record_status(a.status, kStatusInvalid);
            }
        }
        const int full = valid ? pages_of(keep) : 0, rest = valid ? keep - full * a.page_size : 0;
        long long total, wanted;
        const long long need = block_sum_before(rest > 0, s_need, wanted) + asked;
        const bool granted = valid && (rest == 0 || need < free);
        int page = -1;
        if (granted && rest > 0) {
            const long long at = head_at + need;
            page = a.ring[at < a.pages ? at : at - a.pages];
        }
        const long long first = block_sum_before(granted ? full + (rest > 0) : 0, s_warp, total);
        s_first[tid] = first;
        s_full[tid] = full;
        s_source[tid] = source;
        s_page[tid] = page;
        if (blockIdx.x == 0 && tid < n) {
            int from = -1;
            if (granted && rest > 0) {
                from = a.table[source * a.table_stride + full];
                if (from < 0 || from >= a.pages || page < 0 || page >= a.pages) {
                    record_status(a.status, kStatusInvalid);
                    from = -1;
                }
            }
            a.new_lens[b] = granted ? keep : len;
            a.copies[b] = from;
            a.copies[static_cast<long long>(a.B) + b] = from < 0 ? -1 : page;
            a.copies[2ll * a.B + b] = from < 0 ? 0 : rest;
        }
        __syncthreads();
        for (long long r = static_cast<long long>(blockIdx.x) * kThreads + tid; r < total; r += static_cast<long long>(gridDim.x) * kThreads) {
            const int i = last_at_most(s_first, n, r), index = static_cast<int>(r - s_first[i]);
            const bool shared = index < s_full[i];
            const int id = shared ? a.table[s_source[i] * a.table_stride + index] : s_page[i];
            a.table[(base + i) * a.table_stride + index] = id;
            if (id >= 0 && id < a.pages) {
                if (shared)
                    atomicAdd(a.holders + id, 1);
                else
                    a.holders[id] = 1;
            } else {
                record_status(a.status, kStatusInvalid);
            }
        }
        used = min(asked + wanted, free);
        asked += wanted;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.range_out[0] = head + used;
        a.range_out[1] = tail;
    }
}

// ----------------------------------------------------------------- compact
// Which pages are in use as bits in shared memory, with the number of them
// before every 128: ranks and the k-th of a kind are then a search there, and
// each CTA finds every answer by itself.  The k-th page in use that lies at or
// past the number of those in use goes to the k-th free one before it.
// Reading all holders again in every CTA costs less than launches that hand
// results on (32 KB for 8000 pages).  5.6 µs for 300 pages, 9.9 for 8000.
constexpr int kBlockPages = 128;

struct Bits {
    const uint32_t* words;
    const int* before;  // pages in use before each 128
    int blocks, live;

    __device__ __forceinline__ bool in_use(int id) const { return words[id >> 5] >> (id & 31) & 1; }
    __device__ __forceinline__ int rank(int id) const {  // pages in use before id
        int r = before[id / kBlockPages];
        for (int w = id / kBlockPages * 4; w < id >> 5; ++w) r += __popc(words[w]);
        return r + __popc(words[id >> 5] & ((1u << (id & 31)) - 1));
    }
    // Id of the k-th page in use (USED) or free page.
    template <bool USED>
    __device__ __forceinline__ int select(int k) const {
        int lo = 0, hi = blocks;
        auto count = [&](int block) { return USED ? before[block] : block * kBlockPages - before[block]; };
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (count(mid) <= k)
                lo = mid;
            else
                hi = mid;
        }
        k -= count(lo);
        int w = lo * 4;
        uint32_t word = USED ? words[w] : ~words[w];
        for (int i = 0; i < 3 && k >= __popc(word); ++i) {
            k -= __popc(word);
            ++w;
            word = USED ? words[w] : ~words[w];
        }
        int bit = 0;
#pragma unroll
        for (int half = 16; half > 0; half >>= 1) {
            const int low = __popc(word >> bit & ((1u << half) - 1));
            if (k >= low) {
                k -= low;
                bit += half;
            }
        }
        return w * 32 + bit;
    }
};

__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(KvCompactArgs a) {
    extern __shared__ uint32_t s_words[];
    __shared__ long long s_warp[33];
    pdl_start();
    const int tid = threadIdx.x, lane = tid & 31;
    const int pages = static_cast<int>(a.pages), blocks = (pages + kBlockPages - 1) / kBlockPages;
    int* const s_before = reinterpret_cast<int*>(s_words + 4 * blocks);
    const int padded = blocks * kBlockPages;
#pragma unroll 4
    for (int id = tid; id < padded; id += kThreads) {
        const unsigned word = __ballot_sync(~0u, id < pages && a.holders[id] > 0);  // (a warp's ids are in or past `padded` together)
        if (lane == 0) s_words[id >> 5] = word;
    }
    __syncthreads();
    long long live = 0;
    for (int base = 0; base < blocks; base += kThreads) {
        const int i = base + tid;
        int n = 0;
        if (i < blocks)
            for (int w = 0; w < 4; ++w) n += __popc(s_words[4 * i + w]);
        long long total;
        const long long before = block_sum_before(n, s_warp, total);
        if (i < blocks) s_before[i] = static_cast<int>(live + before);
        live += total;
        __syncthreads();
    }
    const Bits bits = {s_words, s_before, blocks, static_cast<int>(live)};
    const int used = bits.live, stay = used < pages ? bits.rank(used) : used, moves = used - stay;
    const long long head = a.range[0];
    const long long head_at = static_cast<long long>(static_cast<uint64_t>(head) % static_cast<uint64_t>(a.pages));
    const Divide pages_of = {a.page_mul, a.page_shift};
    const long long step = static_cast<long long>(gridDim.x) * kThreads, me = static_cast<long long>(blockIdx.x) * kThreads + tid;

    const int half = pages / 2;
    for (long long k = me; k < half; k += step) {
        const bool there = k < moves;
        a.copies[k] = there ? bits.select<true>(stay + static_cast<int>(k)) : -1;
        a.copies[half + k] = there ? bits.select<false>(static_cast<int>(k)) : -1;
        a.copies[2ll * half + k] = there ? a.page_size : 0;
    }
    for (long long i = me; i < pages; i += step) {
        const int id = static_cast<int>(i);
        int n = 0;
        if (id < used) n = a.holders[bits.in_use(id) ? id : bits.select<true>(stay + id - bits.rank(id))];
        a.new_holders[id] = n;
        const long long at = head_at + i;
        a.ring[at < pages ? at : at - pages] = i < pages - used ? used + id : -1;
    }
    const long long most = static_cast<long long>(a.width) * a.page_size, entries = static_cast<long long>(a.B) * a.width;
    for (long long i = me; i < entries; i += step) {
        const int b = static_cast<int>(i / a.width), c = static_cast<int>(i - static_cast<long long>(b) * a.width);
        const int len = a.lens[b];
        if ((len < 0 || len > most) && c == 0) record_status(a.status, kStatusInvalid);
        const int have = len > 0 && len <= most ? pages_of(len - 1) + 1 : 0;
        int id = a.table[b * a.table_stride + c];
        if (c < have) {
            if (id < 0 || id >= pages || !bits.in_use(id))
                record_status(a.status, kStatusInvalid);
            else if (id >= used)
                id = bits.select<false>(bits.rank(id) - stay);
        }
        a.new_table[b * a.new_stride + c] = id;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.range_out[0] = head;
        a.range_out[1] = head + pages - used;
    }
}

// -------------------------------------------------------------------- copy
constexpr int kCopyThreads = 256, kCopyUnits = 4, kList = 2048;
constexpr int kPiece = kCopyThreads * kCopyUnits;  // 16-byte units that a CTA copies at a time

struct CopyShape {
    KvCopyArgs a;
    bool heads_inside;   // a token's heads lie closer than a head's tokens
    uint32_t chunk_mul, inner_mul;
    int chunk_shift, inner_shift;
    int pieces;          // of keys or values of a whole page
    uint32_t piece_mul;  // divide_by(pieces of a copy)
    int piece_shift;
};

// A CTA first lists the copies that there are (the others are −1), then takes
// every gridDim.x-th piece of 16 KB of them.  Units in the order of memory; a
// thread asks for all of a piece's before it writes the first.  Bound by HBM: 2000
// pages of 64 KB 44 µs, 0.88 of the rate of a plain copy, one copy for eight
// forks 3.4, by latency.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ CopyShape s) {
    __shared__ int s_from[kList], s_to[kList], s_tokens[kList];
    __shared__ int s_warp[kCopyThreads / 32];
    pdl_start();
    const KvCopyArgs& a = s.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Divide over_chunks = {s.chunk_mul, s.chunk_shift}, over_inner = {s.inner_mul, s.inner_shift}, over_pieces = {s.piece_mul, s.piece_shift};
    const bool q8 = a.k_scales != nullptr;
    const int per_copy = 2 * s.pieces + (q8 ? 1 : 0);
    long long turn = blockIdx.x;  // of the next piece that is this CTA's, from the list's first on
    for (int base = 0; base < a.n; base += kList) {
        int count = 0;
        __syncthreads();  // the list before has been used
        constexpr int kMine = kList / kCopyThreads;
        int from[kMine], to[kMine], tokens[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int i = base + j * kCopyThreads + tid;
            from[j] = i < a.n ? a.copies[i] : -1;
            to[j] = i < a.n ? a.copies[static_cast<long long>(a.n) + i] : -1;
            tokens[j] = i < a.n ? a.copies[2ll * a.n + i] : 0;
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            bool there = from[j] != -1 || to[j] != -1;
            if (there && (from[j] < 0 || from[j] >= a.pages || to[j] < 0 || to[j] >= a.pages || tokens[j] < 0 || tokens[j] > a.page_size)) {
                record_status(a.status, kStatusInvalid);
                there = false;
            }
            there = there && tokens[j] > 0 && from[j] != to[j];
            const unsigned votes = __ballot_sync(~0u, there);
            if (lane == 0) s_warp[warp] = __popc(votes);
            __syncthreads();
            int at = count + __popc(votes & ((1u << lane) - 1));
            for (int w = 0; w < kCopyThreads / 32; ++w) {
                if (w < warp) at += s_warp[w];
                count += s_warp[w];
            }
            if (there) {
                s_from[at] = from[j];
                s_to[at] = to[j];
                s_tokens[at] = tokens[j];
            }
            __syncthreads();
        }
        const long long all = static_cast<long long>(count) * per_copy;
        for (; turn < all; turn += gridDim.x) {
            const int j = over_pieces(static_cast<int>(turn)), part = static_cast<int>(turn) - j * per_copy;
            const long long src = s_from[j], dst = s_to[j];
            const int n = s_tokens[j];
            if (part < 2 * s.pieces) {
                const bool key = part < s.pieces;
                uint8_t* const memory = static_cast<uint8_t*>(key ? a.k : a.v);
                const int u0 = (key ? part : part - s.pieces) * kPiece + tid, units = n * a.kv_heads * a.chunks;
                uint4 x[kCopyUnits];
                long long off[kCopyUnits];
#pragma unroll
                for (int i = 0; i < kCopyUnits; ++i) {
                    const int u = u0 + i * kCopyThreads;
                    off[i] = -1;
                    if (u >= units) continue;
                    const int row = over_chunks(u), c = u - row * a.chunks;
                    int token, head;
                    if (s.heads_inside) {
                        token = over_inner(row);
                        head = row - token * a.kv_heads;
                    } else {
                        head = row / n;
                        token = row - head * n;
                    }
                    off[i] = token * a.token_stride + head * a.head_stride + c * 16;
                    x[i] = ld_stream(memory + src * a.page_stride + off[i]);
                }
#pragma unroll
                for (int i = 0; i < kCopyUnits; ++i)
                    if (off[i] >= 0) *reinterpret_cast<uint4*>(memory + dst * a.page_stride + off[i]) = x[i];
            } else {
                const long long page = static_cast<long long>(a.kv_heads) * a.page_size;
                for (int u = tid; u < n * a.kv_heads; u += kCopyThreads) {
                    const int head = u / n;
                    const long long at = static_cast<long long>(head) * a.page_size + u - head * n;
                    const __nv_bfloat16 k = a.k_scales[src * page + at], v = a.v_scales[src * page + at];
                    a.k_scales[dst * page + at] = k;
                    a.v_scales[dst * page + at] = v;
                }
            }
        }
        turn -= all;
    }
}

}  // namespace

cudaError_t launch_kv_release(const KvPagesArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.B) * a.width;
    if (!a.last) {
        return launch_pass(kv_release_kernel, 1, kThreads, 0, stream, true, a);
    }
    auto ctas = [&](int64_t each) { return static_cast<int>(std::min<int64_t>((entries + each - 1) / each, dev.sm_count)); };
    const cudaError_t err = launch_pass(kv_let_go_kernel, ctas(kThreads), kThreads, 0, stream, true, a);
    return err != cudaSuccess ? err : launch_pass(kv_give_back_kernel, ctas(kThreads), kThreads, 0, stream, true, a);
}

// The number of entries that are let go of, a word for each page and a bit for each entry of the table, where more pages may
// go back than one CTA should see to.
size_t kv_held_workspace_bytes(int32_t B, int32_t width, int64_t pages) {
    const int64_t entries = static_cast<int64_t>(B) * width;
    return entries <= kFewEntries ? 0 : sizeof(long long) + static_cast<size_t>(pages + (entries + 31) / 32) * 4;
}

cudaError_t launch_kv_fork(KvForkArgs a, const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    const int64_t blocks = (static_cast<int64_t>(a.B) * a.width + 4 * kThreads - 1) / (4 * kThreads);
    return launch_pass(kv_fork_kernel, static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, dev.sm_count))), kThreads, 0, stream, true, a);
}

cudaError_t launch_kv_compact(KvCompactArgs a, const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    const int64_t blocks = (a.pages + kBlockPages - 1) / kBlockPages;
    const size_t smem = static_cast<size_t>(blocks) * 5 * 4;
    if (smem > 40 * 1024) {  // (one value for every call: another thread's call may set it in between)
        const cudaError_t err = cudaFuncSetAttribute(kv_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostCompacted / kBlockPages * 5 * 4);
        if (err != cudaSuccess) return err;
    }
    const int64_t work = std::max<int64_t>(a.pages, static_cast<int64_t>(a.B) * a.width);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((work + kThreads - 1) / kThreads, dev.sm_count));
    return launch_pass(kv_compact_kernel, static_cast<int>(grid), kThreads, smem, stream, true, a);
}

cudaError_t launch_kv_copy(const KvCopyArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    CopyShape s = {};
    s.a = a;
    s.heads_inside = a.kv_heads > 1 && a.head_stride < a.token_stride;
    divide_by(a.chunks, &s.chunk_mul, &s.chunk_shift);
    divide_by(a.kv_heads, &s.inner_mul, &s.inner_shift);
    const int64_t units = static_cast<int64_t>(a.page_size) * a.kv_heads * a.chunks;
    s.pieces = static_cast<int>((units + kPiece - 1) / kPiece);
    const int per_copy = 2 * s.pieces + (a.k_scales ? 1 : 0);
    divide_by(per_copy, &s.piece_mul, &s.piece_shift);
    const int64_t most = static_cast<int64_t>(a.n) * per_copy;
    const int grid = static_cast<int>(std::min<int64_t>(most, 8 * dev.sm_count));
    return launch_pass(kv_copy_kernel, grid, kCopyThreads, 0, stream, true, s);
}

}  // namespace w4
