// Internal declarations of the paged key-value cache's operators (host side
// and kernel arguments).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_internal.h"

namespace w4 {

struct KvPagesArgs {
    const int32_t* lens;
    const int32_t* target;
    int32_t B;
    int32_t page_size;
    int32_t* ring;
    int64_t pages;
    const int64_t* range;
    int32_t* table;
    int64_t table_stride;
    int32_t width;
    int64_t T;
    int32_t* holders;  // nullptr: every page has one
    long long* given;  // nullptr where the table has few entries; else the number of entries that are let go of,
    unsigned* last;    // a word for each page,
    unsigned* marks;   // and a bit for each entry that is let go of
    int32_t* new_lens;
    int32_t* starts;
    int64_t* slots;
    int32_t* positions;
    int64_t* range_out;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

// bf16 rows [tokens, heads, head_dim], strides in elements.
struct Rows {
    __nv_bfloat16* data;
    int64_t token_stride;
    int64_t head_stride;
};

struct KvAppendArgs {
    Rows q, q_out, k, v;
    int32_t q_heads, kv_heads, head_dim;
    int64_t T;
    const int32_t* positions;
    int64_t axis_stride;
    const float* cos;
    const float* sin;
    int64_t rows;
    int32_t rotary;
    int32_t axes;
    int32_t paired;
    void* k_cache;
    void* v_cache;
    __nv_bfloat16* k_scales;
    __nv_bfloat16* v_scales;
    int64_t pages;
    int64_t page_stride, cache_token_stride, cache_head_stride;
    int32_t page_size;
    const int64_t* slots;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

// Normalisation of the rows that turn: x · (mean(x²) + eps)^−½ · (weight + offset).
struct KvNorm {
    const void* q_weight;  // bf16 or fp32 [head_dim]
    const void* k_weight;
    bool bf16;
    float offset;
    float eps;
    float inv_dim;   // 1 / head_dim
};

struct KvForkArgs {
    const int32_t* lens;
    const int32_t* source;
    const int32_t* keep;
    int32_t B;
    int32_t page_size;
    int32_t* table;
    int64_t table_stride;
    int32_t width;
    int32_t* holders;
    const int32_t* ring;
    int64_t pages;
    const int64_t* range;
    int32_t* new_lens;
    int32_t* copies;  // [3, B]
    int64_t* range_out;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

struct KvCompactArgs {
    const int32_t* lens;
    int32_t B;
    int32_t page_size;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* holders;
    int64_t pages;
    const int64_t* range;
    int32_t* new_table;
    int64_t new_stride;
    int32_t* new_holders;
    int32_t* ring;
    int64_t* range_out;
    int32_t* copies;  // [3, pages / 2]
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

// Pages that the compaction knows of at once, a bit for each in shared memory.
constexpr int64_t kMostCompacted = 1 << 20;
// 16-byte units of a page's keys that a copy can count.
constexpr int64_t kMostCopied = 1 << 28;

struct KvCopyArgs {
    void* k;
    void* v;
    __nv_bfloat16* k_scales;  // nullptr: format 16
    __nv_bfloat16* v_scales;
    int64_t pages;
    int64_t page_stride, token_stride, head_stride;  // bytes
    int32_t page_size, kv_heads, chunks;             // 16-byte chunks of a row
    const int32_t* copies;  // [3, n]
    int32_t n;
    unsigned* status;
};

// Axis of each frequency (rotary ≤ 256), two bits each, eight to a word.
struct Axes {
    uint16_t of[16];
};

struct AttnArgs {
    Rows q, out;
    int32_t B;
    int64_t T;
    int32_t q_heads, kv_heads, head_dim;
    const void* k;
    const void* v;
    const __nv_bfloat16* k_scales;
    const __nv_bfloat16* v_scales;
    int64_t pages;
    int64_t page_stride, token_stride, head_stride;
    int32_t page_size;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* lens;
    const int32_t* starts;  // nullptr: T / B rows each
    float scale;
    int64_t window;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
    // Prefixes that groups of requests share take two passes, each of which leaves its rows' sums behind, and a kernel that
    // joins them: kPrefixes, whose "requests" are the groups (B, table and lens are theirs), and kOwn, over each request's
    // tokens behind its prefix.
    int32_t pass;
    int32_t requests;             // kPrefixes: of the batch
    int32_t groups;               // kOwn
    const int32_t* group_starts;  // [groups + 1], requests of each group
    const int32_t* prefix_lens;   // kOwn: [groups]
    long long most_prefix;        // kOwn: tokens that a row of the prefixes' table holds
    // [T · q_heads]: reference and sum of the weights.  kOwn: what the row is, a RowKind.  kPrefixes: parts that the sums
    // are still in (0: none), and where the first of them is.
    float4* sums;
    float* sum_values;  // [T · q_heads, head_dim]
};
enum : int32_t { kAlone = 0, kPrefixes = 1, kOwn = 2 };
enum RowKind : int32_t { kRowAlone = 0, kRowShared = 1, kRowEmpty = 2 };
// Tokens of a prefix, and rows of a batch that shares them: their sum stays below 2³¹.
constexpr int32_t kMostShared = 1 << 30;

// What a call of attention with shared prefixes is told about its groups.
struct SharedArgs {
    int32_t groups;
    const int32_t* starts;  // [groups + 1]
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* lens;
};

// n / by = (n · mul) >> shift for every n < 2³¹: mul = ⌈2^shift / by⌉ with shift
// = 31 + l and 2^l ≥ by errs by less than n / 2^(31 + l) < 1 / by, and fits 32 bits.
inline void divide_by(int32_t by, uint32_t* mul, int32_t* shift) {
    int l = 0;
    while ((int64_t{1} << l) < by) ++l;
    *shift = 31 + l;
    *mul = static_cast<uint32_t>(((uint64_t{1} << *shift) + static_cast<uint64_t>(by) - 1) / static_cast<uint64_t>(by));
}

// The axis of each of the `frequencies`: the axes' sections in blocks, or cycled.
inline Axes axes_of(int frequencies, int axes, const int32_t sections[4], bool cycled) {
    Axes out = {};
    int used[4] = {0, 0, 0, 0};
    for (int i = 0, turn = 0; i < frequencies; ++i) {
        while (used[turn % axes] == sections[turn % axes]) ++turn;
        const int axis = turn % axes;
        out.of[i >> 3] |= static_cast<uint16_t>(axis << (2 * (i & 7)));
        ++used[axis];
        if (cycled) ++turn;
    }
    return out;
}

// Arguments are already validated by the C ABI layer; the divisors are filled in here.
cudaError_t launch_kv_pages(KvPagesArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_kv_append(KvAppendArgs a, const int32_t sections[4], bool cycled, bool q8, const DeviceInfo& dev,
                             cudaStream_t stream);
cudaError_t launch_kv_append_norm(KvAppendArgs a, const KvNorm& norm, const int32_t sections[4], bool cycled, bool q8,
                                  const DeviceInfo& dev, cudaStream_t stream);
// Adds to the launch of w4_kv_pages the pages that requests let go of (their holders are a.holders).
cudaError_t launch_kv_release(const KvPagesArgs& a, const DeviceInfo& dev, cudaStream_t stream);
size_t kv_held_workspace_bytes(int32_t B, int32_t width, int64_t pages);
cudaError_t launch_kv_fork(KvForkArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_kv_compact(KvCompactArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_kv_copy(const KvCopyArgs& a, const DeviceInfo& dev, cudaStream_t stream);
size_t attn_decode_workspace_bytes(int32_t B, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, bool q8);
cudaError_t launch_attn_decode(AttnArgs a, bool q8, void* workspace, const DeviceInfo& dev,
                               cudaStream_t stream);
size_t attn_shared_workspace_bytes(int32_t B, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, bool q8,
                                   int32_t groups);
cudaError_t launch_attn_shared(AttnArgs a, const SharedArgs& shared, bool q8, void* workspace, const DeviceInfo& dev,
                               cudaStream_t stream);

}  // namespace w4
