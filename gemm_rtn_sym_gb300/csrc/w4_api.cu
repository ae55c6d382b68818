// C ABI of the library (declared in include/w4.h): argument checks, kernel
// choice, launches and the per-device status word of the bounded waits.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <vector>

#include <cuda_runtime.h>

#include "w4.h"
#include "w4_device.cuh"
#include "w4_internal.h"
#include "w4_kv.h"

namespace w4 {
namespace {

// One status word per device (written by kernels whose bounded waits ran out).
__device__ unsigned g_status_word = 0;

constexpr int kMaxDevices = 64;
DeviceInfo g_info[kMaxDevices];
bool g_info_ready[kMaxDevices];
std::mutex g_info_mutex;

// Smallest M that goes to the tensor-core kernel: under W4_PATH_AUTO for one
// matrix, and in grouped plans.  Measured crossovers on the 4B-class stack,
// the 27B-class layer and the 2560×9216 matrix (M = 17, 20, 24, 28, 32): the
// small-M kernel is faster up to M = 24 (three token tiles per pass; e.g.
// grouped stack 621 against 665 µs at M = 24), the tensor-core tile from
// M = 28 (grouped stack 665 against 815 µs; 2560×9216 alone 10.5 against
// 11.5 µs), in one launch per matrix and in grouped launches alike.
constexpr int64_t kTensorMinM = 25;
constexpr int64_t kGroupedTensorMinM = 25;

// Largest N or K of the GPTQ calls: their fp64 tile products run 64-row tiles
// on a grid at most 65535 tiles high.
constexpr int64_t kGptqMaxDim = int64_t{65535} * 64;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return na != 0 && nb != 0 && pa < pb + nb && pb < pa + na;
}

int check_sizes(int64_t N, int64_t K) {
    if (N < 0 || K < 0) return W4_ERR_INVALID_ARG;
    if (K % 128 != 0) return W4_ERR_UNSUPPORTED;
    if (N > 0 && K > (int64_t{1} << 62) / N) return W4_ERR_INVALID_ARG;
    return W4_OK;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }

bool valid_group(int32_t group) { return group == 32 || group == 64 || group == 128; }

}  // namespace

const DeviceInfo* device_info(cudaError_t* err) {
    int dev = 0;
    *err = cudaGetDevice(&dev);
    if (*err != cudaSuccess) return nullptr;
    if (dev < 0 || dev >= kMaxDevices) {
        *err = cudaErrorInvalidDevice;
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_info_mutex);
    if (!g_info_ready[dev]) {
        DeviceInfo info;
        if ((*err = cudaDeviceGetAttribute(&info.sm_count, cudaDevAttrMultiProcessorCount, dev)) ||
            (*err = cudaDeviceGetAttribute(&info.cc_major, cudaDevAttrComputeCapabilityMajor, dev)) ||
            (*err = cudaDeviceGetAttribute(&info.cc_minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
            (*err = cudaDeviceGetAttribute(&info.max_smem_optin,
                                           cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) ||
            (*err = cudaGetSymbolAddress(reinterpret_cast<void**>(&info.status), g_status_word)))
            return nullptr;
        g_info[dev] = info;
        g_info_ready[dev] = true;
    }
    *err = cudaSuccess;
    return &g_info[dev];
}

}  // namespace w4

using namespace w4;

extern "C" {

size_t w4_packed_bytes(int64_t N, int64_t K) {
    if (check_sizes(N, K) != W4_OK) return 0;
    return static_cast<size_t>(N) * static_cast<size_t>(K) / 2;
}

size_t w4_scales_bytes(int64_t N, int64_t K, int32_t group) {
    if (!valid_group(group) || check_sizes(N, K) != W4_OK) return 0;
    return static_cast<size_t>(N) * static_cast<size_t>(K / group) * 2;
}

size_t w4_zeros_bytes(int64_t N, int64_t K, int32_t group) {
    if (!valid_group(group) || check_sizes(N, K) != W4_OK) return 0;
    return static_cast<size_t>(N) * static_cast<size_t>(K / group);
}

}  // extern "C"

namespace {

// Symmetric RTN (asym false), asymmetric RTN (zeros written), or symmetric
// RTN of the channel-scaled weights (scaled, group 128 only).
int quantize_impl(const void* W, int64_t N, int64_t K, int32_t group, const float* channel_scales,
                  bool scaled, bool asym, void* packed, void* scales, void* zeros, void* stream) {
    if (!valid_group(group) || (scaled && group != 128)) return W4_ERR_UNSUPPORTED;
    if (const int s = check_sizes(N, K)) return s;
    if (N == 0 || K == 0) return W4_OK;
    if (!W || !packed || !scales || (scaled && !channel_scales) || (asym && !zeros)) return W4_ERR_INVALID_ARG;
    if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales, 2) ||
        (scaled && !aligned(channel_scales, 16)))
        return W4_ERR_MISALIGNED;
    const size_t wb = static_cast<size_t>(N * K) * 2, pb = w4_packed_bytes(N, K),
                 sb = w4_scales_bytes(N, K, group), cb = scaled ? static_cast<size_t>(K) * 4 : 0,
                 zb = asym ? w4_zeros_bytes(N, K, group) : 0;
    if (overlaps(W, wb, packed, pb) || overlaps(W, wb, scales, sb) || overlaps(packed, pb, scales, sb) ||
        overlaps(channel_scales, cb, packed, pb) || overlaps(channel_scales, cb, scales, sb) ||
        overlaps(zeros, zb, W, wb) || overlaps(zeros, zb, packed, pb) || overlaps(zeros, zb, scales, sb))
        return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    return to_status(launch_quantize(W, N, K, group, packed, scales, asym ? zeros : nullptr,
                                     scaled ? channel_scales : nullptr, *dev, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int w4_quantize_rtn(const void* W, int64_t N, int64_t K, int32_t group, void* packed, void* scales,
                    void* stream) {
    return quantize_impl(W, N, K, group, nullptr, false, false, packed, scales, nullptr, stream);
}

int w4_quantize_rtn_asym(const void* W, int64_t N, int64_t K, int32_t group, void* packed, void* scales,
                         void* zeros, void* stream) {
    return quantize_impl(W, N, K, group, nullptr, false, true, packed, scales, zeros, stream);
}

int w4_quantize_rtn_scaled(const void* W, int64_t N, int64_t K, int32_t group, const float* s, void* packed,
                           void* scales, void* stream) {
    return quantize_impl(W, N, K, group, s, true, false, packed, scales, nullptr, stream);
}

size_t w4_gptq_factor_workspace_bytes(int64_t K) {
    if (check_sizes(1, K) != W4_OK || K == 0 || K > kGptqMaxDim) return 0;
    return gptq_factor_workspace_bytes(K);
}

int w4_gptq_factor(const float* H, int64_t K, double damp, double* U, void* workspace, size_t workspace_bytes,
                   void* stream) {
    if (const int s = check_sizes(1, K)) return s;
    if (K == 0) return W4_OK;
    if (K > kGptqMaxDim || static_cast<double>(K) * K > 1e18) return W4_ERR_UNSUPPORTED;
    if (!(damp >= 0.0) || damp > 1e30) return W4_ERR_INVALID_ARG;
    if (!H || !U || !workspace) return W4_ERR_INVALID_ARG;
    if (!aligned(H, 4) || !aligned(U, 8) || !aligned(workspace, 256)) return W4_ERR_MISALIGNED;
    const size_t hb = static_cast<size_t>(K) * K * 4, ub = static_cast<size_t>(K) * K * 8;
    if (overlaps(H, hb, U, ub) || overlaps(workspace, workspace_bytes, H, hb) ||
        overlaps(workspace, workspace_bytes, U, ub))
        return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    switch (launch_gptq_factor(H, K, damp, U, workspace, workspace_bytes, *dev, static_cast<cudaStream_t>(stream))) {
        case 0: return W4_OK;
        case 2: return W4_ERR_INVALID_ARG;
        default: return W4_ERR_CUDA;
    }
}

size_t w4_gptq_workspace_bytes(int64_t N, int64_t K) {
    if (check_sizes(N, K) != W4_OK || N == 0 || K == 0 || N > INT32_MAX || K > INT32_MAX) return 0;
    if (static_cast<double>(N) * K > 1e18) return 0;
    return gptq_workspace_bytes(N, K);
}

int w4_gptq_quantize(const void* W, int64_t N, int64_t K, int32_t group, const double* U, void* packed,
                     void* scales, void* workspace, size_t workspace_bytes, void* stream) {
    if (!valid_group(group)) return W4_ERR_UNSUPPORTED;
    if (const int s = check_sizes(N, K)) return s;
    if (N == 0 || K == 0) return W4_OK;
    if (N > kGptqMaxDim || K > kGptqMaxDim) return W4_ERR_UNSUPPORTED;
    if (!W || !U || !packed || !scales || !workspace) return W4_ERR_INVALID_ARG;
    if (!aligned(W, 16) || !aligned(U, 8) || !aligned(packed, 16) || !aligned(scales, 2) || !aligned(workspace, 256))
        return W4_ERR_MISALIGNED;
    const size_t wb = static_cast<size_t>(N * K) * 2, ub = static_cast<size_t>(K) * K * 8,
                 pb = w4_packed_bytes(N, K), sb = w4_scales_bytes(N, K, group);
    const void* outs[2] = {packed, scales};
    const size_t ob[2] = {pb, sb};
    for (int i = 0; i < 2; ++i)
        if (overlaps(outs[i], ob[i], W, wb) || overlaps(outs[i], ob[i], U, ub) ||
            overlaps(outs[i], ob[i], workspace, workspace_bytes))
            return W4_ERR_INVALID_ARG;
    if (overlaps(packed, pb, scales, sb) || overlaps(workspace, workspace_bytes, W, wb) ||
        overlaps(workspace, workspace_bytes, U, ub))
        return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    switch (launch_gptq(W, N, K, group, U, packed, scales, workspace, workspace_bytes, *dev,
                        static_cast<cudaStream_t>(stream))) {
        case 0: return W4_OK;
        case 2: return W4_ERR_INVALID_ARG;
        default: return W4_ERR_CUDA;
    }
}

int w4_scale_activations(const void* x, int64_t M, int64_t K, const float* s, void* x_out, void* stream) {
    if (M < 0) return W4_ERR_INVALID_ARG;
    if (const int st = check_sizes(M, K)) return st;
    if (M == 0 || K == 0) return W4_OK;
    if (!x || !s || !x_out) return W4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(s, 16) || !aligned(x_out, 16)) return W4_ERR_MISALIGNED;
    const size_t xb = static_cast<size_t>(M * K) * 2, cb = static_cast<size_t>(K) * 4;
    if ((x != x_out && overlaps(x, xb, x_out, xb)) || overlaps(s, cb, x_out, xb)) return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    return to_status(launch_scale_activations(x, M, K, s, x_out, *dev, static_cast<cudaStream_t>(stream)));
}

int w4_gemm_path_for(int64_t M, int64_t N, int64_t K) {
    if (M < 0) return -W4_ERR_INVALID_ARG;
    if (const int s = check_sizes(N, K)) return -s;
    return M >= kTensorMinM ? W4_PATH_TENSOR : W4_PATH_SMALL_M;
}

namespace {

// affine: the w4_gemm_affine formats (group 32/64/128, zeros or nullptr);
// otherwise the symmetric group-128 format.
int gemm_impl(const void* x, int64_t M, int64_t N, int64_t K, int32_t group, const void* packed,
              const void* scales, const void* zeros, void* y, void* stream, int32_t path, bool affine) {
    if (affine && !valid_group(group)) return W4_ERR_UNSUPPORTED;
    if (M < 0) return W4_ERR_INVALID_ARG;
    if (const int s = check_sizes(N, K)) return s;
    if (M > 0 && K > (int64_t{1} << 62) / M) return W4_ERR_INVALID_ARG;
    if (M > 0 && N > (int64_t{1} << 62) / M) return W4_ERR_INVALID_ARG;
    if (path < W4_PATH_AUTO || path > W4_PATH_TENSOR) return W4_ERR_INVALID_ARG;
    // Tensor-map coordinates are 32-bit.
    if (N > INT32_MAX || K > INT32_MAX || M > INT32_MAX) return W4_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return W4_OK;
    if (!y) return W4_ERR_INVALID_ARG;
    if (!aligned(y, 2)) return W4_ERR_MISALIGNED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t yb = static_cast<size_t>(M * N) * 2;
    if (K == 0) return to_status(cudaMemsetAsync(y, 0, yb, st));
    if (!x || !packed || !scales) return W4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 2)) return W4_ERR_MISALIGNED;
    const size_t xb = static_cast<size_t>(M * K) * 2, pb = w4_packed_bytes(N, K),
                 sb = w4_scales_bytes(N, K, affine ? group : 128),
                 zb = affine && zeros ? w4_zeros_bytes(N, K, group) : 0;
    if (overlaps(y, yb, x, xb) || overlaps(y, yb, packed, pb) || overlaps(y, yb, scales, sb) ||
        overlaps(y, yb, zeros, zb))
        return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    if (path == W4_PATH_AUTO) path = M >= kTensorMinM ? W4_PATH_TENSOR : W4_PATH_SMALL_M;
    // The symmetric group-128 format has its own kernels (offset MMA chain in
    // the small-M path); w4_gemm_affine with group 128 and no zeros uses them.
    if (affine && (group != 128 || zeros)) {
        if (path == W4_PATH_TENSOR)
            return to_status(launch_gemm_tc_affine(x, M, N, K, group, packed, scales, zeros, y, *dev, st));
        return to_status(launch_gemv_affine(x, M, N, K, group, packed, scales, zeros, y, *dev, st));
    }
    if (path == W4_PATH_TENSOR)
        return to_status(launch_gemm_tc(x, M, N, K, packed, scales, y, *dev, st));
    return to_status(launch_gemv(x, M, N, K, packed, scales, y, *dev, st));
}

}  // namespace

int w4_gemm_ex(const void* x, int64_t M, int64_t N, int64_t K, const void* packed, const void* scales,
               void* y, void* stream, int32_t path) {
    return gemm_impl(x, M, N, K, 128, packed, scales, nullptr, y, stream, path, false);
}

int w4_gemm(const void* x, int64_t M, int64_t N, int64_t K, const void* packed, const void* scales,
            void* y, void* stream) {
    return gemm_impl(x, M, N, K, 128, packed, scales, nullptr, y, stream, W4_PATH_AUTO, false);
}

int w4_gemm_affine(const void* x, int64_t M, int64_t N, int64_t K, int32_t group, const void* packed,
                   const void* scales, const void* zeros, void* y, void* stream, int32_t path) {
    return gemm_impl(x, M, N, K, group, packed, scales, zeros, y, stream, path, true);
}

namespace {

// Checks one grouped problem like w4_gemm does.
int check_grouped_problem(const w4_gemm_problem& p) {
    if (p.M < 1 || p.N < 1 || p.K < 128) return W4_ERR_INVALID_ARG;
    if (const int s = check_sizes(p.N, p.K)) return s;
    if (p.N > INT32_MAX || p.K > INT32_MAX || p.M > INT32_MAX || p.K > (int64_t{1} << 62) / p.M ||
        p.N > (int64_t{1} << 62) / p.M)
        return W4_ERR_UNSUPPORTED;
    if (!p.x || !p.packed || !p.scales || !p.y) return W4_ERR_INVALID_ARG;
    if (!aligned(p.x, 16) || !aligned(p.packed, 16) || !aligned(p.scales, 2) || !aligned(p.y, 2))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

size_t out_bytes(const w4_gemm_problem& p) { return static_cast<size_t>(p.M * p.N) * 2; }

bool is_tensor(const w4_gemm_problem& p) { return p.M >= kGroupedTensorMinM; }

size_t round128(size_t v) { return (v + 127) / 128 * 128; }

}  // namespace

namespace {

size_t grouped_plan_bytes_impl(int32_t count, const w4_gemm_problem* problems) {
    if (count < 1 || !problems) return 0;
    int64_t small_items = 0, tc_items = 0;
    int32_t n_small = 0, n_tc = 0;
    for (int32_t i = 0; i < count; ++i) {
        const w4_gemm_problem& p = problems[i];
        if (check_grouped_problem(p) != W4_OK) return 0;
        if (is_tensor(p)) {
            ++n_tc;
            tc_items += tc_grouped_items(GroupedSpec{p.x, p.M, p.N, p.K, p.packed, p.scales, p.y, nullptr});
        } else {
            ++n_small;
            small_items += (p.N + 63) / 64;
        }
    }
    if (small_items > INT32_MAX || tc_items > INT32_MAX) return 0;
    // Sized for the largest grids a plan can use (one CTA per item), so that
    // the answer does not depend on the device.
    size_t bytes = 0;
    if (n_small) bytes += round128(grouped_plan_bytes(n_small, small_items, static_cast<int32_t>(small_items)));
    if (n_tc) bytes += tc_grouped_plan_bytes(n_tc, tc_items, static_cast<int32_t>(tc_items));
    return bytes;
}

// Validates the problems (against each other and, when device_memory is not
// NULL, against the plan memory), builds the plan image and fills every field
// of *plan except device_plan.  group: the codes' group size (32, 64, 128);
// zeros: NULL, or count pointers (each NULL or int8 [N, K/group]).  Group 128
// without zeros is the symmetric format's own path (format 0).
int grouped_prepare(const void* device_memory, size_t bytes, int32_t count, const w4_gemm_problem* problems,
                    int32_t group, const void* const* zeros, std::vector<uint8_t>* image, w4_grouped_plan* plan) {
    if (!valid_group(group)) return W4_ERR_UNSUPPORTED;
    bool any_zeros = false;
    for (int32_t i = 0; zeros && i < count; ++i) any_zeros = any_zeros || zeros[i] != nullptr;
    const int format = group == 128 && !any_zeros ? 0 : group;
    int64_t max_m = 1;
    std::vector<GroupedSpec> small, tc;
    for (int32_t i = 0; i < count; ++i) {
        const w4_gemm_problem& p = problems[i];
        if (const int s = check_grouped_problem(p)) return s;
        if (p.K % group != 0) return W4_ERR_UNSUPPORTED;
        const size_t yb = out_bytes(p);
        for (int32_t j = 0; j < count; ++j) {
            const w4_gemm_problem& q = problems[j];
            const void* qz = zeros ? zeros[j] : nullptr;
            const size_t xb = static_cast<size_t>(q.M * q.K) * 2, pb = w4_packed_bytes(q.N, q.K),
                         sb = w4_scales_bytes(q.N, q.K, group), zb = qz ? w4_zeros_bytes(q.N, q.K, group) : 0;
            if (overlaps(p.y, yb, q.x, xb) || overlaps(p.y, yb, q.packed, pb) || overlaps(p.y, yb, q.scales, sb) ||
                overlaps(p.y, yb, qz, zb))
                return W4_ERR_INVALID_ARG;
            if (j != i && overlaps(p.y, yb, q.y, out_bytes(q))) return W4_ERR_INVALID_ARG;
            if (device_memory &&
                (overlaps(device_memory, bytes, q.x, xb) || overlaps(device_memory, bytes, q.packed, pb) ||
                 overlaps(device_memory, bytes, q.scales, sb) || overlaps(device_memory, bytes, q.y, out_bytes(q)) ||
                 overlaps(device_memory, bytes, qz, zb)))
                return W4_ERR_INVALID_ARG;
        }
        const GroupedSpec sp{p.x, p.M, p.N, p.K, p.packed, p.scales, p.y, zeros ? zeros[i] : nullptr};
        if (is_tensor(p)) {
            tc.push_back(sp);
        } else {
            small.push_back(sp);
            max_m = std::max(max_m, p.M);
        }
    }
    const int token_rows = grouped_token_rows(max_m);
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    if (dev->cc_major < 10) return W4_ERR_UNSUPPORTED;
    std::vector<uint8_t> tc_image;
    int64_t n_items = 0, n_tc_items = 0;
    int32_t n_ctas = 0, n_tc_ctas = 0;
    image->clear();
    if (!small.empty()) {
        const int ctas = grouped_ctas(token_rows, format, *dev);
        if (ctas < 1) return W4_ERR_CUDA;
        if (grouped_plan_build(small.data(), static_cast<int32_t>(small.size()), token_rows, format, ctas,
                               dev->sm_count, image, &n_items, &n_ctas) != cudaSuccess)
            return W4_ERR_CUDA;
        image->resize(round128(image->size()), 0);
    }
    const size_t tc_offset = image->size();
    if (!tc.empty()) {
        if (tc_grouped_plan_build(tc.data(), static_cast<int32_t>(tc.size()), format, dev->sm_count, &tc_image,
                                  &n_tc_items, &n_tc_ctas) != cudaSuccess)
            return W4_ERR_CUDA;
        image->insert(image->end(), tc_image.begin(), tc_image.end());
    }
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return W4_ERR_CUDA;
    int max_bm = 0;
    if (!tc.empty()) std::memcpy(&max_bm, tc_image.data() + 12, sizeof(int));  // TcHeader::max_bm
    plan->device_plan = nullptr;
    plan->bytes = image->size();
    plan->count = count;
    plan->device = device;
    plan->items = static_cast<int32_t>(n_items);
    plan->ctas = n_ctas;
    plan->token_rows = small.empty() ? 0 : token_rows;
    plan->tc_items = static_cast<int32_t>(n_tc_items);
    plan->tc_ctas = n_tc_ctas;
    plan->tc_max_bm = max_bm;
    plan->tc_offset = tc_offset;
    plan->format = format;
    return W4_OK;
}

int grouped_plan_init_impl(w4_grouped_plan* plan, void* device_memory, size_t bytes, int32_t count,
                           const w4_gemm_problem* problems, int32_t group, const void* const* zeros) {
    if (!plan || !device_memory || count < 1 || !problems) return W4_ERR_INVALID_ARG;
    if (!aligned(device_memory, 128)) return W4_ERR_MISALIGNED;
    std::vector<uint8_t> image;
    w4_grouped_plan p;
    if (const int s = grouped_prepare(device_memory, bytes, count, problems, group, zeros, &image, &p)) return s;
    if (bytes < image.size()) return W4_ERR_INVALID_ARG;
    if (cudaMemcpy(device_memory, image.data(), image.size(), cudaMemcpyHostToDevice) != cudaSuccess)
        return W4_ERR_CUDA;
    p.device_plan = device_memory;
    *plan = p;
    return W4_OK;
}

}  // namespace

size_t w4_grouped_plan_bytes(int32_t count, const w4_gemm_problem* problems) {
    return grouped_plan_bytes_impl(count, problems);
}

size_t w4_grouped_plan_bytes_affine(int32_t count, const w4_gemm_problem* problems, int32_t group,
                                    const void* const* zeros) {
    (void)zeros;  // the plan's size does not depend on the format
    if (!valid_group(group)) return 0;
    for (int32_t i = 0; problems && i < count; ++i)
        if (problems[i].K % group != 0) return 0;
    return grouped_plan_bytes_impl(count, problems);
}

int w4_grouped_plan_init(w4_grouped_plan* plan, void* device_memory, size_t bytes, int32_t count,
                         const w4_gemm_problem* problems) {
    return grouped_plan_init_impl(plan, device_memory, bytes, count, problems, 128, nullptr);
}

int w4_grouped_plan_init_affine(w4_grouped_plan* plan, void* device_memory, size_t bytes, int32_t count,
                                const w4_gemm_problem* problems, int32_t group, const void* const* zeros) {
    return grouped_plan_init_impl(plan, device_memory, bytes, count, problems, group, zeros);
}

int w4_gemm_grouped(const w4_grouped_plan* plan, void* stream) {
    if (!plan || !plan->device_plan) return W4_ERR_INVALID_ARG;
    const bool has_small = plan->items > 0, has_tc = plan->tc_items > 0;
    if (!has_small && !has_tc) return W4_ERR_INVALID_ARG;
    if (plan->format != 0 && !valid_group(plan->format)) return W4_ERR_INVALID_ARG;
    if (has_small && (plan->ctas < 1 || plan->ctas > plan->items ||
                      grouped_token_rows(plan->token_rows) != plan->token_rows))
        return W4_ERR_INVALID_ARG;
    if (has_tc && (plan->tc_ctas < 1 || plan->tc_ctas > plan->tc_items || plan->tc_max_bm < 16 ||
                   plan->tc_max_bm > 256 || plan->tc_offset % 128 != 0 || plan->tc_offset >= plan->bytes))
        return W4_ERR_INVALID_ARG;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return W4_ERR_CUDA;
    if (device != plan->device) return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (has_small)
        if (const int s = to_status(
                launch_grouped(plan->device_plan, plan->ctas, plan->token_rows, plan->format, *dev, st)))
            return s;
    if (has_tc)
        return to_status(launch_tc_grouped(static_cast<const uint8_t*>(plan->device_plan) + plan->tc_offset,
                                           plan->tc_ctas, plan->tc_max_bm, plan->format, *dev, st));
    return W4_OK;
}

int w4_gemm_grouped_noalloc(int32_t count, const w4_gemm_problem* problems, void* stream) {
    if (count < 1 || !problems) return W4_ERR_INVALID_ARG;
    std::vector<uint8_t> image;
    w4_grouped_plan p;
    if (const int s = grouped_prepare(nullptr, 0, count, problems, 128, nullptr, &image, &p)) return s;
    void* mem = nullptr;
    size_t cap = 0;
    if (static_plan_memory(&mem, &cap) != cudaSuccess) return W4_ERR_CUDA;
    if (image.size() > cap) return W4_ERR_UNSUPPORTED;
    // Stream-ordered: the copy lands after the stream's earlier work (a
    // previous call's kernels no longer read the array).  From pageable
    // memory, the source has been staged when the call returns, so `image`
    // may be released.
    if (cudaMemcpyAsync(mem, image.data(), image.size(), cudaMemcpyHostToDevice, static_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
        return W4_ERR_CUDA;
    p.device_plan = mem;
    return w4_gemm_grouped(&p, stream);
}

namespace {

// The cache's kernels count requests, tokens and rows in 32 bits, and a loop's
// last step may go past them by less than 2¹⁶ (a block of threads, a grid, a
// tile of rows).
constexpr int64_t kMostCounted = 0x7fff0000;

// Memory of strided rows: `bytes` in all.  Level 0, the outermost, has count[0]
// blocks of inner[0] ≤ stride[0] bytes, stride[0] bytes apart; level 1 says the
// same of each such block, and so on.  A block of the last level is solid.
struct Region {
    const void* p = nullptr;
    int64_t bytes = 0;
    int levels = 0;
    int64_t count[3] = {}, stride[3] = {}, inner[3] = {};
};

Region plain(const void* p, size_t bytes) {
    Region r;
    r.p = p;
    r.bytes = p ? static_cast<int64_t>(std::min(bytes, size_t{1} << 62)) : 0;
    return r;
}

// Whether a block of `a` (of `a_bytes`, of level la on) and one of `b` that
// starts `off` bytes after it share a byte.  Blocks that repeat at one stride
// (slices of a fused projection's output, keys and values side by side in a
// page, a token or a row) may interleave; blocks wider than the stride of what
// they lie among count as meeting it.
bool blocks_meet(const Region& a, int la, int64_t a_bytes, const Region& b, int lb, int64_t b_bytes, int64_t off) {
    if (off >= a_bytes || -off >= b_bytes) return false;
    const int64_t sa = la < a.levels ? a.stride[la] : 0, sb = lb < b.levels ? b.stride[lb] : 0, s = std::max(sa, sb);
    if (s == 0) return true;
    const bool in_a = sa == s, in_b = sb == s;
    const int64_t na = in_a ? a.count[la] : 1, nb = in_b ? b.count[lb] : 1;
    const int64_t ea = in_a ? a.inner[la] : a_bytes, eb = in_b ? b.inner[lb] : b_bytes;
    if (ea > s || eb > s) return true;
    // Block j of b lies off + (j − i)·s after block i of a: only the two k = j − i around −off / s can meet.
    const int64_t at = (off % s + s) % s;
    for (const int64_t d : {at, at - s}) {
        const int64_t k = (d - off) / s;
        if (k > -na && k < nb && blocks_meet(a, la + in_a, ea, b, lb + in_b, eb, d)) return true;
    }
    return false;
}

// Whether two regions share a byte.
bool meets(const Region& a, const Region& b) {
    if (!overlaps(a.p, static_cast<size_t>(a.bytes), b.p, static_cast<size_t>(b.bytes))) return false;
    const uintptr_t off = reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p);
    return blocks_meet(a, 0, a.bytes, b, 0, b.bytes, static_cast<int64_t>(off));
}

struct Dim {
    int64_t n, stride;
};

// The region of rows of `row` elements of `size` bytes over `count` (≤ 3)
// dimensions, in any order of the strides.  W4_ERR_INVALID_ARG where two
// places share memory or sizes overflow, W4_ERR_MISALIGNED where a row would
// not start on 16 bytes.
int strided(const void* p, Dim* dims, int count, int64_t row, int64_t size, Region* out) {
    std::sort(dims, dims + count, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    Region r;
    int64_t extent = row;
    for (int i = 0; i < count; ++i) {
        const Dim& d = dims[i];
        if (d.n <= 1) continue;
        if (d.stride < extent || d.stride > ((int64_t{1} << 59) - extent) / (d.n - 1)) return W4_ERR_INVALID_ARG;
        if (d.stride * size % 16 != 0) return W4_ERR_MISALIGNED;
        for (int l = r.levels++; l > 0; --l) r.count[l] = r.count[l - 1], r.stride[l] = r.stride[l - 1], r.inner[l] = r.inner[l - 1];
        r.count[0] = d.n;
        r.stride[0] = d.stride * size;
        r.inner[0] = extent * size;
        extent += (d.n - 1) * d.stride;
    }
    if (!aligned(p, 16)) return W4_ERR_MISALIGNED;
    r.p = p;
    r.bytes = extent * size;
    *out = r;
    return W4_OK;
}

int rows_region(const w4_rows* r, int64_t T, int32_t heads, int32_t head_dim, Region* out) {
    if (!r || !r->data) return W4_ERR_INVALID_ARG;
    Dim dims[2] = {{T, r->token_stride}, {heads, r->head_stride}};
    return strided(r->data, dims, 2, head_dim, 2, out);
}

// k, v, k_scales, v_scales of a cache; the scales' regions are empty for format 16.
int cache_regions(const w4_kv_cache* c, Region (&out)[4]) {
    if (!c || c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1) return W4_ERR_INVALID_ARG;
    if (c->head_dim % 16 != 0 || c->head_dim > 256 || (c->format != 16 && c->format != 8)) return W4_ERR_UNSUPPORTED;
    // Page ids are 32-bit; (pages · kv_heads · page_size) scales and every slot fit 62 bits.
    if (c->pages > INT32_MAX || c->pages * c->page_size > (int64_t{1} << 61) / c->kv_heads) return W4_ERR_UNSUPPORTED;
    const bool q8 = c->format == 8;
    if (!c->k || !c->v || (q8 && (!c->k_scales || !c->v_scales))) return W4_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        Dim dims[3] = {{c->pages, c->page_stride}, {c->page_size, c->token_stride}, {c->kv_heads, c->head_stride}};
        if (const int s = strided(i ? c->v : c->k, dims, 3, c->head_dim, q8 ? 1 : 2, &out[i])) return s;
    }
    const size_t sb = q8 ? static_cast<size_t>(c->pages * c->page_size * c->kv_heads) * 2 : 0;
    if (q8 && (!aligned(c->k_scales, 2) || !aligned(c->v_scales, 2))) return W4_ERR_MISALIGNED;
    out[2] = plain(q8 ? c->k_scales : nullptr, sb);
    out[3] = plain(q8 ? c->v_scales : nullptr, sb);
    return W4_OK;
}

// Whether any output meets another or an input; `twin` (or −1) is the input
// that output 0 may be.
bool any_meet(const Region* outs, int n_out, const Region* ins, int n_in, int twin = -1) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (meets(outs[i], outs[j])) return true;
        for (int j = 0; j < n_in; ++j)
            if (!(i == 0 && j == twin) && meets(outs[i], ins[j])) return true;
    }
    return false;
}

bool same_rows(const w4_rows* a, const w4_rows* b) {
    return a->data == b->data && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

Rows to_rows(const w4_rows* r) { return {static_cast<__nv_bfloat16*>(r->data), r->token_stride, r->head_stride}; }

int usable_device(const DeviceInfo** dev) {
    cudaError_t err;
    *dev = device_info(&err);
    if (!*dev) return W4_ERR_CUDA;
    return (*dev)->cc_major < 10 ? W4_ERR_UNSUPPORTED : W4_OK;
}

bool table_fits(int32_t B, int64_t stride, int32_t width) { return B <= 1 || (stride >= width && stride <= (int64_t{1} << 59) / B); }

size_t table_bytes(int32_t B, int64_t stride, int32_t width) {
    return B > 0 ? (static_cast<size_t>(B - 1) * static_cast<size_t>(B > 1 ? stride : 0) + width) * 4 : 0;
}

int kv_pages(const int32_t* lens, const int32_t* target, int32_t B, int32_t page_size, int32_t* free_pages,
             int64_t pages, const int64_t* free_range, int32_t* block_table, int64_t table_stride, int32_t width,
             int64_t T, bool held, int32_t* holders, int32_t* new_lens, int32_t* starts, int64_t* slots,
             int32_t* positions, int64_t* free_range_out, void* workspace, size_t workspace_bytes, void* stream) {
    if (B < 0 || T < 0 || page_size < 1 || pages < 1 || width < 1) return W4_ERR_INVALID_ARG;
    if (B > kMostCounted || T > INT32_MAX || pages > INT32_MAX || (held && static_cast<int64_t>(B) * width > kMostCounted)) return W4_ERR_UNSUPPORTED;
    if (!free_pages || !free_range || !starts || !free_range_out || (held && !holders)) return W4_ERR_INVALID_ARG;
    const size_t need = held ? kv_held_workspace_bytes(B, width, pages) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4_ERR_INVALID_ARG;
    if (need > 0 && !aligned(workspace, 256)) return W4_ERR_MISALIGNED;
    if (B > 0 && (!lens || !target || !block_table || !new_lens)) return W4_ERR_INVALID_ARG;
    if (T > 0 && (!slots || !positions)) return W4_ERR_INVALID_ARG;
    if (!table_fits(B, table_stride, width)) return W4_ERR_INVALID_ARG;
    const void* fours[] = {lens, target, free_pages, block_table, new_lens, starts, positions, holders};
    const void* eights[] = {free_range, slots, free_range_out};
    for (const void* p : fours)
        if (!aligned(p, 4)) return W4_ERR_MISALIGNED;
    for (const void* p : eights)
        if (!aligned(p, 8)) return W4_ERR_MISALIGNED;
    const size_t b4 = static_cast<size_t>(B) * 4, t4 = static_cast<size_t>(T) * 4;
    const Region outs[] = {plain(block_table, table_bytes(B, table_stride, width)), plain(free_pages, static_cast<size_t>(pages) * 4),
                           plain(new_lens, b4), plain(starts, b4 + 4), plain(slots, 2 * t4), plain(positions, t4),
                           plain(free_range_out, 16), plain(holders, static_cast<size_t>(pages) * 4),
                           plain(need > 0 ? workspace : nullptr, workspace_bytes)};
    const Region ins[] = {plain(lens, b4), plain(target, b4), plain(free_range, 16)};
    if (any_meet(outs, 9, ins, 3)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    long long* const given = need > 0 ? static_cast<long long*>(workspace) : nullptr;
    unsigned* const words = given ? reinterpret_cast<unsigned*>(given + 1) : nullptr;
    const KvPagesArgs a = {lens, target, B, page_size, free_pages, pages, free_range, block_table, table_stride, width,
                           T, holders, given, words, words ? words + pages : nullptr, new_lens, starts, slots, positions, free_range_out, dev->status, 0, 0};
    return to_status(launch_kv_pages(a, *dev, static_cast<cudaStream_t>(stream)));
}

// norm: nullptr for rows that enter as they are.
int kv_append(const w4_kv_cache* cache, const w4_rope* rope, const w4_norm* norm, int64_t T, int32_t q_heads, const w4_rows* q,
              const w4_rows* q_out, const w4_rows* k, const w4_rows* v, const int64_t* slots, void* stream) {
    if (T < 0 || q_heads < 0 || !rope) return W4_ERR_INVALID_ARG;
    Region outs[5], ins[9];
    if (const int s = cache_regions(cache, *reinterpret_cast<Region(*)[4]>(&outs[1]))) return s;
    if (T > kMostCounted || q_heads > 65536 || cache->kv_heads > 65536) return W4_ERR_UNSUPPORTED;
    const w4_rope& r = *rope;
    if (r.rotary < 0 || r.rotary > cache->head_dim) return W4_ERR_INVALID_ARG;
    if (r.rotary % 16 != 0) return W4_ERR_UNSUPPORTED;
    if (r.rotary > 0) {
        if (r.axes < 1 || r.axes > 4) return W4_ERR_UNSUPPORTED;
        int64_t sum = 0;
        for (int i = 0; i < r.axes; ++i) {
            if (r.sections[i] < 0) return W4_ERR_INVALID_ARG;
            sum += r.sections[i];
        }
        if (sum != r.rotary / 2 || r.rows < 1 || r.rows > INT32_MAX || r.axis_stride < 0 ||
            (r.axis_stride > 0 && r.axis_stride < T) || r.axis_stride > (int64_t{1} << 59))
            return W4_ERR_INVALID_ARG;
    }
    if (norm) {
        if (norm->format != 16 && norm->format != 32) return W4_ERR_UNSUPPORTED;
        if (!(norm->eps >= 1e-20f && norm->eps <= 3e38f)) return W4_ERR_INVALID_ARG;
    }
    if (T == 0) return W4_OK;
    if (!slots || (r.rotary > 0 && (!r.positions || !r.cos || !r.sin))) return W4_ERR_INVALID_ARG;
    if (norm) {
        if (!norm->k_weight || (q_heads > 0 && !norm->q_weight)) return W4_ERR_INVALID_ARG;
        const size_t size = norm->format / 8;
        if (!aligned(norm->k_weight, size) || (q_heads > 0 && !aligned(norm->q_weight, size))) return W4_ERR_MISALIGNED;
        ins[7] = plain(norm->k_weight, size * cache->head_dim);
        ins[8] = plain(q_heads > 0 ? norm->q_weight : nullptr, size * cache->head_dim);
    }
    if (!aligned(slots, 8)) return W4_ERR_MISALIGNED;
    if (r.rotary > 0 && (!aligned(r.positions, 4) || !aligned(r.cos, 16) || !aligned(r.sin, 16)))
        return W4_ERR_MISALIGNED;
    const int32_t H = cache->kv_heads, d = cache->head_dim;
    if (const int s = rows_region(k, T, H, d, &ins[0])) return s;
    if (const int s = rows_region(v, T, H, d, &ins[1])) return s;
    ins[2] = plain(slots, static_cast<size_t>(T) * 8);
    const size_t table = r.rotary > 0 ? static_cast<size_t>(r.rows) * (r.rotary / 2) * 4 : 0;
    ins[3] = plain(r.positions, r.rotary > 0 ? static_cast<size_t>((r.axes - 1) * r.axis_stride + T) * 4 : 0);
    ins[4] = plain(r.cos, table);
    ins[5] = plain(r.sin, table);
    if (q_heads > 0) {
        if (const int s = rows_region(q, T, q_heads, d, &ins[6])) return s;
        if (const int s = rows_region(q_out, T, q_heads, d, &outs[0])) return s;
    }
    if (any_meet(outs, 5, ins, 9, q_heads > 0 && same_rows(q, q_out) ? 6 : -1)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    KvAppendArgs a = {};
    if (q_heads > 0) {
        a.q = to_rows(q);
        a.q_out = to_rows(q_out);
    }
    a.k = to_rows(k);
    a.v = to_rows(v);
    a.q_heads = q_heads;
    a.kv_heads = H;
    a.head_dim = d;
    a.T = T;
    a.positions = r.positions;
    a.axis_stride = r.axis_stride;
    a.cos = r.cos;
    a.sin = r.sin;
    a.rows = r.rows;
    a.rotary = r.rotary;
    a.axes = r.axes;
    a.paired = r.paired != 0;
    a.k_cache = cache->k;
    a.v_cache = cache->v;
    a.k_scales = static_cast<__nv_bfloat16*>(cache->k_scales);
    a.v_scales = static_cast<__nv_bfloat16*>(cache->v_scales);
    a.pages = cache->pages;
    a.page_stride = cache->page_stride;
    a.cache_token_stride = cache->token_stride;
    a.cache_head_stride = cache->head_stride;
    a.page_size = cache->page_size;
    a.slots = slots;
    a.status = dev->status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!norm) return to_status(launch_kv_append(a, r.sections, r.cycled != 0, cache->format == 8, *dev, st));
    const KvNorm n = {q_heads > 0 ? norm->q_weight : nullptr, norm->k_weight, norm->format == 16,
                      norm->unit_offset ? 1.f : 0.f, norm->eps, 1.f / static_cast<float>(d)};
    return to_status(launch_kv_append_norm(a, n, r.sections, r.cycled != 0, cache->format == 8, *dev, st));
}

// shared: nullptr for requests on their own.
int attn_decode(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads, const w4_rows* q,
                const w4_rows* out, const int32_t* block_table, int64_t table_stride, int32_t width,
                const int32_t* lens, const int32_t* starts, const SharedArgs* shared, float scale, int64_t window,
                void* workspace, size_t workspace_bytes, void* stream) {
    if (B < 0 || T < 0 || q_heads < 1 || width < 1 || window < 0 || !(scale - scale == 0.f)) return W4_ERR_INVALID_ARG;
    if (shared && (shared->groups < 0 || shared->width < 1)) return W4_ERR_INVALID_ARG;
    Region outs[2], ins[11];
    if (const int s = cache_regions(cache, *reinterpret_cast<Region(*)[4]>(&ins[1]))) return s;
    if (q_heads % cache->kv_heads != 0) return W4_ERR_INVALID_ARG;
    if (q_heads > 65536 || B > kMostCounted || T > kMostCounted / q_heads) return W4_ERR_UNSUPPORTED;
    if (shared && (shared->groups > kMostCounted || T > kMostShared)) return W4_ERR_UNSUPPORTED;
    if (B > 0 && !starts && T % B != 0) return W4_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return W4_OK;
    const bool groups = shared && shared->groups > 0;
    if (!block_table || !lens || !workspace || (groups && (!shared->starts || !shared->table || !shared->lens))) return W4_ERR_INVALID_ARG;
    if (!table_fits(B, table_stride, width) || (groups && !table_fits(shared->groups, shared->table_stride, shared->width)))
        return W4_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(workspace, 256) ||
        (groups && (!aligned(shared->starts, 4) || !aligned(shared->table, 4) || !aligned(shared->lens, 4))))
        return W4_ERR_MISALIGNED;
    const int32_t H = cache->kv_heads, d = cache->head_dim;
    const bool q8 = cache->format == 8;
    const size_t need = groups ? attn_shared_workspace_bytes(B, T, q_heads, H, d, q8, shared->groups)
                               : attn_decode_workspace_bytes(B, T, q_heads, H, d, q8);
    if (workspace_bytes < need) return W4_ERR_INVALID_ARG;
    if (const int s = rows_region(q, T, q_heads, d, &ins[0])) return s;
    if (const int s = rows_region(out, T, q_heads, d, &outs[0])) return s;
    outs[1] = plain(workspace, workspace_bytes);
    ins[5] = plain(block_table, table_bytes(B, table_stride, width));
    ins[6] = plain(lens, static_cast<size_t>(B) * 4);
    ins[7] = plain(starts, static_cast<size_t>(B) * 4 + 4);
    if (groups) {
        ins[8] = plain(shared->starts, static_cast<size_t>(shared->groups) * 4 + 4);
        ins[9] = plain(shared->table, table_bytes(shared->groups, shared->table_stride, shared->width));
        ins[10] = plain(shared->lens, static_cast<size_t>(shared->groups) * 4);
    }
    if (any_meet(outs, 2, ins, 11, same_rows(q, out) ? 0 : -1)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    AttnArgs a = {};
    a.q = to_rows(q);
    a.out = to_rows(out);
    a.B = B;
    a.T = T;
    a.q_heads = q_heads;
    a.kv_heads = H;
    a.head_dim = d;
    a.k = cache->k;
    a.v = cache->v;
    a.k_scales = static_cast<const __nv_bfloat16*>(cache->k_scales);
    a.v_scales = static_cast<const __nv_bfloat16*>(cache->v_scales);
    a.pages = cache->pages;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.page_size = cache->page_size;
    a.table = block_table;
    a.table_stride = table_stride;
    a.width = width;
    a.lens = lens;
    a.starts = starts;
    a.scale = scale;
    a.window = window;
    a.status = dev->status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return to_status(groups ? launch_attn_shared(a, *shared, q8, workspace, *dev, st) : launch_attn_decode(a, q8, workspace, *dev, st));
}

bool attn_workspace_known(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads) {
    return cache && B >= 0 && T >= 0 && q_heads >= 1 && cache->kv_heads >= 1 && cache->head_dim >= 1 &&
           cache->head_dim <= 256 && cache->head_dim % 16 == 0 && q_heads % cache->kv_heads == 0;
}

}  // namespace

int w4_kv_pages(const int32_t* lens, const int32_t* target, int32_t B, int32_t page_size, int32_t* free_pages,
                int64_t pages, const int64_t* free_range, int32_t* block_table, int64_t table_stride, int32_t width,
                int64_t T, int32_t* new_lens, int32_t* starts, int64_t* slots, int32_t* positions,
                int64_t* free_range_out, void* stream) {
    return kv_pages(lens, target, B, page_size, free_pages, pages, free_range, block_table, table_stride, width, T, false,
                    nullptr, new_lens, starts, slots, positions, free_range_out, nullptr, 0, stream);
}

size_t w4_kv_pages_held_workspace_bytes(int32_t B, int32_t width, int64_t pages) {
    return B < 0 || width < 1 || pages < 1 || pages > INT32_MAX || static_cast<int64_t>(B) * width > kMostCounted
               ? 0 : kv_held_workspace_bytes(B, width, pages);
}

int w4_kv_pages_held(const int32_t* lens, const int32_t* target, int32_t B, int32_t page_size, int32_t* free_pages,
                     int64_t pages, const int64_t* free_range, int32_t* block_table, int64_t table_stride,
                     int32_t width, int64_t T, int32_t* holders, int32_t* new_lens, int32_t* starts, int64_t* slots,
                     int32_t* positions, int64_t* free_range_out, void* workspace, size_t workspace_bytes, void* stream) {
    return kv_pages(lens, target, B, page_size, free_pages, pages, free_range, block_table, table_stride, width, T, true,
                    holders, new_lens, starts, slots, positions, free_range_out, workspace, workspace_bytes, stream);
}

int w4_kv_append(const w4_kv_cache* cache, const w4_rope* rope, int64_t T, int32_t q_heads, const w4_rows* q,
                 const w4_rows* q_out, const w4_rows* k, const w4_rows* v, const int64_t* slots, void* stream) {
    return kv_append(cache, rope, nullptr, T, q_heads, q, q_out, k, v, slots, stream);
}

int w4_kv_append_norm(const w4_kv_cache* cache, const w4_rope* rope, const w4_norm* norm, int64_t T, int32_t q_heads,
                      const w4_rows* q, const w4_rows* q_out, const w4_rows* k, const w4_rows* v,
                      const int64_t* slots, void* stream) {
    if (!norm) return W4_ERR_INVALID_ARG;
    return kv_append(cache, rope, norm, T, q_heads, q, q_out, k, v, slots, stream);
}

int w4_kv_fork(const int32_t* lens, const int32_t* source, const int32_t* keep, int32_t B, int32_t page_size,
               int32_t* block_table, int64_t table_stride, int32_t width, int32_t* holders, const int32_t* free_pages,
               int64_t pages, const int64_t* free_range, int32_t* new_lens, int32_t* copies, int64_t* free_range_out,
               void* stream) {
    if (B < 0 || page_size < 1 || pages < 1 || width < 1) return W4_ERR_INVALID_ARG;
    if (B > kMostCounted || pages > INT32_MAX) return W4_ERR_UNSUPPORTED;
    if (!free_pages || !free_range || !free_range_out || !holders) return W4_ERR_INVALID_ARG;
    if (B > 0 && (!lens || !source || !keep || !block_table || !new_lens || !copies)) return W4_ERR_INVALID_ARG;
    if (!table_fits(B, table_stride, width)) return W4_ERR_INVALID_ARG;
    const void* fours[] = {lens, source, keep, block_table, holders, free_pages, new_lens, copies};
    const void* eights[] = {free_range, free_range_out};
    for (const void* p : fours)
        if (!aligned(p, 4)) return W4_ERR_MISALIGNED;
    for (const void* p : eights)
        if (!aligned(p, 8)) return W4_ERR_MISALIGNED;
    const size_t b4 = static_cast<size_t>(B) * 4, p4 = static_cast<size_t>(pages) * 4;
    const Region outs[] = {plain(block_table, table_bytes(B, table_stride, width)), plain(holders, p4), plain(new_lens, b4),
                           plain(copies, 3 * b4), plain(free_range_out, 16)};
    const Region ins[] = {plain(lens, b4), plain(source, b4), plain(keep, b4), plain(free_pages, p4), plain(free_range, 16)};
    if (any_meet(outs, 5, ins, 5)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    const KvForkArgs a = {lens, source, keep, B, page_size, block_table, table_stride, width, holders, free_pages, pages,
                          free_range, new_lens, copies, free_range_out, dev->status, 0, 0};
    return to_status(launch_kv_fork(a, *dev, static_cast<cudaStream_t>(stream)));
}

int w4_kv_compact(const int32_t* lens, int32_t B, int32_t page_size, const int32_t* block_table, int64_t table_stride,
                  int32_t width, const int32_t* holders, int64_t pages, const int64_t* free_range, int32_t* new_table,
                  int64_t new_stride, int32_t* new_holders, int32_t* free_pages, int64_t* free_range_out,
                  int32_t* copies, void* stream) {
    if (B < 0 || page_size < 1 || pages < 1 || width < 1) return W4_ERR_INVALID_ARG;
    if (B > kMostCounted || pages > kMostCompacted) return W4_ERR_UNSUPPORTED;
    if (!holders || !free_range || !new_holders || !free_pages || !free_range_out || (pages > 1 && !copies)) return W4_ERR_INVALID_ARG;
    if (B > 0 && (!lens || !block_table || !new_table)) return W4_ERR_INVALID_ARG;
    if (!table_fits(B, table_stride, width) || !table_fits(B, new_stride, width)) return W4_ERR_INVALID_ARG;
    const void* fours[] = {lens, block_table, holders, new_table, new_holders, free_pages, copies};
    const void* eights[] = {free_range, free_range_out};
    for (const void* p : fours)
        if (!aligned(p, 4)) return W4_ERR_MISALIGNED;
    for (const void* p : eights)
        if (!aligned(p, 8)) return W4_ERR_MISALIGNED;
    const size_t p4 = static_cast<size_t>(pages) * 4;
    const Region outs[] = {plain(new_table, table_bytes(B, new_stride, width)), plain(new_holders, p4), plain(free_pages, p4),
                           plain(free_range_out, 16), plain(copies, static_cast<size_t>(pages / 2) * 12)};
    const Region ins[] = {plain(lens, static_cast<size_t>(B) * 4), plain(block_table, table_bytes(B, table_stride, width)),
                          plain(holders, p4), plain(free_range, 16)};
    if (any_meet(outs, 5, ins, 4)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    const KvCompactArgs a = {lens, B, page_size, block_table, table_stride, width, holders, pages, free_range, new_table,
                             new_stride, new_holders, free_pages, free_range_out, copies, dev->status, 0, 0};
    return to_status(launch_kv_compact(a, *dev, static_cast<cudaStream_t>(stream)));
}

int w4_kv_copy(const w4_kv_cache* cache, const int32_t* copies, int32_t n, void* stream) {
    if (n < 0) return W4_ERR_INVALID_ARG;
    Region outs[4];
    if (const int s = cache_regions(cache, outs)) return s;
    const int64_t size = cache->format == 8 ? 1 : 2, chunks = cache->head_dim * size / 16;
    if (n > kMostCounted || cache->page_size > kMostCopied / chunks / cache->kv_heads) return W4_ERR_UNSUPPORTED;
    if (n == 0) return W4_OK;
    if (!copies) return W4_ERR_INVALID_ARG;
    if (!aligned(copies, 4)) return W4_ERR_MISALIGNED;
    const Region in = plain(copies, static_cast<size_t>(n) * 12);
    if (any_meet(outs, 4, &in, 1)) return W4_ERR_INVALID_ARG;
    const DeviceInfo* dev;
    if (const int s = usable_device(&dev)) return s;
    KvCopyArgs a = {};
    a.k = cache->k;
    a.v = cache->v;
    a.k_scales = cache->format == 8 ? static_cast<__nv_bfloat16*>(cache->k_scales) : nullptr;
    a.v_scales = cache->format == 8 ? static_cast<__nv_bfloat16*>(cache->v_scales) : nullptr;
    a.pages = cache->pages;
    a.page_stride = cache->page_stride * size;
    a.token_stride = cache->token_stride * size;
    a.head_stride = cache->head_stride * size;
    a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads;
    a.chunks = static_cast<int32_t>(chunks);
    a.copies = copies;
    a.n = n;
    a.status = dev->status;
    return to_status(launch_kv_copy(a, *dev, static_cast<cudaStream_t>(stream)));
}

size_t w4_attn_decode_workspace_bytes(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads) {
    if (!attn_workspace_known(cache, B, T, q_heads)) return 0;
    return attn_decode_workspace_bytes(B, T, q_heads, cache->kv_heads, cache->head_dim, cache->format == 8);
}

int w4_attn_decode(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads, const w4_rows* q,
                   const w4_rows* out, const int32_t* block_table, int64_t table_stride, int32_t width,
                   const int32_t* lens, const int32_t* starts, float scale, int64_t window, void* workspace,
                   size_t workspace_bytes, void* stream) {
    return attn_decode(cache, B, T, q_heads, q, out, block_table, table_stride, width, lens, starts, nullptr, scale, window,
                       workspace, workspace_bytes, stream);
}

size_t w4_attn_decode_shared_workspace_bytes(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads,
                                             int32_t groups) {
    if (!attn_workspace_known(cache, B, T, q_heads) || groups < 0 || T > kMostShared) return 0;
    const bool q8 = cache->format == 8;
    return groups > 0 ? attn_shared_workspace_bytes(B, T, q_heads, cache->kv_heads, cache->head_dim, q8, groups)
                      : attn_decode_workspace_bytes(B, T, q_heads, cache->kv_heads, cache->head_dim, q8);
}

int w4_attn_decode_shared(const w4_kv_cache* cache, int32_t B, int64_t T, int32_t q_heads, const w4_rows* q,
                          const w4_rows* out, const int32_t* block_table, int64_t table_stride, int32_t width,
                          const int32_t* lens, const int32_t* starts, int32_t groups, const int32_t* group_starts,
                          const int32_t* prefix_table, int64_t prefix_stride, int32_t prefix_width,
                          const int32_t* prefix_lens, float scale, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const SharedArgs shared = {groups, group_starts, prefix_table, prefix_stride, prefix_width, prefix_lens};
    return attn_decode(cache, B, T, q_heads, q, out, block_table, table_stride, width, lens, starts, &shared, scale, 0,
                       workspace, workspace_bytes, stream);
}

int w4_last_device_status(void* stream) {
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned host = 0;
    if (cudaMemcpyAsync(&host, dev->status, sizeof(host), cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return W4_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return W4_ERR_CUDA;
    if (host != 0) {
        const unsigned zero = 0;
        if (cudaMemcpyAsync(dev->status, &zero, sizeof(zero), cudaMemcpyHostToDevice, st) != cudaSuccess ||
            cudaStreamSynchronize(st) != cudaSuccess)
            return W4_ERR_CUDA;
    }
    return static_cast<int>(host);
}

int w4_wait_probe(int64_t limit_ns, int32_t arrive, void* stream) {
    if (limit_ns < 0) return W4_ERR_INVALID_ARG;
    cudaError_t err;
    const DeviceInfo* dev = device_info(&err);
    if (!dev) return W4_ERR_CUDA;
    return to_status(launch_wait_probe(limit_ns, arrive, *dev, static_cast<cudaStream_t>(stream)));
}

const char* w4_status_string(int status) {
    switch (status) {
        case W4_OK: return "W4_OK";
        case W4_ERR_INVALID_ARG: return "W4_ERR_INVALID_ARG: invalid argument";
        case W4_ERR_UNSUPPORTED: return "W4_ERR_UNSUPPORTED: unsupported size, group or device";
        case W4_ERR_MISALIGNED: return "W4_ERR_MISALIGNED: pointer alignment";
        case W4_ERR_CUDA: return "W4_ERR_CUDA: CUDA runtime error";
        case W4_ERR_TIMEOUT: return "W4_ERR_TIMEOUT: a bounded device wait ran out";
        case W4_ERR_NUMERIC: return "W4_ERR_NUMERIC: a factorization failed (matrix not positive definite)";
        default: return "unknown w4 status";
    }
}

}  // extern "C"
