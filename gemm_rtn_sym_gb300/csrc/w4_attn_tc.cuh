// Pieces of the tensor-core kernels of attention over the paged cache: tiles in
// shared and tensor memory, waits that end, ring positions, codes of 8 bits.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_attn_common.cuh"
#include "w4_device.cuh"
#include "w4_tcgen05.cuh"

namespace w4 {

// Byte of 16-byte chunk c of row r in a tile of ROWS rows: columns of 128 bytes, 128-byte swizzle.
template <int ROWS>
__device__ __forceinline__ uint32_t place(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * ROWS * 128 + r * 128 + (((c ^ r) & 7) << 4));
}

// Descriptor of values as the B operand: tokens along K, values along N, in
// blocks of 64 values `block` bytes apart, eight tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t values_desc(uint32_t saddr, uint32_t block) {
    return static_cast<uint64_t>((saddr & 0x3FFFF) >> 4) | static_cast<uint64_t>(block >> 4) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Ties the registers of an earlier tmem_ld32_async to the wait before it.
__device__ __forceinline__ void reg_fence32(uint32_t (&v)[32]) {
    asm volatile(""
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]));
}

// 32 columns of the thread's lane; in registers after tmem_wait_ld() and reg_fence32().
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    tmem_ld32_async(taddr, v);
    tmem_wait_ld();
    reg_fence32(v);
}

// Tiles that an item's tokens fall in, from the sixteen on that its first lies in: none in a request without tokens.
template <int TT>
__device__ __forceinline__ int tiles_of(const Item& it) {
    return max(0, (it.tok1 - (it.tok0 & ~15) + TT - 1) / TT);
}

// Waits, as a warp, for a phase; where the wait runs out, reports it, gives what is in
// flight once more as long, and lets the caller go on without waiting.
__device__ __forceinline__ void wait_or_report(uint32_t bar, uint32_t parity, bool& alive, unsigned* status) {
    if (!alive || __all_sync(~0u, mbar_wait(bar, parity))) return;
    record_status(status, kStatusTimeout);
    alive = false;
    mbar_wait(bar, parity);
    __syncwarp();
}

// A ring position that goes round `n` places: the place, and the parity of the round.
struct Turn {
    int place = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int n) {
        if (++place == n) place = 0, round ^= 1;
    }
};

// Four codes as bf16, exactly: 0x4300 | m is 128 + m for the lower seven bits m, and 128 or 256 goes off for the sign.
__device__ __forceinline__ uint2 codes_bf16(uint32_t w) {
    const uint32_t m = w & 0x7F7F7F7Fu, sign = w & 0x80808080u;
    auto pair = [&](uint32_t sel) {
        const uint32_t from = __byte_perm(m, 0x43434343u, sel), off = __byte_perm(sign, 0x43434343u, sel);
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&from), *reinterpret_cast<const __nv_bfloat162*>(&off));
        return *reinterpret_cast<const uint32_t*>(&v);
    };
    return make_uint2(pair(0x4140), pair(0x4342));
}

}  // namespace w4
