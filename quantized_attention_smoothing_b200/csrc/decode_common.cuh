// decode_common.cuh -- what the decode kernels share: exact conversions of
// e4m3 and E2M1 cache codes to bf16, swizzled-row addressing, barriers, and
// the tensor maps of the paged caches. Internal to libsage; included inside
// no namespace, defines everything in sage::dec.
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>

#include "sage_internal.h"
#include "sage_ptx.cuh"

namespace sage {
namespace dec {

constexpr int kKeys = 128;                   // keys per tile
constexpr float kLog2e = 1.4426950408889634f;

// Head size D (64 or 128): an e4m3 row of Q, K or V is D bytes, stored
// with the swizzle of that span (128B or 64B); a bf16 V row is 2 D bytes,
// one or two 64-channel 128B-swizzled atoms.
// The 16-byte chunk c of row r of a D-byte swizzled e4m3 row tile.
template <int D>
__device__ __forceinline__ int e4m3_chunk(int c, int r) {
    return D == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3));
}

// Non-blocking test of the phase with the given parity.
__device__ __forceinline__ bool mbar_test_wait(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    return ok != 0;
}

constexpr int al1024(int x) { return (x + 1023) & ~1023; }

// e4m3 codes -> bf16 with exactly the same values, integer operations only.
// A code's 7 magnitude bits placed at bf16 bits 4..10 and its sign at bit 15
// read as a bf16 of value x * 2^-120 (exponent field e of a normal code kept,
// a subnormal code a bf16 subnormal), and the bf16 product by 2^120 is exact.
// `sel` picks the two code bytes of `w` (0x1404: bytes 0, 1; 0x3424: 2, 3).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w, uint32_t sel) {
    const uint32_t t = __byte_perm(w, 0u, sel);          // code bytes at bits 8..15 and 24..31
    const uint32_t bits = ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(bits), "r"(0x7B807B80u));   // 2^120
    return r;
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The e4m3 codes byte m of `a` and byte m of `b` as one bf16 pair (low half
// from `a`), exactly, as in e4m3x2_to_bf16x2; m = 0..3.
template <int m>
__device__ __forceinline__ uint32_t e4m3_pick_to_bf16x2(uint32_t a, uint32_t b) {
    const uint32_t t = __byte_perm(a, b, (m << 4) | ((4 + m) << 12));   // bytes 1 and 3; 0, 2 unused
    return bf16x2_mul(((t >> 4) & 0x07F007F0u) | (t & 0x80008000u), 0x7B807B80u);
}

// Eight E2M1 codes (OCP MX: sign, two exponent bits, one mantissa bit),
// nibble i of `w` (bits 4i .. 4i + 3) holding element i, as four bf16 pairs:
// pair m = (element m, element m + 4), each times the bf16 pair `c2`.
// A code's three magnitude bits placed at bf16 bits 6..8 and its sign at bit
// 15 read as a bf16 of value x * 2^-126 (exponent field = the code's, a
// zero-exponent code a bf16 subnormal), so c2 = 2^(E - 1) gives x * 2^(E -
// 127) in one exact product while that is a bf16 value.
__device__ __forceinline__ void e2m1x8_to_bf16(uint32_t w, uint32_t c2, uint32_t* o) {
    const uint32_t a0 = w << 6, a1 = w << 2, a2 = w >> 2, a3 = w >> 6;
    const uint32_t s0 = w << 12, s1 = w << 8, s2 = w << 4, s3 = w;
    o[0] = bf16x2_mul((a0 & 0x01C001C0u) | (s0 & 0x80008000u), c2);
    o[1] = bf16x2_mul((a1 & 0x01C001C0u) | (s1 & 0x80008000u), c2);
    o[2] = bf16x2_mul((a2 & 0x01C001C0u) | (s2 & 0x80008000u), c2);
    o[3] = bf16x2_mul((a3 & 0x01C001C0u) | (s3 & 0x80008000u), c2);
}

// One MX block (32 E2M1 codes, 16 bytes: elements 8g .. 8g + 7 in word g)
// times 2^(E - 127), E its e8m0 scale code, as 16 bf16 pairs: pair 4g + m =
// (element 8g + m, element 8g + m + 4). E is read as min(E, 252), the largest
// exponent whose values (up to 6 * 2^125) are finite in bf16, so that cache
// bytes the window masks (slots past ctx) cannot turn a zero weight into a
// NaN; a larger E (and E = 255, NaN) lies outside the contract.
__device__ __forceinline__ void e2m1_block_to_bf16(uint4 u, uint32_t E, uint32_t (&o)[16]) {
    E = min(E, 252u);
    const uint32_t lo = E <= 128u ? E + 126u : 253u;                  // 2^(E - 1), or 2^126 then 2^(E - 127)
    const uint32_t c2 = (lo << 7) | (lo << 23);
    e2m1x8_to_bf16(u.x, c2, o);
    e2m1x8_to_bf16(u.y, c2, o + 4);
    e2m1x8_to_bf16(u.z, c2, o + 8);
    e2m1x8_to_bf16(u.w, c2, o + 12);
    if (E > 128u) {
        const uint32_t c3 = (E << 7) | (E << 23);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = bf16x2_mul(o[k], c3);
    }
}

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// Barrier `id` (1..15) of `count` threads (whole warps).
__device__ __forceinline__ void named_sync(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// CTA-wide barrier in its non-aligned form: the threads may reach it from
// different code (each thread arrives exactly once).
__device__ __forceinline__ void bar_sync_all(int count) {
    asm volatile("bar.sync 0, %0;" ::"r"(count) : "memory");
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The cache [num_pages, Hk, page, D] e4m3 as a 3-D map {D bytes, page
// rows, num_pages * Hk}; one box = one page of one kv head (or `box_rows` rows
// of it), with the swizzle of a D-byte row (128B or 64B).
inline bool encode_cache(CUtensorMap* map, const void* ptr, int num_pages, int Hk, int page, int D,
                         int box_rows = 0) {
    auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page),
                                static_cast<cuuint64_t>(num_pages) * Hk};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page) * D};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(box_rows ? box_rows : page), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The transposed V cache [num_pages, Hk, D, page = 128] as a 3-D map
// {128 key bytes, D channel rows, num_pages * Hk}; one box = one page of
// one kv head as [channel][key], 128B swizzle (or half a page, `box_keys` 64,
// 64B swizzle).
inline bool encode_cache_vt(CUtensorMap* map, const void* ptr, int num_pages, int Hk, int D, int box_keys = kKeys) {
    auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kKeys), static_cast<cuuint64_t>(D),
                                static_cast<cuuint64_t>(num_pages) * Hk};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kKeys), static_cast<cuuint64_t>(D) * kKeys};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_keys), static_cast<cuuint32_t>(D), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box_keys == kKeys ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The MXFP4 cache codes [num_pages, Hk, page, D / 2] bytes (two E2M1 codes a
// byte) as a 3-D map {D / 2 bytes, page rows, num_pages * Hk}; one box = one
// page of one kv head (or `box_rows` rows of it), 64B swizzle (D = 128:
// 64-byte rows).
inline bool encode_cache_mx(CUtensorMap* map, const void* ptr, int num_pages, int Hk, int page, int D,
                            int box_rows = 0) {
    auto enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc || D != 128) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D / 2), static_cast<cuuint64_t>(page),
                                static_cast<cuuint64_t>(num_pages) * Hk};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D / 2), static_cast<cuuint64_t>(page) * (D / 2)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(D / 2), static_cast<cuuint32_t>(box_rows ? box_rows : page), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Streaming multiprocessors of the current device (queried once per device).
inline int device_sms() {
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    std::lock_guard<std::mutex> lock(mu);
    int& c = cache[dev];
    if (c == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = 1;
        }
        c = n;
    }
    return c;
}

}  // namespace dec
}  // namespace sage
