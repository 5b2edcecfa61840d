// append.cu -- the quantised write into the paged KV cache: the new tokens'
// K, smoothed by a fixed per-head mean and rotated, and V, quantised to the
// cache's format and stored at the slots of a slot map.
//
// For token n and kv head h, with x = butterfly(K[n, h] - mean[h]) for K (the
// fp32 stages of the quantisation kernels) and x = V[n, h]:
//   FP8, one scale a token   a = max|x|, scale = a / 448,
//                            code = e4m3_rn_sat(x * (448 / a))
//   FP8, one scale in all    code = e4m3_rn_sat(x * (1 / scale))
//   MXFP4                    blocks of 32: E = floor(log2 a) - 2 in [-127, 125],
//                            code = e2m1_rn_sat(x * 2^-E), scale byte E + 127
// A constant subtracted from every key of a head shifts a query's logits by
// one number, which softmax drops, so the mean needs no place in the cache;
// it only has to be the same for all tokens that are attended together.
//
// The floor is HBM: 4 D bytes read and 2 D + 8 written per (token, head). A row
// is held by D / 16 threads, thread q with elements 8 q .. + 7 of the row's lower
// and of its upper half: every load and store of a warp is then whole 128-byte
// (32-byte) lines, the butterfly's stages 1, 2, 4 and the last are register
// arithmetic (f32x2 pairs) and those between shuffles. K and V of a row are
// loaded together before either is used. 32760 tokens of 8 heads take 46.5 us,
// 4.4 TB/s: the schedulers issue in 75 % of the cycles (592 instructions a warp),
// HBM is at 43 % of its nominal rate under the profiler. (With 32 consecutive elements a thread, 16-byte
// accesses 64 bytes apart, 74.5 us, 2.7 TB/s.)
#include <cstdint>

#include <cuda.h>

#include "sage_internal.h"
#include "sage_ptx.cuh"
#include "quant_rows.cuh"

namespace sage {
namespace {

using namespace qrow;

__device__ unsigned g_append_err;

constexpr int kThreads = 128;

struct AppendParams {
    const uint16_t* k;
    const uint16_t* v;
    int64_t ks_n, ks_h, ks_d, vs_n, vs_h, vs_d;      // strides (elements)
    const float* mean;                               // [Hk, D] or null
    const int32_t* slots;
    uint8_t* kc;
    uint8_t* vc;
    float* ksc;
    float* vsc;
    uint8_t* ksf;
    uint8_t* vsf;
    int rows;                                        // N * Hk
    int N, Hk, lg_page, num_slots;
    int vec, v_trans;
};

// Eight consecutive elements of a row, as bf16 bits.
__device__ __forceinline__ uint4 load8(const uint16_t* src, int64_t sd, int vec) {
    if (vec) return __ldg(reinterpret_cast<const uint4*>(src));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __ldg(src + 2 * i * sd) | (static_cast<uint32_t>(__ldg(src + (2 * i + 1) * sd)) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void to_pairs(uint4 u, uint64_t (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = p2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ float amax8(const uint64_t (&x)[4]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = fmax3(a, fabsf(p2lo(x[i])), fabsf(p2hi(x[i])));
    return a;
}

// e4m3 codes of x * r, four a word.
__device__ __forceinline__ uint2 codes_e4m3(const uint64_t (&x)[4], float r) {
    const uint64_t r2 = p2(r, r);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t a = p2mul(x[2 * i], r2), b = p2mul(x[2 * i + 1], r2);
        w[i] = e4m3x2_rn_satfinite(p2lo(a), p2hi(a)) |
               (static_cast<uint32_t>(e4m3x2_rn_satfinite(p2lo(b), p2hi(b))) << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Eight E2M1 codes of an MX block whose largest value is a; sf: its e8m0 byte.
__device__ __forceinline__ uint32_t codes_e2m1(const uint64_t (&x)[4], float a, uint32_t& sf) {
    const int ef = static_cast<int>(__float_as_uint(a) >> 23);            // a >= +0
    const int E = ef == 0 ? -127 : min(max(ef - 129, -127), 125);         // (infinite a: as the largest finite)
    const float sc = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);   // 2^-E
    const uint64_t s2 = p2(sc, sc);
    sf = static_cast<uint32_t>(E + 127);
    return a == 0.0f ? 0u : e2m1x8(p2mul(x[0], s2), p2mul(x[1], s2), p2mul(x[2], s2), p2mul(x[3], s2));
}

constexpr int kFmtToken = 0, kFmtTensor = 1, kFmtMx = 2;

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 10) append_kernel(const AppendParams p) {
    constexpr int LP = D / 16;                        // threads per row
    const int gt = blockIdx.x * kThreads + threadIdx.x;
    const int row = gt / LP, q = gt % LP;
    pdl_wait();
    pdl_launch_dependents();
    const bool in = row < p.rows;
    // rows token by token; over a transposed V head by head, so that a warp's
    // single-byte stores to a channel are neighbours where its tokens' slots are
    int n = 0, h = 0;
    if (in) {
        const int d = p.v_trans ? p.N : p.Hk, a = row / d, b = row - a * d;
        n = p.v_trans ? b : a;
        h = p.v_trans ? a : b;
    }
    const int slot = in ? __ldg(p.slots + n) : -1;
    const bool ok = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && q == 0) atomicCAS(&g_append_err, 0u, kErrRangeCode | (1u << 8));
    // (every thread takes the shuffles below; a row without a slot holds zeros.
    // Loads that do not wait for the slot measured 2 % slower.)
    uint4 wk[2] = {}, wv[2] = {};
    if (ok) {
        const uint16_t* k = p.k + n * p.ks_n + h * p.ks_h + 8 * q * p.ks_d;
        const uint16_t* v = p.v + n * p.vs_n + h * p.vs_h + 8 * q * p.vs_d;
#pragma unroll
        for (int c = 0; c < 2; ++c) wk[c] = load8(k + c * (D / 2) * p.ks_d, p.ks_d, p.vec);
#pragma unroll
        for (int c = 0; c < 2; ++c) wv[c] = load8(v + c * (D / 2) * p.vs_d, p.vs_d, p.vec);
    }
    uint64_t x[2][4];                                 // elements D / 2 c + 8 q ..
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        to_pairs(wk[c], x[c]);
        if (p.mean != nullptr) {
            const float4* m = reinterpret_cast<const float4*>(p.mean + h * D + c * (D / 2) + 8 * q);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 mv = __ldg(m + i);
                x[c][2 * i] = p2sub(x[c][2 * i], p2(mv.x, mv.y));
                x[c][2 * i + 1] = p2sub(x[c][2 * i + 1], p2(mv.z, mv.w));
            }
        }
        butterfly_pairs<8>(x[c]);                     // stages 1, 2, 4
    }
#pragma unroll
    for (int st = 1; st < LP; st <<= 1) {             // stages 8 .. D / 4, across the row's threads
        const bool upper = (q & st) != 0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t y = __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(x[c][i]), st);
                x[c][i] = upper ? p2sub(y, x[c][i]) : p2add(x[c][i], y);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {                     // stage D / 2
        const uint64_t a = x[0][i], b = x[1][i];
        x[0][i] = p2add(a, b);
        x[1][i] = p2sub(a, b);
    }
    const int page = slot >> p.lg_page, off = slot & ((1 << p.lg_page) - 1);
    const int64_t tok = (((int64_t)page * p.Hk + h) << p.lg_page) + off;      // (page, head, offset)
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        if (kv == 1) {
            to_pairs(wv[0], x[0]);
            to_pairs(wv[1], x[1]);
        }
        uint8_t* cache = kv == 0 ? p.kc : p.vc;
        if constexpr (FMT == kFmtMx) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float a = amax8(x[c]);                // of four threads' 32 elements
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                uint32_t sf;
                const uint32_t w = codes_e2m1(x[c], a, sf);
                if (ok) {
                    *reinterpret_cast<uint32_t*>(cache + tok * (D / 2) + c * (D / 4) + 4 * q) = w;
                    if ((q & 3) == 0)
                        (kv == 0 ? p.ksf : p.vsf)[tok * (D / 32) + c * (D / 64) + (q >> 2)] = static_cast<uint8_t>(sf);
                }
            }
        } else {
            float r;
            if constexpr (FMT == kFmtTensor) {
                r = __fdiv_rn(1.0f, __ldg(kv == 0 ? p.ksc : p.vsc));
            } else {
                float a = fmaxf(amax8(x[0]), amax8(x[1]));
#pragma unroll
                for (int st = 1; st < LP; st <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, st));
                r = e4m3_inv_scale(a);
                if (ok && q == 0) (kv == 0 ? p.ksc : p.vsc)[tok] = __fdiv_rn(a, 448.0f);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint2 w = codes_e4m3(x[c], r);
                if (!ok) continue;
                if (kv == 1 && p.v_trans) {
                    // V^T [page, head, D, 128]: channel rows, one byte a token
                    uint8_t* dst = cache + (((int64_t)page * p.Hk + h) * D + c * (D / 2) + 8 * q) * 128 + off;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[i * 128] = static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
                } else {
                    *reinterpret_cast<uint2*>(cache + tok * D + c * (D / 2) + 8 * q) = w;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
    AppendParams p;
    p.k = static_cast<const uint16_t*>(a.k.ptr);
    p.v = static_cast<const uint16_t*>(a.v.ptr);
    p.ks_n = a.k.stride[1];
    p.ks_h = a.k.stride[2];
    p.ks_d = a.k.stride[3];
    p.vs_n = a.v.stride[1];
    p.vs_h = a.v.stride[2];
    p.vs_d = a.v.stride[3];
    p.mean = a.k_mean;
    p.slots = a.slot_map;
    p.kc = a.k_cache;
    p.vc = a.v_cache;
    p.ksc = a.k_scale;
    p.vsc = a.v_scale;
    p.ksf = a.k_sf;
    p.vsf = a.v_sf;
    p.rows = (int)(a.k.size[1] * a.k.size[2]);
    p.N = (int)a.k.size[1];
    p.Hk = (int)a.k.size[2];
    p.lg_page = 31 - __builtin_clz(static_cast<unsigned>(a.page_size));
    p.num_slots = a.num_pages * a.page_size;
    p.vec = view_vec8(a.k) && view_vec8(a.v) ? 1 : 0;
    p.v_trans = (a.kv_flags & 2) ? 1 : 0;
    const int D = (int)a.k.size[3];
    const bool tensor = (a.kv_flags & 1) != 0;
    const dim3 grid((unsigned)ceil_div((int64_t)p.rows * (D / 16), kThreads)), block(kThreads);
    if (a.mx) return launch_pdl(append_kernel<128, kFmtMx>, grid, block, 0, s, p);
    if (D == 128)
        return tensor ? launch_pdl(append_kernel<128, kFmtTensor>, grid, block, 0, s, p)
                      : launch_pdl(append_kernel<128, kFmtToken>, grid, block, 0, s, p);
    return tensor ? launch_pdl(append_kernel<64, kFmtTensor>, grid, block, 0, s, p)
                  : launch_pdl(append_kernel<64, kFmtToken>, grid, block, 0, s, p);
}

unsigned read_clear_append_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_append_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_append_err, &zero, sizeof zero);
    return v;
}

}  // namespace sage
