// shared.cu -- decode attention of a batch whose sequences begin with the
// same prefix: the prefix's keys and values are read once for the query rows
// of all sequences.
//
// Softmax over [prefix | own keys] splits: with (m, l, O) = (max, sum of
// exp2(x - m), sum of exp2(x - m) v) of each part, the whole is
//   M = max m_i,  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// So every part of every row may be computed anywhere, and the launches are
//   1. the prefix's keys against the B T G rows of each kv head: with few rows
//      (at most 64) decode.cu's kernel, its rows taken across sequences; else
//      prefix_kernel below, 128 or 256 rows a CTA;
//   2. each sequence's own keys, decode.cu's kernel with keys from L on; it
//      reads nothing of 1, so its CTAs start as those of 1 leave;
//   3. shared_merge_kernel.
// What bounds 1: reading K and V once is cheap (the point of the operator);
// for rows R and keys L the SMs do 2 R L D FP8 + 2 R L D bf16 MACs and R L
// exponentials. At 128 rows x 128 keys that is 256 + 512 tensor cycles and
// 1024 MUFU cycles an SM, so the exponential bounds a full tile and the two
// row groups of a CTA keep it busy in turn.
#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>

#include "decode_common.cuh"
#include "sage_internal.h"
#include "sage_ptx.cuh"

namespace sage {
namespace {

using namespace dec;

__device__ unsigned g_shared_err;

constexpr int kFewRows = 64;                 // rows that decode.cu's kernel takes

// ------------------------------------------------------------------- merge

struct MergeParams {
    const float2* pre_stat;                  // [Hk n_rt][np][pre_rows]
    const float* pre_o;                      // [Hk n_rt][np][D][pre_rows]
    const float2* own_stat;                  // [B Hk][ns][64]
    const float* own_o;                      // [B Hk][ns][D][64]
    const int32_t* plen;
    int cap_prefix, np, ns, pre_rows, n_rt;
    int n_rows, R, T, G, Hk;
    __nv_bfloat16* out;
    int64_t os0, os1, os2, os3;
};

// CTA: 32 rows (lane = row: partials are channel-major, so a warp reads 128
// contiguous bytes a channel) x kCh channels; its eight warps share out the
// parts and are combined through shared memory.
constexpr int kCh = 16;

template <int D>
__global__ void __launch_bounds__(256) shared_merge_kernel(const MergeParams p) {
    __shared__ float2 st[8][32];
    __shared__ float acc_s[8][kCh][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d0 = blockIdx.y * kCh, hk = blockIdx.z;
    const int n = blockIdx.x * 32 + lane;
    const bool in = n < p.n_rows;
    const int nn = in ? n : p.n_rows - 1;
    const int b = nn / p.R, rr = nn % p.R;
    const int L = max(0, min(*p.plen, p.cap_prefix));
    const int np = L > 0 ? shared_splits((L + kKeys - 1) / kKeys, p.np) : 0;
    const size_t part_p = ((size_t)hk * p.n_rt + nn / p.pre_rows) * p.np, part_o = ((size_t)b * p.Hk + hk) * p.ns;
    const int r = nn % p.pre_rows;
    float M = -INFINITY, l = 0.0f, acc[kCh];
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc[k] = 0.0f;
    for (int e = warp; e < np + p.ns; e += 8) {
        const bool pre = e < np;
        const size_t part = pre ? part_p + e : part_o + (e - np);
        const int rows = pre ? p.pre_rows : 64, row = pre ? r : rr;
        const float2 s = __ldcg((pre ? p.pre_stat : p.own_stat) + part * rows + row);
        const float* o = (pre ? p.pre_o : p.own_o) + (part * D + d0) * rows + row;
        float v[kCh];
#pragma unroll
        for (int k = 0; k < kCh; ++k) v[k] = __ldcg(o + k * rows);
        if (s.x == -INFINITY) continue;          // (a part without keys has no O)
        const float m = fmaxf(M, s.x);
        const float wa = M == -INFINITY ? 0.0f : ex2_approx(M - m), wb = ex2_approx(s.x - m);
        l = fmaf(l, wa, wb * s.y);
#pragma unroll
        for (int k = 0; k < kCh; ++k) acc[k] = fmaf(acc[k], wa, wb * v[k]);
        M = m;
    }
    st[warp][lane] = make_float2(M, l);
    __syncthreads();
    float Mt = -INFINITY, lt = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) Mt = fmaxf(Mt, st[w][lane].x);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float2 s = st[w][lane];
        if (s.x != -INFINITY) lt = fmaf(ex2_approx(s.x - Mt), s.y, lt);
    }
    const float scale = M == -INFINITY ? 0.0f : ex2_approx(M - Mt) / lt;     // lt > 0 where some M is finite
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc_s[warp][k][lane] = acc[k] * scale;
    __syncthreads();
    // thread: row, two channels
    const int row = threadIdx.x >> 3, c2 = 2 * (threadIdx.x & 7);
    const int n2 = blockIdx.x * 32 + row;
    if (n2 >= p.n_rows) return;
    float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        y0 += acc_s[w][c2][row];
        y1 += acc_s[w][c2 + 1][row];
    }
    const int b2 = n2 / p.R, r2 = n2 % p.R, t = r2 / p.G, h = hk * p.G + r2 % p.G;
    __nv_bfloat16* dst = p.out + b2 * p.os0 + t * p.os1 + h * p.os2 + (int64_t)(d0 + c2) * p.os3;
    dst[0] = __float2bfloat16_rn(y0);
    dst[p.os3] = __float2bfloat16_rn(y1);
}

// ------------------------------------------------------------------ prefix

// The query rows of every sequence as the A operand of QK, once for all CTAs:
// row n = (b T + t) G + g of kv head hk rotated (fp32 butterfly) and quantised
// to e4m3 with scale max|q_hat| / 448 (the operations of decode.cu), written
// as images of the shared-memory operand: per 128-row tile [128][D] codes in
// the swizzle of a D-byte row, or (MXFP4 cache) the codes' exact bf16 values,
// two 64-channel atoms [128][128 B], channels in the converters' order for K.
// (In the prefix CTAs themselves this took 14500 cycles, 4 passes of 64 rows,
// repeated by every split.) Four threads a row.
struct QueryParams {
    const uint16_t* q;
    int64_t qs0, qs1, qs2, qs3;
    int q_vec, n_rows, rows_pad, R, G;
    uint8_t* img;
    float* scale;
};

template <int D, bool MX>
__global__ void __launch_bounds__(128) query_kernel(const QueryParams p) {
    constexpr int kQe = D / 4, kLgQe = D == 128 ? 5 : 4, kQRow = MX ? 2 * D : D;
    pdl_launch_dependents();
    const int n = blockIdx.x * 32 + (threadIdx.x >> 2), qq = threadIdx.x & 3, hk = blockIdx.y;
    const bool in = n < p.n_rows;
    const int nn = in ? n : 0, b = nn / p.R, r = nn % p.R;
    pdl_wait();
    const uint16_t* src =
        p.q + b * p.qs0 + (r / p.G) * p.qs1 + (int64_t)(hk * p.G + r % p.G) * p.qs2 + (int64_t)(qq * kQe) * p.qs3;
    float x[kQe];
    if (p.q_vec) {
#pragma unroll
        for (int c = 0; c < kQe / 8; ++c) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + c);
            const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * c + 2 * e] = __uint_as_float(wd[e] << 16);
                x[8 * c + 2 * e + 1] = __uint_as_float(wd[e] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < kQe; ++d) x[d] = __uint_as_float(static_cast<uint32_t>(__ldg(src + d * p.qs3)) << 16);
    }
#pragma unroll
    for (int lg = 0; lg < kLgQe; ++lg) {
        const int hh = 1 << lg;
#pragma unroll
        for (int kk = 0; kk < kQe / 2; ++kk) {
            const int j = ((kk >> lg) << (lg + 1)) + (kk & (hh - 1));
            const float a = x[j], c = x[j + hh];
            x[j] = __fadd_rn(a, c);
            x[j + hh] = __fsub_rn(a, c);
        }
    }
#pragma unroll
    for (int st = 1; st <= 2; st <<= 1) {
        const bool upper = (qq & st) != 0;
#pragma unroll
        for (int j = 0; j < kQe; ++j) {
            const float y = __shfl_xor_sync(0xffffffffu, x[j], st);
            x[j] = upper ? __fsub_rn(y, x[j]) : __fadd_rn(x[j], y);
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int d = 0; d < kQe; ++d) amax = fmaxf(amax, fabsf(x[d]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (!in) return;
    const float s = amax != 0.0f ? __fdiv_rn(amax, 448.0f) : 0.0f, rr = amax != 0.0f ? __fdiv_rn(448.0f, amax) : 0.0f;
    if (qq == 0) p.scale[(size_t)hk * p.rows_pad + n] = s;
    const int qg = n & 127;                       // row of its 128-row tile
    uint8_t* img = p.img + ((size_t)hk * p.rows_pad + (n & ~127)) * kQRow;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 16 * c + 4 * e;
            const uint32_t lo16 = e4m3x2_rn_satfinite(__fmul_rn(x[d], rr), __fmul_rn(x[d + 1], rr));
            const uint32_t hi16 = e4m3x2_rn_satfinite(__fmul_rn(x[d + 2], rr), __fmul_rn(x[d + 3], rr));
            w4[e] = amax != 0.0f ? (lo16 | (hi16 << 16)) : 0u;
        }
        const int chunk = (D / 64) * qq + c;
        if constexpr (MX) {
            // pair m of eight channels = (channel m, channel m + 4)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int k8 = 2 * chunk + hh;
                const uint32_t wa = w4[2 * hh], wb = w4[2 * hh + 1];
                *reinterpret_cast<uint4*>(img + (k8 >> 3) * (128 * 128) + qg * 128 + (((k8 & 7) ^ (qg & 7)) << 4)) =
                    make_uint4(e4m3_pick_to_bf16x2<0>(wa, wb), e4m3_pick_to_bf16x2<1>(wa, wb),
                               e4m3_pick_to_bf16x2<2>(wa, wb), e4m3_pick_to_bf16x2<3>(wa, wb));
            }
        } else {
            *reinterpret_cast<uint4*>(img + qg * D + (e4m3_chunk<D>(chunk, qg) << 4)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
    }
}

// CTA = 16 warps:
//   warps 0-7   softmax, two groups of four; thread = one query row (TMEM lane)
//               and all 128 keys of a unit, so the row statistics need no
//               shuffles;
//   warps 8-11  V converters: e4m3 -> exact bf16 (MXFP4: K and V);
//   warp 12     K/V producer (one TMA box per page), warps 13 and 15 MMA
//               issuers of groups 0 and 1, warp 14 scale producer.
// A unit is one 128-row x 64-key block of S: half h of a key tile, for group g.
// RG = 2 (256 rows a CTA): group g holds rows 128 g .., and the units of tile
// i, w = 4 i + 2 h + g, are its two halves for both groups, so a tile is loaded
// and converted once for 256 rows. RG = 1 (128 rows): both groups hold the
// same rows, group g takes the tiles of parity g, the units of tile i are
// w = 2 i + h, and the groups' (m, l, O) are combined at the end.
// Per unit: S = Q8 K8^T (TMEM, fp32, M = 128, N = 64) -> y = S k_scale -> row
// max -> p = 2^(y c - m) -> P = bf16(p v_scale), written over S's own columns
// as the A operand (in TMEM) of O += P V. S buffer [g][h] is used by every
// fourth unit, so a group computes on one half while the products of the
// other run: PV(w), then QK(w + 3) once PV(w - 1), which read P from that
// buffer, has completed. (One 128-key unit a group in flight, its softmax
// waiting for both products: 1800 of 5500 cycles a unit spent waiting, and 128
// logits a thread spilled; 120 us against 62 us for 4096 rows x 32768 keys.)
// The running max is only raised when a row's new maximum exceeds it by more
// than 8 (base 2): p then stays below 2^8, which fp32 sums and bf16 weights
// hold as exactly as values below one, and most tiles leave O alone.
constexpr int kScStages = 8;                 // scale ring
constexpr int kThreads = 512;
constexpr int kConvWarp0 = 8, kTmaWarp = 12, kMmaWarp0 = 13, kScaleWarp = 14, kMmaWarp1 = 15;
// 256 x 168 + 128 x 96 + 128 x 80 <= 512 x 128 registers, the launch's own
constexpr int kRegsSoft = 168, kRegsConv = 96, kRegsProd = 80;
static_assert(256 * kRegsSoft + 128 * kRegsConv + 128 * kRegsProd <= kThreads * 128, "register split");
constexpr float kLazyMax = 8.0f;
// one pair of exponentials in 2 kPolyEvery goes to the FMA pipe
constexpr int kPolyEvery = 4;

struct PrefixParams {
    const uint8_t* q_img;                    // [Hk n_rt][RG] 128-row operand tiles, from query_kernel
    const float* q_scale;                    // [Hk n_rt][128 RG]
    const float* ksc;
    const float* vsc;
    int per_tensor, v_trans;
    const uint8_t* ksf8;
    const uint8_t* vsf8;
    const int32_t* ptab;
    const int32_t* plen;
    const int32_t* ctx;
    int T, Hk, G, R, n_rows, page, lg_page, cap_prefix, cap_rows, num_pages, window, np, n_rt;
    float logit_scale_log2;
    float2* stat;                            // [Hk n_rt][np][128 RG]
    float* o;                                // [Hk n_rt][np][D][128 RG]
};

template <int D, bool MX, int RG>
struct SmP {
    static constexpr int kRowsCta = 128 * RG;
    // K / V ring; even with RG = 1, so that a group's tiles always come in the same slots
    static constexpr int kStages = RG == 2 ? 3 : 4;
    static constexpr int kQRow = MX ? 2 * D : D;                     // bytes of a query row
    static constexpr int kKStage = MX ? kKeys * D / 2 : kKeys * D;
    static constexpr int kSfStage = MX ? kKeys * D / 32 : 0;
    static constexpr int kQ = 0;                                     // e4m3 [rows][D]; MX bf16 [group][2 atoms][128][128 B]
    static constexpr int kK = kQ + kRowsCta * kQRow;
    static constexpr int kV = kK + kStages * kKStage;
    static constexpr int kKsf = kV + kStages * kKStage;
    static constexpr int kVsf = kKsf + kStages * kSfStage;
    static constexpr int kKb = MX ? al1024(kVsf + kStages * kSfStage) : kVsf;
    static constexpr int kKbBuf = MX ? kKeys * 2 * D : 0;
    static constexpr int kVb = kKb + kKbBuf;                         // [2] bf16 V, D / 64 atoms [128][128 B]
    static constexpr int kVbBuf = kKeys * 2 * D;
    static constexpr int kScale = kVb + 2 * kVbBuf;                  // [slot][k | v][128] fp32
    static constexpr int kScSlot = MX ? 0 : 2 * kKeys;
    static constexpr int kMeta = kScale + kScStages * kScSlot * 4;   // [slot] bad-page mask
    static constexpr int kSpan = kMeta + kScStages * 4;              // [8 warps] lowest, highest key any row sees
    static constexpr int kBar = kSpan + 2 * 8 * 4;
    static constexpr int kKvFull = 0, kKvEmpty = kKvFull + kStages, kSFull = kKvEmpty + kStages, kPReady = kSFull + 4,
                         kPvDone = kPReady + 4, kVReady = kPvDone + 4, kVFree = kVReady + 2, kFinal = kVFree + 2,
                         kQReady = kFinal + 2, kScFull = kQReady + 1, kScEmpty = kScFull + kScStages,
                         kKbReady = kScEmpty + kScStages, kKbFree = kKbReady + 2, kNumBars = kKbFree + 1;
    static constexpr int kMisc = kBar + kNumBars * 8;                // TMEM base, abort flag
    static constexpr int kBytes = kMisc + 16;
    // RG = 1: the other group's half of O, [D][128] fp32, over the code stages
    static constexpr int kX = kK;
    static constexpr int kXStat = kX + 128 * D * 4;                  // [2 groups][128] (m, l)
    static_assert(RG == 2 || kXStat + 2 * 128 * 8 <= kVb, "exchange area");
    static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kVb % 1024 == 0 && kKb % 1024 == 0, "swizzled tiles");
    static_assert(kBar % 8 == 0 && kKsf % 16 == 0 && kScale % 16 == 0, "alignment");
    static_assert(kBytes + 1024 <= 227 * 1024, "shared memory");
};

// D[tmem] (+)= A[tmem] * B[smem], bf16 x bf16 -> fp32 (A: lane = row, a
// 32-bit column two consecutive keys).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of the converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(pred));
    return pred != 0;
}

// 16 consecutive 32-bit TMEM columns of this thread's lane, loaded and waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int D, bool MX, int RG>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PrefixParams p) {
    using Sm = SmP<D, MX, RG>;
    constexpr int kRowsCta = Sm::kRowsCta, kStages = Sm::kStages;
    constexpr uint32_t kOCol = 256;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer: the accesses stay shared-memory ones)
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sm::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sm::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sm::kMisc + 4);
    int* meta = reinterpret_cast<int*>(sm + Sm::kMeta);
    int* span = reinterpret_cast<int*>(sm + Sm::kSpan);
    float* scl = reinterpret_cast<float*>(sm + Sm::kScale);
    const int split = blockIdx.x, hk = blockIdx.y / p.n_rt, rt = blockIdx.y % p.n_rt;
    const int row0 = rt * kRowsCta;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kMmaWarp1) {
        for (int i = lane; i < Sm::kNumBars; i += 32) {
            uint32_t cnt = 1;                                                          // expect_tx; commits
            if (i >= Sm::kKvEmpty && i < Sm::kKvEmpty + kStages) cnt = MX ? 4 : RG + 4; // (QK commits +) converters
            if (i >= Sm::kPReady && i < Sm::kPReady + 4) cnt = 4;                      // softmax group
            if (i >= Sm::kVReady && i < Sm::kVReady + 2) cnt = 4;                      // converters
            if (i >= Sm::kScFull && i < Sm::kScFull + kScStages) cnt = 1 + 32;
            if (i >= Sm::kScEmpty && i < Sm::kScEmpty + kScStages) cnt = 4 * RG;       // the groups that read the tile
            if (i >= Sm::kKbReady && i < Sm::kKbReady + 2) cnt = 4;
            if (i >= Sm::kVFree && i < Sm::kVFree + 2) cnt = RG;                       // the groups' PV commits
            if (i == Sm::kKbFree) cnt = RG;                                            // their QK commits
            mbar_init(&bars[i], cnt);
        }
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    pdl_wait();
    pdl_launch_dependents();

    int L = *p.plen;
    if (L > p.cap_prefix || L < 0) {
        if (tid == 0 && split == 0) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
        L = max(0, min(L, p.cap_prefix));
    }
    // the softmax thread's row, and the keys of the prefix that it sees
    const int g = (warp >> 2) & 1;
    const int r = RG == 2 ? (tid & 255) : (tid & 127);
    const int n = row0 + r;
    const bool rv = n < p.n_rows;
    int key_lo = INT32_MAX, key_hi = -1;
    if (warp < 8 && rv) {
        const int ctx = max(0, min(__ldg(p.ctx + n / p.R), p.cap_rows));
        const int pq = ctx - p.T + (n % p.R) / p.G;
        key_lo = max(0, pq - p.window + 1);
        key_hi = min(pq, L - 1);
        if (key_hi < key_lo) {
            key_lo = INT32_MAX;
            key_hi = -1;
        }
    }
    if (warp < 8) {
        const int lo = __reduce_min_sync(0xffffffffu, key_lo), hi = __reduce_max_sync(0xffffffffu, key_hi);
        if (lane == 0) {
            span[warp] = lo;
            span[8 + warp] = hi;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int lo = INT32_MAX, hi = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = min(lo, span[i]);
        hi = max(hi, span[8 + i]);
    }
    // key tiles [t0, t0 + n_all) that some row of the CTA sees; this split's share
    const int t0 = hi >= 0 ? lo / kKeys : 0;
    const int n_all = hi >= 0 ? hi / kKeys + 1 - t0 : 0;
    const int nsp = shared_splits(n_all, p.np);
    const int tb = t0 + (int)((int64_t)min(split, nsp) * n_all / nsp);
    const int nt = t0 + (int)((int64_t)min(split + 1, nsp) * n_all / nsp) - tb;
    const int ppt = kKeys / p.page;
    const size_t part = (size_t)blockIdx.y * p.np + split;

    if (warp >= kTmaWarp) {
      reg_dealloc<kRegsProd>();
      if (warp == kTmaWarp || warp == kScaleWarp) {
        // ------------------------------------------------------------ producers
        // (as decode.cu's: lane j of chunk c looks up page 32 c + j of the
        // CTA's pages; a page that holds no key below L is not looked up)
        const bool kv = warp == kTmaWarp;
        const float ks_t = !MX && !kv && p.per_tensor ? __ldg(p.ksc) : 1.0f;
        const float vs_t = !MX && !kv && p.per_tensor ? __ldg(p.vsc) : 1.0f;
        int chunk = -1, phys = 0, issued = 0;
        bool bad = false;
        if (kv && lane == 0 && nt > 0) {
            mbar_arrive_expect_tx(&bars[Sm::kQReady], kRowsCta * Sm::kQRow);
            bulk_load(sm + Sm::kQ, p.q_img + (size_t)blockIdx.y * kRowsCta * Sm::kQRow, kRowsCta * Sm::kQRow,
                      &bars[Sm::kQReady]);
        }
        __syncwarp();
        for (int i = 0; i < nt; ++i) {
            const int s = i % kStages, c = i % kScStages;
            const bool free_slot =
                kv ? mbar_wait(&bars[Sm::kKvEmpty + s], ((i / kStages) & 1) ^ 1, abort_flag, &g_shared_err, 1)
                   : mbar_wait(&bars[Sm::kScEmpty + c], ((i / kScStages) & 1) ^ 1, abort_flag, &g_shared_err, 2);
            if (!warp_all(free_slot)) break;
            if ((i * ppt) / 32 != chunk) {
                chunk = (i * ppt) / 32;
                const int lp = tb * ppt + 32 * chunk + lane;
                phys = 0;
                bad = false;
                if (lp < (tb + nt) * ppt && lp * p.page < L) {
                    const int pg = __ldg(p.ptab + lp);
                    if (pg < 0 || pg >= p.num_pages) {
                        bad = true;
                        if (kv) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
                    } else {
                        phys = pg;
                    }
                }
            }
            const int slot0 = (i * ppt) % 32;
            const bool mine = lane >= slot0 && lane < slot0 + ppt;
            if (kv) {
                if (lane == slot0)
                    mbar_arrive_expect_tx(&bars[Sm::kKvFull + s], 2 * (Sm::kKStage + Sm::kSfStage));
                __syncwarp();
                if (mine) {
                    const int z = phys * p.Hk + hk, q = lane - slot0;
                    constexpr int kRowB = Sm::kKStage / kKeys;
                    tma_load_3d(sm + Sm::kK + s * Sm::kKStage + q * p.page * kRowB, &tmK, &bars[Sm::kKvFull + s], 0, 0, z);
                    tma_load_3d(sm + Sm::kV + s * Sm::kKStage + q * p.page * kRowB, &tmV, &bars[Sm::kKvFull + s], 0, 0, z);
                    if constexpr (MX) {
                        constexpr int kSfB = D / 32;
                        const int64_t off = (int64_t)z * p.page * kSfB;
                        bulk_load(sm + Sm::kKsf + s * Sm::kSfStage + q * p.page * kSfB, p.ksf8 + off, p.page * kSfB,
                                  &bars[Sm::kKvFull + s]);
                        bulk_load(sm + Sm::kVsf + s * Sm::kSfStage + q * p.page * kSfB, p.vsf8 + off, p.page * kSfB,
                                  &bars[Sm::kKvFull + s]);
                    }
                }
            } else {
                const unsigned badm = __ballot_sync(0xffffffffu, mine && bad) >> slot0;
                if (lane == 0) {
                    meta[c] = static_cast<int>(badm);
                    mbar_arrive(&bars[Sm::kScFull + c]);
                }
                if constexpr (MX) {
                    mbar_arrive(&bars[Sm::kScFull + c]);
                } else {
                    float* dst = scl + c * Sm::kScSlot + 4 * lane;       // keys 4 lane .. 4 lane + 3
                    if (p.per_tensor) {
                        *reinterpret_cast<float4*>(dst) = make_float4(ks_t, ks_t, ks_t, ks_t);
                        *reinterpret_cast<float4*>(dst + kKeys) = make_float4(vs_t, vs_t, vs_t, vs_t);
                        mbar_arrive(&bars[Sm::kScFull + c]);
                    } else {
                        const int pq = __shfl_sync(0xffffffffu, phys, slot0 + 4 * lane / p.page);
                        const int64_t src = ((int64_t)pq * p.Hk + hk) * p.page + (4 * lane) % p.page;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            cp_async_4(dst + e, p.ksc + src + e);
                            cp_async_4(dst + kKeys + e, p.vsc + src + e);
                        }
                        cp_async_mbar_arrive(&bars[Sm::kScFull + c]);
                    }
                }
            }
            issued = i + 1;
        }
        // no copy of this CTA may land after it exits
        if (kv) {
            if (nt > 0) mbar_wait_drain(&bars[Sm::kQReady], 0);
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait_drain(&bars[Sm::kKvFull + i % kStages], (i / kStages) & 1);
        } else {
            for (int i = max(0, issued - kScStages); i < issued; ++i)
                mbar_wait_drain(&bars[Sm::kScFull + i % kScStages], (i / kScStages) & 1);
        }
      } else {
        // ------------------------------------------------------------ MMA issuers
        // One warp per group: a unit's issue is some hundred dependent
        // instructions, and one warp for both groups was the slowest of all
        // (1130 cycles a unit against 1490 of softmax for two). The whole
        // warp runs the loop, so that the descriptors stay in uniform
        // registers; one elected lane issues.
        const int gu = warp == kMmaWarp1 ? 1 : 0;
        const int mt = RG == 2 ? nt : (nt - gu + 1) / 2;         // the group's tiles: j -> RG == 2 ? j : 2 j + gu
        if (mt > 0) {
            constexpr uint32_t kIdescQK = umma_idesc(1, MX ? 1 : 0, 128, 64);
            const uint32_t idesc_pv = umma_idesc(1, 1, 128, D) | (p.v_trans ? 0u : 1u << 16);   // V: B MN-major
            const uint64_t qd = umma_desc_kmajor(smem_u32(sm + Sm::kQ), MX ? 128 : D) +
                                (RG == 2 ? gu : 0) * ((128 * Sm::kQRow) >> 4);
            const uint64_t kd0 = MX ? umma_desc_kmajor(smem_u32(sm + Sm::kKb), 128)
                                    : umma_desc_kmajor(smem_u32(sm + Sm::kK), D);
            const uint64_t vlbo = (p.v_trans || D == 64)
                                      ? 0ull
                                      : (static_cast<uint64_t>((kKeys * 128) >> 4) << 16) - (1ull << 16);
            const uint64_t vd0 = umma_desc_kmajor(smem_u32(sm + Sm::kVb), 128) + vlbo;
            // V, 16 keys on: 2048 bytes (MN-major), or 32 bytes inside a V^T atom of 64 keys
            const uint32_t vstep = p.v_trans ? 2 : 128, vhalf = p.v_trans ? (D * 128) >> 4 : 4 * 128;
            const uint32_t ts = tmem + 128 * gu, to = tmem + kOCol + 128 * gu;
            uint64_t* s_full = &bars[Sm::kSFull + 2 * gu];
            uint64_t* p_ready = &bars[Sm::kPReady + 2 * gu];
            uint64_t* pv_done = &bars[Sm::kPvDone + 2 * gu];
            int ks = RG == 2 ? 0 : gu;                          // ring slot and phase of the tile QK is at
            uint32_t kph = 0;
            auto k_ready = [&](int i) -> bool {
                const bool r = MX ? mbar_wait(&bars[Sm::kKbReady + (i & 1)], (i >> 1) & 1, abort_flag, &g_shared_err, 3)
                                  : mbar_wait(&bars[Sm::kKvFull + ks], kph, abort_flag, &g_shared_err, 3);
                tc_fence_after();
                return warp_all(r);
            };
            // S(i, h) = Q K(i, h)^T; after the second half, the tile's K is done with
            auto issue_qk = [&](int h) {
                const uint64_t kd = MX ? kd0 + h * ((64 * 128) >> 4)
                                       : kd0 + static_cast<uint32_t>(ks * (Sm::kKStage >> 4) + h * ((64 * D) >> 4));
                if (elect_one()) {
                    if constexpr (MX) {
#pragma unroll
                        for (int st = 0; st < D / 16; ++st)
                            mma_bf16_ss(ts + 64 * h, qd + (st >> 2) * ((128 * 128) >> 4) + 2 * (st & 3),
                                        kd + (st >> 2) * ((kKeys * 128) >> 4) + 2 * (st & 3), kIdescQK,
                                        st > 0 ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            mma_f8_ss(ts + 64 * h, qd + 2 * kk, kd + 2 * kk, kIdescQK, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(s_full + h);
                    if (h == 1) mma_commit(MX ? &bars[Sm::kKbFree] : &bars[Sm::kKvEmpty + ks]);
                }
                __syncwarp();
                if (h == 1) {
                    ks += RG == 2 ? 1 : 2;
                    if (ks >= kStages) {
                        ks -= kStages;
                        kph ^= 1;
                    }
                }
            };
            bool ok = warp_all(mbar_wait(&bars[Sm::kQReady], 0, abort_flag, &g_shared_err, 4));
            if (ok) ok = k_ready(RG == 2 ? 0 : gu);
            if (ok) {
                issue_qk(0);
                issue_qk(1);
            }
            for (int j = 0; ok && j < mt; ++j) {
                const int i = RG == 2 ? j : 2 * j + gu, vb = i & 1;
                const uint32_t ph = j & 1;
                ok = warp_all(mbar_wait(&bars[Sm::kVReady + vb], (i >> 1) & 1, abort_flag, &g_shared_err, 5));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (ok) ok = warp_all(mbar_wait(p_ready + h, ph, abort_flag, &g_shared_err, 6));
                    if (!ok) break;
                    // O += P(i, h) V(i, h): 4 steps of 16 keys
                    tc_fence_after();
                    const uint64_t vd = vd0 + static_cast<uint32_t>(vb * (Sm::kVbBuf >> 4) + h * vhalf);
                    if (elect_one()) {
#pragma unroll
                        for (int st = 0; st < 4; ++st)
                            mma_bf16_ts(to, ts + 64 * h + 8 * st, vd + st * vstep, idesc_pv,
                                        (j > 0 || h > 0 || st > 0) ? 1u : 0u);
                        mma_commit(pv_done + h);
                        if (h == 1) mma_commit(&bars[Sm::kVFree + vb]);
                    }
                    __syncwarp();
                    // the next tile's S(h) takes the columns that P(h) holds
                    if (j + 1 < mt) {
                        if (h == 0) ok = k_ready(RG == 2 ? j + 1 : 2 * (j + 1) + gu);
                        if (ok) ok = warp_all(mbar_wait(pv_done + h, ph, abort_flag, &g_shared_err, 7));
                        if (ok) issue_qk(h);
                    }
                }
            }
            if (elect_one()) mma_commit(&bars[Sm::kFinal + gu]);
            __syncwarp();
            mbar_wait_drain(&bars[Sm::kFinal + gu], 0);
        }
      }
    } else if (warp < 8) {
      reg_alloc<kRegsSoft>();
        // ------------------------------------------------------------ softmax
        // base-2 logit = (S k_scale) cq; cq >= FLT_MIN keeps a masked -inf
        const float cq = fmaxf(rv ? __ldg(p.q_scale + (size_t)blockIdx.y * kRowsCta + r) * p.logit_scale_log2 : 0.0f, FLT_MIN);
        const uint64_t cq2 = f2_pack(cq, cq);
        const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t to = trow + kOCol + 128 * g;
        const bool idle = __all_sync(0xffffffffu, !rv);      // 32 rows of padding: the warp only keeps time
        float m_run = -INFINITY;
        uint64_t l2 = f2_pack(0.0f, 0.0f);
        bool ok = true;
        const int my_units = RG == 2 ? 2 * nt : 2 * ((nt - g + 1) / 2);
        for (int k = 0; k < my_units; ++k) {
            const int h = k & 1, i = RG == 2 ? k >> 1 : 2 * (k >> 1) + g, c = i % kScStages;
            const uint32_t ts = trow + 64 * (2 * g + h);
            ok = warp_all(mbar_wait(&bars[Sm::kSFull + 2 * g + h], (k >> 1) & 1, abort_flag, &g_shared_err, 8));
            if (ok && h == 0)
                ok = warp_all(mbar_wait(&bars[Sm::kScFull + c], (i / kScStages) & 1, abort_flag, &g_shared_err, 9));
            if (!ok) break;
            if (!idle) {
                tc_fence_after();
                const int key0 = (tb + i) * kKeys + 64 * h;
                const int badm = meta[c];
                const float4* ks = reinterpret_cast<const float4*>(scl + c * Sm::kScSlot + 64 * h);
                const float4* vs = ks + kKeys / 4;
                // y = S k_scale of keys 4 q .. 4 q + 3 of 32 loaded columns
                auto scaled = [&](const uint32_t (&x)[32], int cc, int q, uint64_t& y01, uint64_t& y23) {
                    y01 = f2_pack(__uint_as_float(x[4 * q]), __uint_as_float(x[4 * q + 1]));
                    y23 = f2_pack(__uint_as_float(x[4 * q + 2]), __uint_as_float(x[4 * q + 3]));
                    if constexpr (!MX) {
                        const float4 s = ks[8 * cc + q];
                        y01 = f2_mul(y01, f2_pack(s.x, s.y));
                        y23 = f2_mul(y23, f2_pack(s.z, s.w));
                    }
                };
                // two words of P from the logits' base-2 exponents; l += p (a
                // masked key's exponent is -inf, which only MUFU makes exactly 0)
                auto weigh = [&](auto masked, uint64_t e01, uint64_t e23, int cc, int q, uint64_t& l, uint32_t* w) {
                    float a, b, p0, p1, p2, p3;
                    f2_unpack(e01, a, b);
                    if (!decltype(masked)::value && q % kPolyEvery == kPolyEvery - 1) {
                        exp2_poly_x2(a, b, p0, p1);
                    } else {
                        p0 = ex2_approx(a);
                        p1 = ex2_approx(b);
                    }
                    f2_unpack(e23, a, b);
                    p2 = ex2_approx(a);
                    p3 = ex2_approx(b);
                    uint64_t p01 = f2_pack(p0, p1), p23 = f2_pack(p2, p3);
                    l = f2_add(l, f2_add(p01, p23));
                    if constexpr (!MX) {
                        const float4 v = vs[8 * cc + q];
                        p01 = f2_mul(p01, f2_pack(v.x, v.y));
                        p23 = f2_mul(p23, f2_pack(v.z, v.w));
                    }
                    f2_unpack(p01, p0, p1);
                    f2_unpack(p23, p2, p3);
                    const __nv_bfloat162 b01 = __floats2bfloat162_rn(p0, p1), b23 = __floats2bfloat162_rn(p2, p3);
                    w[2 * q] = *reinterpret_cast<const uint32_t*>(&b01);
                    w[2 * q + 1] = *reinterpret_cast<const uint32_t*>(&b23);
                };
                uint32_t x0[32], x1[32];
                tmem_ld32(ts, x0);
                tmem_ld32(ts + 32, x1);
                tmem_wait_ld(x0);
                tmem_wait_ld(x1);
                // Most units are inside every row's window and raise no row's
                // maximum by much, so their weights are computed against the
                // running one while the unit's own is still being found: one
                // pass in which loads, FMA and MUFU overlap. Where the unit
                // turns out to need more, nothing of the pass is kept.
                bool slow = k == 0 || !__all_sync(0xffffffffu, !rv || (key0 >= key_lo && key0 + 63 <= key_hi && badm == 0));
                if (!slow) {
                    const float sub = m_run == -INFINITY ? 0.0f : m_run;
                    const uint64_t nsub2 = f2_pack(-sub, -sub);
                    uint64_t l = l2;
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t w[2][16];
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            uint64_t y01, y23;
                            scaled(cc == 0 ? x0 : x1, cc, q, y01, y23);
                            float a, b;
                            f2_unpack(y01, a, b);
                            m4[2 * (q & 1)] = fmax3(m4[2 * (q & 1)], a, b);
                            f2_unpack(y23, a, b);
                            m4[2 * (q & 1) + 1] = fmax3(m4[2 * (q & 1) + 1], a, b);
                            weigh(std::false_type{}, f2_fma(y01, cq2, nsub2), f2_fma(y23, cq2, nsub2), cc, q, l, w[cc]);
                        }
                    }
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * cq;
                    slow = __any_sync(0xffffffffu, rv && mx > m_run + kLazyMax);
                    if (!slow) {
                        l2 = l;
                        tmem_st16(ts, w[0]);
                        tmem_st16(ts + 16, w[1]);
                    }
                }
                if (slow) {
                    const int clo = key_lo - key0, chi = key_hi - key0;
                    uint64_t y[32];
                    float mx = -INFINITY;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t x[32];
                        tmem_ld32(ts + 32 * cc, x);
                        tmem_wait_ld(x);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            scaled(x, cc, q, y[16 * cc + 2 * q], y[16 * cc + 2 * q + 1]);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int j = 32 * cc + 4 * q + 2 * e;
                                const int bad0 = (badm >> ((64 * h + j) >> p.lg_page)) & 1;    // (a page has >= 16 keys)
                                float a, b;
                                f2_unpack(y[16 * cc + 2 * q + e], a, b);
                                if (j < clo || j > chi || bad0) a = -INFINITY;
                                if (j + 1 < clo || j + 1 > chi || bad0) b = -INFINITY;
                                mx = fmax3(mx, a, b);
                                y[16 * cc + 2 * q + e] = f2_pack(a, b);
                            }
                        }
                    }
                    mx = mx == -INFINITY ? -INFINITY : mx * cq;
                    float alpha = 1.0f;
                    if (mx > m_run + kLazyMax) {              // (a first key too: m_run = -inf)
                        alpha = m_run == -INFINITY ? 1.0f : ex2_approx(m_run - mx);
                        l2 = f2_mul(l2, f2_pack(alpha, alpha));
                        m_run = mx;
                    }
                    // O of the rows whose maximum was raised, once the group's
                    // last PV has completed
                    if (__any_sync(0xffffffffu, alpha != 1.0f)) {
                        if (k > 0)
                            ok = warp_all(mbar_wait(&bars[Sm::kPvDone + 2 * g + (h ^ 1)], ((k - 1) >> 1) & 1, abort_flag,
                                                    &g_shared_err, 14));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int hf = 0; hf < D / 16; ++hf) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * hf, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tmem_st16(to + 16 * hf, o);
                        }
                    }
                    const float sub = m_run == -INFINITY ? 0.0f : m_run;
                    const uint64_t nsub2 = f2_pack(-sub, -sub);
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t w[16];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            weigh(std::true_type{}, f2_fma(y[16 * cc + 2 * q], cq2, nsub2),
                                  f2_fma(y[16 * cc + 2 * q + 1], cq2, nsub2), cc, q, l2, w);
                        tmem_st16(ts + 16 * cc, w);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[Sm::kPReady + 2 * g + h]);
                if (h == 1) mbar_arrive(&bars[Sm::kScEmpty + c]);
            }
        }
        if (ok && my_units > 0)
            ok = warp_all(mbar_wait(&bars[Sm::kPvDone + 2 * g + 1], ((my_units - 1) >> 1) & 1, abort_flag,
                                    &g_shared_err, 10));
        float l0, l1;
        f2_unpack(l2, l0, l1);
        float l = l0 + l1;
        if (!ok || my_units == 0 || m_run == -INFINITY) {
            m_run = -INFINITY;
            l = 0.0f;
        }
        tc_fence_after();
        // channel of TMEM column j (MX: the order of the converted V rows)
        auto chan = [](int j) { return MX ? (j & ~7) + ((j >> 1) & 3) + 4 * (j & 1) : j; };
        float* po = p.o + part * D * kRowsCta + r;
        if constexpr (RG == 2) {
            p.stat[part * kRowsCta + r] = make_float2(m_run, l);
            if (my_units > 0 && !idle) {
#pragma unroll
                for (int hf = 0; hf < D / 32; ++hf) {
                    uint32_t o[32];
                    tmem_ld32(to + 32 * hf, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) po[chan(32 * hf + j) * kRowsCta] = __uint_as_float(o[j]);
                }
            }
            tc_fence_before();
        } else {
            // each group hands the half of O that the other one finishes to it
            float2* xs = reinterpret_cast<float2*>(sm + Sm::kXStat);
            float* xo = reinterpret_cast<float*>(sm + Sm::kX);
            tc_fence_before();
            bar_sync_all(kThreads);                  // the code stages are free
            tc_fence_after();
            xs[128 * g + r] = make_float2(m_run, l);
            const int give = (D / 2) * (1 - g), keep = (D / 2) * g;
            if (my_units > 0 && !idle) {
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    uint32_t o[32];
                    tmem_ld32(to + give + 32 * hf, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) xo[(give + 32 * hf + j) * 128 + r] = __uint_as_float(o[j]);
                }
            }
            named_sync(1, 256);
            const float2 other = xs[128 * (1 - g) + r];
            const float M = fmaxf(m_run, other.x);
            const float wa = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - M);
            const float wb = other.x == -INFINITY ? 0.0f : ex2_approx(other.x - M);
            if (g == 0) p.stat[part * 128 + r] = make_float2(M, wa * l + wb * other.y);
            if (nt > 0 && !idle) {
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    uint32_t o[32];
                    tmem_ld32(to + keep + 32 * hf, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int col = keep + 32 * hf + j;
                        // (a group without a key in the row has no O)
                        float y = m_run == -INFINITY ? 0.0f : wa * __uint_as_float(o[j]);
                        if (other.x != -INFINITY) y = fmaf(wb, xo[col * 128 + r], y);
                        po[chan(col) * 128] = y;
                    }
                }
            }
            tc_fence_before();
        }
    } else {
      reg_dealloc<kRegsConv>();
        // ------------------------------------------------------------ converters
        // lane -> cache row (key; V^T: channel) 32 cw + lane of the tile
        const int row = 32 * (warp - kConvWarp0) + lane;
        for (int i = 0; i < nt; ++i) {
            const int s = i % kStages, vb = i & 1;
            bool ok = warp_all(mbar_wait(&bars[Sm::kKvFull + s], (i / kStages) & 1, abort_flag, &g_shared_err, 11));
            if constexpr (MX) {
                if (ok && i >= 1) ok = warp_all(mbar_wait(&bars[Sm::kKbFree], (i - 1) & 1, abort_flag, &g_shared_err, 12));
                if (!ok) break;
                const uint8_t* krow = sm + Sm::kK + s * Sm::kKStage + row * 64;
                const uint32_t esc = *reinterpret_cast<const uint32_t*>(sm + Sm::kKsf + s * Sm::kSfStage + row * 4);
                uint8_t* dst = sm + Sm::kKb + row * 128;
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t o[16];
                    e2m1_block_to_bf16(*reinterpret_cast<const uint4*>(krow + (e4m3_chunk<64>(blk, row) << 4)),
                                       (esc >> (8 * blk)) & 0xFFu, o);
                    uint8_t* atom = dst + (blk >> 1) * (kKeys * 128);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(atom + (((4 * (blk & 1) + q) ^ (row & 7)) << 4)) =
                            make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[Sm::kKbReady + vb]);
            }
            if (ok && i >= 2) ok = warp_all(mbar_wait(&bars[Sm::kVFree + vb], ((i - 2) >> 1) & 1, abort_flag, &g_shared_err, 13));
            if (!ok) break;
            uint8_t* dst = sm + Sm::kVb + vb * Sm::kVbBuf + row * 128;
            if constexpr (MX) {
                const uint8_t* vrow = sm + Sm::kV + s * Sm::kKStage + row * 64;
                const uint32_t esc = *reinterpret_cast<const uint32_t*>(sm + Sm::kVsf + s * Sm::kSfStage + row * 4);
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t o[16];
                    e2m1_block_to_bf16(*reinterpret_cast<const uint4*>(vrow + (e4m3_chunk<64>(blk, row) << 4)),
                                       (esc >> (8 * blk)) & 0xFFu, o);
                    uint8_t* atom = dst + (blk >> 1) * (kKeys * 128);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(atom + (((4 * (blk & 1) + q) ^ (row & 7)) << 4)) =
                            make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
            } else {
                // 16-byte chunk c of the code row (V: 16 channels of a key;
                // V^T: 16 keys of a channel) -> two chunks of the bf16 row
                auto convert = [&](auto width_c, int atom_b) {
                    constexpr int kWidth = decltype(width_c)::value;
                    const uint8_t* vrow = sm + Sm::kV + s * Sm::kKStage + row * kWidth;
                    uint4 u[kWidth / 16];
#pragma unroll
                    for (int c = 0; c < kWidth / 16; ++c)
                        u[c] = *reinterpret_cast<const uint4*>(vrow + (e4m3_chunk<kWidth>(c, row) << 4));
#pragma unroll
                    for (int c = 0; c < kWidth / 16; ++c) {
                        uint8_t* at = dst + (c >> 2) * atom_b;
                        const int ch = 2 * (c & 3);
                        *reinterpret_cast<uint4*>(at + ((ch ^ (row & 7)) << 4)) =
                            make_uint4(e4m3x2_to_bf16x2(u[c].x, 0x1404u), e4m3x2_to_bf16x2(u[c].x, 0x3424u),
                                       e4m3x2_to_bf16x2(u[c].y, 0x1404u), e4m3x2_to_bf16x2(u[c].y, 0x3424u));
                        *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (row & 7)) << 4)) =
                            make_uint4(e4m3x2_to_bf16x2(u[c].z, 0x1404u), e4m3x2_to_bf16x2(u[c].z, 0x3424u),
                                       e4m3x2_to_bf16x2(u[c].w, 0x1404u), e4m3x2_to_bf16x2(u[c].w, 0x3424u));
                    }
                };
                if (p.v_trans) {
                    if (row < D) convert(std::integral_constant<int, kKeys>{}, D * 128);
                } else {
                    convert(std::integral_constant<int, D>{}, kKeys * 128);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[Sm::kVReady + vb]);
                mbar_arrive(&bars[Sm::kKvEmpty + s]);
            }
        }
    }
    __syncwarp();
    if (RG == 1 && warp >= 8) bar_sync_all(kThreads);            // (the softmax warps were there above)
    __syncwarp();
    tc_fence_before();
    bar_sync_all(kThreads);
    if (warp == kMmaWarp0) {                         // TMEM is read by nobody any more
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ launch

// Where the partials of the two parts lie in the workspace.
struct SharedPlan {
    int pre_rows, n_rt, np, ns;              // rows a prefix CTA has, tiles of them, their splits; own splits
    size_t pre_stat, pre_o, own_stat, own_o, q_img, q_scale, bytes;
};

SharedPlan shared_plan(int B, int T, int H, int Hk, int D) {
    SharedPlan w;
    const int64_t rows = (int64_t)B * T * (H / Hk);
    w.pre_rows = rows <= kFewRows ? kFewRows : (rows <= 256 ? 128 : 256);
    w.n_rt = (int)ceil_div(rows, w.pre_rows);
    const int sms = device_sms();
    w.np = (int)std::max<int64_t>(1, sms / ((int64_t)w.n_rt * Hk));
    w.ns = (int)std::max<int64_t>(1, std::min<int64_t>(16, sms / ((int64_t)B * Hk)));
    const size_t pre = (size_t)w.n_rt * Hk * w.np * w.pre_rows, own = (size_t)B * Hk * w.ns * 64;
    w.pre_stat = 0;
    w.own_stat = w.pre_stat + pre * sizeof(float2);
    w.pre_o = w.own_stat + own * sizeof(float2);
    w.own_o = w.pre_o + pre * D * sizeof(float);
    w.q_img = w.own_o + own * D * sizeof(float);
    const size_t q_rows = w.pre_rows == kFewRows ? 0 : (size_t)Hk * w.n_rt * w.pre_rows;
    w.q_scale = w.q_img + q_rows * 2 * D;                    // (bf16 images for an MXFP4 cache)
    w.bytes = w.q_scale + q_rows * sizeof(float);
    return w;
}

template <int D, bool MX, int RG>
cudaError_t launch_prefix(const DecodeSharedArgs& sa, const SharedPlan& w, const SharedPart& part, cudaStream_t s) {
    const DecodeArgs& a = sa.d;
    constexpr int kSmem = SmP<D, MX, RG>::kBytes + 1024;
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    QueryParams qp;
    qp.q = static_cast<const uint16_t*>(a.q.ptr);
    qp.qs0 = a.q.stride[0];
    qp.qs1 = a.q.stride[1];
    qp.qs2 = a.q.stride[2];
    qp.qs3 = a.q.stride[3];
    qp.q_vec = view_vec8(a.q) ? 1 : 0;
    qp.G = a.H / a.Hk;
    qp.R = a.T * qp.G;
    qp.n_rows = a.B * qp.R;
    qp.rows_pad = w.n_rt * w.pre_rows;
    qp.img = ws + w.q_img;
    qp.scale = reinterpret_cast<float*>(ws + w.q_scale);
    cudaError_t e = launch_pdl(query_kernel<D, MX>, dim3((unsigned)ceil_div(qp.n_rows, 32), a.Hk), dim3(128), 0, s, qp);
    if (e != cudaSuccess) return e;
    PrefixParams p = {};
    p.q_img = qp.img;
    p.q_scale = qp.scale;
    p.ksc = a.k_scale;
    p.vsc = a.v_scale;
    p.per_tensor = (a.kv_flags & 1) ? 1 : 0;
    p.v_trans = (!MX && (a.kv_flags & 2)) ? 1 : 0;
    p.ksf8 = a.k_sf;
    p.vsf8 = a.v_sf;
    p.ptab = sa.prefix_table;
    p.plen = sa.prefix_len;
    p.ctx = a.ctx_lens;
    p.T = a.T;
    p.Hk = a.Hk;
    p.G = a.H / a.Hk;
    p.R = a.T * p.G;
    p.n_rows = a.B * p.R;
    p.page = a.page_size;
    p.lg_page = 31 - __builtin_clz(static_cast<unsigned>(a.page_size));
    p.cap_prefix = sa.max_prefix_pages * a.page_size;
    p.cap_rows = a.max_pages * a.page_size;
    p.num_pages = a.num_pages;
    p.window = a.window;
    p.np = w.np;
    p.n_rt = w.n_rt;
    p.logit_scale_log2 = a.softmax_scale / static_cast<float>(D) * kLog2e;
    p.stat = part.stat;
    p.o = part.o;
    CUtensorMap tk, tv;
    const bool ok = MX ? encode_cache_mx(&tk, a.k_cache, a.num_pages, a.Hk, a.page_size, D) &&
                             encode_cache_mx(&tv, a.v_cache, a.num_pages, a.Hk, a.page_size, D)
                       : encode_cache(&tk, a.k_cache, a.num_pages, a.Hk, a.page_size, D) &&
                             (p.v_trans ? encode_cache_vt(&tv, a.v_cache, a.num_pages, a.Hk, D)
                                        : encode_cache(&tv, a.v_cache, a.num_pages, a.Hk, a.page_size, D));
    if (!ok) return cudaErrorInvalidValue;
    auto kern = prefix_kernel<D, MX, RG>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(w.np, w.n_rt * a.Hk), dim3(kThreads), kSmem, s, tk, tv, p);
}

}  // namespace

size_t decode_shared_ws_bytes(int B, int T, int H, int Hk, int D) { return shared_plan(B, T, H, Hk, D).bytes; }

cudaError_t launch_decode_shared(const DecodeSharedArgs& sa, cudaStream_t s) {
    const DecodeArgs& a = sa.d;
    const SharedPlan w = shared_plan(a.B, a.T, a.H, a.Hk, a.D);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    SharedPart part = {};
    part.prefix_table = sa.prefix_table;
    part.prefix_len = sa.prefix_len;
    part.max_prefix_pages = sa.max_prefix_pages;
    part.pre = 1;
    part.nsplit = w.np;
    part.n_rt = w.n_rt;
    part.stat = reinterpret_cast<float2*>(ws + w.pre_stat);
    part.o = reinterpret_cast<float*>(ws + w.pre_o);
    cudaError_t e;
    if (w.pre_rows == kFewRows) {
        e = launch_decode_part(a, part, s);
    } else if (w.pre_rows == 128) {
        e = a.mx ? launch_prefix<128, true, 1>(sa, w, part, s)
                 : (a.D == 128 ? launch_prefix<128, false, 1>(sa, w, part, s)
                               : launch_prefix<64, false, 1>(sa, w, part, s));
    } else {
        e = a.mx ? launch_prefix<128, true, 2>(sa, w, part, s)
                 : (a.D == 128 ? launch_prefix<128, false, 2>(sa, w, part, s)
                               : launch_prefix<64, false, 2>(sa, w, part, s));
    }
    if (e != cudaSuccess) return e;
    MergeParams m = {};
    m.pre_stat = part.stat;
    m.pre_o = part.o;
    part.pre = 0;
    part.nsplit = w.ns;
    part.stat = reinterpret_cast<float2*>(ws + w.own_stat);
    part.o = reinterpret_cast<float*>(ws + w.own_o);
    part.late_wait = 1;
    e = launch_decode_part(a, part, s);
    if (e != cudaSuccess) return e;
    m.own_stat = part.stat;
    m.own_o = part.o;
    m.plen = sa.prefix_len;
    m.cap_prefix = sa.max_prefix_pages * a.page_size;
    m.np = w.np;
    m.ns = w.ns;
    m.pre_rows = w.pre_rows;
    m.n_rt = w.n_rt;
    m.T = a.T;
    m.G = a.H / a.Hk;
    m.R = a.T * m.G;
    m.n_rows = a.B * m.R;
    m.Hk = a.Hk;
    m.out = static_cast<__nv_bfloat16*>(a.out);
    m.os0 = a.out_stride[0];
    m.os1 = a.out_stride[1];
    m.os2 = a.out_stride[2];
    m.os3 = a.out_stride[3];
    const dim3 grid((unsigned)ceil_div(m.n_rows, 32), (unsigned)(a.D / kCh), (unsigned)a.Hk);
    // a plain stream-ordered launch: it starts after both parts
    if (a.D == 128) shared_merge_kernel<128><<<grid, 256, 0, s>>>(m);
    else shared_merge_kernel<64><<<grid, 256, 0, s>>>(m);
    return cudaGetLastError();
}

unsigned read_clear_shared_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_shared_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_shared_err, &zero, sizeof zero);
    return v;
}

}  // namespace sage
