// shared.cu -- decode attention of a batch whose sequences begin with the
// same prefix: the prefix's keys and values are read once for the query rows
// of all sequences.
//
// Softmax over [prefix | own keys] splits: with (m, l, O) = (max, sum of
// exp2(x - m), sum of exp2(x - m) v) of each part, the whole is
//   M = max m_i,  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// So every part of every row may be computed anywhere, and the launches are
//   1. query_kernel: the query rows rotated and quantised;
//   2. prefix_kernel: the prefix's keys against the B T G rows of each kv head,
//      128 or 256 rows a CTA (with at most 64 rows, rows_kernel does 1 and 2);
//   3. rows_kernel: each sequence's own keys; it reads nothing of 2, so its
//      CTAs run on the SMs that 2 leaves over and start as those of 2 leave;
//   4. shared_merge_kernel.
// What bounds 2: reading K and V once is cheap (the point of the operator);
// for rows R and keys L the SMs do 2 R L D FP8 + 2 R L D fp16 FLOPs and R L
// exponentials: 31 us of tensor time and 30 us of MUFU for 4096 rows, 32768
// keys and D 128, where the kernel takes 74. No pipe is full (MUFU 39 %,
// tensor 33 %, issue 44 %): a unit of 128 rows x 64 keys is a chain of 2250
// cycles in two softmax warps a scheduler, and what was tried against that
// (four warps a scheduler, turns, earlier loads of S, fewer exponentials on
// MUFU, naps instead of polls, PV without its wait) gained nothing or lost.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_common.cuh"
#include "sage_internal.h"
#include "sage_ptx.cuh"

namespace sage {
namespace {

using namespace dec;

__device__ unsigned g_shared_err;

constexpr int kFewRows = 64;                 // rows that rows_kernel takes
constexpr int kBlk = 64;                     // keys that a warp of it takes at a time

// The splits, of at most nsplit, that n key tiles (prefix_kernel) or blocks
// (rows_kernel) are shared out among: none gets fewer than a CTA works on at
// once (2^lg_at_once), which would only make more partials to combine.
__host__ __device__ inline int used_splits(int n, int nsplit, int lg_at_once) {
    const int want = (n + (1 << lg_at_once) - 1) >> lg_at_once;
    return want < 1 ? 1 : (want < nsplit ? want : nsplit);
}

// The share [first, last) of split `split` of n things among nsp (none for
// split >= nsp).
__device__ __forceinline__ void share_out(int n, int nsp, int split, int& first, int& last) {
    const int q = (int)((unsigned)n / (unsigned)nsp), rem = n - q * nsp, s = min(split, nsp);
    first = s * q + min(s, rem);
    last = s < nsp ? first + q + (s < rem ? 1 : 0) : first;
}

// n / d as a multiplication: exact while n d < 2^32 (mul = ceil(2^32 / d)).
struct FastDiv {
    uint32_t mul;                            // 0: d = 1
};
inline FastDiv fast_div_by(int64_t d) { return {d <= 1 ? 0u : (uint32_t)(((int64_t(1) << 32) + d - 1) / d)}; }
__device__ __forceinline__ int fast_div(int n, FastDiv d) { return d.mul == 0 ? n : (int)__umulhi((uint32_t)n, d.mul); }

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^e for |e| <= 252 (two normal factors, so that no half of it underflows).
__device__ __forceinline__ float pow2i(int e) {
    const int a = e / 2, b = e - a;
    return __int_as_float((a + 127) << 23) * __int_as_float((b + 127) << 23);
}

// The e4m3 pair in the low (high) half of w as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_lo_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// A mask of the n lowest bytes of a word (n <= 0: none, n >= 4: all).
__device__ __forceinline__ uint32_t low_bytes(int n) {
    return n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
}

// An FP8 cache's value scales are taken relative to a power of two, 2^e, so
// that what they are multiplied into fits fp16 (which keeps 11 bits where bf16
// would keep 8): the converted V rows of prefix_kernel, the weights of
// rows_kernel. e is the exponent of the first tile's largest scale and is
// raised when a later tile has one over 2^kScaleRoom times as large, O
// following by an exact power of two. Slots that hold no key of the part
// count as zero, whatever they hold.
constexpr int kScaleRoom = 4;
constexpr int kNoExp = -1000;
// The exponent to use from a tile on whose largest scale is vmax.
__device__ __forceinline__ int scale_exp(int e, float vmax) {
    const int ev = vmax > 0.0f ? max(-120, min(120, (int)(__float_as_uint(vmax) >> 23) - 126)) : kNoExp;
    return ev > (e == kNoExp ? kNoExp : e + kScaleRoom) ? ev : e;
}

// The running max is only raised when a row's new maximum exceeds it by more
// than this (base 2): p then stays below 2^8, which fp32 sums and 16-bit
// weights hold as exactly as values below one, and most tiles leave O alone.
constexpr float kLazyMax = 8.0f;

// Partials are laid out [D / 4][rows][4 channels] fp32: a warp whose lanes are
// rows writes and reads 512 contiguous bytes with one 16-byte access a lane
// (channel by channel, 128 bytes at a time, the 128 KB of a prefix CTA took
// 5000 cycles to leave it).

// ------------------------------------------------------------------- merge

struct MergeParams {
    const float2* pre_stat;                  // [Hk n_rt][np][pre_rows]
    const float* pre_o;                      // [Hk n_rt][np][D / 4][pre_rows][4]
    const float2* own_stat;                  // [B Hk][ns][64]
    const float* own_o;                      // [B Hk][ns][D / 4][64][4]
    const int32_t* plen;
    const int32_t* ctx;
    int cap_prefix, cap_rows, window, np, ns, pre_rows, n_rt;
    int unit, lg_at_once;                    // keys of a tile or block of the prefix part, used_splits' third
    int lg_unit, lg_own;                     // a sequence's own: log2 of its unit, used_splits' third
    int n_rows, R, T, G, Hk;
    __nv_bfloat16* out;
    int64_t os0, os1, os2, os3;
};

// Blocks [first, first + n) (of 2^lg keys) of a sequence's own keys, those of
// [L, ctx) that one of its T query tokens sees, and the lowest and highest such
// key.
__device__ __forceinline__ void own_keys(int ctx, int L, int T, int window, int lg, int& lo, int& hi, int& first, int& n) {
    lo = max(L, ctx - T - window + 1);
    hi = lo < ctx ? ctx - 1 : -1;
    first = hi >= 0 ? lo >> lg : 0;
    n = hi >= 0 ? (hi >> lg) + 1 - first : 0;
}

// CTA: 32 rows (lane = row) x kCh channels; its W warps share out the parts
// and are combined through shared memory. A part's O is requested together
// with its statistics, kAtOnce parts at a time, and dropped where the row has
// no key in it (it then holds anything): with so few parts a warp, two
// dependent trips to L2 were most of the time.
constexpr int kCh = 16;

template <int D, int W>
__global__ void __launch_bounds__(32 * W) shared_merge_kernel(const MergeParams p) {
    __shared__ float2 st[W][32];
    __shared__ float acc_s[W][kCh][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d0 = blockIdx.y * kCh, hk = blockIdx.z;
    const int n = blockIdx.x * 32 + lane;
    const int nn = min(n, p.n_rows - 1);
    const int b = nn / p.R, rr = nn - b * p.R;
    const int rt = nn / p.pre_rows, r = nn - rt * p.pre_rows;
    pdl_wait();
    const int ctx = max(0, min(__ldg(p.ctx + b), p.cap_rows));
    const int L = max(0, min(__ldg(p.plen), p.cap_prefix));
    const int np = L > 0 ? used_splits((L + p.unit - 1) / p.unit, p.np, p.lg_at_once) : 0;
    int lo, hi, first, n_own;
    own_keys(ctx, L, p.T, p.window, p.lg_unit, lo, hi, first, n_own);
    const int parts = np + (n_own > 0 ? used_splits(n_own, p.ns, p.lg_own) : 0);
    const int most = __reduce_max_sync(0xffffffffu, parts);
    const size_t part_p = ((size_t)hk * p.n_rt + rt) * p.np, part_o = ((size_t)b * p.Hk + hk) * p.ns;
    float M = -INFINITY, l = 0.0f, acc[kCh];
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc[k] = 0.0f;
    constexpr int kAtOnce = 4;
    for (int e0 = warp; e0 < most; e0 += W * kAtOnce) {
        float2 s[kAtOnce];
        float v[kAtOnce][kCh];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int e = e0 + W * i;
            s[i] = make_float2(-INFINITY, 0.0f);
            if (e < parts) {
                const bool pre = e < np;
                const int rows = pre ? p.pre_rows : 64, row = pre ? r : rr;
                const size_t part = pre ? part_p + e : part_o + e - np;
                s[i] = __ldcg((pre ? p.pre_stat : p.own_stat) + part * rows + row);
                const float4* o = reinterpret_cast<const float4*>(pre ? p.pre_o : p.own_o) + (part * (D / 4) + d0 / 4) * rows + row;
#pragma unroll
                for (int k = 0; k < kCh / 4; ++k) {
                    const float4 x = __ldcg(o + k * rows);
                    v[i][4 * k] = x.x;
                    v[i][4 * k + 1] = x.y;
                    v[i][4 * k + 2] = x.z;
                    v[i][4 * k + 3] = x.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (s[i].x == -INFINITY) continue;
            const float m = fmaxf(M, s[i].x);
            const float wa = M == -INFINITY ? 0.0f : ex2_approx(M - m), wb = ex2_approx(s[i].x - m);
            l = fmaf(l, wa, wb * s[i].y);
#pragma unroll
            for (int k = 0; k < kCh; ++k) acc[k] = fmaf(acc[k], wa, wb * v[i][k]);
            M = m;
        }
    }
    st[warp][lane] = make_float2(M, l);
    __syncthreads();
    float Mt = -INFINITY, lt = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) Mt = fmaxf(Mt, st[w][lane].x);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float2 s = st[w][lane];
        if (s.x != -INFINITY) lt = fmaf(ex2_approx(s.x - Mt), s.y, lt);
    }
    const float scale = M == -INFINITY ? 0.0f : ex2_approx(M - Mt) / lt;     // lt > 0 where some M is finite
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc_s[warp][k][lane] = acc[k] * scale;
    __syncthreads();
    // thread: row, two channels
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
        const int row = (threadIdx.x >> 3) + 4 * W * i, c2 = 2 * (threadIdx.x & 7);
        const int n2 = blockIdx.x * 32 + row;
        if (n2 >= p.n_rows) return;
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            y0 += acc_s[w][c2][row];
            y1 += acc_s[w][c2 + 1][row];
        }
        const int b2 = n2 / p.R, r2 = n2 % p.R, t = r2 / p.G, h = hk * p.G + r2 % p.G;
        __nv_bfloat16* dst = p.out + b2 * p.os0 + t * p.os1 + h * p.os2 + (int64_t)(d0 + c2) * p.os3;
        dst[0] = __float2bfloat16_rn(y0);
        dst[p.os3] = __float2bfloat16_rn(y1);
    }
}

// ------------------------------------------------------------------ prefix

// The query rows of every sequence, once for all CTAs: row n = (b T + t) G + g
// of kv head hk rotated (fp32 butterfly) and quantised to e4m3 with scale
// max|q_hat| / 448 (the operations of decode.cu). The codes go out row by row
// for rows_kernel, and for prefix_kernel as images of its shared-memory
// operand: per 128-row tile [128][D] codes in the swizzle of a D-byte row, or
// (MXFP4 cache) the codes' exact bf16 values, two 64-channel atoms [128][128 B],
// channels in the converters' order for K.
// (In the prefix CTAs themselves this took 14500 cycles, 4 passes of 64 rows,
// repeated by every split.) Four threads a row.
struct QueryParams {
    const uint16_t* q;
    int64_t qs0, qs1, qs2, qs3;
    int q_vec, n_rows, rows_pad, R, G;
    uint8_t* codes;                          // [Hk][rows_pad][D]
    uint8_t* img;
    float* scale;                            // [Hk][rows_pad]
};

// Quarter qq of a query row (src: its first element), held by four neighbouring
// threads: the row rotated and quantised, this quarter's codes four a word.
// Returns the row's scale.
template <int D>
__device__ __forceinline__ float quantise_quarter(const uint16_t* src, int64_t sd, bool vec, int qq, uint32_t (&w)[D / 16]) {
    constexpr int kQe = D / 4, kLgQe = D == 128 ? 5 : 4;
    float x[kQe];
    if (vec) {
#pragma unroll
        for (int c = 0; c < kQe / 8; ++c) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + c);
            const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * c + 2 * e] = __uint_as_float(wd[e] << 16);
                x[8 * c + 2 * e + 1] = __uint_as_float(wd[e] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < kQe; ++d) x[d] = __uint_as_float(static_cast<uint32_t>(__ldg(src + d * sd)) << 16);
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
    const float rr = e4m3_inv_scale(amax);
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
        const uint32_t lo16 = e4m3x2_rn_satfinite(__fmul_rn(x[4 * e], rr), __fmul_rn(x[4 * e + 1], rr));
        const uint32_t hi16 = e4m3x2_rn_satfinite(__fmul_rn(x[4 * e + 2], rr), __fmul_rn(x[4 * e + 3], rr));
        w[e] = amax != 0.0f ? (lo16 | (hi16 << 16)) : 0u;
    }
    return amax != 0.0f ? __fdiv_rn(amax, 448.0f) : 0.0f;
}

template <int D, bool MX>
__global__ void __launch_bounds__(128) query_kernel(const QueryParams p) {
    constexpr int kQe = D / 4, kQRow = MX ? 2 * D : D;
    pdl_launch_dependents();
    const int n = blockIdx.x * 32 + (threadIdx.x >> 2), qq = threadIdx.x & 3, hk = blockIdx.y;
    const bool in = n < p.n_rows;
    const int nn = in ? n : 0, b = nn / p.R, r = nn % p.R;
    pdl_wait();
    uint32_t w4[D / 16];
    const float s = quantise_quarter<D>(p.q + b * p.qs0 + (r / p.G) * p.qs1 + (int64_t)(hk * p.G + r % p.G) * p.qs2 +
                                            (int64_t)(qq * kQe) * p.qs3, p.qs3, p.q_vec, qq, w4);
    if (!in) return;
    if (qq == 0) p.scale[(size_t)hk * p.rows_pad + n] = s;
    const int qg = n & 127;                       // row of its 128-row tile
    uint8_t* img = p.img + ((size_t)hk * p.rows_pad + (n & ~127)) * kQRow;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const int chunk = (D / 64) * qq + c;
        const uint4 u = make_uint4(w4[4 * c], w4[4 * c + 1], w4[4 * c + 2], w4[4 * c + 3]);
        *reinterpret_cast<uint4*>(p.codes + ((size_t)hk * p.rows_pad + n) * D + 16 * chunk) = u;
        if constexpr (MX) {
            // pair m of eight channels = (channel m, channel m + 4)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int k8 = 2 * chunk + hh;
                const uint32_t wa = w4[4 * c + 2 * hh], wb = w4[4 * c + 2 * hh + 1];
                *reinterpret_cast<uint4*>(img + (k8 >> 3) * (128 * 128) + qg * 128 + (((k8 & 7) ^ (qg & 7)) << 4)) =
                    make_uint4(e4m3_pick_to_bf16x2<0>(wa, wb), e4m3_pick_to_bf16x2<1>(wa, wb),
                               e4m3_pick_to_bf16x2<2>(wa, wb), e4m3_pick_to_bf16x2<3>(wa, wb));
            }
        } else {
            *reinterpret_cast<uint4*>(img + qg * D + (e4m3_chunk<D>(chunk, qg) << 4)) = u;
        }
    }
}

// CTA = 16 warps:
//   warps 0-7   softmax, two groups of four; thread = one query row (TMEM lane)
//               and all 64 keys of a unit, so the row statistics need no
//               shuffles;
//   warps 8-11  V converters: e4m3 -> fp16, the value's scale multiplied in
//               (MXFP4: K and V -> bf16, exactly);
//   warp 12     K/V producer (one TMA box per page), warps 13 and 15 MMA
//               issuers of groups 0 and 1, warp 14 scale producer.
// A unit is one 128-row x 64-key block of S: half h of a key tile, for group g.
// RG = 2 (256 rows a CTA): group g holds rows 128 g .., and the units of tile
// i, w = 4 i + 2 h + g, are its two halves for both groups, so a tile is loaded
// and converted once for 256 rows. RG = 1 (128 rows): both groups hold the
// same rows, group g takes the tiles of parity g, the units of tile i are
// w = 2 i + h, and the groups' (m, l, O) are combined at the end.
// Per unit: S = Q8 K8^T (TMEM, fp32, M = 128, N = 64) -> y = S k_scale ->
// p = 2^(y c - m) -> P = fp16(p) (MXFP4: bf16(p)), over S's own columns as the
// A operand (in TMEM) of O += P V. S buffer [g][h] is used by every fourth
// unit, so a group computes on one half while the products of the other run:
// PV(w), then QK(w + 3) once PV(w - 1), which read P from that buffer, has
// completed. (One 128-key unit a group in flight, its softmax waiting for both
// products: 1800 of 5500 cycles a unit spent waiting, and 128 logits a thread
// spilled. The value scales multiplied into P instead of V, and the unit's
// maximum taken instead of its sum checked: 100.2 us against 97.2 for a call
// of 4096 rows and 32768 keys.)
constexpr int kScStages = 8;                 // scale ring
constexpr int kThreads = 512;
constexpr int kConvWarp0 = 8, kTmaWarp = 12, kMmaWarp0 = 13, kScaleWarp = 14, kMmaWarp1 = 15;
// 256 x 168 + 128 x 96 + 128 x 80 <= 512 x 128 registers, the launch's own
constexpr int kRegsSoft = 168, kRegsConv = 96, kRegsProd = 80;
static_assert(256 * kRegsSoft + 128 * kRegsConv + 128 * kRegsProd <= kThreads * 128, "register split");
// A unit's 64 weights against the running max: where they add up to more than
// kMaxSum some logit is over 2 above it, and the max is raised wherever that is
// so (kRaise); where a row's first ones add up to less than kMinSum its max is
// taken first. The sum l keeps the fp32 weights, so the 16-bit ones must not
// lose bits beside it: fp16 (FP8 cache) holds 2^-24 at least, so the first
// unit's have to add up to 1 (the largest is then 2^-6 or more, and no weight
// is off by more than 2^-25 of l); bf16 (MXFP4) has the range of fp32.
constexpr float kMaxSum = 256.0f, kRaise = 2.0f;
template <bool MX>
constexpr float kMinSum = MX ? 0x1p-54f : 1.0f;
// one pair of exponentials in 2 kPolyEvery goes to the FMA pipe
constexpr int kPolyEvery = 4;

struct PrefixParams {
    const uint8_t* q_img;                    // [Hk n_rt][RG] 128-row operand tiles, from query_kernel
    const uint8_t* codes;                    // OWN: [Hk][rows_pad][D]
    const float* q_scale;                    // [Hk][rows_pad]
    const float* ksc;
    const float* vsc;
    int per_tensor, v_trans;
    const uint8_t* ksf8;
    const uint8_t* vsf8;
    const int32_t* ptab;
    const int32_t* plen;
    const int32_t* ctx;
    FastDiv div_r, div_g;
    int T, Hk, R, n_rows, rows_pad, page, lg_page, max_pages, cap_prefix, cap_rows, num_pages, window, np, n_rt;
    float logit_scale_log2;
    float2* stat;                            // [Hk n_rt][np][128 RG]; OWN: [B Hk][np][64]
    float* o;                                // [Hk n_rt][np][D / 4][128 RG][4]; OWN: [B Hk][np][D / 4][64][4]
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
    static constexpr int kVb = kKb + kKbBuf;                         // [2] V, fp16 (MX: bf16), D / 64 atoms [128][128 B]
    static constexpr int kVbBuf = kKeys * 2 * D;
    static constexpr int kScale = kVb + 2 * kVbBuf;                  // [slot] k [128] fp32, v [128] fp16
    static constexpr int kScSlot = MX ? 0 : kKeys + kKeys / 2;
    static constexpr int kMeta = kScale + kScStages * kScSlot * 4;   // [slot] bad-page mask; exponent of the value scales
    static constexpr int kSpan = kMeta + 2 * kScStages * 4;              // [8 warps] lowest, highest key any row sees
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

// D[tmem] (+)= A[tmem] * B[smem], fp16 or bf16 (both operands the same, as idesc
// says) -> fp32 (A: lane = row, a 32-bit column two consecutive keys).
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
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

// OWN (RG = 1): a sequence's own keys instead, its rows (more than 32 of them)
// in the lower half of the tile, on a grid [B Hk][splits]; launched behind the
// prefix's kernel, of which it reads nothing.
template <int D, bool MX, int RG, bool OWN>
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
    const int split = blockIdx.x, seq = OWN ? blockIdx.y / p.Hk : 0;
    const int hk = OWN ? blockIdx.y - seq * p.Hk : blockIdx.y / p.n_rt;
    const int row0 = OWN ? seq * p.R : blockIdx.y % p.n_rt * kRowsCta, row_end = OWN ? row0 + p.R : p.n_rows;
    constexpr int kRowsOut = OWN ? 64 : kRowsCta;    // of a partial
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kMmaWarp1) {
        for (int i = lane; i < Sm::kNumBars; i += 32) {
            uint32_t cnt = 1;                                                          // expect_tx; commits
            if (i >= Sm::kKvEmpty && i < Sm::kKvEmpty + kStages) cnt = MX ? 4 : RG + 4; // (QK commits +) converters
            if (i >= Sm::kPReady && i < Sm::kPReady + 4) cnt = 4;                      // softmax group
            if (i >= Sm::kVReady && i < Sm::kVReady + 2) cnt = 4;                      // converters
            if (i >= Sm::kScFull && i < Sm::kScFull + kScStages) cnt = 32;
            if (i >= Sm::kScEmpty && i < Sm::kScEmpty + kScStages) cnt = 4 * RG + (MX ? 0 : 4);   // softmax groups, converters
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
    if (!OWN) pdl_wait();
    pdl_launch_dependents();

    // what the set-up reads, requested together: the length, and the softmax
    // thread's row
    int L = *p.plen;
    const int g = (warp >> 2) & 1;
    const int r = RG == 2 ? (tid & 255) : (tid & 127);
    const int n = row0 + r;
    const bool rv = n < row_end;
    int ctx = 0;
    float q_scale = 0.0f;
    if (warp < 8 && rv) {
        ctx = __ldg(p.ctx + fast_div(n, p.div_r));
        q_scale = __ldcg(p.q_scale + (size_t)hk * p.rows_pad + n);
    }
    const float ks_t = !MX && p.per_tensor ? __ldg(p.ksc) : 1.0f, vs_t = !MX && p.per_tensor ? __ldg(p.vsc) : 1.0f;
    if (L > p.cap_prefix || L < 0) {
        if (tid == 0 && split == 0) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
        L = max(0, min(L, p.cap_prefix));
    }
    if constexpr (OWN) {
        if (tid == 0 && split == 0 && (ctx < 0 || ctx > p.cap_rows)) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
        // the query operand, from the codes (a tile's image has its rows elsewhere)
        for (int idx = tid; idx < p.R * (D / 16); idx += kThreads) {
            const int row = idx / (D / 16), ch = idx % (D / 16);
            const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p.codes + ((size_t)hk * p.rows_pad + row0 + row) * D) + ch);
            if constexpr (MX) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int k8 = 2 * ch + hh;
                    const uint32_t wa = hh ? u.z : u.x, wb = hh ? u.w : u.y;
                    *reinterpret_cast<uint4*>(sm + Sm::kQ + (k8 >> 3) * (128 * 128) + row * 128 + (((k8 & 7) ^ (row & 7)) << 4)) =
                        make_uint4(e4m3_pick_to_bf16x2<0>(wa, wb), e4m3_pick_to_bf16x2<1>(wa, wb),
                                   e4m3_pick_to_bf16x2<2>(wa, wb), e4m3_pick_to_bf16x2<3>(wa, wb));
                }
            } else {
                *reinterpret_cast<uint4*>(sm + Sm::kQ + row * D + (e4m3_chunk<D>(ch, row) << 4)) = u;
            }
        }
        fence_proxy_async_smem();
    }
    // the keys of the part that the row sees
    int key_lo = INT32_MAX, key_hi = -1;
    if (warp < 8 && rv) {
        const int pq = max(0, min(ctx, p.cap_rows)) - p.T + fast_div(n - fast_div(n, p.div_r) * p.R, p.div_g);
        key_lo = max(OWN ? L : 0, pq - p.window + 1);
        key_hi = OWN ? pq : min(pq, L - 1);
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
    int tb, te;
    share_out(n_all, used_splits(n_all, p.np, RG == 1 ? 1 : 0), split, tb, te);
    const int nt = te - tb;
    tb += t0;
    // keys that are there: the prefix's, or those that a row sees (a sequence's
    // pages may hold anything below L)
    const int there = OWN ? lo : 0, gone = OWN ? hi + 1 : L;
    const int32_t* ptab = p.ptab + (OWN ? (int64_t)seq * p.max_pages : 0);
    const int ppt = kKeys / p.page;
    const size_t part = (size_t)blockIdx.y * p.np + split;

    if (warp >= kTmaWarp) {
      reg_dealloc<kRegsProd>();
      if (warp == kTmaWarp || warp == kScaleWarp) {
        // ------------------------------------------------------------ producers
        // (as decode.cu's: lane j of chunk c looks up page 32 c + j of the
        // CTA's pages; a page that holds no key of the part is not looked up)
        const bool kv = warp == kTmaWarp;
        int chunk = -1, phys = 0, issued = 0, vexp = kNoExp;
        bool bad = false, found = false;
        if (OWN && kv && lane == 0 && nt > 0) mbar_arrive(&bars[Sm::kQReady]);
        if (!OWN && kv && lane == 0 && nt > 0) {
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
                bad = found = false;
                if (lp < (tb + nt) * ppt && lp * p.page < gone && (!OWN || (lp + 1) * p.page > there)) {
                    const int pg = __ldg(ptab + lp);
                    if (pg < 0 || pg >= p.num_pages) {
                        bad = true;
                        if (kv) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
                    } else {
                        phys = pg;
                        found = true;
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
                    // FP8: a page without a key of the part, or off the cache, is read
                    // as zeros (a coordinate off the map): what its stand-in holds
                    // could be NaN codes, which a weight of zero does not cancel
                    const int z = MX || found ? phys * p.Hk + hk : -1, q = lane - slot0;
                    constexpr int kRowB = Sm::kKStage / kKeys;
                    for (int y = 0; y < p.page; y += 64) {                   // boxes of at most 64 rows
                        const int at = s * Sm::kKStage + (q * p.page + y) * kRowB;
                        tma_load_3d(sm + Sm::kK + at, &tmK, &bars[Sm::kKvFull + s], 0, y, z);
                        if (!p.v_trans) tma_load_3d(sm + Sm::kV + at, &tmV, &bars[Sm::kKvFull + s], 0, y, z);
                    }
                    if (p.v_trans) tma_load_3d(sm + Sm::kV + s * Sm::kKStage, &tmV, &bars[Sm::kKvFull + s], 0, 0, z);
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
                if (lane == 0) meta[c] = static_cast<int>(badm);
                if (MX || p.per_tensor) {
                    if (lane == 0) meta[kScStages + c] = 0;
                    mbar_arrive(&bars[Sm::kScFull + c]);
                } else {
                    // keys 4 lane .. 4 lane + 3: k_scale, and v_scale relative to
                    // 2^vexp, zero where the slot holds no key of the part
                    float ks[4], vs[4];
                    const int pq = __shfl_sync(0xffffffffu, phys, slot0 + 4 * lane / p.page);
                    const int64_t src = ((int64_t)pq * p.Hk + hk) * p.page + (4 * lane) % p.page;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ks[e] = __ldg(p.ksc + src + e);
                        vs[e] = __ldg(p.vsc + src + e);
                    }
                    const int key = (tb + i) * kKeys + 4 * lane;
                    const bool off_page = (badm >> (4 * lane / p.page)) & 1;
                    float vmax = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (key + e < lo || key + e > hi || off_page) vs[e] = 0.0f;
                        vmax = fmaxf(vmax, vs[e]);
                    }
                    // (a scale is not negative: its bits order like its value)
                    vexp = scale_exp(vexp, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vmax))));
                    const float f = vexp == kNoExp ? 0.0f : pow2i(-vexp);
                    float* dst = scl + c * Sm::kScSlot + 4 * lane;
                    *reinterpret_cast<float4*>(dst) = make_float4(ks[0], ks[1], ks[2], ks[3]);
                    *reinterpret_cast<uint2*>(scl + c * Sm::kScSlot + kKeys + 2 * lane) =
                        make_uint2(f16x2(vs[0] * f, vs[1] * f), f16x2(vs[2] * f, vs[3] * f));
                    if (lane == 0) meta[kScStages + c] = vexp;
                    mbar_arrive(&bars[Sm::kScFull + c]);
                }
            }
            issued = i + 1;
        }
        // no copy of this CTA may land after it exits
        if (kv) {
            if (nt > 0) mbar_wait_drain(&bars[Sm::kQReady], 0);
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait_drain(&bars[Sm::kKvFull + i % kStages], (i / kStages) & 1);
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
            const uint32_t idesc_pv = umma_idesc(1, MX ? 1 : 0, 128, D) | (p.v_trans ? 0u : 1u << 16);   // bf16 | fp16; V: B MN-major
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
                            mma_f16_ts(to, ts + 64 * h + 8 * st, vd + st * vstep, idesc_pv,
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
        const float cq = fmaxf(q_scale * p.logit_scale_log2 * ks_t, FLT_MIN);
        const uint64_t cq2 = f2_pack(cq, cq);
        const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t to = trow + kOCol + 128 * g;
        const bool idle = __all_sync(0xffffffffu, !rv);      // 32 rows of padding: the warp only keeps time
        const bool tensor = MX || p.per_tensor;              // logits without a scale of their own
        // A row starts from m = 0, which holds for its first maximum too unless
        // that is far off; l = 0 says that it has seen no key.
        float m_run = 0.0f;
        uint64_t l2 = f2_pack(0.0f, 0.0f);
        int vexp = kNoExp;                           // FP8: O is in units of 2^vexp
        bool ok = true;
        const int my_units = RG == 2 ? 2 * nt : 2 * ((nt - g + 1) / 2);
        for (int k = 0; k < my_units; ++k) {
            const int h = k & 1, i = RG == 2 ? k >> 1 : 2 * (k >> 1) + g, c = i % kScStages;
            const uint32_t ts = trow + 64 * (2 * g + h);
            ok = warp_all(mbar_wait(&bars[Sm::kSFull + 2 * g + h], (k >> 1) & 1, abort_flag, &g_shared_err, 8));
            if (!ok) break;
            if (h == 0) ok = warp_all(mbar_wait(&bars[Sm::kScFull + c], (i / kScStages) & 1, abort_flag, &g_shared_err, 9));
            if (!ok) break;
            if (!idle) {
                // (behind the wait for the scales: before it, or before the last
                // unit's sum is checked, the loads measured 4 to 7 % slower)
                uint32_t x0[32], x1[32];
                tc_fence_after();
                const int key0 = (tb + i) * kKeys + 64 * h;
                const int badm = meta[c];
                const float4* ks = reinterpret_cast<const float4*>(scl + c * Sm::kScSlot + 64 * h);
                // y = S k_scale of keys 4 q .. 4 q + 3 of 32 loaded columns
                auto scaled = [&](bool plain, const uint32_t (&x)[32], int cc, int q, uint64_t& y01, uint64_t& y23) {
                    y01 = f2_pack(__uint_as_float(x[4 * q]), __uint_as_float(x[4 * q + 1]));
                    y23 = f2_pack(__uint_as_float(x[4 * q + 2]), __uint_as_float(x[4 * q + 3]));
                    if (!plain) {
                        const float4 s = ks[8 * cc + q];
                        y01 = f2_mul(y01, f2_pack(s.x, s.y));
                        y23 = f2_mul(y23, f2_pack(s.z, s.w));
                    }
                };
                // two words of P from the logits' base-2 exponents; l += p (a
                // masked key's exponent is -inf, which only MUFU makes exactly 0)
                auto weigh = [&](auto masked, uint64_t e01, uint64_t e23, int q, uint64_t& l, uint32_t* w) {
                    float a, b, p0, p1, p2, p3;
                    f2_unpack(e01, a, b);
                    if (!decltype(masked)::value && q % kPolyEvery == kPolyEvery - 1) {
                        exp2_poly_x2(fminf(a, 127.0f), fminf(b, 127.0f), p0, p1);
                    } else {
                        p0 = ex2_approx(a);
                        p1 = ex2_approx(b);
                    }
                    f2_unpack(e23, a, b);
                    p2 = ex2_approx(a);
                    p3 = ex2_approx(b);
                    l = f2_add(l, f2_add(f2_pack(p0, p1), f2_pack(p2, p3)));
                    w[2 * q] = MX ? bf16x2(p0, p1) : f16x2(p0, p1);
                    w[2 * q + 1] = MX ? bf16x2(p2, p3) : f16x2(p2, p3);
                };
                // Most units are wholly seen, or not at all, by every row and
                // raise no row's maximum by much, so their weights are computed
                // against the running one, and their sum tells whether that was
                // right: no weight is above 2^8 where 64 of them add up to no
                // more. Where the unit turns out to need its own maximum,
                // nothing of the pass is kept.
                const int ve = MX ? 0 : meta[kScStages + c];
                if (vexp == kNoExp) vexp = ve;               // (no key before: O holds zeros)
                const bool none = key_hi < key0 || key_lo > key0 + 63, all = key_lo <= key0 && key_hi >= key0 + 63;
                bool slow = ve != vexp || badm != 0 || key0 + 63 >= gone || (OWN && key0 < there) || !__all_sync(0xffffffffu, none || all);
                tmem_ld64_wait(ts, x0, x1);
                auto fast = [&](auto plain) {
                    const uint64_t nsub2 = f2_pack(-m_run, -m_run);
                    uint64_t lu[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
                    uint32_t w[2][16];
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            uint64_t y01, y23;
                            scaled(decltype(plain)::value, cc == 0 ? x0 : x1, cc, q, y01, y23);
                            weigh(std::false_type{}, f2_fma(y01, cq2, nsub2), f2_fma(y23, cq2, nsub2), q, lu[q & 1], w[cc]);
                        }
                    }
                    const uint64_t lsum = f2_add(lu[0], lu[1]);
                    float a, b;
                    f2_unpack(lsum, a, b);
                    a += b;
                    slow = __any_sync(0xffffffffu, all && (a > kMaxSum || (l2 == 0 && a < kMinSum<MX>)));
                    if (!slow) {
                        if (__any_sync(0xffffffffu, none)) {
#pragma unroll
                            for (int q = 0; q < 32; ++q) w[q / 16][q % 16] = none ? 0u : w[q / 16][q % 16];
                        }
                        if (!none) l2 = f2_add(l2, lsum);
                        tmem_st16(ts, w[0]);
                        tmem_st16(ts + 16, w[1]);
                    }
                };
                if (!slow) {
                    if (tensor) fast(std::true_type{});
                    else fast(std::false_type{});
                }
                if (slow) {
                    const int clo = key_lo - key0, chi = key_hi - key0;
                    uint64_t y[32];
                    float mx = -INFINITY;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t x[32];
                        tmem_ld32_wait(ts + 32 * cc, x);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            scaled(tensor, x, cc, q, y[16 * cc + 2 * q], y[16 * cc + 2 * q + 1]);
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
                    if (l2 == 0) {
                        if (mx > -INFINITY) m_run = mx;       // its first key (O is zero)
                    } else if (mx > m_run + kRaise) {
                        alpha = ex2_approx(m_run - mx);
                        l2 = f2_mul(l2, f2_pack(alpha, alpha));
                        m_run = mx;
                    }
                    if (ve != vexp) {
                        alpha *= pow2i(vexp - ve);
                        vexp = ve;
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
                    const uint64_t nsub2 = f2_pack(-m_run, -m_run);
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t w[16];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            weigh(std::true_type{}, f2_fma(y[16 * cc + 2 * q], cq2, nsub2),
                                  f2_fma(y[16 * cc + 2 * q + 1], cq2, nsub2), q, l2, w);
                        tmem_st16(ts + 16 * cc, w);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
            }
            if (!ok) break;
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
        if (!ok || l == 0.0f) {                      // (no key seen)
            m_run = -INFINITY;
            l = 0.0f;
        }
        const float unit = MX || vexp == kNoExp ? 1.0f : vs_t * pow2i(vexp);
        tc_fence_after();
        // four channels, of columns j .. of O (MX: the eight columns of a group
        // hold channels 0 4 1 5 2 6 3 7)
        float4* po = reinterpret_cast<float4*>(p.o) + part * (D / 4) * kRowsOut + r;
        auto put = [&](int col, const float (&y)[32]) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                po[(col + j) / 4 * kRowsOut] = MX ? make_float4(y[j], y[j + 2], y[j + 4], y[j + 6])
                                                  : make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                po[((col + j) / 4 + 1) * kRowsOut] = MX ? make_float4(y[j + 1], y[j + 3], y[j + 5], y[j + 7])
                                                        : make_float4(y[j + 4], y[j + 5], y[j + 6], y[j + 7]);
            }
        };
        if constexpr (RG == 2) {
            p.stat[part * kRowsCta + r] = make_float2(m_run, l);
            if (my_units > 0 && !idle) {
#pragma unroll
                for (int hf = 0; hf < D / 32; ++hf) {
                    uint32_t o[32];
                    tmem_ld32_wait(to + 32 * hf, o);
                    float y[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(o[j]) * unit;
                    put(32 * hf, y);
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
                    tmem_ld32_wait(to + give + 32 * hf, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) xo[(give + 32 * hf + j) * 128 + r] = __uint_as_float(o[j]) * unit;
                }
            }
            named_sync(1, 256);
            const float2 other = xs[128 * (1 - g) + r];
            const float M = fmaxf(m_run, other.x);
            const float wa = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - M);
            const float wb = other.x == -INFINITY ? 0.0f : ex2_approx(other.x - M);
            if (g == 0 && r < kRowsOut) p.stat[part * kRowsOut + r] = make_float2(M, wa * l + wb * other.y);
            if (nt > 0 && !idle) {
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    uint32_t o[32];
                    tmem_ld32_wait(to + keep + 32 * hf, o);
                    float y[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        // (a group without a key in the row has no O)
                        y[j] = m_run == -INFINITY ? 0.0f : wa * unit * __uint_as_float(o[j]);
                        if (other.x != -INFINITY) y[j] = fmaf(wb, xo[(keep + 32 * hf + j) * 128 + r], y[j]);
                    }
                    put(keep + 32 * hf, y);
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
                // V^T: 16 keys of a channel) -> two chunks of the fp16 row;
                // slots without a key of the part count as zeros, the others'
                // scales (relative to 2^vexp, rounded to fp16) are multiplied in
                const int c8 = i % kScStages;
                if (!warp_all(mbar_wait(&bars[Sm::kScFull + c8], (i / kScStages) & 1, abort_flag, &g_shared_err, 16))) break;
                const uint8_t* vsc = reinterpret_cast<const uint8_t*>(scl + c8 * Sm::kScSlot + kKeys);
                const uint32_t vs_row = p.per_tensor || p.v_trans
                                            ? 0u : 0x10001u * *reinterpret_cast<const uint16_t*>(vsc + 2 * row);
                const int left = gone - (tb + i) * kKeys, skip = OWN ? there - (tb + i) * kKeys : 0;   // keys [skip, left)
                auto convert = [&](auto width_c, auto trans_c, int atom_b) {
                    constexpr bool kTrans = decltype(trans_c)::value;
                    constexpr int kWidth = decltype(width_c)::value;
                    const uint8_t* vrow = sm + Sm::kV + s * Sm::kKStage + row * kWidth;
                    uint4 u[kWidth / 16];
#pragma unroll
                    for (int c = 0; c < kWidth / 16; ++c)
                        u[c] = *reinterpret_cast<const uint4*>(vrow + (e4m3_chunk<kWidth>(c, row) << 4));
                    if (left < kKeys || (OWN && skip > 0)) {
#pragma unroll
                        for (int c = 0; c < kWidth / 16; ++c) {
                            const int n = kTrans ? left - 16 * c : (row < left && row >= skip ? 16 : 0);
                            const int m = OWN && kTrans ? skip - 16 * c : 0;
                            u[c].x &= low_bytes(n) & ~low_bytes(m);
                            u[c].y &= low_bytes(n - 4) & ~low_bytes(m - 4);
                            u[c].z &= low_bytes(n - 8) & ~low_bytes(m - 8);
                            u[c].w &= low_bytes(n - 12) & ~low_bytes(m - 12);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kWidth / 16; ++c) {
                        uint8_t* at = dst + (c >> 2) * atom_b;
                        const int ch = 2 * (c & 3);
                        uint32_t f[8] = {e4m3_lo_to_f16x2(u[c].x), e4m3_hi_to_f16x2(u[c].x), e4m3_lo_to_f16x2(u[c].y),
                                         e4m3_hi_to_f16x2(u[c].y), e4m3_lo_to_f16x2(u[c].z), e4m3_hi_to_f16x2(u[c].z),
                                         e4m3_lo_to_f16x2(u[c].w), e4m3_hi_to_f16x2(u[c].w)};
                        if (!p.per_tensor) {
                            uint32_t v8[8];
                            if (kTrans) {
                                const uint4 a = *reinterpret_cast<const uint4*>(vsc + 32 * c);
                                const uint4 b = *reinterpret_cast<const uint4*>(vsc + 32 * c + 16);
                                v8[0] = a.x, v8[1] = a.y, v8[2] = a.z, v8[3] = a.w;
                                v8[4] = b.x, v8[5] = b.y, v8[6] = b.z, v8[7] = b.w;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = f16x2_mul(f[e], kTrans ? v8[e] : vs_row);
                        }
                        *reinterpret_cast<uint4*>(at + ((ch ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                };
                if (p.v_trans) {
                    if (row < D) convert(std::integral_constant<int, kKeys>{}, std::true_type{}, D * 128);
                } else {
                    convert(std::integral_constant<int, D>{}, std::false_type{}, kKeys * 128);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[Sm::kVReady + vb]);
                mbar_arrive(&bars[Sm::kKvEmpty + s]);
                if (!MX) mbar_arrive(&bars[Sm::kScEmpty + i % kScStages]);
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
    if (OWN) pdl_wait();                             // this grid ends after the one before it
}

// -------------------------------------------------------------- few rows

// Up to 64 query rows against a run of keys: a sequence's own rows against its
// own keys [L, ctx), and, where the whole batch has no more rows than that,
// all rows against the prefix. With 16 rows a key costs 4 D FLOPs a byte of
// cache, far from what a tensor pipe is bound by; what counts is latency and
// bytes in flight. So no TMEM and no roles: a warp takes 16 rows and 64 keys
// at a time through mma fragments (FP8: fp16, MXFP4: bf16, both exact), and
// two or three CTAs of four independent warps share an SM.
// One lane copies a warp's blocks (a TMA box of K or V per page, scales by
// cp.async): the next block's K is on its way while this one's softmax and PV
// run, the next V while the next QK runs, one stage of each being enough.
// Pages without a key are read as zeros (a coordinate off the map), and the
// slots of V without a key are zeroed: a NaN code there must not meet a weight
// of zero. A call is latency, not throughput: one block a warp and straight
// code, so what counts is how few instructions there are, at 4 to 7 cycles
// each. (With the fragments loaded straight from global memory, or with 16-byte
// cp.async, 64-bit divisions and a rolled epilogue, a call took 19000 cycles
// for one block a warp; decode.cu's kernel, one CTA an SM, 27 us for 256
// sequences of at most 512 own keys.)
// Fragments. The order of the summed index is free as long as both operands
// have the same, and so is the order of output columns; with thread (g, c) =
// (lane / 4, lane % 4):
//   S = Q K^T  summed index: thread c holds the run d = c D / 4 .. of its key
//              (16 or 32 contiguous bytes), 4 elements a step; column n of
//              n-tile j is key 8 j + n, or, over a transposed V, key
//              16 (n / 2) + 2 j + n % 2, so that thread c's columns are the 16
//              consecutive keys 16 c ..
//   O = P V    step s of 16 keys = n-tiles 2 s and 2 s + 1, whose S registers
//              are P's A operand; thread (g, c) holds V of the keys of its S
//              columns (V^T: four bytes of a 16-byte run) and channels
//              D g / 8 .., one per n-tile, converted exactly in registers.
// With the boxes' swizzles these reads take every bank once, those of a
// 64-byte V row (V^T) twice.
constexpr int kRowsWarps = 4;

// log2 of the key slices that its four warps make with this many rows
__host__ __device__ inline int lg_slices(int rows) { return rows <= 16 ? 2 : (rows <= 32 ? 1 : 0); }

struct RowsParams {
    const uint8_t* q8;                       // [Hk][rows_pad][D] e4m3 codes
    const float* q_scale;                    // [Hk][rows_pad]
    const uint16_t* q;                       // or (q8 null) the queries, which every CTA quantises for its rows
    int64_t qs0, qs1, qs2, qs3;
    int q_vec;
    const float* ksc;
    const float* vsc;
    const uint8_t* ksf;
    const uint8_t* vsf;
    int per_tensor;
    const int32_t* ptab;                     // [B, max_pages]
    const int32_t* prefix;
    const int32_t* plen;
    const int32_t* ctx;
    int B, T, Hk, G, R, n_rows, rows_pad, lg_page, max_pages, cap_prefix, num_pages, window;
    int np, ns;                              // splits of the prefix part (0: not here), of a sequence's own
    FastDiv div_np, div_ns, div_hk, div_r, div_g;
    float logit_scale_log2;
    float2* pre_stat;                        // [Hk][np][64]
    float* pre_o;                            // [Hk][np][D / 4][64][4]
    float2* own_stat;                        // [B Hk][ns][64]
    float* own_o;
    int late_wait;                           // launched behind prefix_kernel, of which it reads nothing
};

template <int D, bool MX, bool VT>
struct SmR {
    static constexpr int kSteps = D / 16;                            // QK steps
    static constexpr int kRow = MX ? D / 2 : D;                      // bytes of a cache row
    static constexpr int kPitch = 17;                                // rows of a staged O
    static constexpr int kKBytes = kBlk * kRow, kVBytes = VT ? D * kBlk : kBlk * kRow;
    // a warp's K and V, later its O; then all warps' scales [k | v][64]
    static constexpr int kStage = al1024(kKBytes + kVBytes > D * kPitch * 4 ? kKBytes + kVBytes : D * kPitch * 4);
    static constexpr int kScale = kRowsWarps * kStage;
    static constexpr int kStat = kScale + kRowsWarps * 2 * 4 * kBlk;
    static constexpr int kSpan = kStat + kRowsWarps * 16 * 8;        // lowest, highest key any row sees
    static constexpr int kQs = kSpan + 8;                            // [64] query scales
    static constexpr int kBar = kQs + 64 * 4;                        // [warp][k | v], then [warp] abort flags
    static constexpr int kQf = (kBar + kRowsWarps * 20 + 15) & ~15;  // [m-tile][step][lane] query fragments
    // with m-tiles of 16 rows; three CTAs an SM with one, two with more
    static constexpr int bytes(int mts) { return 1024 + kQf + mts * kSteps * 32 * 16; }
    static_assert(kKBytes % 1024 == 0 && kBar % 8 == 0, "alignment");
    static_assert(3 * (bytes(1) + 1024) <= 228 * 1024 && 2 * (bytes(4) + 1024) <= 228 * 1024, "CTAs an SM");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// A copy of 4 bytes, the destination zeroed instead where !in.
__device__ __forceinline__ void cp_async_4_or_zero(void* dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool MX, bool VT>
__global__ void __launch_bounds__(32 * kRowsWarps, 3)
    rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const RowsParams p) {
    using Sm = SmR<D, MX, VT>;
    constexpr int kSteps = Sm::kSteps, kRow = Sm::kRow, kPitch = Sm::kPitch;
    constexpr int kNt = D / 8;                   // n-tiles of O = channels a thread has of a V row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    uint8_t* st = sm + warp * Sm::kStage;
    float* sc = reinterpret_cast<float*>(sm + Sm::kScale) + warp * 2 * kBlk;
    uint4* qf = reinterpret_cast<uint4*>(sm + Sm::kQf);
    auto stat_s = reinterpret_cast<float2(*)[16]>(sm + Sm::kStat);
    int* span = reinterpret_cast<int*>(sm + Sm::kSpan);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Sm::kBar) + 2 * warp;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Sm::kBar + kRowsWarps * 16) + warp;
    if (lane == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (!p.late_wait) pdl_wait();
    pdl_launch_dependents();

    const bool pre = (int)blockIdx.x < p.np * p.Hk;
    const int bi = pre ? blockIdx.x : blockIdx.x - p.np * p.Hk;
    const int nsplit = pre ? p.np : p.ns;
    const int item = fast_div(bi, pre ? p.div_np : p.div_ns), split = bi - item * nsplit;
    const int b = pre ? 0 : fast_div(item, p.div_hk), hk = item - b * p.Hk;
    const int rows = pre ? p.n_rows : p.R;
    const int n0 = b * p.R;                                   // first row (pre: b = 0)
    // warps: m-tile (16 rows) x key slice
    const int mts = (rows + 15) >> 4, lg_s = lg_slices(rows), slices = 1 << lg_s;
    const int mt = warp >> lg_s, slice = warp & (slices - 1);
    const bool live = mt < mts;
    // everything the set-up reads, requested together
    int L = *p.plen;
    const int r0 = 16 * mt + g;
    int ctx[2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
        ctx[r] = pre ? (r0 + 8 * r < rows ? __ldg(p.ctx + fast_div(r0 + 8 * r, p.div_r)) : 0) : __ldg(p.ctx + b);
    uint4 u[2][D / 64];
    float cq[2];                                 // base-2 logit = (S k_scale) cq; > 0 keeps a masked -inf
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const bool in = p.q8 != nullptr && live && r0 + 8 * r < rows;
        const size_t n = (size_t)hk * p.rows_pad + n0 + r0 + 8 * r;
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
            u[r][k] = in ? __ldcg(reinterpret_cast<const uint4*>(p.q8 + n * D + c * (D / 4)) + k)
                         : make_uint4(0u, 0u, 0u, 0u);
        cq[r] = in ? __ldcg(p.q_scale + n) : 0.0f;
    }
    const float ks_t = !MX && p.per_tensor ? __ldg(p.ksc) : 1.0f, vs_t = !MX && p.per_tensor ? __ldg(p.vsc) : 1.0f;

    if (L < 0 || L > p.cap_prefix) {
        if (tid == 0 && split == 0) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
        L = max(0, min(L, p.cap_prefix));
    }
    const int cap = p.max_pages << p.lg_page;
    if (!pre && tid == 0 && split == 0 && (ctx[0] < 0 || ctx[0] > cap)) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
    // keys that rows r0 and r0 + 8 see of this part
    int klo[2], khi[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        klo[r] = INT32_MAX;
        khi[r] = -1;
        if (r0 + 8 * r < rows) {
            ctx[r] = max(0, min(ctx[r], cap));
            const int n = r0 + 8 * r, rr = pre ? n - fast_div(n, p.div_r) * p.R : n;
            const int pq = ctx[r] - p.T + fast_div(rr, p.div_g);
            const int a = max(pre ? 0 : L, pq - p.window + 1), e = pre ? min(pq, L - 1) : pq;
            if (e >= a) {
                klo[r] = a;
                khi[r] = e;
            }
        }
    }
    // [lo, hi]: keys that any row sees (a sequence's T rows see all of its keys
    // from the first one's window on)
    int lo, hi, blk0, n_all;
    if (pre) {
        if (tid == 0) {
            span[0] = INT32_MAX;
            span[1] = -1;
        }
        __syncthreads();
        lo = __reduce_min_sync(0xffffffffu, live ? min(klo[0], klo[1]) : INT32_MAX);
        hi = __reduce_max_sync(0xffffffffu, live ? max(khi[0], khi[1]) : -1);
        if (lane == 0) {
            atomicMin(span, lo);
            atomicMax(span + 1, hi);
        }
        __syncthreads();
        lo = span[0];
        hi = span[1];
        blk0 = hi >= 0 ? lo / kBlk : 0;
        n_all = hi >= 0 ? hi / kBlk + 1 - blk0 : 0;
    } else {
        own_keys(max(0, min(ctx[0], cap)), L, p.T, p.window, 6, lo, hi, blk0, n_all);
    }
    int first, last;
    share_out(n_all, used_splits(n_all, nsplit, lg_s), split, first, last);
    first += blk0;
    last += blk0;
    const size_t part = (size_t)item * nsplit + split;
    float2* stat = (pre ? p.pre_stat : p.own_stat) + part * 64;
    float* out = (pre ? p.pre_o : p.own_o) + part * D * 64;
    if (first >= last) {                                      // (most CTAs of a short call)
        if (tid < rows) stat[tid] = make_float2(-INFINITY, 0.0f);
        if (p.late_wait) pdl_wait();
        return;
    }

    const int32_t* tab = pre ? p.prefix : p.ptab + (int64_t)b * p.max_pages;
    const int lgp = min(p.lg_page, 6);                        // keys of one page inside a block (log2)
    // Pages of a block, lane i holding page i: its number, or -1 where it holds
    // no key of [lo, hi] or is off the cache (bad)
    struct Pages {
        int k0, phys;
        bool bad;
    };
    auto lookup = [&](int blk) {
        Pages f{blk * kBlk, -1, false};
        const int lp = (f.k0 >> p.lg_page) + lane;
        if (lane < (kBlk >> lgp) && (lp << p.lg_page) <= hi && ((lp + 1) << p.lg_page) > lo) {
            f.phys = __ldg(tab + lp);
            f.bad = f.phys < 0 || f.phys >= p.num_pages;
        }
        return f;
    };
    // a block's K (V) codes and scales into the stage
    auto copy = [&](const Pages& f, bool v) {
        const bool found = f.phys >= 0 && !f.bad;
        const int in0 = f.k0 & ((1 << p.lg_page) - 1);        // block's offset in a larger page
        if (lane == 0) mbar_arrive_expect_tx(&bar[v], v ? Sm::kVBytes : Sm::kKBytes);
        __syncwarp();
        if (lane < (kBlk >> lgp)) {
            const int z = found ? f.phys * p.Hk + hk : -1;
            uint8_t* dst = st + (v ? Sm::kKBytes : 0) + (lane << lgp) * kRow;
            if (VT && v) tma_load_3d(dst, &tmV, &bar[1], in0, 0, z);
            else tma_load_3d(dst, v ? &tmV : &tmK, &bar[v], 0, in0, z);
        }
        if (MX || !p.per_tensor) {
            const uint8_t* src = MX ? (v ? p.vsf : p.ksf) : reinterpret_cast<const uint8_t*>(v ? p.vsc : p.ksc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int o = lane + 32 * i;
                const int pg = __shfl_sync(0xffffffffu, found ? f.phys : -1, o >> lgp);
                const int64_t t = (((int64_t)max(pg, 0) * p.Hk + hk) << p.lg_page) + in0 + (o & ((1 << lgp) - 1));
                cp_async_4_or_zero(sc + (v ? kBlk : 0) + o, src + 4 * t, pg >= 0 && f.k0 + o >= lo && f.k0 + o <= hi);
            }
        }
        cp_async_commit();
    };
    uint32_t phase[2] = {0, 0};
    bool ok = true;
    int landing = 0;                                          // copies in flight: 1 K, 2 V
    // K (V) of the present block has landed
    auto landed = [&](int v) {
        ok = warp_all(mbar_wait(&bar[v], phase[v], abort_flag, &g_shared_err, 15));
        if (!ok) return;
        phase[v] ^= 1;
        landing &= ~(1 << v);
        cp_async_wait<1>();
        __syncwarp();
    };
    Pages pg = {0, -1, false};
    __syncwarp();
    if (live && first + slice < last) {
        pg = lookup(first + slice);
        copy(pg, false);
        copy(pg, true);
        landing = 3;
    }
    // the query codes as A fragments in shared memory, thread (g, c) holding the
    // run c D / 4 .. of rows g and g + 8: their exact fp16 values (an e4m3
    // mma.sync is made of conversions and fp16 products on this machine, the
    // queries' anew for every key tile); for an MXFP4 cache bf16, pairs
    // (m, m + 4) of eight channels as e2m1_block_to_bf16 orders K's
    float* qs = reinterpret_cast<float*>(sm + Sm::kQs);
    if (p.q8 == nullptr) {
        // four threads a row, which write what the other branch writes below
        const int qq = tid & 3;
        for (int rr = tid >> 2; (rr & ~7) < 16 * mts; rr += 8 * kRowsWarps) {
            const int n = rr < rows ? n0 + rr : n0, bb = pre ? fast_div(n, p.div_r) : b, ro = n - bb * p.R;
            const int t = fast_div(ro, p.div_g);
            uint32_t w[kSteps];
            const float x = quantise_quarter<D>(p.q + bb * p.qs0 + t * p.qs1 + (int64_t)(hk * p.G + ro - t * p.G) * p.qs2 +
                                                    (int64_t)(qq * (D / 4)) * p.qs3, p.qs3, p.q_vec, qq, w);
            if (qq == 0) qs[rr] = rr < rows ? x : 0.0f;
            uint32_t* dst = reinterpret_cast<uint32_t*>(qf + ((rr >> 4) * kSteps * 32 + 4 * (rr & 7) + qq)) + ((rr >> 3) & 1);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                uint32_t a, c2;
                if constexpr (MX) {
                    const uint32_t wa = w[s & ~1], wb = w[s | 1];
                    a = (s & 1) ? e4m3_pick_to_bf16x2<2>(wa, wb) : e4m3_pick_to_bf16x2<0>(wa, wb);
                    c2 = (s & 1) ? e4m3_pick_to_bf16x2<3>(wa, wb) : e4m3_pick_to_bf16x2<1>(wa, wb);
                } else {
                    a = e4m3_lo_to_f16x2(w[s]);
                    c2 = e4m3_hi_to_f16x2(w[s]);
                }
                dst[s * 128] = rr < rows ? a : 0u;
                dst[s * 128 + 2] = rr < rows ? c2 : 0u;
            }
        }
    } else if (live && slice == 0) {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(u[0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(u[1]);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            uint4 a;
            if constexpr (MX) {
                const int k = s & ~1;
                if ((s & 1) == 0)
                    a = make_uint4(e4m3_pick_to_bf16x2<0>(w0[k], w0[k + 1]), e4m3_pick_to_bf16x2<0>(w1[k], w1[k + 1]),
                                   e4m3_pick_to_bf16x2<1>(w0[k], w0[k + 1]), e4m3_pick_to_bf16x2<1>(w1[k], w1[k + 1]));
                else
                    a = make_uint4(e4m3_pick_to_bf16x2<2>(w0[k], w0[k + 1]), e4m3_pick_to_bf16x2<2>(w1[k], w1[k + 1]),
                                   e4m3_pick_to_bf16x2<3>(w0[k], w0[k + 1]), e4m3_pick_to_bf16x2<3>(w1[k], w1[k + 1]));
            } else {
                a = make_uint4(e4m3_lo_to_f16x2(w0[s]), e4m3_lo_to_f16x2(w1[s]), e4m3_hi_to_f16x2(w0[s]),
                               e4m3_hi_to_f16x2(w1[s]));
            }
            qf[(mt * kSteps + s) * 32 + lane] = a;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (p.q8 == nullptr && live) cq[r] = qs[r0 + 8 * r];
        cq[r] = fmaxf(cq[r] * p.logit_scale_log2, FLT_MIN);
    }

    // key (of the block) of element x of this thread's pair in n-tile j
    auto key_of = [&](int j, int x) { return VT ? 16 * c + 2 * j + x : 8 * j + 2 * c + x; };
    float O[kNt][4];
#pragma unroll
    for (int t = 0; t < kNt; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[t][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int vexp = kNoExp;                                        // FP8: O is in units of 2^vexp
    for (int blk = first + slice; live && blk < last; blk += slices) {
        const int k0 = blk * kBlk;
        const bool more = blk + slices < last;
        Pages next = {0, -1, false};
        if (more) next = lookup(blk + slices);
        const unsigned badm = __ballot_sync(0xffffffffu, pg.bad);
        if (pg.bad) atomicCAS(&g_shared_err, 0u, kErrRangeCode);
        // ---- S = Q K^T
        landed(0);
        if (!ok) break;
        float S[8][4];
        constexpr int kAt = MX ? 2 : 4, kRun = MX ? 1 : D / 64;        // n-tiles at a time; 16-byte runs of a key
#pragma unroll
        for (int j0 = 0; j0 < 8; j0 += kAt) {
            uint32_t kb[kAt][MX ? 16 : 4 * kRun];
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int o = VT ? 16 * (g >> 1) + 2 * (j0 + j) + (g & 1) : 8 * (j0 + j) + g;
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    const uint4 x =
                        *reinterpret_cast<const uint4*>(st + o * kRow + (e4m3_chunk<kRow>(kRun * c + k, o) << 4));
                    if constexpr (MX) {
                        e2m1_block_to_bf16(x, reinterpret_cast<const uint8_t*>(sc)[4 * o + c], kb[j]);
                    } else {
                        kb[j][4 * k] = x.x;
                        kb[j][4 * k + 1] = x.y;
                        kb[j][4 * k + 2] = x.z;
                        kb[j][4 * k + 3] = x.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) S[j0 + j][e] = 0.0f;
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint4 a = qf[(mt * kSteps + s) * 32 + lane];
#pragma unroll
                for (int j = 0; j < kAt; ++j) {
                    if constexpr (MX) mma_16816(S[j0 + j], a, kb[j][2 * s], kb[j][2 * s + 1]);
                    else mma_16816_f16(S[j0 + j], a, e4m3_lo_to_f16x2(kb[j][s]), e4m3_hi_to_f16x2(kb[j][s]));
                }
            }
        }
        // ---- scales of keys 16 c .., masks, maxima
        if constexpr (!MX) {
            if (p.per_tensor) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[j][e] *= ks_t;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 s = *reinterpret_cast<const float2*>(sc + key_of(j, 0));
                    S[j][0] *= s.x;
                    S[j][1] *= s.y;
                    S[j][2] *= s.x;
                    S[j][3] *= s.y;
                }
            }
        }
        __syncwarp();
        if (more) {
            copy(next, false);                                // K's stage is free
            landing |= 1;
        } else {
            cp_async_commit();
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int a = klo[r] - k0, e = khi[r] - k0;       // key o of the block is seen for a <= o <= e
            if (!__all_sync(0xffffffffu, a <= 0 && e >= kBlk - 1 && badm == 0)) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int o = key_of(j, x);
                        if (o < a || o > e || ((badm >> (o >> lgp)) & 1)) S[j][2 * r + x] = -INFINITY;
                    }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; k += 2) mx = fmax3(mx, S[k >> 1][2 * r], S[k >> 1][2 * r + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = mx == -INFINITY ? -INFINITY : mx * cq[r];
            const bool raise = mx > m[r] + kLazyMax;          // (a first key too)
            const float alpha = raise && m[r] != -INFINITY ? ex2_approx(m[r] - mx) : 1.0f;
            if (raise) m[r] = mx;
            if (__any_sync(0xffffffffu, alpha != 1.0f)) {
                l[r] *= alpha;
#pragma unroll
                for (int t = 0; t < kNt; ++t) {
                    O[t][2 * r] *= alpha;
                    O[t][2 * r + 1] *= alpha;
                }
            }
            const float sub = m[r] == -INFINITY ? 0.0f : m[r];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float x = ex2_approx(fmaf(S[k >> 1][2 * r + (k & 1)], cq[r], -sub));
                l[r] += x;
                S[k >> 1][2 * r + (k & 1)] = x;
            }
        }
        landed(1);
        if (!ok) break;
        // slots of found pages that no row sees: zeros (of a transposed V, below)
        const bool edge = lo > k0 || hi < k0 + kBlk - 1;
        if (!MX && !VT && edge) {
            for (int o = lane; o < kBlk; o += 32)
                if (k0 + o < lo || k0 + o > hi) {
#pragma unroll
                    for (int i = 0; i < kRow / 16; ++i)
                        *reinterpret_cast<uint4*>(st + Sm::kKBytes + o * kRow + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                }
            fence_proxy_async_smem();                         // (before the next copy into the stage)
            __syncwarp();
        }
        if constexpr (!MX) {
            // value scales relative to 2^vexp (those of slots without a key are zero)
            float vs[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 x = p.per_tensor ? make_float2(vs_t, vs_t)
                                              : *reinterpret_cast<const float2*>(sc + kBlk + key_of(j, 0));
                vs[2 * j] = x.x;
                vs[2 * j + 1] = x.y;
            }
            float vmax = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; k += 2) vmax = fmax3(vmax, vs[k], vs[k + 1]);
            vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
            vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
            const int ne = scale_exp(vexp, vmax);
            if (ne != vexp) {
                if (vexp != kNoExp) {
                    const float f = pow2i(vexp - ne);
#pragma unroll
                    for (int t = 0; t < kNt; ++t)
#pragma unroll
                        for (int x = 0; x < 4; ++x) O[t][x] *= f;
                }
                vexp = ne;
            }
            const float f = vexp == kNoExp ? 0.0f : pow2i(-vexp);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                S[k >> 1][k & 1] *= vs[k] * f;
                S[k >> 1][2 + (k & 1)] *= vs[k] * f;
            }
        }
        // ---- O += P V
        if constexpr (VT) {
            uint4 pa[4];
#pragma unroll
            for (int s = 0; s < 4; ++s)
                pa[s] = make_uint4(f16x2(S[2 * s][0], S[2 * s][1]), f16x2(S[2 * s][2], S[2 * s][3]),
                                   f16x2(S[2 * s + 1][0], S[2 * s + 1][1]), f16x2(S[2 * s + 1][2], S[2 * s + 1][3]));
            // of keys 16 c .., no row sees those outside [va, ve]
            const int va = lo - k0 - 16 * c, ve = hi - k0 - 16 * c;
#pragma unroll
            for (int t = 0; t < kNt; ++t) {
                uint4 x = *reinterpret_cast<const uint4*>(st + Sm::kKBytes + (kNt * g + t) * kBlk +
                                                          (e4m3_chunk<64>(c, t) << 4));
                if (edge) {
                    x.x &= low_bytes(ve + 1) & ~low_bytes(va);
                    x.y &= low_bytes(ve - 3) & ~low_bytes(va - 4);
                    x.z &= low_bytes(ve - 7) & ~low_bytes(va - 8);
                    x.w &= low_bytes(ve - 11) & ~low_bytes(va - 12);
                }
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) mma_16816_f16(O[t], pa[s], e4m3_lo_to_f16x2(w[s]), e4m3_hi_to_f16x2(w[s]));
            }
        } else {
            constexpr int kW = kRow / 32;                     // words of a value's run
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t w[4][kW];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int o = 16 * s + 2 * c + (k & 1) + 8 * (k >> 1);
                    const uint8_t* row = st + Sm::kKBytes + o * kRow;
                    if constexpr (kW == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(row + (e4m3_chunk<kRow>(g, o) << 4));
                        w[k][0] = x.x;
                        w[k][1] = x.y;
                        w[k][kW - 2] = x.z;
                        w[k][kW - 1] = x.w;
                    } else {
                        const uint2 x =
                            *reinterpret_cast<const uint2*>(row + (e4m3_chunk<kRow>(g >> 1, o) << 4) + 8 * (g & 1));
                        w[k][0] = x.x;
                        w[k][1] = x.y;
                    }
                }
                auto pair = [](float x, float y) { return MX ? bf16x2(x, y) : f16x2(x, y); };
                const uint4 a = make_uint4(pair(S[2 * s][0], S[2 * s][1]), pair(S[2 * s][2], S[2 * s][3]),
                                           pair(S[2 * s + 1][0], S[2 * s + 1][1]),
                                           pair(S[2 * s + 1][2], S[2 * s + 1][3]));
                if constexpr (MX) {
                    // 16 channels of four keys: pairs (channel m, m + 4) of eight
                    // first, then the same channel of two keys side by side
                    uint32_t x[4][8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t E = min((uint32_t) reinterpret_cast<const uint8_t*>(
                            sc + kBlk)[4 * (16 * s + 2 * c + (k & 1) + 8 * (k >> 1)) + (g >> 1)], 252u);
                        const uint32_t e1 = E <= 128u ? E + 126u : 253u;
#pragma unroll
                        for (int q = 0; q < 2; ++q) e2m1x8_to_bf16(w[k][q], (e1 << 7) | (e1 << 23), x[k] + 4 * q);
                        if (E > 128u) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) x[k][q] = bf16x2_mul(x[k][q], (E << 7) | (E << 23));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        const int q = 4 * (t >> 3) + (t & 3);
                        const uint32_t sel = (t & 4) ? 0x7632u : 0x5410u;
                        mma_16816(O[t], a, __byte_perm(x[0][q], x[1][q], sel), __byte_perm(x[2][q], x[3][q], sel));
                    }
                } else {
                    // byte pairs (key 0, key 1) and (key 2, key 3) of two channels
                    // at a time
#pragma unroll
                    for (int t = 0; t < kNt; t += 2) {
                        const uint32_t sel = (t & 2) ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(w[0][t >> 2], w[1][t >> 2], sel);
                        const uint32_t y = __byte_perm(w[2][t >> 2], w[3][t >> 2], sel);
                        mma_16816_f16(O[t], a, e4m3_lo_to_f16x2(x), e4m3_lo_to_f16x2(y));
                        mma_16816_f16(O[t + 1], a, e4m3_hi_to_f16x2(x), e4m3_hi_to_f16x2(y));
                    }
                }
            }
        }
        __syncwarp();
        if (more) {
            copy(next, true);                                 // V's stage is free
            landing |= 2;
        } else {
            cp_async_commit();
        }
        pg = next;
    }
    // ---- the warp's (m, l, O), staged [channel][row] over its stage; the
    // slices combined
    cp_async_wait<0>();
    if (landing & 1) mbar_wait_drain(&bar[0], phase[0]);      // (after a time-out alone)
    if (landing & 2) mbar_wait_drain(&bar[1], phase[1]);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (c == 0) stat_s[warp][g + 8 * r] = make_float2(m[r], l[r]);
    }
    float* os = reinterpret_cast<float*>(st);
    const float unit = MX || vexp == kNoExp ? 1.0f : pow2i(vexp);
#pragma unroll
    for (int t = 0; t < kNt; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) os[(kNt * (2 * c + (e & 1)) + t) * kPitch + g + 8 * (e >> 1)] = O[t][e] * unit;
    __syncthreads();
    // thread: row tid % 16 of an m-tile, channels 4 (tid / 16 + 8 i) ..
    const int r = tid & 15;
    for (int t = 0; t < mts; ++t) {
        const float2* ss = &stat_s[t << lg_s][r];
        float M = -INFINITY, ls = 0.0f;
        for (int s = 0; s < slices; ++s) M = fmaxf(M, ss[16 * s].x);
        float y[kNt];
#pragma unroll
        for (int k = 0; k < kNt; ++k) y[k] = 0.0f;
        for (int s = 0; s < slices; ++s) {
            const float2 x = ss[16 * s];
            const float wt = x.x == -INFINITY ? 0.0f : ex2_approx(x.x - M);
            const float* o = reinterpret_cast<const float*>(sm + ((t << lg_s) + s) * Sm::kStage) + (tid >> 4) * 4 * kPitch + r;
            ls = fmaf(wt, x.y, ls);
#pragma unroll
            for (int k = 0; k < kNt; ++k) y[k] = fmaf(wt, o[(32 * (k >> 2) + (k & 3)) * kPitch], y[k]);
        }
        if (16 * t + r < rows) {
            if (tid < 16) stat[16 * t + r] = make_float2(M, ls);
#pragma unroll
            for (int k = 0; k < kNt; k += 4)
                reinterpret_cast<float4*>(out)[(2 * k + (tid >> 4)) * 64 + 16 * t + r] =
                    make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
        }
    }
    if (p.late_wait) pdl_wait();                              // this grid ends after the one before it
}

// ------------------------------------------------------------------ launch

// How a batch's work is cut, and where its pieces lie in the workspace.
struct SharedPlan {
    int pre_rows, n_rt, np, ns;              // rows of a prefix CTA, tiles of them, their splits; a sequence's splits
    int rows_pad, own_tc;                    // own_tc: a sequence's own keys by prefix_kernel too
    size_t pre_stat, pre_o, own_stat, own_o, codes, img, q_scale, bytes;
};

// The most that a batch of these sizes may be cut into, whatever its lengths,
// and the layout that has room for it.
SharedPlan shared_plan(int B, int T, int H, int Hk, int D) {
    SharedPlan w;
    const int64_t rows = (int64_t)B * T * (H / Hk), sms = device_sms(), items = (int64_t)B * Hk;
    const bool few = rows <= kFewRows;
    w.pre_rows = few ? kFewRows : (rows <= 128 ? 128 : 256);
    w.n_rt = (int)ceil_div(rows, w.pre_rows);
    // one CTA an SM for prefix_kernel, two or three for rows_kernel
    w.np = (int)std::max<int64_t>(1, (few ? 2 * sms : sms) / ((int64_t)w.n_rt * Hk));
    w.ns = (int)std::max<int64_t>(1, std::min<int64_t>(32, (few ? 1 : (T * (H / Hk) > 16 ? 2 : 3)) * sms / items));
    w.rows_pad = few ? (int)rows : w.n_rt * w.pre_rows;
    w.own_tc = 0;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) & ~(size_t)255;
        return o;
    };
    // (in 128-row CTAs no more than in 256-row ones: at most one an SM, or one
    // a row tile)
    const size_t pre = std::max<size_t>((size_t)w.n_rt * Hk * w.np, few ? 0 : sms) * w.pre_rows, own = (size_t)items * w.ns * 64;
    const size_t q_rows = (size_t)Hk * (few ? 128 : w.rows_pad);    // (up to 64 rows may go to prefix_kernel too)
    w.pre_stat = take(pre * sizeof(float2));
    w.own_stat = take(own * sizeof(float2));
    w.pre_o = take(pre * D * sizeof(float));
    w.own_o = take(own * D * sizeof(float));
    w.codes = take(q_rows * D);
    w.img = take(q_rows * 2 * D);                            // (bf16 images for an MXFP4 cache)
    w.q_scale = take(q_rows * sizeof(float));
    w.bytes = at;
    return w;
}

// The cut of a call, by its estimated time. A prefix CTA has an SM to itself;
// the sequences' own CTAs run on the SMs left over, or behind it; 128 or 256
// rows a CTA trade partials for conversions of V; and the own keys of sequences
// of many rows may go to prefix_kernel too. So the most CTAs are not the least
// time: MXFP4 B32 behind 16384 tokens takes 37.8 us with 128 prefix CTAs of two
// tiles and 27.8 with 86 of three; B16 T4 window 4096 36.8 with 64 + 256 CTAs,
// 30.1 with 16 + 256, and 24.1 with 32 + 64, own keys by prefix_kernel. The
// model's constants (microseconds; tiles are 128 keys, blocks 64 keys a warp)
// are fitted to 70 batches of 65 to 4096 rows over all their cuts: its choice
// is 2 % slower than the best one on average, 29 % at worst. The lengths are on
// the device; the tables' sizes stand for them, and a sequence's own keys for
// half of what its table has room for (only the time depends on that).
void choose_cut(const DecodeSharedArgs& sa, SharedPlan& w) {
    const DecodeArgs& a = sa.d;
    const int sms = device_sms(), R = a.T * (a.H / a.Hk), lg_s = lg_slices(R), per_sm = R > 16 ? 2 : 3;
    const int64_t rows = (int64_t)a.B * R, items = (int64_t)a.B * a.Hk;
    const int64_t cap_pre = (int64_t)sa.max_prefix_pages * a.page_size, cap_row = (int64_t)a.max_pages * a.page_size;
    const int64_t seen = std::min<int64_t>(cap_row, (int64_t)a.window + a.T);
    const int tiles = (int)std::max<int64_t>(1, std::min(ceil_div(cap_pre, kKeys), ceil_div(seen, kKeys) + 1));
    const int blocks = (int)ceil_div(std::max<int64_t>(kBlk, std::min(cap_row - cap_pre + a.page_size, seen)), kBlk);
    const int half = std::max(1, blocks / 2);                              // of an average sequence
    const float d64 = a.D == 64 ? 0.7f : 1.0f;
    const float pre_fixed[3] = {0.0f, 4.1f, 6.4f}, tile[3] = {0.0f, a.mx ? 2.75f : 1.48f * d64, a.mx ? 3.37f : 1.79f * d64};
    const float merge_bytes = 3.5e6f;                                      // a microsecond
    // own keys by rows_kernel, by prefix_kernel: a CTA, a block (tile); CTAs an
    // SM; the share of the SMs left over that they get beside the prefix
    const float own_fixed[2] = {2.8f, 5.8f};
    const float own_unit[2] = {(a.mx ? 5.56f : 2.16f * d64) * (R > 16 ? 0.84f : 1.0f), 2.0f * (a.mx ? 1.95f : 1.03f * d64)};
    const int fit[2] = {per_sm, 1};
    const float beside[2] = {0.34f, 0.2f};
    const float whole = 0.53f;                                             // of a last wave that is not full
    const SharedPlan most = w;
    float best = FLT_MAX;
    if (w.pre_rows == kFewRows) {
        // rows_kernel for both parts, one launch fewer. With over 16 rows a
        // block costs twice what it does beside a prefix (64 rows behind 29932
        // tokens, 8 heads of 64: 51.8 us, 32.1 by prefix_kernel), but a call of one
        // block a warp is 3.5 us shorter (9.2 against 12.6).
        const int lg = lg_slices((int)rows);
        w.np = used_splits((int)ceil_div(cap_pre, kBlk), w.np, lg);
        w.ns = used_splits((int)ceil_div(cap_row, kBlk), w.ns, lg_s);
        if (rows <= 16) return;
        const int64_t pre_blocks = std::min(ceil_div(cap_pre, kBlk), ceil_div(seen, kBlk) + 1);
        best = (a.mx ? 6.0f : 3.6f) * ceil_div(pre_blocks, (int64_t)w.np << lg) - 1.5f;
    }
    for (int rg = rows <= 128 ? 1 : 2; rg >= 1; --rg) {
        const int64_t units = ceil_div(rows, 128 * rg) * a.Hk;            // row tiles of all heads
        if (rg == 1 && most.pre_rows != 128 && units > sms) continue;      // (the layout's bound)
        const int np_max = (int)std::max<int64_t>(1, sms / units), step = rg == 1 ? 2 : 1;
        int per = (int)ceil_div(std::max(ceil_div(tiles, np_max), (int64_t)step), step) * step;
        for (int n = 0; n < 7; ++n, per += std::max(step, per / 4 / step * step)) {
            const int np = (int)ceil_div(tiles, per);
            const float ctas = (float)units * np, tp = pre_fixed[rg] + per * tile[rg];
            const float waves = std::ceil(ctas / sms);
            for (int v = 0; v < (R > 32 ? 2 : 1); ++v) {
                const int lg = v ? 1 : lg_s, units_max = v ? (blocks + 1) / 2 + 1 : blocks, units_mean = std::max(1, v ? (half + 1) / 2 : half);
                const float slots = std::max(0.0f, sms - ctas) * fit[v], all = (float)sms * fit[v];
                for (int ns = 1;; ns = std::min(2 * ns, most.ns)) {
                    const int used = used_splits(units_mean, ns, lg), least = used_splits(units_max, ns, lg);
                    const float longest = own_fixed[v] + own_unit[v] * ceil_div(units_max, (int64_t)least << lg);
                    const float mean = own_fixed[v] + own_unit[v] * ceil_div(units_mean, (int64_t)used << lg);
                    const float n_own = (float)items * used;
                    auto run = [&](float n) { return mean * (std::ceil(n / all) * whole + n / all * (1.0f - whole)); };
                    float t = std::max(waves * tp, longest);
                    if (ctas >= sms) {
                        t = waves * tp + std::max(run(n_own), longest);
                    } else if (n_own > slots) {
                        const float done = (std::floor(tp / mean) * whole + tp / mean * (1.0f - whole)) * slots * beside[v];
                        if (n_own > done) t = std::max(tp + std::max(mean, run(n_own - done)), longest);
                    }
                    t += (ctas * 128 * rg + n_own * R) * a.D * 4 / merge_bytes;
                    if (t < best) {
                        best = t;
                        w.pre_rows = 128 * rg;
                        w.n_rt = (int)(units / a.Hk);
                        w.np = np;
                        w.ns = ns;
                        w.own_tc = v;
                        w.rows_pad = w.n_rt * w.pre_rows;
                    }
                    if (ns == most.ns) break;
                }
            }
            if (np == 1) break;
        }
    }
}

template <int D, bool MX, int RG, bool OWN>
cudaError_t launch_prefix(const DecodeSharedArgs& sa, const SharedPlan& w, const CUtensorMap& tk, const CUtensorMap& tv,
                          cudaStream_t s) {
    const DecodeArgs& a = sa.d;
    constexpr int kSmem = SmP<D, MX, RG>::kBytes + 1024;
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    PrefixParams p = {};
    p.q_img = ws + w.img;
    p.q_scale = reinterpret_cast<const float*>(ws + w.q_scale);
    p.ksc = a.k_scale;
    p.vsc = a.v_scale;
    p.per_tensor = (a.kv_flags & 1) ? 1 : 0;
    p.v_trans = (!MX && (a.kv_flags & 2)) ? 1 : 0;
    p.ksf8 = a.k_sf;
    p.vsf8 = a.v_sf;
    p.codes = ws + w.codes;
    p.rows_pad = w.rows_pad;
    p.max_pages = a.max_pages;
    p.ptab = OWN ? a.page_table : sa.prefix_table;
    p.plen = sa.prefix_len;
    p.ctx = a.ctx_lens;
    p.T = a.T;
    p.Hk = a.Hk;
    p.R = a.T * (a.H / a.Hk);
    p.div_r = fast_div_by(p.R);
    p.div_g = fast_div_by(a.H / a.Hk);
    p.n_rows = a.B * p.R;
    p.page = a.page_size;
    p.lg_page = 31 - __builtin_clz(static_cast<unsigned>(a.page_size));
    p.cap_prefix = sa.max_prefix_pages * a.page_size;
    p.cap_rows = a.max_pages * a.page_size;
    p.num_pages = a.num_pages;
    p.window = std::min(a.window, INT32_MAX - 64);           // (positions start at -T: no wrap)
    p.np = OWN ? w.ns : w.np;
    p.n_rt = w.n_rt;
    p.logit_scale_log2 = a.softmax_scale / static_cast<float>(D) * kLog2e;
    p.stat = reinterpret_cast<float2*>(ws + (OWN ? w.own_stat : w.pre_stat));
    p.o = reinterpret_cast<float*>(ws + (OWN ? w.own_o : w.pre_o));
    const cudaError_t e = allow_smem<prefix_kernel<D, MX, RG, OWN>>(kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefix_kernel<D, MX, RG, OWN>, OWN ? dim3(w.ns, a.B * a.Hk) : dim3(w.np, w.n_rt * a.Hk), dim3(kThreads), kSmem, s, tk, tv, p);
}

template <int D, bool MX>
cudaError_t launch_shared_d(const DecodeSharedArgs& sa, cudaStream_t s) {
    const DecodeArgs& a = sa.d;
    // (a function of the sizes alone: a serving loop's next call has the same)
    const int sizes[] = {device_sms(), a.B, a.T, a.H, a.Hk, a.page_size, a.max_pages, a.window, sa.max_prefix_pages};
    static thread_local int last[9] = {};
    static thread_local SharedPlan w;
    if (!std::equal(sizes, sizes + 9, last)) {
        w = shared_plan(a.B, a.T, a.H, a.Hk, D);
        choose_cut(sa, w);
        std::copy(sizes, sizes + 9, last);
    }
    const bool few = w.pre_rows == kFewRows;
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    QueryParams q = {};
    q.q = static_cast<const uint16_t*>(a.q.ptr);
    q.qs0 = a.q.stride[0];
    q.qs1 = a.q.stride[1];
    q.qs2 = a.q.stride[2];
    q.qs3 = a.q.stride[3];
    q.q_vec = view_vec8(a.q) ? 1 : 0;
    q.G = a.H / a.Hk;
    q.R = a.T * q.G;
    q.n_rows = a.B * q.R;
    q.rows_pad = w.rows_pad;
    q.codes = ws + w.codes;
    q.img = ws + w.img;
    q.scale = reinterpret_cast<float*>(ws + w.q_scale);
    cudaError_t e = cudaSuccess;
    if (!few) e = launch_pdl(query_kernel<D, MX>, dim3((unsigned)ceil_div(q.n_rows, 32), a.Hk), dim3(128), 0, s, q);
    if (e != cudaSuccess) return e;
    // boxes of half a 128-token page; a transposed V also whole, for prefix_kernel
    CUtensorMap tk, tv, tv128;
    const bool vt = !MX && (a.kv_flags & 2);
    const int box = std::min(a.page_size, kBlk);
    const bool ok = MX ? encode_cache_mx(&tk, a.k_cache, a.num_pages, a.Hk, a.page_size, D, box) &&
                             encode_cache_mx(&tv, a.v_cache, a.num_pages, a.Hk, a.page_size, D, box)
                       : encode_cache(&tk, a.k_cache, a.num_pages, a.Hk, a.page_size, D, box) &&
                             (vt ? encode_cache_vt(&tv, a.v_cache, a.num_pages, a.Hk, D, kBlk) &&
                                       (few || encode_cache_vt(&tv128, a.v_cache, a.num_pages, a.Hk, D))
                                 : encode_cache(&tv, a.v_cache, a.num_pages, a.Hk, a.page_size, D, box));
    if (!ok) return cudaErrorInvalidValue;
    if (!few) {
        const CUtensorMap& tvp = vt ? tv128 : tv;
        e = w.pre_rows == 128 ? launch_prefix<D, MX, 1, false>(sa, w, tk, tvp, s) : launch_prefix<D, MX, 2, false>(sa, w, tk, tvp, s);
        if (e == cudaSuccess && w.own_tc) e = launch_prefix<D, MX, 1, true>(sa, w, tk, tvp, s);
        if (e != cudaSuccess) return e;
    }
    RowsParams r = {};
    r.q8 = few ? nullptr : q.codes;
    r.q_scale = q.scale;
    r.q = q.q;
    r.qs0 = q.qs0;
    r.qs1 = q.qs1;
    r.qs2 = q.qs2;
    r.qs3 = q.qs3;
    r.q_vec = q.q_vec;
    r.ksc = a.k_scale;
    r.vsc = a.v_scale;
    r.ksf = a.k_sf;
    r.vsf = a.v_sf;
    r.per_tensor = (a.kv_flags & 1) ? 1 : 0;
    r.ptab = a.page_table;
    r.prefix = sa.prefix_table;
    r.plen = sa.prefix_len;
    r.ctx = a.ctx_lens;
    r.B = a.B;
    r.T = a.T;
    r.Hk = a.Hk;
    r.G = q.G;
    r.R = q.R;
    r.n_rows = q.n_rows;
    r.rows_pad = w.rows_pad;
    r.lg_page = 31 - __builtin_clz(static_cast<unsigned>(a.page_size));
    r.max_pages = a.max_pages;
    r.cap_prefix = sa.max_prefix_pages * a.page_size;
    r.num_pages = a.num_pages;
    r.window = std::min(a.window, INT32_MAX - 64);
    r.np = few ? w.np : 0;
    r.ns = w.ns;
    r.logit_scale_log2 = a.softmax_scale / static_cast<float>(D) * kLog2e;
    r.pre_stat = reinterpret_cast<float2*>(ws + w.pre_stat);
    r.pre_o = reinterpret_cast<float*>(ws + w.pre_o);
    r.own_stat = reinterpret_cast<float2*>(ws + w.own_stat);
    r.own_o = reinterpret_cast<float*>(ws + w.own_o);
    r.late_wait = few ? 0 : 1;
    r.div_np = fast_div_by(r.np);
    r.div_ns = fast_div_by(r.ns);
    r.div_hk = fast_div_by(r.Hk);
    r.div_r = fast_div_by(r.R);
    r.div_g = fast_div_by(r.G);
    const dim3 grid((unsigned)(r.np * a.Hk + (int64_t)w.ns * a.B * a.Hk)), block(32 * kRowsWarps);
    const int mts = (int)ceil_div(few ? q.n_rows : q.R, 16);
    if (w.own_tc) {
        // (launched above)
    } else if (vt) {
        using Sm = SmR<D, false, true>;
        e = allow_smem<rows_kernel<D, false, true>>(Sm::bytes(4));
        if (e == cudaSuccess) e = launch_pdl(rows_kernel<D, false, true>, grid, block, Sm::bytes(mts), s, tk, tv, r);
    } else {
        using Sm = SmR<D, MX, false>;
        e = allow_smem<rows_kernel<D, MX, false>>(Sm::bytes(4));
        if (e == cudaSuccess) e = launch_pdl(rows_kernel<D, MX, false>, grid, block, Sm::bytes(mts), s, tk, tv, r);
    }
    if (e != cudaSuccess) return e;
    MergeParams m = {};
    m.pre_stat = r.pre_stat;
    m.pre_o = r.pre_o;
    m.own_stat = r.own_stat;
    m.own_o = r.own_o;
    m.plen = sa.prefix_len;
    m.cap_prefix = r.cap_prefix;
    m.np = w.np;
    m.ns = w.ns;
    m.pre_rows = w.pre_rows;
    m.n_rt = w.n_rt;
    m.unit = few ? kBlk : kKeys;
    m.lg_at_once = few ? lg_slices(q.n_rows) : (w.pre_rows == 128 ? 1 : 0);
    m.T = a.T;
    m.G = q.G;
    m.R = q.R;
    m.n_rows = q.n_rows;
    m.Hk = a.Hk;
    m.out = static_cast<__nv_bfloat16*>(a.out);
    m.os0 = a.out_stride[0];
    m.os1 = a.out_stride[1];
    m.os2 = a.out_stride[2];
    m.os3 = a.out_stride[3];
    m.ctx = a.ctx_lens;
    m.cap_rows = a.max_pages * a.page_size;
    m.window = r.window;
    m.lg_unit = w.own_tc ? 7 : 6;
    m.lg_own = w.own_tc ? 1 : lg_slices(q.R);
    // (four warps hold all of sixteen parts at once)
    const dim3 mg((unsigned)ceil_div(m.n_rows, 32), D / kCh, a.Hk);
    return w.np + w.ns <= 16 ? launch_pdl(shared_merge_kernel<D, 4>, mg, dim3(128), 0, s, m)
                             : launch_pdl(shared_merge_kernel<D, 8>, mg, dim3(256), 0, s, m);
}

}  // namespace

size_t decode_shared_ws_bytes(int B, int T, int H, int Hk, int D) { return shared_plan(B, T, H, Hk, D).bytes; }

cudaError_t launch_decode_shared(const DecodeSharedArgs& a, cudaStream_t s) {
    if (a.d.mx) return a.d.D == 128 ? launch_shared_d<128, true>(a, s) : cudaErrorInvalidValue;
    switch (a.d.D) {
        case 64: return launch_shared_d<64, false>(a, s);
        case 128: return launch_shared_d<128, false>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

unsigned read_clear_shared_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_shared_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_shared_err, &zero, sizeof zero);
    return v;
}

}  // namespace sage
