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

// ------------------------------------------------------------------ launch

// Where the partials of the two parts lie in the workspace.
struct SharedPlan {
    int pre_rows, n_rt, np, ns;              // rows a prefix CTA has, tiles of them, their splits; own splits
    size_t pre_stat, pre_o, own_stat, own_o, bytes;
};

SharedPlan shared_plan(int B, int T, int H, int Hk, int D) {
    SharedPlan w;
    const int64_t rows = (int64_t)B * T * (H / Hk);
    w.pre_rows = kFewRows;
    w.n_rt = (int)ceil_div(rows, w.pre_rows);
    const int sms = device_sms();
    w.np = (int)std::max<int64_t>(1, sms / ((int64_t)w.n_rt * Hk));
    w.ns = (int)std::max<int64_t>(1, std::min<int64_t>(16, sms / ((int64_t)B * Hk)));
    const size_t pre = (size_t)w.n_rt * Hk * w.np * w.pre_rows, own = (size_t)B * Hk * w.ns * 64;
    w.pre_stat = 0;
    w.own_stat = w.pre_stat + pre * sizeof(float2);
    w.pre_o = w.own_stat + own * sizeof(float2);
    w.own_o = w.pre_o + pre * D * sizeof(float);
    w.bytes = w.own_o + own * D * sizeof(float);
    return w;
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
    cudaError_t e = launch_decode_part(a, part, s);
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
