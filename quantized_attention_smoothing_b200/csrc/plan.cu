// plan.cu -- one serving step's bookkeeping of the paged KV cache, on the
// GPU: from the lengths of a batch's requests, the pages they take from and
// give back to a free list, their block tables, and the slot (page * page
// size + offset) of every new token. The tables are what sage_attn_decode
// and sage_attn_decode_shared read, the slots where sage_kv_append writes.
//
// Request b holds cached_b tokens and adds new_b (new_b < 0: it has ended).
// With P the shared prefix's tokens,
//   start_b = P where cached_b = 0 < new_b, else cached_b
//   held_b  = ceil(start_b / page), need_b = ceil((start_b + new_b) / page) - held_b
//   gone_b  = held_b - prefix_pages for a request that has ended
// and three exclusive sums over the requests (tokens, need, gone) place
// everything: the pages given back are pushed on the free list in request
// order, the new ones popped from its top, the new tokens numbered in a row.
//
// The arithmetic is a scan of at most 8192 requests; what it costs is
// latency: one launch, three dependent trips to memory (lengths; free-list
// and table entries; stores). So one cluster of up to 8 CTAs does all of it:
// every CTA reads all lengths and makes the same sums for itself (B / 1024
// lengths a thread), then the CTAs share out the entries to write. The
// cluster barrier between the reads of the lengths and the writes of the new
// ones lets the outputs be the inputs' own buffers. A long slot map (over
// kInlineTokens) is left to a second launch over the whole GPU, which finds
// everything in the first one's outputs: position of token t of request b =
// ctx_b - (offset_{b+1} - t).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "sage_internal.h"
#include "sage_ptx.cuh"

namespace sage {
namespace {

__device__ unsigned g_plan_err;

constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr int kRowsPer = kPlanMaxRows / kThreads;      // lengths a thread sums at most
// slots the cluster writes itself: 8 CTAs x 1024 threads x 4 slots, twice
constexpr int kInlineTokens = 65536;
constexpr int kSlotThreads = 256, kSlotPer = 2048;     // slot kernel: slots per CTA

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// For U numbers at once, the row whose range [off[b], off[b + 1]) holds i
// (off[0] = 0 <= i < off[n]): the last b with off[b] <= i. step: the largest
// power of two below n (0 for n = 1).
template <int U>
__device__ __forceinline__ void find_rows(const int* off, int n, int step, const int* i, int* b) {
#pragma unroll
    for (int u = 0; u < U; ++u) b[u] = 0;
    for (; step > 0; step >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = b[u] + step;
            if (x < n && off[x] <= i[u]) b[u] = x;
        }
    }
}

__device__ __forceinline__ int first_step(int n) { return n > 1 ? 1 << (31 - __clz(n - 1)) : 0; }

struct Sum3 {
    long long tok, need, gone;
};

__device__ __forceinline__ Sum3 warp_scan(Sum3 v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, v.tok, d);
        const long long b = __shfl_up_sync(0xffffffffu, v.need, d);
        const long long c = __shfl_up_sync(0xffffffffu, v.gone, d);
        if (lane >= d) {
            v.tok += a;
            v.need += b;
            v.gone += c;
        }
    }
    return v;
}

struct PlanParams {
    const int32_t* cached;
    const int32_t* fresh;                   // new_lens
    const int32_t* prefix;
    int32_t* free_list;
    const int32_t* free_count;
    int32_t* table;
    int32_t* ctx;
    int32_t* free_count_out;
    int32_t* offsets;
    int32_t* slots;
    int B, max_pages, lg_page, num_pages, max_tokens, prefix_pages;
    int inline_slots;
};

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanParams p) {
    extern __shared__ int sm[];
    int* tok_off = sm;                       // [B + 1] exclusive sums
    int* need_off = tok_off + p.B + 1;
    int* gone_off = need_off + p.B + 1;
    int* start_of = gone_off + p.B + 1;      // [B] start_b, ~start_b for a request that joins
    __shared__ Sum3 warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster_rank(), nthr = cluster_size() * kThreads, gtid = rank * kThreads + tid;
    const int lg = p.lg_page, page = 1 << lg;
    const int P = p.prefix_pages << lg, cap = p.max_pages << lg;

    pdl_wait();
    pdl_launch_dependents();
    const int fc = *p.free_count;
    // ---- lengths of this thread's rows, and their sums
    const int per = (p.B + kThreads - 1) / kThreads, b0 = tid * per;
    int own_tok[kRowsPer], own_need[kRowsPer], own_gone[kRowsPer];   // (used only when every sum fits)
    Sum3 mine = {0, 0, 0};
    bool bad = fc < 0 || fc > p.num_pages;
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        own_tok[i] = (int)mine.tok;
        own_need[i] = (int)mine.need;
        own_gone[i] = (int)mine.gone;
        if (i < per && b0 + i < p.B) {
            const int b = b0 + i, have = p.cached[b], add = p.fresh[b];
            const bool joins = have == 0 && add > 0;
            const int start = joins ? P : have;
            bad |= have < 0 || start > cap || (have > 0 && have < P) || (add > 0 && add > cap - start);
            start_of[b] = joins ? ~start : start;
            const int held = (start + page - 1) >> lg;
            if (add >= 0) {
                mine.tok += add;
                mine.need += (int)(((unsigned)start + (unsigned)add + page - 1) >> lg) - held;
            } else {
                mine.gone += max(0, held - p.prefix_pages);
            }
        }
    }
    const Sum3 incl = warp_scan(mine, lane);
    if (lane == 31) warp_sum[warp] = incl;
    bad = __syncthreads_or(bad);
    const Sum3 tot = warp_scan(warp_sum[lane], lane);    // every warp sums the warps' totals
    const int before = (warp + 31) & 31;                 // lane of the warps before this one
    Sum3 base = {__shfl_sync(0xffffffffu, tot.tok, before), __shfl_sync(0xffffffffu, tot.need, before),
                 __shfl_sync(0xffffffffu, tot.gone, before)};
    if (warp == 0) base = {0, 0, 0};
    base.tok += incl.tok - mine.tok;
    base.need += incl.need - mine.need;
    base.gone += incl.gone - mine.gone;
    const long long n_tok = __shfl_sync(0xffffffffu, tot.tok, 31);
    const long long n_need = __shfl_sync(0xffffffffu, tot.need, 31);
    const long long n_gone = __shfl_sync(0xffffffffu, tot.gone, 31);
    // all or nothing: too few pages, slots or table entries, or a length out
    // of range, and the step changes nothing
    bad |= n_tok > p.max_tokens || n_need > fc + n_gone || fc + n_gone > p.num_pages;
    if (bad) {
        if (rank == 0 && tid == 0) atomicCAS(&g_plan_err, 0u, kErrRangeCode | (1u << 8));
        // (a copy onto itself where the outputs are the inputs' buffers)
        for (int b = gtid; b < p.B; b += nthr) p.ctx[b] = p.cached[b];
        for (int b = gtid; b <= p.B; b += nthr) p.offsets[b] = 0;
        // (64-bit: a slot map may be as long as a 32-bit length says)
        for (int64_t t = gtid; t < p.max_tokens; t += nthr) p.slots[t] = -1;
        if (gtid == 0) *p.free_count_out = fc;
        return;
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        if (i < per && b0 + i < p.B) {
            tok_off[b0 + i] = (int)base.tok + own_tok[i];
            need_off[b0 + i] = (int)base.need + own_need[i];
            gone_off[b0 + i] = (int)base.gone + own_gone[i];
        }
    }
    if (tid == 0) {
        tok_off[p.B] = (int)n_tok;
        need_off[p.B] = (int)n_need;
        gone_off[p.B] = (int)n_gone;
    }
    __syncthreads();
    cluster_arrive();                        // this CTA has read the lengths and the count

    const int na = (int)n_need, nf = (int)n_gone, top = fc + nf;
    auto start_at = [&](int b) {
        const int s = start_of[b];
        return s < 0 ? ~s : s;
    };
    // U things a thread at a time, searches and loads of all of them before
    // any store: with many things the loops are bound by their chains of
    // dependent accesses (62000 new entries: 17.9 us one by one, 11.7 with four
    // at a time), with few by the searches themselves, dummies' included
    const int step = first_step(p.B);
    // the i-th pages given back
    auto gone_pages = [&](auto u_c, const int* i, const bool* in, int* pg) {
        constexpr int U = decltype(u_c)::value;
        int b[U];
        find_rows<U>(gone_off, p.B, step, i, b);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (in[u]) pg[u] = p.table[(int64_t)b[u] * p.max_pages + p.prefix_pages + i[u] - gone_off[b[u]]];
    };
    // the k-th pages handed out
    auto new_pages = [&](auto u_c, const int* k, const bool* in, int* pg) {
        constexpr int U = decltype(u_c)::value;
        int g[U];
        bool back[U], any = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = top - 1 - k[u];
            back[u] = in[u] && at >= fc;
            g[u] = max(0, at - fc);
            any |= back[u];
            if (in[u] && at < fc) pg[u] = p.free_list[at];
        }
        if (any) gone_pages(u_c, g, back, pg);
    };
    // body(u_c, first, stride) for the things first, first + stride, .. of n
    auto batches = [&](int n, auto body) {
        int i = gtid;
        for (; i + 3 * (int64_t)nthr < n; i += 4 * nthr) body(std::integral_constant<int, 4>{}, i);
        for (; i < n; i += nthr) body(std::integral_constant<int, 1>{}, i);
    };
    // ---- new table entries
    batches(na, [&](auto u_c, int k0) {
        constexpr int U = decltype(u_c)::value;
        int k[U], b[U], pg[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = true;
            k[u] = k0 + u * nthr;
        }
        find_rows<U>(need_off, p.B, step, k, b);
        new_pages(u_c, k, in, pg);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int held = (start_at(b[u]) + page - 1) >> lg;
            p.table[(int64_t)b[u] * p.max_pages + held + k[u] - need_off[b[u]]] = pg[u];
        }
    });
    // ---- the prefix's entries for the requests that join
    if (p.prefix_pages > 0) {
        for (int b = gtid >> 5; b < p.B; b += nthr >> 5)
            if (start_of[b] < 0)
                for (int e = lane; e < p.prefix_pages; e += 32)
                    p.table[(int64_t)b * p.max_pages + e] = p.prefix[e];
    }
    // ---- pages given back and not handed out again stay on the list
    batches(nf - na, [&](auto u_c, int i0) {
        constexpr int U = decltype(u_c)::value;
        int i[U], pg[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = true;
            i[u] = i0 + u * nthr;
        }
        gone_pages(u_c, i, in, pg);
#pragma unroll
        for (int u = 0; u < U; ++u) p.free_list[fc + i[u]] = pg[u];
    });
    // ---- slots
    if (p.inline_slots) {
        batches((int)n_tok, [&](auto u_c, int t0) {
            constexpr int U = decltype(u_c)::value;
            int t[U], b[U], k[U], pg[U], pos[U];
            bool fresh[U], any = false;
#pragma unroll
            for (int u = 0; u < U; ++u) t[u] = t0 + u * nthr;
            find_rows<U>(tok_off, p.B, step, t, b);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int start = start_at(b[u]), held = (start + page - 1) >> lg;
                pos[u] = start + t[u] - tok_off[b[u]];
                const int e = pos[u] >> lg;
                fresh[u] = e >= held;
                k[u] = fresh[u] ? need_off[b[u]] + e - held : 0;
                any |= fresh[u];
                if (!fresh[u]) pg[u] = p.table[(int64_t)b[u] * p.max_pages + e];
            }
            if (any) new_pages(u_c, k, fresh, pg);
#pragma unroll
            for (int u = 0; u < U; ++u) p.slots[t[u]] = (pg[u] << lg) + (pos[u] & (page - 1));
        });
        for (int t = (int)n_tok + gtid; t < p.max_tokens; t += nthr) p.slots[t] = -1;
    }
    cluster_wait();                          // every CTA has read the lengths
    for (int b = gtid; b < p.B; b += nthr) {
        // (own row, read above: the new length needs new_b again, which is
        // not written; an ended row keeps nothing)
        const int add = p.fresh[b];
        p.ctx[b] = add < 0 ? 0 : start_at(b) + add;
        p.offsets[b] = tok_off[b];
    }
    if (gtid == 0) {
        p.offsets[p.B] = tok_off[p.B];
        *p.free_count_out = top - na;
    }
}

// The slots of a long map from the first launch's outputs: thread = 4
// consecutive slots at a time, the requests' token offsets in shared memory.
__global__ void __launch_bounds__(kSlotThreads) slot_kernel(const int32_t* __restrict__ offsets,
                                                            const int32_t* __restrict__ ctx,
                                                            const int32_t* __restrict__ table, int32_t* slots, int B,
                                                            int max_pages, int lg, int max_tokens, int vec) {
    extern __shared__ int off[];
    pdl_wait();
    pdl_launch_dependents();
    for (int b = threadIdx.x; b <= B; b += kSlotThreads) off[b] = __ldg(offsets + b);
    __syncthreads();
    const int n_tok = off[B], step = first_step(B);
    constexpr int U = kSlotPer / (4 * kSlotThreads);     // runs of four slots a thread
    int t[U], b[U], last[U];                             // position of token x: last + x
    const int64_t t00 = (int64_t)blockIdx.x * kSlotPer + 4 * threadIdx.x;
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = (int)min(t00 + u * 4 * kSlotThreads, (int64_t)max(n_tok - 1, 0));
    find_rows<U>(off, B, step, t, b);
#pragma unroll
    for (int u = 0; u < U; ++u) last[u] = __ldg(ctx + b[u]) - off[b[u] + 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t t0 = t00 + u * 4 * kSlotThreads;
        int s[4] = {-1, -1, -1, -1};
        if (t0 < n_tok) {
            int e = -1, pg = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = (int)t0 + i;
                if (x < n_tok) {
                    if (x >= off[b[u] + 1]) {
                        do ++b[u];
                        while (x >= off[b[u] + 1]);
                        last[u] = __ldg(ctx + b[u]) - off[b[u] + 1];
                        e = -1;
                    }
                    const int pos = last[u] + x;
                    if ((pos >> lg) != e) {
                        e = pos >> lg;
                        pg = __ldg(table + (int64_t)b[u] * max_pages + e);
                    }
                    s[i] = (pg << lg) + (pos & ((1 << lg) - 1));
                }
            }
        }
        if (vec && t0 + 4 <= max_tokens) {
            *reinterpret_cast<int4*>(slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < max_tokens) slots[t0 + i] = s[i];
        }
    }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
    PlanParams p;
    p.cached = a.cached_lens;
    p.fresh = a.new_lens;
    p.prefix = a.prefix_table;
    p.free_list = a.free_list;
    p.free_count = a.free_count;
    p.table = a.page_table;
    p.ctx = a.ctx_lens;
    p.free_count_out = a.free_count_out;
    p.offsets = a.token_offsets;
    p.slots = a.slot_map;
    p.B = a.B;
    p.max_pages = a.max_pages;
    p.lg_page = 31 - __builtin_clz(static_cast<unsigned>(a.page_size));
    p.num_pages = a.num_pages;
    p.max_tokens = a.max_tokens;
    p.prefix_pages = a.prefix_pages;
    p.inline_slots = a.max_tokens <= kInlineTokens ? 1 : 0;
    const size_t smem = (4 * (size_t)a.B + 3) * sizeof(int);
    cudaError_t e = allow_smem<plan_kernel>((4 * kPlanMaxRows + 3) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    // one CTA for every 1024 slots, rows and (as a guess) table entries
    const int64_t items = (p.inline_slots ? a.max_tokens : kInlineTokens) + (int64_t)a.B;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    unsigned n = 1;
    while (n < kMaxCluster && (int64_t)n * kThreads < items) n *= 2;
    attr[1].val.clusterDim.x = n;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
    if (e != cudaSuccess || p.inline_slots) return e;
    const int vec = reinterpret_cast<uintptr_t>(a.slot_map) % 16 == 0 ? 1 : 0;
    return launch_pdl(slot_kernel, dim3((unsigned)ceil_div(a.max_tokens, kSlotPer)), dim3(kSlotThreads),
                      ((size_t)a.B + 1) * sizeof(int), s, p.offsets, p.ctx, p.table, p.slots, p.B, p.max_pages,
                      p.lg_page, p.max_tokens, vec);
}

unsigned read_clear_plan_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_plan_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_plan_err, &zero, sizeof zero);
    return v;
}

}  // namespace sage
