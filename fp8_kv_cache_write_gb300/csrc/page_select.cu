// page_select.cu -- the pages a decode query reads: a cheap score of every page from its
// 8-bit bounds (page_bounds.cu), and the `budget` pages with the highest scores.
//
// For sequence b and KV head h with the query heads g of its group,
//     u = [sum_g max(q_g, 0), sum_g min(q_g, 0)]            2 D values, 8 bits: c = rint(u / s)
//     score(page) = fp32(sum_d c_d hi_d + c_{D+d} lo_d) * bounds_scale
// an estimate, off by half a step of the codes, of the sum over the group's heads of the
// largest logit a key between the page's extremes could have (up to the factor s, which all
// pages of a head share).  Because the sum over heads
// moves into the query, a page costs one product of 2 D bytes whatever the group's size.
// The products are whole numbers (below 2^23, exact in fp32), so the score has one
// rounding, does not depend on the order of the sums, and the selection is reproducible:
// ties go to the lower page.
//
// Bound: HBM for the bounds (2 D + 4 bytes a page and head) in large batches, latency for
// one request.  Split: two kernels, the second launched early.
//   * Scores: a CTA takes 512 pages of one (sequence, KV head), a warp 32 of them at once, so
//     that every byte the CTA reads is in flight together and the query's codes are worked
//     out meanwhile.  Scores go to the workspace as sortable 32-bit keys.
//   * Pages: a CTA per (sequence, KV head) keeps its keys in shared memory and narrows
//     [lowest, highest key] to one of 1024 equal bins that holds the last key taken; the few
//     keys of that bin are ranked against each other, where they are many it is narrowed
//     again.  Then every warp writes the pages of its run of keys, in their order.
// Measured: 8 heads of 8192 pages 13.6 us, 64 heads of about 1300 pages 11.3 us, 256 heads of 63
// to 4063 pages at D 64 20.4 us; the two kernels' chains of dependent steps are what is left.
// (One kernel with a cluster per head and histograms summed over its shared memories: 16 and
// 14 us for one request of 8192 pages a head and for 64 heads of 1300, three meetings of the
// cluster taking half of it.)
#include <cuda_runtime.h>

#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace fp8kv {

namespace {

constexpr int kThreads = 512;                // of page_score; page_take: 512 or 1024
constexpr int kTakeWarps = 32;
constexpr int kBins = 1024;
constexpr int kFew = 128;                    // keys of a bin that are ranked one by one
constexpr uint32_t kForced = 0xffffffffu;    // sinks and recent pages: always taken
constexpr uint32_t kNan = 0xfffffffeu;       // a score that is not a number ranks first

// fp32 as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t sortable(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// a + b with the error of the sum in `err` (two-sum; what the sum of the group's heads
// loses is added at the end, so that it is rounded once).
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
    const float s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    err = __fadd_rn(err, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb)));
    return s;
}

// Pages of sequence b (its length may not pass the table).
__device__ __forceinline__ int pages_of(const PageSelectParams& p, int b, bool report_errors) {
    int ctx = p.context_lens[b];
    if (ctx > p.max_blocks_per_seq * kPage) {
        if (report_errors) report(p.err, FP8KV_ERR_BAD_INDEX);
        ctx = p.max_blocks_per_seq * kPage;
    }
    return ctx > 0 ? (ctx + kPage - 1) / kPage : 0;
}

// blockIdx.x: chunk of kThreads pages, then (sequence, KV head).
template <int D>
__global__ void __launch_bounds__(kThreads, 2) page_score_kernel(PageSelectParams p, int chunks) {
    constexpr int kLoads = 2 * D / 64;       // 16-byte pieces of a page's bounds a lane takes
    constexpr int kSubs = 256 / D;           // groups of 8 pages whose pieces are in flight
    __shared__ __align__(16) int8_t code[2 * D];             // the query in 8 bits
    __shared__ float wmax[D / 32];
    const int unit = static_cast<int>(blockIdx.x) / chunks;
    const int b = unit / p.Hkv, h = unit - b * p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quad = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    const int n = pages_of(p, b, h == 0 && blockIdx.x % chunks == 0 && tid == 0);
    const int page = (static_cast<int>(blockIdx.x) - unit * chunks) * kThreads + tid;
    if (n <= p.budget || page - tid >= n) return;            // the whole CTA

    // ---- bounds: a quad of lanes per page, 32 pages a warp
    int blk = -1;
    if (page < n) blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks_per_seq + page];
    const __nv_bfloat16* q = p.q + (static_cast<int64_t>(b) * p.Hq + h * p.G) * D + tid;
    float x0 = tid < D ? __bfloat162float(q[0]) : 0.f;       // (its latency beside the table's)
    const bool ok = blk >= 0 && blk < p.num_blocks;
    const int64_t row = ok ? static_cast<int64_t>(blk) * p.Hkv + h : 0;
    const float scale = ok ? p.bounds_scale[row] : 0.f;
    uint4 x[kSubs][kLoads];
    auto load = [&](int s0) {
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
            const int64_t r = __shfl_sync(0xffffffffu, row, (s0 + sub) * 8 + quad);
            const uint4* src = reinterpret_cast<const uint4*>(p.bounds + r * (2 * D)) + c;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) x[sub][k] = __ldg(src + k * 4);
        }
    };
    load(0);

    // ---- the query's 8-bit codes
    float pos = 0.f, neg = 0.f;
    if (tid < D) {
        float ep = 0.f, en = 0.f;
        for (int g = 0; g < p.G; ++g) {
            pos = two_sum(pos, fmaxf(x0, 0.f), ep);          // NaN counts as 0
            neg = two_sum(neg, fminf(x0, 0.f), en);
            if (g + 1 < p.G) x0 = __bfloat162float(q[static_cast<int64_t>(g + 1) * D]);
        }
        pos = __fadd_rn(pos, ep);
        neg = __fadd_rn(neg, en);
        if (!(pos <= FLT_MAX)) pos = FLT_MAX;                // infinities: the largest number
        if (!(neg >= -FLT_MAX)) neg = -FLT_MAX;
    }
    float a = fmaxf(pos, -neg);
    if (warp < D / 32) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        if (lane == 0) wmax[warp] = a;
    }
    __syncthreads();
    if (tid < D) {
        a = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) a = fmaxf(a, wmax[w]);
        const float s = __fdiv_rn(a, 127.f);
        auto to_code = [&](float v) {
            return s == 0.f ? 0 : max(-127, min(127, __float2int_rn(__fdiv_rn(v, s))));
        };
        code[tid] = static_cast<int8_t>(to_code(pos));
        code[D + tid] = static_cast<int8_t>(to_code(neg));
    }
    __syncthreads();

    // ---- scores
    int dot = 0;
#pragma unroll
    for (int s0 = 0; s0 < 4; s0 += kSubs) {
        if (s0 > 0) load(s0);
        int d[kSubs] = {};
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const uint4 qc = *reinterpret_cast<const uint4*>(&code[(k * 4 + c) * 16]);
#pragma unroll
            for (int sub = 0; sub < kSubs; ++sub) {
                d[sub] = __dp4a(static_cast<int>(x[sub][k].x), static_cast<int>(qc.x), d[sub]);
                d[sub] = __dp4a(static_cast<int>(x[sub][k].y), static_cast<int>(qc.y), d[sub]);
                d[sub] = __dp4a(static_cast<int>(x[sub][k].z), static_cast<int>(qc.z), d[sub]);
                d[sub] = __dp4a(static_cast<int>(x[sub][k].w), static_cast<int>(qc.w), d[sub]);
            }
        }
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
            d[sub] += __shfl_xor_sync(0xffffffffu, d[sub], 1);
            d[sub] += __shfl_xor_sync(0xffffffffu, d[sub], 2);
            const int mine = __shfl_sync(0xffffffffu, d[sub], (lane & 7) * 4);
            if ((lane >> 3) == s0 + sub) dot = mine;
        }
    }
    if (page >= n) return;
    // + 0: a product of -0 ties with one of 0
    const float score = __fadd_rn(__fmul_rn(static_cast<float>(dot), scale), 0.f);
    uint32_t key = score == score ? sortable(score) : kNan;
    if (!ok) {
        report(p.err, FP8KV_ERR_BAD_INDEX);
        key = 0u;                                            // behind every score
    }
    if (page < p.sink || page >= n - p.recent) key = kForced;
    p.keys[static_cast<int64_t>(unit) * p.max_blocks_per_seq + page] = key;
}

struct Shared {
    uint32_t hist[kBins];
    uint2 few[kFew];                         // the keys of the last bin, and their pages
    uint32_t wlo[kTakeWarps], whi[kTakeWarps];
    uint32_t wsum[kTakeWarps];
    uint32_t found[3];                       // bin, keys above it, keys in it
    uint32_t n_few;
    uint32_t wabove[kTakeWarps], wtie[kTakeWarps];
    uint32_t last[2];                        // the last key that is taken, and its page
};

// A CTA per (sequence, KV head).  SMEM: its keys fit the shared memory behind `Shared`.
template <bool SMEM>
__global__ void __launch_bounds__(kTakeWarps * 32, 1) page_take_kernel(PageSelectParams p) {
    extern __shared__ uint4 smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    uint32_t* const copy = reinterpret_cast<uint32_t*>(smem_raw + (sizeof(Shared) + 15) / 16);
    const int unit = static_cast<int>(blockIdx.x);
    const int b = unit / p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
    const uint32_t* const scored = p.keys + static_cast<int64_t>(unit) * p.max_blocks_per_seq;
    const uint32_t* const keys = SMEM ? copy : scored;
    int32_t* out = p.pages + static_cast<int64_t>(unit) * p.budget;
    for (int i = tid; i < kBins; i += threads) sh.hist[i] = 0u;
    if (tid == 0) sh.n_few = 0u;
    // (page_score lets this kernel start after it has itself waited for its predecessor)
    const int n = pages_of(p, b, false);
    pdl_wait();                              // the scores are there
    pdl_trigger();
    if (n <= p.budget) {                     // every page: no scores
        for (int i = tid; i < p.budget; i += threads) out[i] = i < n ? i : -1;
        if (tid == 0) p.counts[unit] = n;
        return;
    }

    uint32_t lo = 0xffffffffu, hi = 0u;
    constexpr int kBatch = 4;                // loads in flight
    for (int i0 = tid; i0 < n; i0 += kBatch * threads) {
        uint32_t k[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (i0 + u * threads < n) k[u] = scored[i0 + u * threads];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i0 + u * threads >= n) break;
            if (SMEM) copy[i0 + u * threads] = k[u];
            if (k[u] != kForced) {
                lo = min(lo, k[u]);
                hi = max(hi, k[u]);
            }
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.wlo[warp] = lo;
        sh.whi[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, lane < warps ? sh.wlo[lane] : 0xffffffffu);
    hi = __reduce_max_sync(0xffffffffu, lane < warps ? sh.whi[lane] : 0u);

    // ---- the bin [lo, hi] that holds the last key taken: keys above it are taken, and `need`
    //      of the in_bin keys in it.  n > budget >= sink + recent, so the forced ranges are
    //      disjoint and more than `need` other pages exist.
    uint32_t need = static_cast<uint32_t>(p.budget - p.sink - p.recent), in_bin = 0u;
    if (need == 0u) lo = hi = kNan;                          // (only the forced ones lie above)
    while (need > 0u) {
        const int shift = max(0, 22 - __clz(hi - lo));       // (hi - lo) >> shift < 1024
#pragma unroll 4
        for (int i = tid; i < n; i += threads) {
            const uint32_t k = keys[i];
            if (k != kForced && k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        // sums from the highest bin down: thread t < 512 holds bins 1023 - 2 t and 1022 - 2 t
        const int at = kBins - 2 - 2 * tid;
        uint2 v = make_uint2(0u, 0u);
        if (at >= 0) v = reinterpret_cast<const uint2*>(sh.hist)[at / 2];
        const uint32_t both = v.x + v.y;
        uint32_t incl = both;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        if (at >= 0) reinterpret_cast<uint2*>(sh.hist)[at / 2] = make_uint2(0u, 0u);
        const uint32_t lower = __reduce_add_sync(0xffffffffu, lane < warp ? sh.wsum[lane] : 0u);
        const uint32_t above = lower + incl - both;          // keys in higher bins
        if (above < need && above + both >= need) {          // one thread of the CTA
            const bool upper = above + v.y >= need;
            sh.found[0] = static_cast<uint32_t>(upper ? at + 1 : at);
            sh.found[1] = upper ? above : above + v.y;
            sh.found[2] = upper ? v.y : v.x;
        }
        __syncthreads();
        need -= sh.found[1];
        in_bin = sh.found[2];
        lo += sh.found[0] << shift;
        const uint32_t width = (1u << shift) - 1u;
        if (hi - lo > width) hi = lo + width;                // (lo + width may pass 32 bits)
        if (shift == 0 || in_bin <= kFew) break;
        __syncthreads();                                     // found[] is read
    }

    // ---- a warp takes a run of keys: how many lie above the bin, and in it; the few of the bin
    const bool few = in_bin <= kFew;
    const int run = ((n + warps - 1) / warps + 31) / 32 * 32;
    const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
    uint32_t above = 0u, tie = 0u;           // of this lane
#pragma unroll 4
    for (int i = r0 + lane; i < r1; i += 32) {
        const uint32_t k = keys[i];
        above += k > hi;
        if (k >= lo && k <= hi && in_bin > 0u) {
            ++tie;
            if (few) sh.few[atomicAdd(&sh.n_few, 1u)] = make_uint2(k, i);
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
        sh.wabove[warp] = above;
        sh.wtie[warp] = tie;
    }
    __syncthreads();
    // ---- the last key taken, by rank among the few (or, of equal ones, the need-th by page)
    if (few && tid < static_cast<int>(in_bin)) {
        const uint2 me = sh.few[tid];
        uint32_t first = 0u;                                 // keys that go before this one
#pragma unroll 4
        for (uint32_t i = 0; i < in_bin; ++i) {
            const uint2 o = sh.few[i];
            first += o.x > me.x || (o.x == me.x && o.y < me.y);
        }
        if (first + 1u == need) {
            sh.last[0] = me.x;
            sh.last[1] = me.y;
        }
    }
    __syncthreads();
    const uint32_t last_key = sh.last[0], last_page = sh.last[1];
    auto of_few = [&](uint32_t k, uint32_t page) {
        return k > last_key || (k == last_key && page <= last_page);
    };
    // pages taken in front of this warp's run
    uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? sh.wabove[lane] : 0u);
    uint32_t tied = __reduce_add_sync(0xffffffffu, lane < warp ? sh.wtie[lane] : 0u);
    if (few) {
        uint32_t taken = 0u;
        for (uint32_t i = lane; i < in_bin; i += 32)
            taken += sh.few[i].y < static_cast<uint32_t>(r0) && of_few(sh.few[i].x, sh.few[i].y);
        at += __reduce_add_sync(0xffffffffu, taken);
    } else {
        at += min(tied, need);
    }

    // ---- the pages in their order
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
    for (int i = r0 + lane; i - lane < r1; i += 32) {
        const bool in = i < r1;
        const uint32_t k = in ? keys[i] : 0u;
        const bool here = in && in_bin > 0u && k >= lo && k <= hi;
        const uint32_t ties = __ballot_sync(0xffffffffu, here);
        const bool part = few ? of_few(k, i) : tied + __popc(ties & below) < need;
        const bool take = in && (k > hi || (here && part));
        const uint32_t taken = __ballot_sync(0xffffffffu, take);
        if (take) {
            const uint32_t w = at + __popc(taken & below);
            if (w < static_cast<uint32_t>(p.budget)) out[w] = i;
        }
        at += __popc(taken);
        tied += __popc(ties);
    }
    if (tid == 0) p.counts[unit] = p.budget;
}

// Keys that a CTA of page_take keeps in shared memory (800 thousand positions); more are read
// from the workspace again.
constexpr int kSmemKeys = 50000;

}  // namespace

cudaError_t launch_page_select(const PageSelectParams& p, int D, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv;
    const int chunks = (p.max_blocks_per_seq + kThreads - 1) / kThreads;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, units * chunks, kThreads, 0, stream);
    cudaError_t e;
    if (D == 64)
        e = cudaLaunchKernelEx(&cfg, page_score_kernel<64>, p, chunks);
    else if (D == 128)
        e = cudaLaunchKernelEx(&cfg, page_score_kernel<128>, p, chunks);
    else
        e = cudaLaunchKernelEx(&cfg, page_score_kernel<256>, p, chunks);
    if (e != cudaSuccess) return e;
    const bool fits = p.max_blocks_per_seq <= kSmemKeys;
    const int base = static_cast<int>((sizeof(Shared) + 15) / 16 * 16);
    static unsigned long long done[64] = {};
    if (fits) {
        e = opt_in_smem(reinterpret_cast<const void*>(page_take_kernel<true>), base + kSmemKeys * 4,
                        done);
        if (e != cudaSuccess) return e;
    }
    // few heads: a CTA of 1024 threads for each, more: two CTAs a SM
    cfg = pdl_config(attr, units, units <= sm_count() ? 1024 : 512,
                     base + (fits ? p.max_blocks_per_seq * 4 : 0), stream);
    return fits ? cudaLaunchKernelEx(&cfg, page_take_kernel<true>, p)
                : cudaLaunchKernelEx(&cfg, page_take_kernel<false>, p);
}

}  // namespace fp8kv
