// page_select.cu -- the pages a decode query reads: a cheap score of every page from its
// 8-bit bounds (page_bounds.cu), and the `budget` pages with the highest scores.
//
// For sequence b and KV head h with the query heads g of its group,
//     u = [sum_g max(q_g, 0), sum_g min(q_g, 0)]            2 D values, 8 bits: c = rint(u / s)
//     score(page) = fp32(sum_d c_d hi_d + c_{D+d} lo_d) * bounds_scale
// the sum over the group's heads of the largest logit a key inside the page's bounds could
// have (up to the factor s, which all pages of a head share).  Because the sum over heads
// moves into the query, a page costs one product of 2 D bytes whatever the group's size.
// The products are whole numbers (below 2^23, exact in fp32), so the score has one
// rounding, does not depend on the order of the sums, and the selection is reproducible:
// ties go to the lower page.
//
// Bound: HBM for the bounds (2 D + 4 bytes a page and head) in large batches, latency for
// one request.  Split: a thread-block cluster takes one (sequence, KV head), its CTAs equal
// runs of pages; scores stay in shared memory as sortable 32-bit keys.  The threshold is
// found by narrowing [lowest, highest key] to one of 1024 equal bins at a time, with
// histograms in shared memory that every CTA sums over the cluster's (distributed shared
// memory): two to three rounds, then each CTA writes its pages behind those of the ranks
// below.  One launch, no workspace, no global atomics.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace fp8kv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr uint32_t kForced = 0xffffffffu;    // sinks and recent pages: always taken
constexpr uint32_t kNan = 0xfffffffeu;       // a score that is not a number ranks first

struct Shared {
    uint32_t hist[2][kBins];
    int8_t code[512];                        // the query in 8 bits, 2 D of them
    float wmax[kWarps];
    uint32_t wlo[kWarps], whi[kWarps];
    uint32_t range[2];                       // this CTA's lowest and highest key
    uint32_t wsum[kWarps];
    uint32_t found[3];                       // bin, keys above it, keys in it
    uint32_t wabove[kWarps], wtie[kWarps];
    uint32_t total[2];                       // this CTA's keys above the threshold, at it
};

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

template <int D>
__global__ void __launch_bounds__(kThreads) page_select_kernel(PageSelectParams p) {
    constexpr int kLoads = 2 * D / 64;       // 16-byte pieces of a page's bounds a lane takes
    extern __shared__ uint4 smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + (sizeof(Shared) + 15) / 16);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int ranks = static_cast<int>(cluster.num_blocks());
    const int unit = static_cast<int>(blockIdx.x) / ranks;
    const int b = unit / p.Hkv, h = unit - b * p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto sync = [&]() {
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    pdl_wait();
    pdl_trigger();

    int ctx = p.context_lens[b];
    if (ctx > p.max_blocks_per_seq * kPage) {
        if (h == 0 && rank == 0 && tid == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        ctx = p.max_blocks_per_seq * kPage;
    }
    const int n = ctx > 0 ? (ctx + kPage - 1) / kPage : 0;
    int32_t* out = p.pages + static_cast<int64_t>(unit) * p.budget;
    if (n <= p.budget) {                     // every page: no scores
        for (int i = rank * kThreads + tid; i < p.budget; i += ranks * kThreads)
            out[i] = i < n ? i : -1;
        if (rank == 0 && tid == 0) p.counts[unit] = n;
        return;                              // the whole cluster
    }
    const int per = (n + ranks - 1) / ranks; // pages of a rank
    const int p0 = min(n, rank * per), mine = min(n, p0 + per) - p0;
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq + p0;

    // ---- the query's 8-bit codes
    float pos = 0.f, neg = 0.f;
    if (tid < D) {
        const __nv_bfloat16* q = p.q + (static_cast<int64_t>(b) * p.Hq + h * p.G) * D + tid;
        float ep = 0.f, en = 0.f;
        for (int g = 0; g < p.G; ++g) {
            const float x = __bfloat162float(q[static_cast<int64_t>(g) * D]);
            pos = two_sum(pos, fmaxf(x, 0.f), ep);           // NaN counts as 0
            neg = two_sum(neg, fminf(x, 0.f), en);
        }
        pos = __fadd_rn(pos, ep);
        neg = __fadd_rn(neg, en);
        if (!(pos <= FLT_MAX)) pos = FLT_MAX;                // infinities: the largest number
        if (!(neg >= -FLT_MAX)) neg = -FLT_MAX;
    }
    float a = fmaxf(pos, -neg);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (lane == 0) sh.wmax[warp] = a;
    for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0u;
    __syncthreads();
    if (tid < D) {
        a = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) a = fmaxf(a, sh.wmax[w]);
        const float s = __fdiv_rn(a, 127.f);
        auto code = [&](float x) {
            return s == 0.f ? 0 : max(-127, min(127, __float2int_rn(__fdiv_rn(x, s))));
        };
        sh.code[tid] = static_cast<int8_t>(code(pos));
        sh.code[D + tid] = static_cast<int8_t>(code(neg));
    }
    __syncthreads();

    // ---- scores: a quad of lanes per page, 32 pages a warp at a time
    const int quad = lane >> 2, c = lane & 3;
    uint4 qc[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        qc[i] = *reinterpret_cast<const uint4*>(&sh.code[(i * 4 + c) * 16]);
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int i0 = warp * 32; i0 < mine; i0 += kThreads) {
        const int i = i0 + lane;
        int blk = -1;
        if (i < mine) blk = table[i];
        const bool ok = blk >= 0 && blk < p.num_blocks;
        const int64_t row = ok ? static_cast<int64_t>(blk) * p.Hkv + h : 0;
        const float scale = ok ? p.bounds_scale[row] : 0.f;
        int dot = 0;
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
            const int64_t r = __shfl_sync(0xffffffffu, row, sub * 8 + quad);
            const uint4* src = reinterpret_cast<const uint4*>(p.bounds + r * (2 * D)) + c;
            uint4 x[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) x[k] = __ldg(src + k * 4);
            int d = 0;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                d = __dp4a(static_cast<int>(x[k].x), static_cast<int>(qc[k].x), d);
                d = __dp4a(static_cast<int>(x[k].y), static_cast<int>(qc[k].y), d);
                d = __dp4a(static_cast<int>(x[k].z), static_cast<int>(qc[k].z), d);
                d = __dp4a(static_cast<int>(x[k].w), static_cast<int>(qc[k].w), d);
            }
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            const int mine_d = __shfl_sync(0xffffffffu, d, (lane & 7) * 4);
            if ((lane >> 3) == sub) dot = mine_d;
        }
        if (i < mine) {
            // + 0: a product of -0 ties with one of 0
            const float score = __fadd_rn(__fmul_rn(static_cast<float>(dot), scale), 0.f);
            uint32_t key = score == score ? sortable(score) : kNan;
            if (!ok) {
                report(p.err, FP8KV_ERR_BAD_INDEX);
                key = 0u;                                    // behind every score
            }
            if (p0 + i < p.sink || p0 + i >= n - p.recent) {
                key = kForced;
            } else {
                lo = min(lo, key);
                hi = max(hi, key);
            }
            keys[i] = key;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (lane == 0) {
        sh.wlo[warp] = lo;
        sh.whi[warp] = hi;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) {
            lo = min(lo, sh.wlo[w]);
            hi = max(hi, sh.whi[w]);
        }
        sh.range[0] = lo;
        sh.range[1] = hi;
    }
    sync();
    for (int r = 0; r < ranks; ++r) {
        const uint32_t* o = ranks > 1 ? cluster.map_shared_rank(sh.range, r) : sh.range;
        const uint32_t l = o[0], u = o[1];
        lo = r == 0 ? l : min(lo, l);
        hi = r == 0 ? u : max(hi, u);
    }

    // ---- the threshold: keys above `top` are taken, and the first `ties` (in page order)
    //      of those equal to it.  n > budget >= sink + recent, so the forced ranges are
    //      disjoint and more than `need` other pages exist.
    uint32_t need = static_cast<uint32_t>(p.budget - p.sink - p.recent);
    uint32_t top = kNan, ties = 0u;
    for (int round = 0; need > 0u; ++round) {
        uint32_t* hist = sh.hist[round & 1];
        const uint32_t span = hi - lo;
        const int shift = max(0, 22 - __clz(span));          // span >> shift < 1024
        for (int i = tid; i < mine; i += kThreads) {
            const uint32_t k = keys[i];
            if (k != kForced && k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1u);
        }
        sync();
        // suffix sums: thread t holds bins 1023 - 2 t and 1022 - 2 t, highest first
        const int at = kBins - 2 - 2 * tid;
        uint2 v = make_uint2(0u, 0u);
        for (int r = 0; r < ranks; ++r) {
            const uint2* o = reinterpret_cast<const uint2*>(
                ranks > 1 ? cluster.map_shared_rank(hist, r) : hist);
            const uint2 x = o[at / 2];
            v.x += x.x;
            v.y += x.y;
        }
        const uint32_t both = v.x + v.y;
        uint32_t incl = both;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        uint32_t above = incl - both;                        // keys in higher bins
        for (int w = 0; w < warp; ++w) above += sh.wsum[w];
        if (above < need && above + both >= need) {          // one thread of the CTA
            const bool upper = above + v.y >= need;
            sh.found[0] = static_cast<uint32_t>(upper ? at + 1 : at);
            sh.found[1] = upper ? above : above + v.y;
            sh.found[2] = upper ? v.y : v.x;
        }
        // the other buffer was last read in the round before, which every CTA has left
        for (int i = tid; i < kBins; i += kThreads) sh.hist[(round & 1) ^ 1][i] = 0u;
        __syncthreads();
        const uint32_t bin = sh.found[0], in_bin = sh.found[2];
        need -= sh.found[1];
        lo += bin << shift;
        const uint32_t width = (1u << shift) - 1u;
        if (hi - lo > width) hi = lo + width;                // (lo + width may pass 32 bits)
        if (shift == 0 || in_bin == need) {
            // every key of the bin is one value, or all of them are taken
            top = shift == 0 ? lo : lo - 1u;
            ties = shift == 0 ? need : 0u;
            if (shift != 0 && lo == 0u) {                    // nothing lies below key 0
                top = 0u;
                ties = 0xffffffffu;
            }
            break;
        }
        __syncthreads();                                     // found[] is read
    }

    // ---- the pages in their order: warp w takes a run of its own
    const int run = ((mine + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int r0 = min(mine, warp * run), r1 = min(mine, r0 + run);
    uint32_t above = 0u, tie = 0u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const uint32_t k = i0 + lane < r1 ? keys[i0 + lane] : 0u;
        const bool in = i0 + lane < r1;
        above += __popc(__ballot_sync(0xffffffffu, in && k > top));
        tie += __popc(__ballot_sync(0xffffffffu, in && k == top));
    }
    if (lane == 0) {
        sh.wabove[warp] = above;
        sh.wtie[warp] = tie;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t sa = 0u, st = 0u;
        for (int w = 0; w < kWarps; ++w) {
            sa += sh.wabove[w];
            st += sh.wtie[w];
        }
        sh.total[0] = sa;
        sh.total[1] = st;
    }
    sync();
    uint32_t na = 0u, nt = 0u;               // keys above, at the threshold, before this run
    for (int r = 0; r < rank; ++r) {
        const uint32_t* o = cluster.map_shared_rank(sh.total, r);
        na += o[0];
        nt += o[1];
    }
    for (int w = 0; w < warp; ++w) {
        na += sh.wabove[w];
        nt += sh.wtie[w];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
        const bool in = i0 + lane < r1;
        const uint32_t k = in ? keys[i0 + lane] : 0u;
        const uint32_t ma = __ballot_sync(0xffffffffu, in && k > top);
        const uint32_t mt = __ballot_sync(0xffffffffu, in && k == top);
        const uint32_t ra = na + __popc(ma & below), rt = nt + __popc(mt & below);
        if (in && (k > top || (k == top && rt < ties))) {
            const uint32_t w = ra + min(rt, ties);
            if (w < static_cast<uint32_t>(p.budget)) out[w] = p0 + i0 + lane;
        }
        na += __popc(ma);
        nt += __popc(mt);
    }
    if (rank == 0 && tid == 0) p.counts[unit] = p.budget;
    if (ranks > 1) cluster.sync();           // the other ranks have read this one's totals
}

template <int D>
cudaError_t launch_d(const PageSelectParams& p, int ranks, int threads_pages,
                     cudaStream_t stream) {
    static unsigned long long done[64] = {};
    const int bytes = static_cast<int>((sizeof(Shared) + 15) / 16 * 16) + threads_pages * 4;
    const void* fn = reinterpret_cast<const void*>(page_select_kernel<D>);
    const cudaError_t e = opt_in_smem(fn, kSelectMaxSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg =
        pdl_config(attr, static_cast<int64_t>(p.B) * p.Hkv * ranks, kThreads, bytes, stream);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, page_select_kernel<D>, p);
}

}  // namespace

static_assert(sizeof(Shared) + kSelectMaxKeys * 4 + 16 <= kSelectMaxSmem, "shared memory");

cudaError_t launch_page_select(const PageSelectParams& p, int D, cudaStream_t stream) {
    // CTAs a (sequence, KV head): as many as fill the SMs about twice, each with at least 64
    // pages' worth of work, and enough that a CTA's keys fit its shared memory
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv;
    int ranks = 1;
    while (ranks < kSelectRanks && (units * ranks * 2 <= 2 * sm_count()) &&
           p.max_blocks_per_seq >= ranks * 2 * 64)
        ranks *= 2;
    while (ranks < kSelectRanks && (p.max_blocks_per_seq + ranks - 1) / ranks > kSelectMaxKeys) ranks *= 2;
    const int keys = (p.max_blocks_per_seq + ranks - 1) / ranks;
    if (D == 64) return launch_d<64>(p, ranks, keys, stream);
    if (D == 128) return launch_d<128>(p, ranks, keys, stream);
    return launch_d<256>(p, ranks, keys, stream);
}

}  // namespace fp8kv
