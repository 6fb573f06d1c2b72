// list_attn.cu -- decode attention of one query token per sequence over a list of pages of
// its own for every KV head: the pages that a selection left (sparse_decode_attn), or, behind
// a shared prefix, all pages of the sequence's own tail (prefix_decode_attn, whose prefix
// part prefix_attn.cu computes once for the whole batch; this kernel joins both).
//
//     o = sum_t softmax(z)_t s_v(t) code_v(t),  z_t = softmax_scale * s_k(t) q . code_k(t)
// over the tokens t below the context length on the listed pages.
//
// Bound: HBM (a page and head of D 128 is 4 KiB of codes) for batches, latency for one
// request: count -> page ids -> block ids -> pages -> join is a chain of dependent loads.
// Split: a unit is (sequence, KV head, up to 8 of its query heads); one CTA takes it, of as
// many warps as give every unit its share of the SMs', and where one CTA is too small for
// that a thread-block cluster of up to 8.  The warps deal the listed pages among themselves,
// and the parts of a unit meet in (distributed) shared memory: one launch, no plan, no
// workspace.  Units get equal shares whatever their lists hold, so among lists (or tails) of
// unequal length the longest decides.  (Clusters of small CTAs instead of
// larger CTAs: 54.4 against 50.6 us on 32 x 8 lists of 256 pages, D 128.)
//   * groups of 9 to 16 query heads are two units, which read a page each: 32 x 8 lists of 256
//     pages at D 128 take 86 us with 16 heads a group, 51 with 4 or 8.
//   * every warp has a ring of pages of its own, filled by 16-byte asynchronous copies from
//     all of its lanes: no barrier between warps until the join, and the wait is the lane's
//     own count of copies.  Pieces are placed by the 128-byte swizzle, so that the fragments
//     are read without bank conflicts.  (Straight from global memory into the fragments'
//     registers, without a ring: 71 us on 32 x 8 lists of 256 pages at D 128, where too little
//     was in flight while a warp computed.)
//   * S^T = K_page Q^T (16 tokens x 8 heads), O^T += V_page^T P^T, f16 operands (e4m3 codes
//     convert exactly, q is scaled by a power of two) or bf16 ones, fp32 accumulation.
//     Weights enter as hi + lo halves: 22 bits (f16), 16 bits (bf16).
//   * per-token V scales: the running reference m follows z_t + log2 s_v(t), so that the
//     weights p_t s_v(t) that enter the product lie below 2^4 whatever the scales are
//     (scales below 2^-100 count as that in the reference, which keeps p finite in fp32).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"
#include "prefix.cuh"

namespace fp8kv {

namespace {

namespace cg = cooperative_groups;

constexpr float kMaxInit = -1.0e30f;     // a reference below any real logit, finite

// Token of fragment row g (and of row g + 8: + 8): after the transposition of P a lane holds
// the weights of tokens c, c + 4 (c + 8, c + 12), whose V rows it loads.
__device__ __forceinline__ int perm8(int g) { return (g >> 1) | ((g & 1) << 2); }

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// hi + lo halves of two weights, both transposed into the B operand's layout.
template <bool BF16>
__device__ __forceinline__ void weight_terms(float w0, float w1, uint32_t& hi, uint32_t& lo) {
    if constexpr (BF16) {
        const uint32_t x = pack_bf16x2(w0, w1);
        const float2 f = unpack_bf16x2(x);
        hi = transposed(x);
        lo = transposed(pack_bf16x2(w0 - f.x, w1 - f.y));
    } else {
        const uint32_t x = pack_f16x2(w0, w1);
        const float2 f = unpack_f16x2(x);
        hi = transposed(x);
        lo = transposed(pack_f16x2(w0 - f.x, w1 - f.y));
    }
}

template <int D, bool BF16>
struct Shape {
    static constexpr int kElem = BF16 ? 2 : 1;
    static constexpr int kRowB = D * kElem;
    static constexpr int kTileB = kPage * kRowB;
    static constexpr int kSegs = kRowB / 64;            // 16-byte pieces of a K row a lane takes
    static constexpr int kPerSeg = 4 / kElem;           // k-steps a piece feeds
    static constexpr int kSteps = D / 16;               // k-steps of S, row tiles of O^T
    static constexpr int kVBytes = kRowB / 8;           // V bytes a lane takes per token
    static constexpr int kVWords = kVBytes / 4;
    static constexpr int kCopies = kTileB / 512;        // 16-byte copies of a lane per tile
    // a stage: K tile, V tile, their scale rows (64 bytes each), the page's first position
    static constexpr int kStageB = 2 * kTileB + 128;
    // warps an SM is to hold (registers and shared memory) and pages in a warp's ring: about
    // 200 KiB an SM in flight
    static constexpr int kSmWarps = kRowB <= 128 ? 16 : kRowB == 256 ? 12 : 6;
    static constexpr int kStages = kRowB == 64 ? 4 : kRowB == 128 ? 3 : 2;
    static constexpr int kWarpB = kStages * kStageB;
    static constexpr int kOStride = D + 4;              // floats of a head's row of partial O
    // the join reuses the rings
    static_assert(8 * (kOStride + 2) * 4 <= kWarpB, "a warp's part fits its ring");
    static constexpr int smem(int warps) { return warps * (kWarpB + kStages * 4); }
    static_assert(smem(kSmWarps) + 1024 <= 227 * 1024, "shared memory");
};

// Byte offset of 16-byte piece c of token row t in a tile under the 128-byte swizzle.  Rows
// of 64 bytes lie two to a line, wider ones as panels of 128 bytes.
template <int ROWB>
__device__ __forceinline__ int piece_at(int t, int c) {
    if constexpr (ROWB == 64) {
        const int r = t >> 1, cc = ((t & 1) << 2) | c;
        return r * 128 + ((cc ^ (r & 7)) << 4);
    } else {
        return (c >> 3) * 2048 + t * 128 + (((c & 7) ^ (t & 7)) << 4);
    }
}

template <int D, bool BF16, bool PT, bool PREFIX>
__global__ void __launch_bounds__(Shape<D, BF16>::kSmWarps * 32)
    list_attn_kernel(ListAttnParams p) {
    using S = Shape<D, BF16>;
    extern __shared__ __align__(128) uint8_t smem[];
    float* const part_o = reinterpret_cast<float*>(smem);   // [warp][8][kOStride], at the end
    const int n_warps = static_cast<int>(blockDim.x) >> 5;
    float* const part_m = part_o + n_warps * 8 * S::kOStride;
    float* const part_l = part_m + n_warps * 8;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int ranks = static_cast<int>(cluster.num_blocks());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int unit = static_cast<int>(blockIdx.x) / ranks;
    const int groups = (p.G + 7) / 8;
    const int bh = unit / groups;                       // (sequence, KV head)
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int head0 = (unit - bh * groups) * 8;         // of the KV head's group
    const int heads = min(8, p.G - head0);

    // Behind a prefix the preceding kernel is prefix_attn, which lets this one start after it
    // has itself waited for its predecessor: only the prefix's partials need the wait (below).
    if constexpr (!PREFIX) pdl_wait();
    pdl_trigger();

    int ctx = p.context_lens[b];
    if (ctx > p.max_blocks_per_seq * kPage) {
        if (h == 0 && rank == 0 && threadIdx.x == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        ctx = p.max_blocks_per_seq * kPage;
    }
    const int n_pages = ctx > 0 ? (ctx + kPage - 1) / kPage : 0;
    int n;
    if constexpr (PREFIX)
        n = n_pages;
    else
        n = p.counts != nullptr ? min(max(p.counts[bh], 0), p.budget) : p.budget;
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks_per_seq;
    const int32_t* list = PREFIX ? nullptr : p.pages + static_cast<int64_t>(bh) * p.budget;

    // ---- the query as the B operand of S^T: head g of the unit
    uint2 qb[S::kSteps];
    float hs0, hs1;                                     // logit factors (base 2) of heads 2c, 2c + 1
    {
        const __nv_bfloat16* q =
            p.q + (static_cast<int64_t>(b) * p.Hq + h * p.G + head0 + g) * D;
#pragma unroll
        for (int ks = 0; ks < S::kSteps; ++ks) {
            const int s = ks / S::kPerSeg, j = ks % S::kPerSeg;
            const int d0 = s * (64 / S::kElem) + c * (16 / S::kElem) + 4 * j;
            qb[ks] = g < heads ? *reinterpret_cast<const uint2*>(q + d0) : make_uint2(0u, 0u);
        }
        float f = p.scale_log2;
        if constexpr (!BF16) {
            float amax = 0.f;
#pragma unroll
            for (int ks = 0; ks < S::kSteps; ++ks) {
                const float2 x = unpack_bf16x2(qb[ks].x), y = unpack_bf16x2(qb[ks].y);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // the power of two that puts max |q| into [2^14, 2^15): exact in f16 but for
            // values 2^-31 and less of the largest
            int e = 0;
            if (amax > 0.f && amax <= 3.4e38f) {
                frexpf(amax, &e);
                e = min(126, max(-126, 15 - e));
            }
            const float up = ldexpf(1.f, e);
#pragma unroll
            for (int ks = 0; ks < S::kSteps; ++ks) {
                const float2 x = unpack_bf16x2(qb[ks].x), y = unpack_bf16x2(qb[ks].y);
                qb[ks].x = pack_f16x2(x.x * up, x.y * up);
                qb[ks].y = pack_f16x2(y.x * up, y.y * up);
            }
            f = f * ldexpf(1.f, -e);
            if constexpr (!PT)
                f *= p.k_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
        }
        hs0 = __shfl_sync(0xffffffffu, f, (2 * c) * 4);
        hs1 = __shfl_sync(0xffffffffu, f, (2 * c + 1) * 4);
    }

    float o[S::kSteps][4];
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = kMaxInit, m1 = kMaxInit, l0 = 0.f, l1 = 0.f;
    constexpr float kLazy = BF16 ? 8.f : 4.f;           // how far logits may pass the reference
    constexpr float kLift = BF16 ? 1.f : 16.f;          // of the f16 weights, into normal numbers
    const int tA = perm8(g), tB = tA + 8;

    // ---- this warp's entries of the list: worker + i * workers, 32 of them looked up at once
    //      (lane j holds the j-th's block and first token), the next 32 while these run
    const int workers = ranks * n_warps, worker = rank * n_warps + warp;
    const int per_warp = n > worker ? (n - worker + workers - 1) / workers : 0;
    auto look_up = [&](int first, int& blk, int& pos) {
        blk = -1;
        pos = 0;
        if (first + lane < per_warp) {
            const int i = worker + (first + lane) * workers;
            const int page = PREFIX ? i : list[i];
            if (page >= 0 && page < n_pages) {
                const int x = table[page];
                if (x >= 0 && x < p.num_blocks) {
                    blk = x;
                    pos = page * kPage;
                } else {
                    report(p.err, FP8KV_ERR_BAD_INDEX);
                }
            }
        }
    };
    int blk, pos, blk_next, pos_next, first = 0;
    look_up(0, blk, pos);
    look_up(32, blk_next, pos_next);
    uint32_t left = __ballot_sync(0xffffffffu, blk >= 0);
    // the next page: its tile, or -1
    auto next = [&](int64_t& tile, int& at) {
        while (left == 0u && first + 32 < per_warp) {
            first += 32;
            blk = blk_next;
            pos = pos_next;
            look_up(first + 32, blk_next, pos_next);
            left = __ballot_sync(0xffffffffu, blk >= 0);
        }
        at = -1;
        if (left != 0u) {
            const int j = __ffs(left) - 1;
            left &= left - 1u;
            tile = static_cast<int64_t>(__shfl_sync(0xffffffffu, blk, j)) * p.Hkv + h;
            at = __shfl_sync(0xffffffffu, pos, j);
        }
    };
    // ---- the ring: stage s holds page i with i % kStages == s
    uint8_t* const ring = smem + warp * S::kWarpB;
    int* const at_of = reinterpret_cast<int*>(smem + n_warps * S::kWarpB) + warp * S::kStages;
    const uint64_t policy = l2_evict_first();           // pages are read once
    auto issue = [&](int stage) {
        int64_t tile;
        int at;
        next(tile, at);
        if (lane == 0) at_of[stage] = at;
        if (at >= 0) {
            const uint8_t* ks = p.k_cache + tile * S::kTileB + lane * 16;
            const uint8_t* vs = p.v_cache + tile * S::kTileB + lane * 16;
            const uint32_t dst = smem_addr(ring + stage * S::kStageB);
#pragma unroll
            for (int i = 0; i < S::kCopies; ++i) {
                const int piece = i * 32 + lane;
                const uint32_t o = piece_at<S::kRowB>(piece / (S::kRowB / 16), piece % (S::kRowB / 16));
                cp_async16_hint(dst + o, ks + i * 512, policy);
                cp_async16_hint(dst + S::kTileB + o, vs + i * 512, policy);
            }
            if constexpr (PT) {
                if (lane < 8)
                    cp_async16_hint(dst + 2 * S::kTileB + lane * 16,
                                    (lane < 4 ? p.k_scale_cache : p.v_scale_cache) + tile * kPage +
                                        (lane & 3) * 4,
                                    policy);
            }
        }
        cp_async_commit();                              // (an empty group behind the last page)
    };
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) issue(i);

    for (int stage = 0;; stage = stage + 1 == S::kStages ? 0 : stage + 1) {
        cp_async_wait<S::kStages - 1>();
        __syncwarp();                                   // every lane's copies have landed
        const int at = at_of[stage];
        if (at < 0) break;
        const uint8_t* kt = ring + stage * S::kStageB;
        const uint8_t* vt = kt + S::kTileB;
        // ---- S^T (rows: tokens tA, tB; columns: heads 2c, 2c + 1)
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S::kSegs; ++s) {
            const uint4 x = *reinterpret_cast<const uint4*>(kt + piece_at<S::kRowB>(tA, 4 * s + c));
            const uint4 y = *reinterpret_cast<const uint4*>(kt + piece_at<S::kRowB>(tB, 4 * s + c));
            const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < S::kPerSeg; ++j) {
                const uint2 qf = qb[s * S::kPerSeg + j];
                if constexpr (BF16) {
                    mma16<true>(z, wx[2 * j], wy[2 * j], wx[2 * j + 1], wy[2 * j + 1], qf.x, qf.y);
                } else {
                    uint32_t xl, xh, yl, yh;
                    f16x2x2_from_e4m3x4(wx[j], xl, xh);
                    f16x2x2_from_e4m3x4(wy[j], yl, yh);
                    mma16<false>(z, xl, yl, xh, yh, qf.x, qf.y);
                }
            }
        }
        // ---- logits; the reference follows z + log2 s_v
        const bool vA = at + tA < ctx, vB = at + tB < ctx;
        float ksA = 1.f, ksB = 1.f, lvA = 0.f, lvB = 0.f, vsA = 1.f, vsB = 1.f;
        if constexpr (PT) {
            const float* scl = reinterpret_cast<const float*>(kt + 2 * S::kTileB);
            ksA = scl[tA];
            ksB = scl[tB];
            vsA = vA ? scl[16 + tA] : 0.f;
            vsB = vB ? scl[16 + tB] : 0.f;
            lvA = fmaxf(__log2f(fabsf(vsA)), -100.f);
            lvB = fmaxf(__log2f(fabsf(vsB)), -100.f);
        }
        z[0] = vA ? z[0] * hs0 * ksA : -CUDART_INF_F;
        z[1] = vA ? z[1] * hs1 * ksA : -CUDART_INF_F;
        z[2] = vB ? z[2] * hs0 * ksB : -CUDART_INF_F;
        z[3] = vB ? z[3] * hs1 * ksB : -CUDART_INF_F;
        float mx0 = fmaxf(z[0] + lvA, z[2] + lvB), mx1 = fmaxf(z[1] + lvA, z[3] + lvB);
        if (__any_sync(0xffffffffu, mx0 > m0 + kLazy || mx1 > m1 + kLazy)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
            }
            const float a0 = mx0 > m0 + kLazy ? ex2(m0 - mx0) : 1.f;
            const float a1 = mx1 > m1 + kLazy ? ex2(m1 - mx1) : 1.f;
            if (mx0 > m0 + kLazy) m0 = mx0;
            if (mx1 > m1 + kLazy) m1 = mx1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a1;
                o[i][2] *= a0;
                o[i][3] *= a1;
            }
        }
        const float p0 = ex2(z[0] - m0), p1 = ex2(z[1] - m1);
        const float p2 = ex2(z[2] - m0), p3 = ex2(z[3] - m1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        uint32_t h0, h1, w0, w1;
        weight_terms<BF16>(p0 * vsA * kLift, p1 * vsA * kLift, h0, w0);
        weight_terms<BF16>(p2 * vsB * kLift, p3 * vsB * kLift, h1, w1);
        // ---- V rows of tokens c, c + 4, c + 8, c + 12: piece j of the lane is piece 8 j + g
        uint32_t v[4][S::kVWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = c + 4 * r;
            if constexpr (S::kVBytes == 8) {
                const uint2 x = *reinterpret_cast<const uint2*>(vt + piece_at<S::kRowB>(t, g >> 1) + (g & 1) * 8);
                v[r][0] = x.x;
                v[r][1] = x.y;
            } else {
#pragma unroll
                for (int j = 0; j < S::kVBytes / 16; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vt + piece_at<S::kRowB>(t, 8 * j + g));
                    v[r][4 * j] = x.x;
                    v[r][4 * j + 1] = x.y;
                    v[r][4 * j + 2] = x.z;
                    v[r][4 * j + 3] = x.w;
                }
            }
        }
        if (at + kPage > ctx) {
            // rows past the sequence may hold any bytes, NaN codes among them
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (at + c + 4 * r >= ctx) {
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) v[r][w] = 0u;
                }
        }
        // ---- O^T += V^T P^T (row g: the lane's value 2 i, row g + 8: 2 i + 1)
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
            uint32_t a0, a1, a2, a3;
            if constexpr (BF16) {
                a0 = __byte_perm(v[0][i], v[1][i], 0x5410);
                a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
                a2 = __byte_perm(v[2][i], v[3][i], 0x5410);
                a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
            } else {
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                f16x2x2_from_e4m3x4(__byte_perm(v[0][i >> 1], v[1][i >> 1], sel), a0, a1);
                f16x2x2_from_e4m3x4(__byte_perm(v[2][i >> 1], v[3][i >> 1], sel), a2, a3);
            }
            mma16<BF16>(o[i], a0, a1, a2, a3, h0, h1);
            mma16<BF16>(o[i], a0, a1, a2, a3, w0, w1);
        }
        __syncwarp();                                   // the stage is read
        issue(stage);
    }
    __syncthreads();                                    // the rings are done with

    // ---- the warps' parts meet in shared memory, the CTAs' in the cluster's
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    {
        float* w = part_o + warp * 8 * S::kOStride;
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
            // value 2 i of the lane's bytes: piece 2 i elem / 16, and its place in the piece
            int d;
            if constexpr (S::kVBytes == 8)
                d = g * 8 + 2 * i;
            else
                d = (8 * (2 * i * S::kElem / 16) + g) * (16 / S::kElem) + (2 * i) % (16 / S::kElem);
            *reinterpret_cast<float2*>(w + (2 * c) * S::kOStride + d) = make_float2(o[i][0], o[i][2]);
            *reinterpret_cast<float2*>(w + (2 * c + 1) * S::kOStride + d) = make_float2(o[i][1], o[i][3]);
        }
        if (g == 0) {
            part_m[warp * 8 + 2 * c] = m0;
            part_m[warp * 8 + 2 * c + 1] = m1;
            part_l[warp * 8 + 2 * c] = l0;
            part_l[warp * 8 + 2 * c + 1] = l1;
        }
    }
    __syncthreads();
    const float v_const = (!BF16 && !PT ? p.v_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0] : 1.f) / kLift;
    // four values of a head at a time; the CTA's own parts, summed into warp 0's place
    constexpr int kQuads = D / 4;
    for (int e = threadIdx.x; e < heads * kQuads; e += blockDim.x) {
        const int head = e / kQuads, d = (e - head * kQuads) * 4;
        float M = part_m[head];
        for (int w = 1; w < n_warps; ++w) M = fmaxf(M, part_m[w * 8 + head]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < n_warps; ++w) {
            const float f = ex2(part_m[w * 8 + head] - M);
            const float4 x = *reinterpret_cast<const float4*>(part_o + (w * 8 + head) * S::kOStride + d);
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        *reinterpret_cast<float4*>(part_o + head * S::kOStride + d) = acc;
    }
    __syncthreads();
    if (threadIdx.x < 8) {
        const int head = threadIdx.x;
        float M = part_m[head], L = 0.f;
        for (int w = 1; w < n_warps; ++w) M = fmaxf(M, part_m[w * 8 + head]);
        for (int w = 0; w < n_warps; ++w) L += ex2(part_m[w * 8 + head] - M) * part_l[w * 8 + head];
        part_m[head] = M;
        part_l[head] = L;
    }
    // ---- a warp per head: the largest reference, the sum, over the prefix's pieces of its row too
    __shared__ float s_ref[8], s_sum[8];
    __shared__ int s_pieces[8];
    if constexpr (PREFIX) {
        if (static_cast<int>(threadIdx.x) < heads) {
            const int len = min(p.prefix_len[0], p.prefix_pages * kPage);
            const PrefixShares shares(len, prefix_keys(D), p.units, p.workers);
            const int64_t row = static_cast<int64_t>(b) * p.G + head0 + threadIdx.x;
            s_pieces[threadIdx.x] =
                shares.tiles > 0
                    ? shares.pieces(static_cast<int64_t>(h) * p.row_tiles + row / kPrefixRows)
                    : 0;
        }
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    if constexpr (PREFIX) pdl_wait();        // the prefix's partials are there
    for (int head = warp; head < heads; head += n_warps) {
        float M = kMaxInit, L = 0.f, m = kMaxInit, l = 0.f;
        if (lane < ranks) {
            m = (ranks > 1 ? cluster.map_shared_rank(part_m, lane) : part_m)[head];
            l = (ranks > 1 ? cluster.map_shared_rank(part_l, lane) : part_l)[head];
            M = m;
        }
        int pieces = 0;
        const float *pm = nullptr, *pl = nullptr;
        if constexpr (PREFIX) {
            const int64_t row = static_cast<int64_t>(b) * p.G + head0 + head;
            pieces = s_pieces[head];
            pm = p.pre_m + (static_cast<int64_t>(h) * p.B * p.G + row) * p.splits;
            pl = p.pre_l + (static_cast<int64_t>(h) * p.B * p.G + row) * p.splits;
            for (int s = lane; s < pieces; s += 32) M = fmaxf(M, pm[s]);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        L = ex2(m - M) * l;
        if constexpr (PREFIX)
            for (int s = lane; s < pieces; s += 32) L += ex2(pm[s] - M) * pl[s];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        if (lane == 0) {
            s_ref[head] = M;
            s_sum[head] = L;
        }
    }
    __syncthreads();
    for (int e = rank * blockDim.x + threadIdx.x; e < heads * kQuads; e += ranks * blockDim.x) {
        const int head = e / kQuads, d = (e - head * kQuads) * 4;
        const float M = s_ref[head], L = s_sum[head];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float f, const float4& x) {
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        };
        for (int r = 0; r < ranks; ++r) {
            const float* om = ranks > 1 ? cluster.map_shared_rank(part_m, r) : part_m;
            const float* oo = ranks > 1 ? cluster.map_shared_rank(part_o, r) : part_o;
            add(ex2(om[head] - M), *reinterpret_cast<const float4*>(oo + head * S::kOStride + d));
        }
        acc.x *= v_const;
        acc.y *= v_const;
        acc.z *= v_const;
        acc.w *= v_const;
        if constexpr (PREFIX) {
            const int64_t row = (static_cast<int64_t>(h) * p.B + b) * p.G + head0 + head;
            const float* pm = p.pre_m + row * p.splits;
            const float* po = p.pre_o + row * p.splits * D + d;
            const int pieces = s_pieces[head];
#pragma unroll 8
            for (int s = 0; s < pieces; ++s)
                add(ex2(pm[s] - M), *reinterpret_cast<const float4*>(po + static_cast<int64_t>(s) * D));
        }
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;   // nothing seen: a zero row
        const int64_t dst = (static_cast<int64_t>(b) * p.Hq + h * p.G + head0 + head) * D + d;
        if (p.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + dst) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + dst) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    if (ranks > 1) cluster.sync();           // nobody leaves while its parts are read
}

// A unit's CTAs and their warps.
struct Plan {
    int warps, ranks;
};

// As many warps a unit as its share of the SMs', while each keeps two pages.  Few units: a
// cluster, as many of its CTAs as have an SM of their own (8 heads of 128 pages: 8 CTAs of 8
// warps 7.7 us, 4 of 16 warps 9.2, 2 of 16 warps 11.3); behind a prefix, whose kernel holds
// the SMs till its end, a cluster is worth its later start only for long tails (4 x 8 tails of
// up to 19 pages: 11.8 us without, 15.9 with clusters of 4).  Then CTAs of an SM's warps, halved
// until they are not above a rank's share, or two or three.
template <int D, bool BF16, bool PREFIX>
Plan plan_of(const ListAttnParams& p, int pages) {
    using S = Shape<D, BF16>;
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((p.G + 7) / 8);
    int64_t share = static_cast<int64_t>(sm_count()) * S::kSmWarps / units;
    if (share > (pages + 1) / 2) share = (pages + 1) / 2;
    Plan pl{S::kSmWarps, 1};
    while (pl.ranks < 8 && units * pl.ranks * 2 <= sm_count() && share >= pl.ranks * 4 &&
           (!PREFIX || pages > pl.ranks * S::kSmWarps * 8))
        pl.ranks *= 2;
    while (pl.warps * pl.ranks > share && pl.warps > 3) pl.warps /= 2;
    return pl;
}

template <int D, bool BF16, bool PT, bool PREFIX>
cudaError_t launch_one(const ListAttnParams& p, const Plan& pl, cudaStream_t stream) {
    using S = Shape<D, BF16>;
    static unsigned long long done[64] = {};
    const void* fn = reinterpret_cast<const void*>(list_attn_kernel<D, BF16, PT, PREFIX>);
    const cudaError_t e = opt_in_smem(fn, S::smem(S::kSmWarps), done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((p.G + 7) / 8);
    cudaLaunchConfig_t cfg =
        pdl_config(attr, units * pl.ranks, pl.warps * 32, S::smem(pl.warps), stream);
    if (pl.ranks > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(pl.ranks);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, list_attn_kernel<D, BF16, PT, PREFIX>, p);
}

template <int D, bool PREFIX>
cudaError_t launch_d(const ListAttnParams& p, int kv_dtype, int pages, cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16)
        return launch_one<D, true, false, PREFIX>(p, plan_of<D, true, PREFIX>(p, pages), stream);
    const Plan pl = plan_of<D, false, PREFIX>(p, pages);
    if (p.scale_mode == FP8KV_SCALE_PER_TOKEN_HEAD)
        return launch_one<D, false, true, PREFIX>(p, pl, stream);
    return launch_one<D, false, false, PREFIX>(p, pl, stream);
}

}  // namespace

cudaError_t launch_list_attn(const ListAttnParams& p, int D, int kv_dtype, cudaStream_t stream) {
    if (p.pages == nullptr) {
        const int pages = p.max_blocks_per_seq;
        if (D == 64) return launch_d<64, true>(p, kv_dtype, pages, stream);
        if (D == 128) return launch_d<128, true>(p, kv_dtype, pages, stream);
        return launch_d<256, true>(p, kv_dtype, pages, stream);
    }
    const int pages = p.budget < p.max_blocks_per_seq ? p.budget : p.max_blocks_per_seq;
    if (D == 64) return launch_d<64, false>(p, kv_dtype, pages, stream);
    if (D == 128) return launch_d<128, false>(p, kv_dtype, pages, stream);
    return launch_d<256, false>(p, kv_dtype, pages, stream);
}

}  // namespace fp8kv
