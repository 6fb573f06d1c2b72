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
// Split: a unit is (sequence, KV head, up to 8 of its query heads); a thread-block cluster
// of 1 to 16 CTAs of 4 warps takes one unit and its warps deal the listed pages among
// themselves.  Lists are of nearly equal length, so no plan is needed, and the parts of a
// unit meet in (distributed) shared memory: one launch, no workspace.
//   * pages go from global memory straight into the fragments of mma.sync: a lane's 16-byte
//     pieces are its A operand once the rows (tokens) and columns (channels) of both products
//     are suitably permuted, so there is no ring in shared memory, no barrier and no copy
//     engine between a page and its product; the next pages' loads are issued as soon as the
//     registers of the current ones are free.
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

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
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

// Cache bytes, read once: past L1.
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(reinterpret_cast<uint64_t>(p)));
    return x;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p) {
    uint2 x;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(x.x), "=r"(x.y)
                 : "l"(reinterpret_cast<uint64_t>(p)));
    return x;
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
    // pages in registers at once: two while both fit beside the accumulators
    static constexpr int kPages = kRowB <= 128 ? 2 : 1;
    static constexpr int kOStride = D + 4;              // floats of a head's row of partial O
    static constexpr int kSmem = kWarps * 8 * (kOStride + 2) * 4;
    static constexpr int kMinCtas = kRowB <= 128 ? 3 : 2;
};

// One page's K (or V) pieces and scales of a lane.
template <int D, bool BF16>
struct Tile {
    using S = Shape<D, BF16>;
    uint4 k[2 * S::kSegs];
    uint32_t v[4][S::kVWords];
    float ks[2], vs[2];
    int pos;                                            // first token; -1: nothing here
};

template <int D, bool BF16, bool PT, bool PREFIX>
__global__ void __launch_bounds__(kThreads, Shape<D, BF16>::kMinCtas)
    list_attn_kernel(ListAttnParams p) {
    using S = Shape<D, BF16>;
    constexpr int NP = S::kPages;
    extern __shared__ float smem[];
    float* const part_o = smem;                         // [warp][8][kOStride]
    float* const part_m = smem + kWarps * 8 * S::kOStride;
    float* const part_l = part_m + kWarps * 8;
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
    const int workers = ranks * kWarps, worker = rank * kWarps + warp;
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
    Tile<D, BF16> t[NP];
    int64_t tile[NP];
    auto load_k = [&](int k) {
        next(tile[k], t[k].pos);
        if (t[k].pos < 0) return;
        const uint8_t* src = p.k_cache + tile[k] * S::kTileB + c * 16;
#pragma unroll
        for (int s = 0; s < S::kSegs; ++s) {
            t[k].k[2 * s] = load16(src + tA * S::kRowB + s * 64);
            t[k].k[2 * s + 1] = load16(src + tB * S::kRowB + s * 64);
        }
        if constexpr (PT) {
            t[k].ks[0] = p.k_scale_cache[tile[k] * kPage + tA];
            t[k].ks[1] = p.k_scale_cache[tile[k] * kPage + tB];
        }
    };
    auto load_v = [&](int k) {
        if (t[k].pos < 0) return;
        const uint8_t* src = p.v_cache + tile[k] * S::kTileB;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint8_t* row = src + (c + 4 * r) * S::kRowB;
            if constexpr (S::kVBytes == 8) {
                const uint2 x = load8(row + g * 8);
                t[k].v[r][0] = x.x;
                t[k].v[r][1] = x.y;
            } else {
                // 16-byte piece j of the lane is piece 8 j + g of the row (whole lines a warp)
#pragma unroll
                for (int j = 0; j < S::kVBytes / 16; ++j) {
                    const uint4 x = load16(row + (8 * j + g) * 16);
                    t[k].v[r][4 * j] = x.x;
                    t[k].v[r][4 * j + 1] = x.y;
                    t[k].v[r][4 * j + 2] = x.z;
                    t[k].v[r][4 * j + 3] = x.w;
                }
            }
        }
        if constexpr (PT) {
            t[k].vs[0] = p.v_scale_cache[tile[k] * kPage + tA];
            t[k].vs[1] = p.v_scale_cache[tile[k] * kPage + tB];
        }
    };
#pragma unroll
    for (int k = 0; k < NP; ++k) load_k(k);
#pragma unroll
    for (int k = 0; k < NP; ++k) load_v(k);

    while (t[0].pos >= 0) {
        // ---- S^T (rows: tokens tA, tB; columns: heads 2c, 2c + 1)
        float z[NP][4];
#pragma unroll
        for (int k = 0; k < NP; ++k) z[k][0] = z[k][1] = z[k][2] = z[k][3] = 0.f;
#pragma unroll
        for (int s = 0; s < S::kSegs; ++s) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                if (k > 0 && t[k].pos < 0) continue;
                const uint4 x = t[k].k[2 * s], y = t[k].k[2 * s + 1];
                const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < S::kPerSeg; ++j) {
                    const uint2 qf = qb[s * S::kPerSeg + j];
                    if constexpr (BF16) {
                        mma16<true>(z[k], wx[2 * j], wy[2 * j], wx[2 * j + 1], wy[2 * j + 1], qf.x,
                                    qf.y);
                    } else {
                        uint32_t xl, xh, yl, yh;
                        f16x2x2_from_e4m3x4(wx[j], xl, xh);
                        f16x2x2_from_e4m3x4(wy[j], yl, yh);
                        mma16<false>(z[k], xl, yl, xh, yh, qf.x, qf.y);
                    }
                }
            }
        }
        // ---- logits; the reference follows z + log2 s_v
        float vs[NP][2], mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
        int at[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            at[k] = t[k].pos;
            // (a page that is not there: every row masked)
            const bool vA = at[k] >= 0 && at[k] + tA < ctx, vB = at[k] >= 0 && at[k] + tB < ctx;
            float ksA = 1.f, ksB = 1.f, lvA = 0.f, lvB = 0.f;
            vs[k][0] = vs[k][1] = 1.f;
            if constexpr (PT) {
                ksA = t[k].ks[0];
                ksB = t[k].ks[1];
                vs[k][0] = vA ? t[k].vs[0] : 0.f;
                vs[k][1] = vB ? t[k].vs[1] : 0.f;
                lvA = fmaxf(__log2f(fabsf(vs[k][0])), -100.f);
                lvB = fmaxf(__log2f(fabsf(vs[k][1])), -100.f);
            }
            z[k][0] = vA ? z[k][0] * hs0 * ksA : -CUDART_INF_F;
            z[k][1] = vA ? z[k][1] * hs1 * ksA : -CUDART_INF_F;
            z[k][2] = vB ? z[k][2] * hs0 * ksB : -CUDART_INF_F;
            z[k][3] = vB ? z[k][3] * hs1 * ksB : -CUDART_INF_F;
            mx0 = fmaxf(mx0, fmaxf(z[k][0] + lvA, z[k][2] + lvB));
            mx1 = fmaxf(mx1, fmaxf(z[k][1] + lvA, z[k][3] + lvB));
        }
        // the K registers are free: the next pages'
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (k > 0 && t[k - 1].pos < 0)
                t[k].pos = -1;
            else
                load_k(k);
        }
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
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (k > 0 && at[k] < 0) continue;
            const float p0 = ex2(z[k][0] - m0), p1 = ex2(z[k][1] - m1);
            const float p2 = ex2(z[k][2] - m0), p3 = ex2(z[k][3] - m1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            uint32_t h0, h1, w0, w1;
            weight_terms<BF16>(p0 * vs[k][0] * kLift, p1 * vs[k][0] * kLift, h0, w0);
            weight_terms<BF16>(p2 * vs[k][1] * kLift, p3 * vs[k][1] * kLift, h1, w1);
            if (at[k] + kPage > ctx) {
                // rows past the sequence may hold any bytes, NaN codes among them
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (at[k] + c + 4 * r >= ctx) {
#pragma unroll
                        for (int w = 0; w < S::kVWords; ++w) t[k].v[r][w] = 0u;
                    }
            }
            // ---- O^T += V^T P^T (row g: the lane's value 2 i, row g + 8: 2 i + 1)
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                uint32_t a0, a1, a2, a3;
                if constexpr (BF16) {
                    a0 = __byte_perm(t[k].v[0][i], t[k].v[1][i], 0x5410);
                    a1 = __byte_perm(t[k].v[0][i], t[k].v[1][i], 0x7632);
                    a2 = __byte_perm(t[k].v[2][i], t[k].v[3][i], 0x5410);
                    a3 = __byte_perm(t[k].v[2][i], t[k].v[3][i], 0x7632);
                } else {
                    const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                    f16x2x2_from_e4m3x4(__byte_perm(t[k].v[0][i >> 1], t[k].v[1][i >> 1], sel), a0, a1);
                    f16x2x2_from_e4m3x4(__byte_perm(t[k].v[2][i >> 1], t[k].v[3][i >> 1], sel), a2, a3);
                }
                mma16<BF16>(o[i], a0, a1, a2, a3, h0, h1);
                mma16<BF16>(o[i], a0, a1, a2, a3, w0, w1);
            }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) load_v(k);
    }

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
    // four values of a head at a time; the CTA's own four parts, summed into warp 0's place
    constexpr int kQuads = D / 4;
    for (int e = threadIdx.x; e < heads * kQuads; e += kThreads) {
        const int head = e / kQuads, d = (e - head * kQuads) * 4;
        float M = part_m[head];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, part_m[w * 8 + head]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
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
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, part_m[w * 8 + head]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) L += ex2(part_m[w * 8 + head] - M) * part_l[w * 8 + head];
        part_m[head] = M;
        part_l[head] = L;
    }
    __shared__ int s_pieces[8];              // the prefix's pieces of each head's row
    if constexpr (PREFIX) {
        pdl_wait();                          // the prefix's partials are there
        if (threadIdx.x < 8) {
            const int len = min(p.prefix_len[0], p.prefix_pages * kPage);
            const PrefixShares shares(len, prefix_keys(D), p.units, p.workers);
            const int64_t row = static_cast<int64_t>(b) * p.G + head0 + threadIdx.x;
            s_pieces[threadIdx.x] =
                shares.tiles > 0 && threadIdx.x < heads
                    ? shares.pieces(static_cast<int64_t>(h) * p.row_tiles + row / kPrefixRows)
                    : 0;
        }
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    for (int e = rank * kThreads + threadIdx.x; e < heads * kQuads; e += ranks * kThreads) {
        const int head = e / kQuads, d = (e - head * kQuads) * 4;
        float M = kMaxInit;
        for (int r = 0; r < ranks; ++r)
            M = fmaxf(M, (ranks > 1 ? cluster.map_shared_rank(part_m, r) : part_m)[head]);
        int64_t row = 0;
        int pieces = 0;
        if constexpr (PREFIX) {
            row = (static_cast<int64_t>(h) * p.B + b) * p.G + head0 + head;
            pieces = s_pieces[head];
            for (int s = 0; s < pieces; ++s) M = fmaxf(M, p.pre_m[row * p.splits + s]);
        }
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float f, const float4& x) {
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        };
        for (int r = 0; r < ranks; ++r) {
            const float* om = ranks > 1 ? cluster.map_shared_rank(part_m, r) : part_m;
            const float* ol = ranks > 1 ? cluster.map_shared_rank(part_l, r) : part_l;
            const float* oo = ranks > 1 ? cluster.map_shared_rank(part_o, r) : part_o;
            const float f = ex2(om[head] - M);
            L += f * ol[head];
            add(f, *reinterpret_cast<const float4*>(oo + head * S::kOStride + d));
        }
        acc.x *= v_const;
        acc.y *= v_const;
        acc.z *= v_const;
        acc.w *= v_const;
        if constexpr (PREFIX) {
#pragma unroll 4
            for (int s = 0; s < pieces; ++s) {
                const float f = ex2(p.pre_m[row * p.splits + s] - M);
                L += f * p.pre_l[row * p.splits + s];
                add(f, *reinterpret_cast<const float4*>(p.pre_o + (row * p.splits + s) * D + d));
            }
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

template <int D, bool BF16, bool PT, bool PREFIX>
cudaError_t launch_one(const ListAttnParams& p, int ranks, cudaStream_t stream) {
    using S = Shape<D, BF16>;
    static unsigned long long done[64] = {};
    const void* fn = reinterpret_cast<const void*>(list_attn_kernel<D, BF16, PT, PREFIX>);
    const cudaError_t e = opt_in_smem(fn, S::kSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((p.G + 7) / 8);
    cudaLaunchConfig_t cfg = pdl_config(attr, units * ranks, kThreads, S::kSmem, stream);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, list_attn_kernel<D, BF16, PT, PREFIX>, p);
}

// CTAs of a unit: as many as fill the SMs' places, while every warp keeps two rounds of
// pages.
template <int D, bool BF16>
int ranks_of(const ListAttnParams& p, int pages) {
    using S = Shape<D, BF16>;
    const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((p.G + 7) / 8);
    int ranks = 1;
    while (ranks < 8 && units * ranks * 2 <= static_cast<int64_t>(sm_count()) * S::kMinCtas &&
           pages > ranks * kWarps * S::kPages)
        ranks *= 2;
    return ranks;
}

template <int D, bool PREFIX>
cudaError_t launch_d(const ListAttnParams& p, int kv_dtype, int pages, cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16)
        return launch_one<D, true, false, PREFIX>(p, ranks_of<D, true>(p, pages), stream);
    const int ranks = ranks_of<D, false>(p, pages);
    if (p.scale_mode == FP8KV_SCALE_PER_TOKEN_HEAD)
        return launch_one<D, false, true, PREFIX>(p, ranks, stream);
    return launch_one<D, false, false, PREFIX>(p, ranks, stream);
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
