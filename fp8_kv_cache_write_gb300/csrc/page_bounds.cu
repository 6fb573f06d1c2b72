// page_bounds.cu -- the largest and smallest value of every channel of a page's keys, in
// 8 bits under one scale a (page, head): what kv_page_select scores a page by.
//
//     hi_d = max_t x_td, lo_d = min_t x_td over the page's tokens below the context length
//     s = fp32(max_d max(|hi_d|, |lo_d|) / 127),  codes rint(fp32(hi_d / s)), rint(fp32(lo_d / s))
//
// with x the keys as cached (fp32 of code * scale).  Maxima and minima do not depend on
// their order and the two quotients are IEEE divides, so the codes are reproducible.
//
// Bound: HBM for prompts (a page and head of D 128 reads 2112 bytes and writes 260).
// Split: a warp takes one (page, head) tile; a lane owns the same 4 to 16 bytes of every
// token row (a 64-byte row: of every other one), so that a column's maximum stays in one
// lane and needs no shuffles, and all of the tile's loads are in flight at once.  Rows past
// the sequence's end are read as its last row, which changes no maximum.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace fp8kv {

namespace {

constexpr int kThreads = 256;

template <int N> struct LanePiece;
template <> struct LanePiece<4> { using T = uint32_t; };
template <> struct LanePiece<8> { using T = uint2; };
template <> struct LanePiece<16> { using T = uint4; };

// 8-bit code of x / s; a zero scale (every value 0, or so small that s rounds to 0) codes 0.
__device__ __forceinline__ uint32_t bound_code(float x, float s) {
    if (s == 0.f) return 0u;
    const int r = __float2int_rn(__fdiv_rn(x, s));
    // only a subnormal s, which holds few bits, can leave [-127, 127]
    return static_cast<uint32_t>(max(-127, min(127, r))) & 0xffu;
}

template <int D, bool BF16, bool PER_TOKEN>
__global__ void __launch_bounds__(kThreads) page_bounds_kernel(PageBoundsParams p) {
    constexpr int kRowB = D * (BF16 ? 2 : 1);
    constexpr int kLanes = kRowB / 4 < 32 ? kRowB / 4 : 32;   // lanes of a row
    constexpr int kB = kRowB / kLanes;                        // bytes of a lane
    constexpr int kAt = 32 / kLanes;                          // rows a warp reads at once
    constexpr int kN = kB / (BF16 ? 2 : 1);                   // values of a lane's piece
    constexpr int kLoads = kPage / kAt;
    using Piece = typename LanePiece<kB>::T;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int64_t bj = item / p.Hkv;
    const int h = static_cast<int>(item - bj * p.Hkv);
    const int b = static_cast<int>(bj / p.pages_per_seq);
    if (b >= p.B) return;
    int ctx = p.context_lens[b];
    if (ctx > p.max_blocks_per_seq * kPage) {
        if (lane == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        ctx = p.max_blocks_per_seq * kPage;
    }
    const int first = p.new_tokens > 0 && ctx > p.new_tokens ? (ctx - p.new_tokens) / kPage : 0;
    const int page = first + static_cast<int>(bj - static_cast<int64_t>(b) * p.pages_per_seq);
    if (page * kPage >= ctx) return;                         // ctx <= 0 too: page >= 0
    const int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks_per_seq + page];
    if (blk < 0 || blk >= p.num_blocks) {
        if (lane == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        return;
    }
    const int last = min(kPage, ctx - page * kPage) - 1;     // the page's last token row
    const int64_t tile = static_cast<int64_t>(blk) * p.Hkv + h;
    const uint8_t* src = p.k_cache + tile * (kPage * kRowB) + (lane % kLanes) * kB;
    Piece raw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        raw[i] = *reinterpret_cast<const Piece*>(src + min(i * kAt + lane / kLanes, last) * kRowB);
    float scale = 1.f;
    if constexpr (PER_TOKEN)
        scale = p.k_scale_cache[tile * kPage + min(lane & 15, last)];
    else if constexpr (!BF16)
        scale = p.k_scale[p.mode == FP8KV_SCALE_PER_HEAD ? h : 0];

    float hi[kN], lo[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        hi[j] = -CUDART_INF_F;
        lo[j] = CUDART_INF_F;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        uint32_t w[kB / 4];
        memcpy(w, &raw[i], kB);
        float x[kN];
        if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < kB / 4; ++j) {
                const float2 a = unpack_bf16x2(w[j]);
                x[2 * j] = a.x;
                x[2 * j + 1] = a.y;
            }
        } else {
            const float s = PER_TOKEN ? __shfl_sync(0xffffffffu, scale, i * kAt + lane / kLanes)
                                      : scale;
            const uint64_t s2 = pack_f32x2(s, s);
#pragma unroll
            for (int j = 0; j < kB / 4; ++j) {
                uint32_t u0, u1;
                f16x2x2_from_e4m3x4(w[j], u0, u1);
                const float2 a = unpack_f16x2(u0), c = unpack_f16x2(u1);
                const float2 a2 = unpack_f32x2(mul_f32x2(pack_f32x2(a.x, a.y), s2));
                const float2 c2 = unpack_f32x2(mul_f32x2(pack_f32x2(c.x, c.y), s2));
                x[4 * j] = a2.x;
                x[4 * j + 1] = a2.y;
                x[4 * j + 2] = c2.x;
                x[4 * j + 3] = c2.y;
            }
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) {                       // NaN is left out
            hi[j] = fmaxf(hi[j], x[j]);
            lo[j] = fminf(lo[j], x[j]);
        }
    }
    if constexpr (kAt == 2) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
            lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
        }
    }
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        if (hi[j] < lo[j]) hi[j] = lo[j] = 0.f;              // nothing but NaN
        hi[j] = fminf(fmaxf(hi[j], -FLT_MAX), FLT_MAX);      // infinities: the largest number
        lo[j] = fminf(fmaxf(lo[j], -FLT_MAX), FLT_MAX);
        a = fmaxf(a, fmaxf(fabsf(hi[j]), fabsf(lo[j])));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    const float s = __fdiv_rn(a, 127.f);
    uint32_t ch[(kN + 3) / 4] = {}, cl[(kN + 3) / 4] = {};
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        ch[j / 4] |= bound_code(hi[j], s) << (8 * (j & 3));
        cl[j / 4] |= bound_code(lo[j], s) << (8 * (j & 3));
    }
    int8_t* dst = p.bounds + tile * (2 * D) + (lane % kLanes) * kN;
    // two rows at a time: both halves of the warp hold the columns, one stores each bound
    if (kAt == 1 || lane < kLanes) memcpy(__builtin_assume_aligned(dst, kN), ch, kN);
    if (kAt == 1 || lane >= kLanes) memcpy(__builtin_assume_aligned(dst + D, kN), cl, kN);
    if (lane == 0) p.bounds_scale[tile] = s;
}

template <int D>
cudaError_t launch_d(const PageBoundsParams& p, int kv_dtype, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.B) * p.pages_per_seq * p.Hkv;
    constexpr int kWarps = kThreads / 32;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, (items + kWarps - 1) / kWarps, kThreads, 0, stream);
    if (kv_dtype == FP8KV_KV_BF16)
        return cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, true, false>, p);
    if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD)
        return cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, false, true>, p);
    return cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, false, false>, p);
}

}  // namespace

cudaError_t launch_page_bounds(const PageBoundsParams& p, int D, int kv_dtype,
                               cudaStream_t stream) {
    if (D == 64) return launch_d<64>(p, kv_dtype, stream);
    if (D == 128) return launch_d<128>(p, kv_dtype, stream);
    return launch_d<256>(p, kv_dtype, stream);
}

}  // namespace fp8kv
