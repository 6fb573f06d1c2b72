// page_bounds.cu -- the largest and smallest value of every channel of a page's keys, in
// 8 bits under one scale a (page, head): what kv_page_select scores a page by.
//
//     hi_d = max_t x_td, lo_d = min_t x_td over the page's tokens below the context length
//     s = fp32(max_d max(|hi_d|, |lo_d|) / 127),  codes rint(fp32(hi_d / s)), rint(fp32(lo_d / s))
//
// with x the keys as cached (fp32 of code * scale).  Maxima and minima do not depend on
// their order and the two quotients are IEEE divides, so the codes are reproducible.
//
// Bound: HBM for prompts (a page and head of D 128 reads 2112 bytes and writes 260); reached are
// the issue slots, with per-token scales (550 warp instructions a page and head).
// Split: a warp takes one (page, head) tile; a lane owns the same 4 to 16 bytes of every
// token row (a 64-byte row: of every other one), so that a column's maximum stays in one
// lane and needs no shuffles, and all of the tile's loads are in flight at once.
//   * Under one scale for all rows the maxima are taken on the codes, as f16 or bf16 pairs,
//     and scaled afterwards: rounding keeps the order.
//   * The quotients' codes come from products with 1 / s, which are within 2^-22 of a quotient
//     of at most 127; the IEEE divides are left to lanes where one lies within 10^-4 of a
//     rounding border.
//   * Rows past the sequence's end are read as its last row, which changes no maximum.
// Measured: 65536 pages and heads of D 128, one scale 37 us = 4.1 TB/s, bf16 47 us = 6.1 TB/s (0.9 of
// the copy rate), with per-token scales 43.3 us = 3.6 TB/s, half of the
// cycles on the pipe that converts, compares and permutes; a decode step's last pages (32 x 8) 2.8 us.
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

__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// n / d for n < 2^31 by a multiplication (the host works out mul and shift).
struct Divisor {
    unsigned d, mul, shift;
    explicit Divisor(unsigned d_) : d(d_), shift(0) {
        while (shift < 31 && (1u << shift) < d) ++shift;
        mul = static_cast<unsigned>(((static_cast<uint64_t>(1) << 32) * ((1u << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned of(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// A lane's pieces of a tile's rows, and the rows' scales (not PER_TOKEN: the one).
template <int D, bool BF16, bool PER_TOKEN>
struct Rows {
    static constexpr int kRowB = D * (BF16 ? 2 : 1);
    static constexpr int kLanes = kRowB / 4 < 32 ? kRowB / 4 : 32;   // lanes of a row
    static constexpr int kB = kRowB / kLanes;                        // bytes of a lane
    static constexpr int kAt = 32 / kLanes;                          // rows a warp reads at once
    static constexpr int kN = kB / (BF16 ? 2 : 1);                   // values of a lane's piece
    static constexpr int kLoads = kPage / kAt;
    static constexpr int kCtas = kB == 4 ? 4 : kB == 8 ? 3 : 2;      // on an SM, by registers
    using Piece = typename LanePiece<kB>::T;
    Piece raw[kLoads];
    float sc[PER_TOKEN ? kLoads : 1];

    // last: the page's last row; those behind it are read as it
    __device__ __forceinline__ void load(const uint8_t* src, const float* scales, int lane, int last) {
        if (last == kPage - 1) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                raw[i] = *reinterpret_cast<const Piece*>(src + (i * kAt + lane / kLanes) * kRowB);
            if constexpr (PER_TOKEN && kAt == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = reinterpret_cast<const float4*>(scales)[i];
                    sc[4 * i] = f.x;
                    sc[4 * i + 1] = f.y;
                    sc[4 * i + 2] = f.z;
                    sc[4 * i + 3] = f.w;
                }
                return;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                raw[i] = *reinterpret_cast<const Piece*>(src + min(i * kAt + lane / kLanes, last) * kRowB);
        }
        if constexpr (PER_TOKEN) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) sc[i] = scales[min(i * kAt + lane / kLanes, last)];
        } else if constexpr (!BF16) {
            sc[0] = *scales;
        }
    }

    // Largest and smallest value of the lane's columns.
    __device__ __forceinline__ void columns(float (&hi)[kN], float (&lo)[kN]) const {
        constexpr int N = kN, kWords = kB / 4;
        if constexpr (PER_TOKEN) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                hi[j] = -CUDART_INF_F;
                lo[j] = CUDART_INF_F;
            }
            // two rows at a time: one packed product and one maximum of three a column
#pragma unroll
            for (int i = 0; i < kLoads; i += 2) {
                uint32_t w0[kWords], w1[kWords];
                memcpy(w0, &raw[i], kB);
                memcpy(w1, &raw[i + 1], kB);
                const uint64_t s2 = pack_f32x2(sc[i], sc[i + 1]);
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    uint32_t u[2], v[2];
                    f16x2x2_from_e4m3x4(w0[j], u[0], u[1]);
                    f16x2x2_from_e4m3x4(w1[j], v[0], v[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 a = unpack_f16x2(u[k]), c = unpack_f16x2(v[k]);
                        const float2 x = unpack_f32x2(mul_f32x2(pack_f32x2(a.x, c.x), s2));
                        const float2 y = unpack_f32x2(mul_f32x2(pack_f32x2(a.y, c.y), s2));
                        const int at = 4 * j + 2 * k;        // NaN is left out
                        hi[at] = max3(hi[at], x.x, x.y);
                        lo[at] = min3(lo[at], x.x, x.y);
                        hi[at + 1] = max3(hi[at + 1], y.x, y.y);
                        lo[at + 1] = min3(lo[at + 1], y.x, y.y);
                    }
                }
            }
        } else {
            constexpr uint32_t kInf = BF16 ? 0x7f807f80u : 0x7c007c00u;
            constexpr int kPairs = N / 2;
            uint32_t h[kPairs], l[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                h[j] = kInf | 0x80008000u;
                l[j] = kInf;
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                uint32_t w[kWords], x[kPairs];
                memcpy(w, &raw[i], kB);
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    if constexpr (BF16)
                        x[j] = w[j];
                    else
                        f16x2x2_from_e4m3x4(w[j], x[2 * j], x[2 * j + 1]);
                }
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {               // NaN is left out
                    h[j] = max_pair(h[j], x[j], BF16);
                    l[j] = min_pair(l[j], x[j], BF16);
                }
            }
            const float s = BF16 ? 1.f : sc[0];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 a = BF16 ? unpack_bf16x2(h[j]) : unpack_f16x2(h[j]);
                const float2 c = BF16 ? unpack_bf16x2(l[j]) : unpack_f16x2(l[j]);
                const float p[2] = {a.x * s, a.y * s}, q[2] = {c.x * s, c.y * s};
#pragma unroll
                for (int k = 0; k < 2; ++k) {                    // (a negative scale swaps them)
                    hi[2 * j + k] = s < 0.f ? q[k] : p[k];
                    lo[2 * j + k] = s < 0.f ? p[k] : q[k];
                }
            }
        }
    }
};

template <int D, bool BF16, bool PER_TOKEN>
__global__ void __launch_bounds__(kThreads, Rows<D, BF16, PER_TOKEN>::kCtas)
    page_bounds_kernel(PageBoundsParams p, unsigned items, Divisor heads, Divisor pages) {
    using R = Rows<D, BF16, PER_TOKEN>;
    constexpr int kRowB = R::kRowB, kLanes = R::kLanes, kAt = R::kAt, kN = R::kN;
    const int lane = threadIdx.x & 31;
    const unsigned stride = gridDim.x * (kThreads / 32);
    unsigned item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    // block and last token row of an item's page (-1: nothing to do)
    auto look_up = [&](unsigned it, int& blk, int& last) {
        blk = -1;
        last = 0;
        if (it >= items) return;
        const unsigned bj = heads.of(it);
        const unsigned b = pages.of(bj);
        int ctx = p.context_lens[b];
        const bool past = ctx > p.max_blocks_per_seq * kPage;
        if (past) ctx = p.max_blocks_per_seq * kPage;
        const int first = p.new_tokens > 0 && ctx > p.new_tokens ? (ctx - p.new_tokens) / kPage : 0;
        const int page = first + static_cast<int>(bj - b * p.pages_per_seq);
        if (page * kPage < ctx) {                            // (no page: ctx <= 0)
            const int x = p.block_table[static_cast<int64_t>(b) * p.max_blocks_per_seq + page];
            const bool ok = x >= 0 && x < p.num_blocks;
            if ((past || !ok) && lane == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
            if (ok) blk = x;
            last = min(kPage, ctx - page * kPage) - 1;
        }
    };
    auto load = [&](R& rows, int64_t tile, int h, int last) {
        rows.load(p.k_cache + tile * (kPage * kRowB) + (lane % kLanes) * R::kB,
                  PER_TOKEN ? p.k_scale_cache + tile * kPage
                  : BF16    ? nullptr
                            : p.k_scale + (p.mode == FP8KV_SCALE_PER_HEAD ? h : 0),
                  lane, last);
    };
    auto finish = [&](const R& rows, int64_t tile) {
        float hi[kN], lo[kN];
        rows.columns(hi, lo);
        if constexpr (kAt == 2) {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
                lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
            }
        }
        float a = 0.f;
        auto magnitude = [&]() {
#pragma unroll
            for (int j = 0; j < kN; ++j) a = max3(a, fabsf(hi[j]), fabsf(lo[j]));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        };
        // infinities, and columns of nothing but NaN (which are infinite too, or NaN), show in
        // the largest magnitude or the test below: they are rare
        bool odd = false;
#pragma unroll
        for (int j = 0; j < kN; ++j) odd |= !(hi[j] >= lo[j]);
        magnitude();
        if (__any_sync(0xffffffffu, odd) || !(a <= FLT_MAX)) {
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                if (!(hi[j] >= lo[j])) hi[j] = lo[j] = 0.f;  // nothing but NaN
                hi[j] = fminf(fmaxf(hi[j], -FLT_MAX), FLT_MAX);   // infinities: the largest number
                lo[j] = fminf(fmaxf(lo[j], -FLT_MAX), FLT_MAX);
            }
            a = 0.f;
            magnitude();
        }
        const float s = __fdiv_rn(a, 127.f);
        const float r = __frcp_rn(s);
        uint32_t yh[kN], yl[kN];
        float off = 0.f;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            // adding 1.5 * 2^23 rounds to a whole number, whose low byte is the sum's; what is
            // left of the value tells how near a border the quotient lies
            const float h = __fmaf_rn(hi[j], r, 12582912.f), l = __fmaf_rn(lo[j], r, 12582912.f);
            yh[j] = __float_as_uint(h);
            yl[j] = __float_as_uint(l);
            off = max3(off, fabsf(__fmaf_rn(__fadd_rn(h, -12582912.f), -s, hi[j])),
                       fabsf(__fmaf_rn(__fadd_rn(l, -12582912.f), -s, lo[j])));
        }
        uint32_t ch[(kN + 3) / 4], cl[(kN + 3) / 4];
        auto pack = [&](const uint32_t(&y)[kN], uint32_t(&c)[(kN + 3) / 4]) {
#pragma unroll
            for (int j = 0; j < kN; j += 4) {
                const uint32_t low = __byte_perm(y[j], y[j + 1], 0x0040);
                c[j / 4] = kN < 4 ? low
                                  : __byte_perm(low, __byte_perm(y[(j + 2) % kN], y[(j + 3) % kN], 0x0040), 0x5410);
            }
        };
        if (!(off < 0.4999f * s) || !(s > 0x1p-100f)) {      // (a zero scale among them)
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                yh[j] = bound_code(hi[j], s);
                yl[j] = bound_code(lo[j], s);
            }
        }
        pack(yh, ch);
        pack(yl, cl);
        int8_t* dst = p.bounds + tile * (2 * D) + (lane % kLanes) * kN;
        // two rows at a time: both halves of the warp hold the columns, one stores each bound
        if (kAt == 1 || lane < kLanes) memcpy(__builtin_assume_aligned(dst, kN), ch, kN);
        if (kAt == 1 || lane >= kLanes) memcpy(__builtin_assume_aligned(dst + D, kN), cl, kN);
        if (lane == 0) p.bounds_scale[tile] = s;
    };
    // a warp's next page is looked up while this one's rows are on their way
    int blk, last, blk_next, last_next;
    look_up(item, blk, last);
    for (; item < items; item += stride) {
        const int h = static_cast<int>(item - heads.of(item) * heads.d);
        const int64_t tile = static_cast<int64_t>(blk) * p.Hkv + h;
        R rows;
        if (blk >= 0) load(rows, tile, h, last);
        look_up(item + stride, blk_next, last_next);
        if (blk >= 0) finish(rows, tile);
        blk = blk_next;
        last = last_next;
    }
}

template <int D, bool BF16, bool PER_TOKEN>
cudaError_t launch_one(const PageBoundsParams& p, cudaStream_t stream) {
    // (the host keeps the items within 31 bits)
    constexpr int kWarps = kThreads / 32;
    const int64_t resident = static_cast<int64_t>(Rows<D, BF16, PER_TOKEN>::kCtas) * sm_count();
    const unsigned items = static_cast<unsigned>(p.B) * p.pages_per_seq * p.Hkv;
    int64_t blocks = (static_cast<int64_t>(items) + kWarps - 1) / kWarps;
    if (blocks > resident) blocks = resident;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, blocks, kThreads, 0, stream);
    return cudaLaunchKernelEx(&cfg, page_bounds_kernel<D, BF16, PER_TOKEN>, p, items, Divisor(p.Hkv),
                              Divisor(p.pages_per_seq));
}

template <int D>
cudaError_t launch_d(const PageBoundsParams& p, int kv_dtype, cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16) return launch_one<D, true, false>(p, stream);
    if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD) return launch_one<D, false, true>(p, stream);
    return launch_one<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_page_bounds(const PageBoundsParams& p, int D, int kv_dtype,
                               cudaStream_t stream) {
    if (D == 64) return launch_d<64>(p, kv_dtype, stream);
    if (D == 128) return launch_d<128>(p, kv_dtype, stream);
    return launch_d<256>(p, kv_dtype, stream);
}

}  // namespace fp8kv
