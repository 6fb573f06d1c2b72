// cache_read.cu -- cached rows back as values: out = code * scale (e4m3), rounded
// once to bf16 or kept in fp32; bf16 caches are copied (or widened).
//
// Bound: HBM.  A row of `width` values reads width bytes (bf16: 2 width), its scale
// and its slot, and writes 2 or 4 width bytes; one multiply a value.
//
// Split: a lane owns 16 values of a row (16 bytes of codes); a block takes a
// tile of whole rows so that a row index is a division by a constant, and every
// thread has its loads of kItems pieces in flight before the first conversion: all
// slots first, then all pieces.
//
// Measured: 131072 tokens of 8 heads of 128, e4m3 to bf16: 120 us = 6.8 TB/s, the copy
// rate (piece by piece, each behind its slot's check: 3 us more; with two 16-byte stores a
// lane, each filling half sectors: 174); 131072 latent rows of 576: 35.3 us = 6.5 TB/s.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace fp8kv {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;                    // 16-value pieces in flight per thread

template <int WIDTH, bool BF16, bool F32, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(ReadParams p, int64_t tiles) {
    constexpr int U = WIDTH / 16;            // pieces of a row
    constexpr int kRows = kThreads * kItems / U;   // rows of a tile
    const int which = blockIdx.x >= tiles;
    // at most 2^30 rows (the host refuses more)
    const int r0 = static_cast<int>((blockIdx.x - (which ? tiles : 0)) * kRows);
    const int rows = static_cast<int>(p.T * p.H);
    const uint8_t* cache = which ? p.cache[1] : p.cache[0];
    void* const out = which ? p.out[1] : p.out[0];
    const float* scale = which ? p.scale[1] : p.scale[0];
    const float* scale_cache = which ? p.scale_cache[1] : p.scale_cache[0];
    pdl_wait();
    pdl_trigger();

    // ALIGNED: rows start at 32-byte boundaries on both sides, and a lane's 16 values
    // move in one 32-byte access (two 16-byte stores with that stride fill half sectors)
    Bytes32 x[kItems];
    float s[kItems];
    bool have[kItems];
    int64_t slot[kItems];
    int head[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int rr = (threadIdx.x + i * kThreads) / U;
        const int r = r0 + rr;
        have[i] = rr < kRows && r < rows;
        slot[i] = -1;                        // negative: padding, a zero row
        head[i] = 0;
        if (have[i]) {
            const unsigned ur = static_cast<unsigned>(r);
            const int t = p.H == 1 ? r : static_cast<int>(ur / static_cast<unsigned>(p.H));
            head[i] = r - t * p.H;
            slot[i] = p.slot_mapping[t];
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int item = threadIdx.x + i * kThreads;
        const int u = item - item / U * U;
#pragma unroll
        for (int w = 0; w < 8; ++w) x[i].w[w] = 0u;
        s[i] = 0.f;
        if (slot[i] < 0 || slot[i] >= p.num_blocks * kPage) continue;
        const int64_t row = ((slot[i] >> 4) * p.H + head[i]) * kPage + (slot[i] & 15);
        if constexpr (BF16) {
            const uint8_t* src = cache + (row * WIDTH + u * 16) * 2;
            if constexpr (ALIGNED) {
                x[i] = load32(src);
            } else {
                *reinterpret_cast<uint4*>(x[i].w) = *reinterpret_cast<const uint4*>(src);
                *reinterpret_cast<uint4*>(x[i].w + 4) = *reinterpret_cast<const uint4*>(src + 16);
            }
        } else {
            *reinterpret_cast<uint4*>(x[i].w) =
                *reinterpret_cast<const uint4*>(cache + row * WIDTH + u * 16);
            s[i] = p.mode == FP8KV_SCALE_PER_TOKEN_HEAD ? scale_cache[row]
                   : scale[p.mode == FP8KV_SCALE_PER_HEAD ? head[i] : 0];
        }
    }
    // behind the loads: the report's store may alias them and would hold them back
#pragma unroll
    for (int i = 0; i < kItems; ++i)
        if (slot[i] >= p.num_blocks * kPage) report(p.err, FP8KV_ERR_BAD_INDEX);
    auto put = [](void* dst, const Bytes32& v) {
        if constexpr (ALIGNED) {
            store32(dst, v);
        } else {
            static_cast<uint4*>(dst)[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
            static_cast<uint4*>(dst)[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
        }
    };
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (!have[i]) continue;
        const int item = threadIdx.x + i * kThreads;
        const int rr = item / U, u = item - rr * U;
        const int64_t at = static_cast<int64_t>(r0 + rr) * WIDTH + u * 16;
        if constexpr (BF16 && !F32) {
            put(static_cast<__nv_bfloat16*>(out) + at, x[i]);
        } else {
            float f[16];
            if constexpr (BF16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 a = unpack_bf16x2(x[i].w[j]);
                    f[2 * j] = a.x;
                    f[2 * j + 1] = a.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t lo, hi;
                    f16x2x2_from_e4m3x4(x[i].w[j], lo, hi);
                    const float2 a = unpack_f16x2(lo), b = unpack_f16x2(hi);
                    f[4 * j] = a.x * s[i];
                    f[4 * j + 1] = a.y * s[i];
                    f[4 * j + 2] = b.x * s[i];
                    f[4 * j + 3] = b.y * s[i];
                }
            }
            Bytes32 o;
            if constexpr (F32) {
                float* dst = static_cast<float*>(out) + at;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.w[j] = __float_as_uint(f[8 * g + j]);
                    put(dst + 8 * g, o);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o.w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
                put(static_cast<__nv_bfloat16*>(out) + at, o);
            }
        }
    }
}

template <int WIDTH, bool BF16, bool F32>
cudaError_t launch_typed(const ReadParams& p, int tensors, cudaStream_t stream) {
    constexpr int kRows = kThreads * kItems / (WIDTH / 16);
    const int64_t tiles = (p.T * p.H + kRows - 1) / kRows;
    bool aligned = true;                     // rows are multiples of 32 bytes
    for (int i = 0; i < tensors; ++i)
        aligned = aligned && reinterpret_cast<uintptr_t>(p.out[i]) % 32 == 0 &&
                  (!BF16 || reinterpret_cast<uintptr_t>(p.cache[i]) % 32 == 0);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(attr, tiles * tensors, kThreads, 0, stream);
    return aligned
               ? cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, BF16, F32, true>, p, tiles)
               : cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, BF16, F32, false>, p, tiles);
}

template <int WIDTH>
cudaError_t launch_width(const ReadParams& p, int tensors, int kv_dtype, int out_f32,
                         cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16)
        return out_f32 ? launch_typed<WIDTH, true, true>(p, tensors, stream)
                       : launch_typed<WIDTH, true, false>(p, tensors, stream);
    return out_f32 ? launch_typed<WIDTH, false, true>(p, tensors, stream)
                   : launch_typed<WIDTH, false, false>(p, tensors, stream);
}

}  // namespace

cudaError_t launch_cache_read(const ReadParams& p, int tensors, int width, int kv_dtype,
                              int out_f32, cudaStream_t stream) {
    switch (width) {
        case 64: return launch_width<64>(p, tensors, kv_dtype, out_f32, stream);
        case 128: return launch_width<128>(p, tensors, kv_dtype, out_f32, stream);
        case 256: return launch_width<256>(p, tensors, kv_dtype, out_f32, stream);
        case 128 + kLatentRope:
            return launch_width<128 + kLatentRope>(p, tensors, kv_dtype, out_f32, stream);
        case 256 + kLatentRope:
            return launch_width<256 + kLatentRope>(p, tensors, kv_dtype, out_f32, stream);
        default: return launch_width<512 + kLatentRope>(p, tensors, kv_dtype, out_f32, stream);
    }
}

}  // namespace fp8kv
