// cache_read.cu -- cached rows back as values: out = code * scale (e4m3), rounded
// once to bf16 or kept in fp32; bf16 caches are copied (or widened).
//
// Bound: HBM.  A row of `width` values reads width bytes (bf16: 2 width), its scale
// and its slot, and writes 2 or 4 width bytes; one multiply a value.
//
// Split: a lane owns 16 values of a row (a 16-byte load of codes); a block takes a
// tile of whole rows so that a row index is a division by a constant, and every
// thread has its loads of kItems pieces in flight before the first conversion.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace fp8kv {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;                    // 16-value pieces in flight per thread

template <int WIDTH, bool BF16, bool F32>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(ReadParams p, int64_t tiles) {
    constexpr int U = WIDTH / 16;            // pieces of a row
    constexpr int kRows = kThreads * kItems / U;   // rows of a tile
    const int which = blockIdx.x >= tiles;
    const int64_t r0 = (blockIdx.x - (which ? tiles : 0)) * kRows;
    const int64_t rows = p.T * p.H;
    const uint8_t* cache = p.cache[which];
    pdl_wait();
    pdl_trigger();

    uint4 x[kItems], y[kItems];
    float s[kItems];
    bool have[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int item = threadIdx.x + i * kThreads;
        const int rr = item / U, u = item - rr * U;
        const int64_t r = r0 + rr;
        x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
        s[i] = 0.f;
        have[i] = rr < kRows && r < rows;
        if (!have[i]) continue;
        const int64_t t = p.H == 1 ? r : r / p.H;
        const int h = static_cast<int>(r - t * p.H);
        const int64_t slot = p.slot_mapping[t];
        if (slot < 0) continue;              // padding: a zero row
        if (slot >= p.num_blocks * kPage) {
            if (u == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
            continue;
        }
        const int64_t row = ((slot >> 4) * p.H + h) * kPage + (slot & 15);
        if constexpr (BF16) {
            const uint4* src = reinterpret_cast<const uint4*>(cache + (row * WIDTH + u * 16) * 2);
            x[i] = src[0];
            y[i] = src[1];
        } else {
            x[i] = *reinterpret_cast<const uint4*>(cache + row * WIDTH + u * 16);
            s[i] = p.mode == FP8KV_SCALE_PER_TOKEN_HEAD ? p.scale_cache[which][row]
                   : p.scale[which][p.mode == FP8KV_SCALE_PER_HEAD ? h : 0];
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (!have[i]) continue;
        const int item = threadIdx.x + i * kThreads;
        const int rr = item / U, u = item - rr * U;
        const int64_t at = (r0 + rr) * WIDTH + u * 16;
        if constexpr (BF16 && !F32) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out[which]) + at);
            dst[0] = x[i];
            dst[1] = y[i];
        } else {
            float f[16];
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            if constexpr (BF16) {
                const uint32_t v[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = unpack_bf16x2(w[j]), b = unpack_bf16x2(v[j]);
                    f[2 * j] = a.x;
                    f[2 * j + 1] = a.y;
                    f[8 + 2 * j] = b.x;
                    f[8 + 2 * j + 1] = b.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t lo, hi;
                    f16x2x2_from_e4m3x4(w[j], lo, hi);
                    const float2 a = unpack_f16x2(lo), b = unpack_f16x2(hi);
                    f[4 * j] = a.x * s[i];
                    f[4 * j + 1] = a.y * s[i];
                    f[4 * j + 2] = b.x * s[i];
                    f[4 * j + 3] = b.y * s[i];
                }
            }
            if constexpr (F32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out[which]) + at);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dst[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            } else {
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
                uint4* dst =
                    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out[which]) + at);
                dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

template <int WIDTH>
cudaError_t launch_width(const ReadParams& p, int tensors, int kv_dtype, int out_f32,
                         cudaStream_t stream) {
    constexpr int kRows = kThreads * kItems / (WIDTH / 16);
    const int64_t tiles = (p.T * p.H + kRows - 1) / kRows;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(attr, tiles * tensors, kThreads, 0, stream);
    if (kv_dtype == FP8KV_KV_BF16)
        return out_f32 ? cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, true, true>, p, tiles)
                       : cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, true, false>, p, tiles);
    return out_f32 ? cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, false, true>, p, tiles)
                   : cudaLaunchKernelEx(&cfg, cache_read_kernel<WIDTH, false, false>, p, tiles);
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
