// rope_write.cu -- rotary positions fused with the cache writes: q and k of the
// paged K/V cache (rope_kv_cache_write), and the shared rotary key and the
// queries' rotary part of the latent cache (latent_cache_write).
//
// What they compute: pairs (x, y) of a row's first rotary_dim values become
//     (x cos a - y sin a, y cos a + x sin a) * mscale,  a = position * theta_i,
// in fp32 from bf16.  Queries are rounded once, to bf16.  Keys are rounded once,
// to the cache's type: the e4m3 scale and codes come from the fp32 values (a
// rotation to bf16 followed by fp8kv_kv_cache_write would round twice).
//
// Bound: HBM.  Per token rope_kv_cache_write reads 2 D (Hq + 2 Hkv) bytes and writes
// 2 D Hq + 2 D Hkv (e4m3) plus the scales; the arithmetic (a few operations per
// byte, one sine and cosine per pair and token) hides behind it.
//
// Split: D / 16 lanes own one row, 16 values each, so both partners of every pair
// and the codes of a row stay in one lane and its scale is a shuffle reduction.  A
// warp takes rows of ONE token, so that its angles are computed once, shared out
// over the rows' lanes, and used for all of them.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace fp8kv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                   // rows a lane keeps in flight

// Stores one row's 16 values of this lane into an e4m3 or bf16 cache row at `dst`
// (the row's first byte).
__device__ __forceinline__ void store_cache16(uint8_t* dst, const RopeUnit& un,
                                              const float (&f)[16], bool bf16, float s) {
    if (bf16) {
        *reinterpret_cast<uint4*>(dst + 2 * un.a) = pack_bf16x8(f);
        *reinterpret_cast<uint4*>(dst + 2 * un.b) = pack_bf16x8(f + 8);
    } else {
        uint32_t w[4];
        e4m3_codes16(f, s, w);
        *reinterpret_cast<uint2*>(dst + un.a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + un.b) = make_uint2(w[2], w[3]);
    }
}

__device__ __forceinline__ float amax16(const float (&f)[16]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(f[i]));
    return a;
}

// Rows of a token in the order q heads, k heads, v heads; warp w of the grid takes
// rows [c * rows_per_warp, ...) of token w / chunks, c = w % chunks.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 2) rope_kv_cache_write_kernel(RopeWriteParams p,
                                                                          int chunks) {
    constexpr int U = D / 16;                // lanes per row
    constexpr int kRows = 32 / U;            // rows per warp at a time
    const int lane = threadIdx.x & 31;
    const int u = lane % U, g = lane / U;
    const unsigned group = ((1u << U) - 1u) << (g * U);
    const int64_t warp =
        static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    const int64_t t = warp / chunks;
    pdl_wait();                              // inputs of earlier kernels are visible
    pdl_trigger();
    if (t >= p.T) return;
    const int rows = p.Hq + 2 * p.Hkv;
    const int r0 = static_cast<int>(warp - t * chunks) * p.rows_per_warp;
    const int r1 = min(rows, r0 + p.rows_per_warp);
    const RopeUnit un = rope_unit<INTERLEAVED>(u, p.rotary_dim);
    const int64_t slot = p.slot_mapping[t];
    const int64_t position = p.positions[t];
    const bool bad = slot >= p.num_blocks * kPage;
    const bool store = slot >= 0 && !bad;    // a negative slot stores nothing (padding)
    if (bad && lane == 0 && r1 > p.Hq) report(p.err, FP8KV_ERR_BAD_INDEX);

    float2 cs[8];
    bool have_angles = false;
    for (int base = r0; base < r1; base += kRows * kUnroll) {
        uint4 xa[kUnroll], xb[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = base + i * kRows + g;
            xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < r1 && (r < p.Hq || store)) {
                const __nv_bfloat16* src =
                    r < p.Hq ? p.q + t * p.q_stride + static_cast<int64_t>(r) * D
                    : r < p.Hq + p.Hkv
                        ? p.k + t * p.k_stride + static_cast<int64_t>(r - p.Hq) * D
                        : p.v + t * p.v_stride + static_cast<int64_t>(r - p.Hq - p.Hkv) * D;
                xa[i] = *reinterpret_cast<const uint4*>(src + un.a);
                xb[i] = *reinterpret_cast<const uint4*>(src + un.b);
            }
        }
        if (!have_angles) {                  // while the first rows' loads are in flight
            rope_share<U>(cs, position, p.freqs, p.rotary_dim, p.mscale, lane);
            have_angles = true;
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = base + i * kRows + g;
            if (r >= r1) continue;           // a row's lanes leave together
            float f[16];
            unpack_bf16x8(xa[i], f);
            unpack_bf16x8(xb[i], f + 8);
            if (un.turns && r < p.Hq + p.Hkv) rope_turn<INTERLEAVED>(f, cs);
            if (r < p.Hq) {
                __nv_bfloat16* dst =
                    p.q_out + t * p.q_out_stride + static_cast<int64_t>(r) * D;
                *reinterpret_cast<uint4*>(dst + un.a) = pack_bf16x8(f);
                *reinterpret_cast<uint4*>(dst + un.b) = pack_bf16x8(f + 8);
                continue;
            }
            if (!store) continue;
            const int which = r >= p.Hq + p.Hkv;           // 0 = K, 1 = V
            const int h = r - p.Hq - (which ? p.Hkv : 0);
            const int64_t row = ((slot >> 4) * p.Hkv + h) * kPage + (slot & 15);
            float s = 1.f;
            if (!p.kv_bf16) {
                if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD) {
                    float a = amax16(f);
#pragma unroll
                    for (int o = U / 2; o > 0; o >>= 1)
                        a = fmaxf(a, __shfl_xor_sync(group, a, o));
                    s = __fdiv_rn(a, 448.0f);
                    if (u == 0) (which ? p.v_scale_cache : p.k_scale_cache)[row] = s;
                } else {
                    const float* sc = which ? p.v_scale : p.k_scale;
                    s = sc[p.mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                }
            }
            uint8_t* cache = static_cast<uint8_t*>(which ? p.v_cache : p.k_cache);
            store_cache16(cache + row * D * (p.kv_bf16 ? 2 : 1), un, f, p.kv_bf16 != 0, s);
        }
    }
}

// ---------------------------------------------------------------- latent cache
// Warp w of the grid: token w / tasks; task 0 stores the token's cache row (lane j
// owns latent values [16j, 16j + 16), lanes 28..31 the 64 rotated ones), task
// i > 0 turns query heads [32 (i - 1), 32 i), 4 lanes a head.
constexpr int kHeadsPerTask = 8 * kUnroll;

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) latent_cache_write_kernel(LatentWriteParams p,
                                                                         int tasks) {
    constexpr int U = kLatentRope / 16;
    const int lane = threadIdx.x & 31;
    const int u = lane % U, g = lane / U;
    const int64_t warp =
        static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    const int64_t t = warp / tasks;
    pdl_wait();
    pdl_trigger();
    if (t >= p.T) return;
    const int task = static_cast<int>(warp - t * tasks);
    const RopeUnit un = rope_unit<INTERLEAVED>(u, kLatentRope);
    const bool turn = p.positions != nullptr;
    float2 cs[8];

    if (task == 0) {
        const int64_t slot = p.slot_mapping[t];
        if (slot < 0) return;                // padding
        if (slot >= p.num_blocks * kPage) {
            if (lane == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
            return;
        }
        const bool latent = lane < p.L / 16;
        const bool key = lane >= 32 - U;
        uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa, ka = xa, kb = xa;
        if (latent) {
            const __nv_bfloat16* src = p.c + t * p.c_stride + lane * 16;
            xa = *reinterpret_cast<const uint4*>(src);
            xb = *reinterpret_cast<const uint4*>(src + 8);
        }
        if (key) {
            const __nv_bfloat16* src = p.k_pe + t * p.k_pe_stride;
            ka = *reinterpret_cast<const uint4*>(src + un.a);
            kb = *reinterpret_cast<const uint4*>(src + un.b);
        }
        if (turn) rope_share<U>(cs, p.positions[t], p.freqs, kLatentRope, p.mscale, lane);
        float f[16], k[16];
        unpack_bf16x8(xa, f);
        unpack_bf16x8(xb, f + 8);
        unpack_bf16x8(ka, k);
        unpack_bf16x8(kb, k + 8);
        if (turn) rope_turn<INTERLEAVED>(k, cs);
        float s = 1.f;
        if (!p.kv_bf16) {
            if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD) {
                float a = fmaxf(amax16(f), amax16(k));   // lanes without a part hold zeros
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                s = __fdiv_rn(a, 448.0f);
                if (lane == 0) p.scale_cache[slot] = s;
            } else {
                s = p.scale[0];
            }
        }
        const int elem = p.kv_bf16 ? 2 : 1;
        uint8_t* row = p.cache + slot * (p.L + kLatentRope) * elem;
        const RopeUnit plain{lane * 16, lane * 16 + 8, false};
        if (latent) store_cache16(row, plain, f, p.kv_bf16 != 0, s);
        if (key) store_cache16(row + p.L * elem, un, k, p.kv_bf16 != 0, s);
        return;
    }

    uint4 xa[kUnroll], xb[kUnroll];
    const int h0 = (task - 1) * kHeadsPerTask + g;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int h = h0 + 8 * i;
        xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.H) {
            const __nv_bfloat16* src = p.q_pe + t * p.q_stride + h * p.q_head_stride;
            xa[i] = *reinterpret_cast<const uint4*>(src + un.a);
            xb[i] = *reinterpret_cast<const uint4*>(src + un.b);
        }
    }
    if (turn) rope_share<U>(cs, p.positions[t], p.freqs, kLatentRope, p.mscale, lane);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int h = h0 + 8 * i;
        if (h >= p.H) continue;
        float f[16];
        unpack_bf16x8(xa[i], f);
        unpack_bf16x8(xb[i], f + 8);
        if (turn) rope_turn<INTERLEAVED>(f, cs);
        __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + h * p.q_out_head_stride;
        *reinterpret_cast<uint4*>(dst + un.a) = pack_bf16x8(f);
        *reinterpret_cast<uint4*>(dst + un.b) = pack_bf16x8(f + 8);
    }
}

template <int D>
cudaError_t launch_rope(const RopeWriteParams& p, int interleaved, int64_t blocks, int chunks,
                        cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(attr, blocks, kThreads, 0, stream);
    return interleaved
               ? cudaLaunchKernelEx(&cfg, rope_kv_cache_write_kernel<D, true>, p, chunks)
               : cudaLaunchKernelEx(&cfg, rope_kv_cache_write_kernel<D, false>, p, chunks);
}

}  // namespace

cudaError_t launch_rope_kv_cache_write(RopeWriteParams p, int D, int interleaved,
                                       cudaStream_t stream, int num_sms) {
    // A warp takes a whole token (its angles computed once) when there are tokens
    // enough to fill the GPU; few tokens are cut into chunks of one load batch.
    const int rows = p.Hq + 2 * p.Hkv;
    const int batch = 32 / (D / 16) * kUnroll;
    const int64_t fill = static_cast<int64_t>(num_sms) * 16;
    int chunks = 1;
    if (p.T < fill) {
        const int64_t want = (fill + p.T - 1) / p.T;
        const int most = (rows + batch - 1) / batch;
        chunks = static_cast<int>(want < most ? want : most);
    }
    p.rows_per_warp = (rows + chunks - 1) / chunks;
    chunks = (rows + p.rows_per_warp - 1) / p.rows_per_warp;
    const int64_t blocks = (p.T * chunks + kThreads / 32 - 1) / (kThreads / 32);
    switch (D) {
        case 64: return launch_rope<64>(p, interleaved, blocks, chunks, stream);
        case 128: return launch_rope<128>(p, interleaved, blocks, chunks, stream);
        default: return launch_rope<256>(p, interleaved, blocks, chunks, stream);
    }
}

cudaError_t launch_latent_cache_write(const LatentWriteParams& p, int interleaved,
                                      cudaStream_t stream, int num_sms) {
    (void)num_sms;
    const int tasks = 1 + (p.q_pe ? (p.H + kHeadsPerTask - 1) / kHeadsPerTask : 0);
    const int64_t blocks = (p.T * tasks + kThreads / 32 - 1) / (kThreads / 32);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(attr, blocks, kThreads, 0, stream);
    return interleaved ? cudaLaunchKernelEx(&cfg, latent_cache_write_kernel<true>, p, tasks)
                       : cudaLaunchKernelEx(&cfg, latent_cache_write_kernel<false>, p, tasks);
}

}  // namespace fp8kv
