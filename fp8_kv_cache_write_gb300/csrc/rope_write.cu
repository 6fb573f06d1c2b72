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
// warp takes rows of ONE token at a time, so that its angles are computed once, shared
// out over the rows' lanes, and used for all of them.
//
// Loads: the reads in flight, not the arithmetic, set the rate, and registers hold too
// few of them.  Every lane copies the pieces it will use itself into shared memory
// (cp.async), kDepth - 1 batches ahead and across tokens, in warps that stay for many
// tokens; what a lane reads back only that lane wrote, so nothing synchronises.
//
// Measured: 32768 tokens, 32 / 8 heads of 128, e4m3 with per-token-head scales: 122 us =
// 6.1 TB/s, 0.90 of the copy rate (plain loads in 16 warps an SM: 141 us; 20 warps, 2 rows
// ahead: 139; asking later tokens' rows into L2 first: 149 to 172).  8 tokens: 3.6 us a
// call in a graph, the latency of two dependent loads.  The latent write keeps one token
// per warp and many warps (32768 tokens, 16 heads: 33.4 us = 5.7 TB/s, 0.84; the ring
// above in persistent warps: 52; the slot's check in front of the loads: 41; 5, 6, 8 CTAs
// an SM for 7: 39, 37, 36; CTAs of 8 warps: 37 to 39): its rows are short, and what is
// left is the issue slots (62 % busy) and the latency between a warp's loads and stores.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace fp8kv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnroll = 2;                   // rows of a load batch per lane
constexpr int kDepth = 4;                    // batches of the ring
constexpr int kBlocksPerSm = 4;              // persistent: more at once is slower (32768
                                             // tokens: 4: 124 us, 5: 131, 6: 136)
constexpr int kLatentBlocksPerSm = 7;

// A warp's ring: [batch][row of the batch, group a or b][lane].
struct Ring {
    uint4 x[kDepth][2 * kUnroll][32];
};

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

// Largest of a warp's non-negative values (their bits are ordered like they are).
__device__ __forceinline__ float warp_max_nonneg(float a) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

__device__ __forceinline__ float amax16(const float (&f)[16]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(f[i]));
    return a;
}

// Rows of a token in the order q heads, k heads, v heads.  An item is rows
// [c * rows_per_item, ...) of a token, c < chunks; warps take items in turn.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    rope_kv_cache_write_kernel(RopeWriteParams p, int chunks) {
    constexpr int U = D / 16;                // lanes per row
    constexpr int kRows = 32 / U;            // rows per warp at a time
    constexpr int kBatch = kRows * kUnroll;
    __shared__ Ring rings[kWarps];
    Ring& ring = rings[threadIdx.x / 32];
    const int lane = threadIdx.x & 31;
    const int u = lane % U, g = lane / U;
    const unsigned group = ((1u << U) - 1u) << (g * U);
    const int warps = gridDim.x * kWarps;
    const int w = blockIdx.x * kWarps + threadIdx.x / 32;
    const int items = static_cast<int>(p.T) * chunks;
    const int rows = p.Hq + 2 * p.Hkv;
    const RopeUnit un = rope_unit<INTERLEAVED>(u, p.rotary_dim);
    pdl_wait();                              // inputs of earlier kernels are visible
    pdl_trigger();
    if (w >= items) return;
    const uint64_t pol = l2_evict_first();   // inputs are read once

    // ---- copies: item `ci` of this warp, its rows from `cr` on, into slot `cslot`
    int ci = w, cslot = 0;
    int cr = (w % chunks) * p.rows_per_item;
    auto copy = [&] {
        if (ci < items) {
            const int c = ci % chunks;
            const int64_t t = ci / chunks;
            const int end = min(rows, (c + 1) * p.rows_per_item);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int r = cr + i * kRows + g;
                if (r >= end) continue;
                const __nv_bfloat16* src =
                    r < p.Hq ? p.q + t * p.q_stride + r * D
                    : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * D
                                       : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * D;
                cp_async16_hint(smem_addr(&ring.x[cslot][2 * i][lane]), src + un.a, pol);
                cp_async16_hint(smem_addr(&ring.x[cslot][2 * i + 1][lane]), src + un.b, pol);
            }
            cr += kBatch;
            if (cr >= end) {
                ci += warps;
                cr = (ci % chunks) * p.rows_per_item;
            }
        }
        cslot = cslot + 1 == kDepth ? 0 : cslot + 1;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) copy();

    int slot_in = 0;                         // ring slot of the next batch
    int64_t next_position = p.positions[w / chunks], next_slot = p.slot_mapping[w / chunks];
    for (int item = w; item < items; item += warps) {
        const int64_t t = item / chunks;
        const int r0 = (item % chunks) * p.rows_per_item;
        const int r1 = min(rows, r0 + p.rows_per_item);
        const int64_t position = next_position, slot = next_slot;
        if (item + warps < items) {
            next_position = p.positions[(item + warps) / chunks];
            next_slot = p.slot_mapping[(item + warps) / chunks];
        }
        const bool bad = slot >= p.num_blocks * kPage;
        const bool store = slot >= 0 && !bad;    // a negative slot stores nothing (padding)
        if (bad && lane == 0 && r1 > p.Hq) report(p.err, FP8KV_ERR_BAD_INDEX);
        const int64_t page_row = (slot >> 4) * p.Hkv * kPage + (slot & 15);
        RopeAngles angles;
        rope_share<U>(angles, position, p.freqs, p.rotary_dim, p.mscale, lane);
        for (int base = r0; base < r1; base += kBatch) {
            copy();
            cp_async_wait<kDepth - 1>();
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int r = base + i * kRows + g;
                if (r >= r1) continue;           // a row's lanes leave together
                float f[16];
                unpack_bf16x8(ring.x[slot_in][2 * i][lane], f);
                unpack_bf16x8(ring.x[slot_in][2 * i + 1][lane], f + 8);
                if (un.turns && r < p.Hq + p.Hkv) rope_turn<INTERLEAVED>(f, angles);
                if (r < p.Hq) {
                    __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + r * D;
                    *reinterpret_cast<uint4*>(dst + un.a) = pack_bf16x8(f);
                    *reinterpret_cast<uint4*>(dst + un.b) = pack_bf16x8(f + 8);
                    continue;
                }
                if (!store) continue;
                const int which = r >= p.Hq + p.Hkv;           // 0 = K, 1 = V
                const int h = r - p.Hq - (which ? p.Hkv : 0);
                const int64_t row = page_row + h * kPage;
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
            slot_in = slot_in + 1 == kDepth ? 0 : slot_in + 1;
        }
    }
}

// ---------------------------------------------------------------- latent cache
// Warp w of the grid: token w / tasks, part w % tasks.  Part 0 stores the token's
// cache row: lane j owns latent values [16j, 16j + 16) and pair j of the rotary key,
// whose angle it computes.  The queries' heads, 4 lanes each (8 pairs a lane, their
// angles fetched from the lanes that have them), are dealt to all parts, or to the
// parts behind the first.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kLatentBlocksPerSm)
    latent_cache_write_kernel(LatentWriteParams p, int tasks) {
    constexpr int U = kLatentRope / 16;
    const int lane = threadIdx.x & 31;
    const int u = lane % U, g = lane / U;
    // at most 2^30 (token, part) pairs: 32-bit arithmetic
    const unsigned warp = blockIdx.x * kWarps + threadIdx.x / 32;
    const unsigned token = tasks == 1 ? warp : warp / static_cast<unsigned>(tasks);
    const int task = static_cast<int>(warp - token * tasks);
    const int64_t t = token;
    pdl_wait();
    pdl_trigger();
    if (t >= p.T) return;
    const bool turn = p.positions != nullptr;
    const RopeUnit un = rope_unit<INTERLEAVED>(u, kLatentRope);
    // heads of this part
    const int parts = tasks > 1 ? tasks - 1 : 1;
    const int per = (p.H + parts - 1) / parts;
    const bool heads = p.q_pe != nullptr && (tasks == 1 || task > 0);
    const int h_lo = heads && task > 0 ? (task - 1) * per : 0;
    const int h_hi = heads ? min(p.H, h_lo + per) : 0;

    uint4 xa[kUnroll], xb[kUnroll];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + 8 * i + g;
            xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h < h_hi) {
                const __nv_bfloat16* src = p.q_pe + t * p.q_stride + h * p.q_head_stride;
                xa[i] = *reinterpret_cast<const uint4*>(src + un.a);
                xb[i] = *reinterpret_cast<const uint4*>(src + un.b);
            }
        }
    };
    if (h_lo < h_hi) load(h_lo);

    int64_t slot = -1;                       // negative: padding, nothing is stored
    uint4 ca = make_uint4(0u, 0u, 0u, 0u), cb = ca;
    float2 k = make_float2(0.f, 0.f);
    const int ka = INTERLEAVED ? 2 * lane : lane;                    // the pair's values
    const int kb = INTERLEAVED ? 2 * lane + 1 : lane + kLatentRope / 2;
    const bool latent = lane < p.L / 16;
    if (task == 0) {
        slot = p.slot_mapping[t];
        if (latent) {
            const __nv_bfloat16* src = p.c + t * p.c_stride + lane * 16;
            ca = *reinterpret_cast<const uint4*>(src);
            cb = *reinterpret_cast<const uint4*>(src + 8);
        }
        const __nv_bfloat16* kp = p.k_pe + t * p.k_pe_stride;
        k = make_float2(__bfloat162float(kp[ka]), __bfloat162float(kp[kb]));
    }
    int64_t position = 0, freq = 0;
    if (turn) {
        position = p.positions[t];
        freq = p.freqs[lane];
    }
    // behind the loads: the report's store may alias them and would hold them back
    if (slot >= p.num_blocks * kPage) {
        if (lane == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        slot = -1;
    }
    float2 mine = make_float2(1.f, 0.f);     // pair `lane`'s cosine and sine
    if (turn) {
        mine = rope_cos_sin(position, freq);
        mine.x *= p.mscale;
        mine.y *= p.mscale;
    }

    if (slot >= 0) {
        if (turn)
            k = make_float2(k.x * mine.x - k.y * mine.y, k.y * mine.x + k.x * mine.y);
        float f[16];
        unpack_bf16x8(ca, f);
        unpack_bf16x8(cb, f + 8);
        const int elem = p.kv_bf16 ? 2 : 1;
        uint8_t* row = p.cache + slot * (p.L + kLatentRope) * elem;
        const RopeUnit plain{lane * 16, lane * 16 + 8, false};
        if (p.kv_bf16) {
            if (latent) store_cache16(row, plain, f, true, 1.f);
            __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(row) + p.L;
            kr[ka] = __float2bfloat16_rn(k.x);
            kr[kb] = __float2bfloat16_rn(k.y);
        } else {
            float s;
            if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD) {
                // lanes without latent values hold zeros
                float a = fmaxf(amax16(f), fmaxf(fabsf(k.x), fabsf(k.y)));
                a = warp_max_nonneg(a);
                s = __fdiv_rn(a, 448.0f);
                if (lane == 0) p.scale_cache[slot] = s;
            } else {
                s = p.scale[0];
            }
            if (latent) {                    // 16 codes, one store
                uint32_t w[4];
                e4m3_codes16(f, s, w);
                *reinterpret_cast<uint4*>(row + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            const uint32_t kc = s != 0.0f ? e4m3x2_by_divide(k.x, k.y, s) : 0u;
            if (INTERLEAVED) {
                *reinterpret_cast<uint16_t*>(row + p.L + ka) = static_cast<uint16_t>(kc);
            } else {
                row[p.L + ka] = static_cast<uint8_t>(kc);
                row[p.L + kb] = static_cast<uint8_t>(kc >> 8);
            }
        }
    }
    if (h_lo >= h_hi) return;                // whole warps

    RopeAngles angles;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float2 m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i].x = __shfl_sync(0xffffffffu, mine.x, 8 * u + e + i);
            m[i].y = __shfl_sync(0xffffffffu, mine.y, 8 * u + e + i);
        }
        angles.set(e / 2, m[0], m[1]);
    }
    for (int h0 = h_lo; h0 < h_hi; h0 += 8 * kUnroll) {
        uint4 ya[kUnroll], yb[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            ya[i] = xa[i];
            yb[i] = xb[i];
        }
        if (h0 + 8 * kUnroll < h_hi) load(h0 + 8 * kUnroll);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + 8 * i + g;
            if (h >= h_hi) continue;
            float f[16];
            unpack_bf16x8(ya[i], f);
            unpack_bf16x8(yb[i], f + 8);
            if (turn) rope_turn<INTERLEAVED>(f, angles);
            __nv_bfloat16* dst = p.q_out + t * p.q_out_stride + h * p.q_out_head_stride;
            *reinterpret_cast<uint4*>(dst + un.a) = pack_bf16x8(f);
            *reinterpret_cast<uint4*>(dst + un.b) = pack_bf16x8(f + 8);
        }
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
    // A warp takes whole tokens (angles computed once) when there are tokens enough for
    // every warp; few tokens are cut into items of one load batch.
    const int rows = p.Hq + 2 * p.Hkv;
    const int batch = 32 / (D / 16) * kUnroll;
    const int64_t fill = static_cast<int64_t>(num_sms) * kBlocksPerSm * kWarps;
    int chunks = 1;
    if (p.T < fill) {
        const int64_t want = (fill + p.T - 1) / p.T;
        const int most = (rows + batch - 1) / batch;
        chunks = static_cast<int>(want < most ? want : most);
    }
    p.rows_per_item = (rows + chunks - 1) / chunks;
    chunks = (rows + p.rows_per_item - 1) / p.rows_per_item;
    int64_t blocks = (p.T * chunks + kWarps - 1) / kWarps;
    if (blocks > fill / kWarps) blocks = fill / kWarps;
    switch (D) {
        case 64: return launch_rope<64>(p, interleaved, blocks, chunks, stream);
        case 128: return launch_rope<128>(p, interleaved, blocks, chunks, stream);
        default: return launch_rope<256>(p, interleaved, blocks, chunks, stream);
    }
}

cudaError_t launch_latent_cache_write(const LatentWriteParams& p, int interleaved,
                                      cudaStream_t stream, int num_sms) {
    // One warp a token when there are tokens enough for every warp; few tokens leave
    // their heads to warps of their own, a load batch each.
    const int batch = 8 * kUnroll;
    const int64_t fill = static_cast<int64_t>(num_sms) * kLatentBlocksPerSm * kWarps;
    const int tasks = p.q_pe == nullptr || p.T >= fill ? 1 : 1 + (p.H + batch - 1) / batch;
    const int64_t blocks = (p.T * tasks + kWarps - 1) / kWarps;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pdl_config(attr, blocks, kThreads, 0, stream);
    return interleaved ? cudaLaunchKernelEx(&cfg, latent_cache_write_kernel<true>, p, tasks)
                       : cudaLaunchKernelEx(&cfg, latent_cache_write_kernel<false>, p, tasks);
}

}  // namespace fp8kv
