// prefix_attn.cu -- the part of decode attention that a batch shares: every query of the
// batch over one common prefix, its pages read once instead of once per sequence.
//
// For KV head h the rows are the R = B G queries of its group over all sequences; with the
// prefix's keys they form one dense attention problem,
//     z = softmax_scale * s_k(t) q . code_k(t),  p = 2^(z - m),  O = sum_t p s_v(t) code_v(t)
// whose partials (O, m, l) list_attn.cu joins with each sequence's own tail.
//
// Bound: HBM for up to 128 rows a head (a 128-key tile of D 128 is 32 KiB of codes, about
// 1440 clocks of an SM's share of the copy rate; its two products take 1024 clocks of the
// tensor pipe), the tensor pipe and the softmax beyond.
// Split: tiles of 128 rows x 128 keys (D 256: 64 keys).  The (head, row tile, key tile)
// units of the call, flattened in that order, are dealt in equal consecutive shares to one
// persistent CTA per SM; a share that crosses a row tile goes on with the next one's queries.
// A row tile's pieces go to slots of their own in the workspace.
//
// Warps of a CTA: 16 for the softmax (a thread owns a quarter of a row's keys), one that
// issues the MMAs, one that brings K and V by TMA, one for scales and masks, 4 for V tiles.
//   * e4m3: S = Q K^T is an e4m3 MMA straight on the cached codes, q in two e4m3 terms under a
//     power of two per row (bf16's 8 bits; exact down to 2^-10 of the row's largest value,
//     beyond that to 2^-17 of it).  V's codes become f16 (exactly) on their way from where
//     bulk copies leave them into swizzled tiles, and the weights are one f16 term: rounded
//     to 2^-12 of a weight, lifted so that weights down to 2^-21 of the largest stay normal.
//     (Keys as f16 too, one MMA: 9400 clocks a tile in all, the conversion of both tiles and
//     the shared memory it moves through being the bound.)
//   * bf16: q, keys and values as they are; the weights are two bf16 terms (2^-16).
//   * the weights go to tensor memory and are the second product's A operand from there.
//   * per-token V scales as in list_attn.cu: the reference m follows z + log2 s_v, so the
//     weights p s_v stay within f16 whatever the scales are.
//   * S is double-buffered: the next tile's Q K^T runs while this one's softmax does.
//   * references move only when a tile exceeds them by 2^8; O is rescaled in tensor memory.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"
#include "prefix.cuh"
#include "tc.cuh"

namespace fp8kv {

namespace {

constexpr int kRows = kPrefixRows;           // query rows of a tile (MMA M)
constexpr int kParts = 4;                    // threads of a row
constexpr int kSoftWarps = 4 * kParts;
constexpr int kMmaWarp = kSoftWarps;
constexpr int kTmaWarp = kSoftWarps + 1;
constexpr int kSclWarp = kSoftWarps + 2;
constexpr int kVWarp = kSoftWarps + 3;       // 4 warps
constexpr int kThreads = (kVWarp + 4) * 32;
constexpr float kMaxInit = -1.0e30f;
constexpr float kLazy = 8.f;                 // binades a logit may pass the reference
constexpr int kScl = 4;                      // slots of the tiles' scales and masks

template <int D, bool BF16>
struct Cfg {
    static constexpr int kKeys = prefix_keys(D);
    static constexpr int kPages = kKeys / kPage;
    static constexpr int kRowB = D * (BF16 ? 2 : 1);          // cached bytes of a row
    static constexpr int kPanelB = kRowB < 128 ? kRowB : 128; // K and Q rows are panels this wide
    static constexpr int kPanels = kRowB / kPanelB;
    static constexpr uint32_t kLayout = kPanelB == 128 ? kLayoutSw128 : kLayoutSw64;
    static constexpr int kRawB = kKeys * kRowB;               // a tile as cached
    static constexpr int kTileB = kKeys * D * 2;              // a 16-bit V tile
    static constexpr int kQTerms = BF16 ? 1 : 2;
    static constexpr int kQB = kRows * kRowB;                 // one term of Q
    static constexpr int kPart = kKeys / kParts;              // keys of a softmax thread
    static constexpr int kPTerms = BF16 ? 2 : 1;
    static constexpr float kLiftLog2 = BF16 ? 0.f : 7.f;      // w <= 2^8: below f16's 2^16
    static constexpr float kLift = BF16 ? 1.f : 128.f;
    // stages: K tiles, V tiles in 16 bits, e4m3 V tiles as cached
    static constexpr int kKS = BF16 ? (D == 64 ? 3 : 2) : 3;
    static constexpr int kVS = BF16 ? (D == 256 ? 2 : 3) : 2;
    static constexpr int kRS = BF16 ? kVS : (D == 256 ? 2 : 3);
    // tensor memory: S twice, the weights (16-bit pairs), O
    static constexpr uint32_t kPCol = 2 * kKeys;
    static constexpr uint32_t kOCol = kPCol + kPTerms * kKeys / 2;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kOCol + D <= kTmemCols, "tensor memory");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kQTerms * kQB;
    static constexpr int kOffV = kOffK + kKS * kRawB;
    static constexpr int kOffRaw = kOffV + kVS * kTileB;      // (bf16: V arrives in place)
    // per tile: key factors, value factors, log2 of the value scales, which keys are there
    static constexpr int kOffScl = kOffRaw + (BF16 ? 0 : kRS * kRawB);
    static constexpr int kOffMask = kOffScl + (BF16 ? 0 : kScl * 3 * 128 * 4);
    static constexpr int kOffPages = kOffMask + kScl * 4 * 4; // which pages a V tile got
    static constexpr int kOffMax = kOffPages + 16;            // [2][parts][128 rows]
    static constexpr int kOffBar = kOffMax + 2 * kParts * 128 * 4;
    static constexpr int kSmem = kOffBar + 48 * 8 + 1024;
    static_assert(kSmem <= 227 * 1024 - 64, "shared memory");
};

enum { kKFull = 0, kKEmpty = 3, kRawFull = 6, kRawEmpty = 9, kVFull = 12, kVEmpty = 15, kSFull = 18,
       kSEmpty = 20, kSclFull = 22, kSclEmpty = 26, kPFull = 30, kPvDone, kQFull, kIdle, kPair,
       kBars = kPair + 4 };
static_assert(kBars <= 48, "barriers");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A from tensor memory (16-bit pairs a column), B from shared memory.
__device__ __forceinline__ void mma_f16kind_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two fp32 values -> their e4m3 codes and the codes of what those miss.
__device__ __forceinline__ void e4m3_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = e4m3x2_from_f32(a, b);
    const float2 h = unpack_f16x2(f16x2_from_e4m3x2(hi));
    lo = e4m3x2_from_f32(a - h.x, b - h.y);
}

// The tiles of a share in order: key tile within the row tile, row tile's head.
struct Walk {
    int tile, tiles, row_tile, row_tiles, head;
    __device__ __forceinline__ Walk(int64_t t, int tiles_, int row_tiles_)
        : tiles(tiles_), row_tiles(row_tiles_) {
        const int64_t u = t / tiles_;
        tile = static_cast<int>(t - u * tiles_);
        head = static_cast<int>(u / row_tiles_);
        row_tile = static_cast<int>(u - static_cast<int64_t>(head) * row_tiles_);
    }
    __device__ __forceinline__ void next() {
        if (++tile < tiles) return;
        tile = 0;
        if (++row_tile < row_tiles) return;
        row_tile = 0;
        ++head;
    }
};

// Waits for a phase; gives up when another thread has, or when the budget ran out.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort,
                                              int32_t* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0u) {
            if (*abort) return false;
            if (global_ns() - t0 > kWaitBudgetNs) {
                *abort = 1;
                report(err, FP8KV_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

template <int D, bool BF16, bool PT>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, PrefixAttnParams p) {
    using C = Cfg<D, BF16>;
    constexpr int KEYS = C::kKeys;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    volatile int* abort = &s_abort;

    pdl_wait();
    pdl_trigger();
    int len = p.prefix_len[0];
    if (len > p.prefix_pages * kPage) {
        if (blockIdx.x == 0 && tid == 0) report(p.err, FP8KV_ERR_BAD_INDEX);
        len = p.prefix_pages * kPage;
    }
    const PrefixShares shares(len, KEYS, p.units, gridDim.x);
    const int T = shares.tiles;                              // key tiles of a row tile
    if (static_cast<int64_t>(blockIdx.x) >= shares.workers) return;   // no tile for this CTA
    const int64_t w0 = shares.begin(blockIdx.x);
    const int n = static_cast<int>(shares.begin(blockIdx.x + 1) - w0);   // its tiles
    const int64_t R = static_cast<int64_t>(p.B) * p.G;       // rows of a head

    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), C::kTmemCols);
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar(kKFull + i), 1);
            mbar_init(bar(kKEmpty + i), 1);
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), 4);
            mbar_init(bar(kVFull + i), 4);
            mbar_init(bar(kVEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kSEmpty + i), kSoftWarps);
        }
        for (int i = 0; i < kScl; ++i) {
            mbar_init(bar(kSclFull + i), 1);
            mbar_init(bar(kSclEmpty + i), kSoftWarps);
        }
        mbar_init(bar(kPFull), kSoftWarps);
        mbar_init(bar(kPvDone), 1);
        mbar_init(bar(kQFull), kSoftWarps);
        mbar_init(bar(kIdle), 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar(kPair + i), kParts);
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // block id of page i of a key tile (-1: none)
    auto fetch = [&](int tile, int i) -> int {
        const int page = tile * C::kPages + i;
        if (i >= C::kPages || page >= (len + kPage - 1) / kPage) return -1;
        const int id = p.prefix_table[page];
        if (id >= 0 && id < p.num_blocks) return id;
        report(p.err, FP8KV_ERR_BAD_INDEX);
        return -1;
    };
    // a warp's wait for a phase, and its arrival
    auto wait = [&](int i, int phase) {
        return __all_sync(0xffffffffu, wait_or_abort(bar(i), phase & 1, abort, p.err));
    };
    auto arrive = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    if (warp >= kVWarp) {
        // =============================== V tiles for the second product
        const int lt = tid - kVWarp * 32;                    // 0 .. 127
        Walk at(w0, T, p.row_tiles);
        for (int j = 0; j < n; ++j, at.next()) {
            const int rs = j % C::kRS, st = j % C::kVS;
            const int left = len - at.tile * KEYS;           // keys of the tile that exist
            if (!wait(kRawFull + rs, j / C::kRS)) break;
            const uint32_t pages = reinterpret_cast<const uint32_t*>(smem + C::kOffPages)[rs];
            // rows that are not there may hold any bytes, NaN among them: zeros
            const bool whole = left >= KEYS && pages == (1u << C::kPages) - 1u;
            auto there = [&](int row) { return ((pages >> (row / kPage)) & 1u) && row < left; };
            uint8_t* dst = smem + C::kOffV + st * C::kTileB;
            if constexpr (BF16) {
                if (!whole)
                    for (int q = lt; q < KEYS * D / 8; q += 128) {
                        const int row = q % KEYS, c = q / KEYS;
                        if (!there(row))
                            *reinterpret_cast<uint4*>(dst + (c / 8) * (KEYS * 128) + row * 128 +
                                                      (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
            } else {
                if (j >= C::kVS && !wait(kVEmpty + st, (j - C::kVS) / C::kVS)) break;
                const uint8_t* raw = smem + C::kOffRaw + rs * C::kRawB;
                constexpr int kChunks = C::kRowB / 16;
#pragma unroll
                for (int k = 0; k < KEYS * kChunks / 128; ++k) {
                    const int q = k * 128 + lt, row = q / kChunks, c = q % kChunks;
                    uint4 x = *reinterpret_cast<const uint4*>(raw + q * 16);
                    if (!whole && !there(row)) x = make_uint4(0u, 0u, 0u, 0u);
                    uint4 a, b;
                    f16x2x2_from_e4m3x4(x.x, a.x, a.y);
                    f16x2x2_from_e4m3x4(x.y, a.z, a.w);
                    f16x2x2_from_e4m3x4(x.z, b.x, b.y);
                    f16x2x2_from_e4m3x4(x.w, b.z, b.w);
                    // 16 values: two 16-byte chunks of panel c / 4; the pieces of odd panels
                    // store theirs the other way round, which keeps a row's stores apart
                    uint8_t* line = dst + (c / 4) * (KEYS * 128) + row * 128;
                    const int flip = (c >> 2) & 1, c0 = (c & 3) * 2 + flip;
                    *reinterpret_cast<uint4*>(line + ((c0 ^ (row & 7)) << 4)) = flip ? b : a;
                    *reinterpret_cast<uint4*>(line + (((c0 ^ 1) ^ (row & 7)) << 4)) = flip ? a : b;
                }
            }
            fence_proxy_async();
            arrive(kVFull + st);
            if constexpr (!BF16) {
                if (lane == 0) mbar_arrive(bar(kRawEmpty + rs));
            }
        }
    } else if (warp == kSclWarp) {
        // =============================== scales and masks, four keys a lane
        Walk at(w0, T, p.row_tiles);
        const bool mine = lane < KEYS / 4;
        auto load = [&](float4& ks, float4& vs, int& valid) {
            const int id = mine ? fetch(at.tile, lane / 4) : -1;
            valid = id < 0 ? 0 : min(4, max(0, len - at.tile * KEYS - 4 * lane));
            if (PT && valid > 0) {
                const int64_t row = (static_cast<int64_t>(id) * p.Hkv + at.head) * kPage + (lane & 3) * 4;
                ks = *reinterpret_cast<const float4*>(p.k_scale_cache + row);
                vs = *reinterpret_cast<const float4*>(p.v_scale_cache + row);
            }
            at.next();
        };
        float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
        int valid = 0;
        load(ks, vs, valid);
        for (int j = 0; j < n; ++j) {
            float4 ks1 = ks, vs1 = vs;
            int valid1 = 0;
            if (j + 1 < n) load(ks1, vs1, valid1);
            const int sl = j % kScl;
            if (j >= kScl && !wait(kSclEmpty + sl, (j - kScl) / kScl)) break;
            uint32_t bits = ((1u << valid) - 1u) << (4 * (lane & 7));
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, off);
            if ((lane & 7) == 0 && mine)
                reinterpret_cast<uint32_t*>(smem + C::kOffMask)[sl * 4 + lane / 8] = bits;
            if (PT && mine) {
                float* scl = reinterpret_cast<float*>(smem + C::kOffScl) + sl * 3 * 128 + 4 * lane;
                const float kk[4] = {ks.x, ks.y, ks.z, ks.w}, vv[4] = {vs.x, vs.y, vs.z, vs.w};
                float f[4], w[4], lg[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a key that is not there has any scales: none of them reaches a sum
                    const float v = i < valid ? vv[i] : 0.f;
                    f[i] = i < valid ? kk[i] * p.scale_log2 : 0.f;
                    w[i] = v * C::kLift;
                    lg[i] = fmaxf(__log2f(fabsf(v)), -100.f);
                }
                *reinterpret_cast<float4*>(scl) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(scl + 128) = make_float4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<float4*>(scl + 256) = make_float4(lg[0], lg[1], lg[2], lg[3]);
            }
            arrive(kSclFull + sl);
            ks = ks1;
            vs = vs1;
            valid = valid1;
        }
    } else if (warp == kTmaWarp) {
        // =============================== K tiles (tensor copies), V tiles (e4m3: as cached)
        if (lane == 0) {
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
        }
        Walk at(w0, T, p.row_tiles);
        int id = fetch(at.tile, lane), k_issued = 0, v_issued = 0;
        for (int j = 0; j < n; ++j) {
            const int h = at.head;
            at.next();
            const int id_next = j + 1 < n ? fetch(at.tile, lane) : -1;
            const uint32_t here = __ballot_sync(0xffffffffu, id >= 0);
            const uint32_t bytes = __popc(here) * (kPage * C::kRowB);
            const int ks = j % C::kKS, rs = j % C::kRS;
            const int64_t tile = static_cast<int64_t>(id) * p.Hkv + h;
            if (j >= C::kKS && !wait(kKEmpty + ks, (j - C::kKS) / C::kKS)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + ks), bytes);
            __syncwarp();
            if (id >= 0)
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_3d(sbase + C::kOffK + ks * C::kRawB + pn * (KEYS * C::kPanelB) +
                                    lane * (kPage * C::kPanelB),
                                &kmap, pn * C::kPanelB, 0, static_cast<int>(tile), bar(kKFull + ks));
            ++k_issued;
            if (j >= C::kRS &&
                !wait((BF16 ? kVEmpty : kRawEmpty) + rs, (j - C::kRS) / C::kRS))
                break;
            if (lane == 0) {
                reinterpret_cast<uint32_t*>(smem + C::kOffPages)[rs] = here;
                mbar_arrive_expect_tx(bar(kRawFull + rs), bytes);
            }
            __syncwarp();
            if (id >= 0) {
                if constexpr (BF16) {
#pragma unroll
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        tma_load_3d(sbase + C::kOffV + rs * C::kTileB + pn * (KEYS * 128) +
                                        lane * (kPage * 128),
                                    &vmap, pn * 128, 0, static_cast<int>(tile), bar(kRawFull + rs));
                } else {
                    bulk_load(sbase + C::kOffRaw + rs * C::kRawB + lane * (kPage * C::kRowB),
                              p.v_cache + tile * (kPage * C::kRowB), kPage * C::kRowB,
                              bar(kRawFull + rs));
                }
            }
            ++v_issued;
            id = id_next;
        }
        // an abort: the copies in flight land before the CTA leaves (bounded waits)
        if (*abort) {
            for (int j = max(0, k_issued - C::kKS); j < k_issued; ++j)
                (void)mbar_wait_bounded(bar(kKFull + j % C::kKS), (j / C::kKS) & 1);
            for (int j = max(0, v_issued - C::kRS); j < v_issued; ++j)
                (void)mbar_wait_bounded(bar(kRawFull + j % C::kRS), (j / C::kRS) & 1);
        }
    } else if (warp == kMmaWarp) {
        // =============================== MMA issuer (one thread)
        if (lane == 0) {
            constexpr uint32_t kFmt = BF16 ? 1u : 0u;        // bf16; e4m3 and f16
            constexpr uint32_t id_qk = instr_desc(kFmt, kFmt, 0, 0, KEYS, kRows);
            constexpr uint32_t id_pv = instr_desc(kFmt, kFmt, 0, 1, D, kRows);
            auto wait1 = [&](int i, int phase) { return wait_or_abort(bar(i), phase & 1, abort, p.err); };
            auto qk = [&](int j) {
                const uint32_t k = sbase + C::kOffK + (j % C::kKS) * C::kRawB;
                constexpr int kPer = C::kPanelB / 32;        // 32-byte steps of a panel
#pragma unroll
                for (int s = 0; s < C::kRowB / 32; ++s) {
                    const uint64_t b = smem_desc(k + (s / kPer) * (KEYS * C::kPanelB) + (s % kPer) * 32,
                                                 16, 8 * C::kPanelB, C::kLayout);
#pragma unroll
                    for (int term = 0; term < C::kQTerms; ++term) {
                        const uint64_t a =
                            smem_desc(sbase + C::kOffQ + term * C::kQB +
                                          (s / kPer) * (kRows * C::kPanelB) + (s % kPer) * 32,
                                      16, 8 * C::kPanelB, C::kLayout);
                        const uint32_t acc = s > 0 || term > 0 ? 1u : 0u;
                        if constexpr (BF16)
                            mma_f16kind(tmem + (j & 1) * KEYS, a, b, id_qk, acc);
                        else
                            mma_f8f6f4(tmem + (j & 1) * KEYS, a, b, id_qk, acc);
                    }
                }
                mma_commit(bar(kSFull + (j & 1)));
                mma_commit(bar(kKEmpty + j % C::kKS));
            };
            auto pv = [&](int j, bool first) {
                const uint32_t v = sbase + C::kOffV + (j % C::kVS) * C::kTileB;
#pragma unroll
                for (int s = 0; s < KEYS / 16; ++s) {        // 16 keys a step
                    // V is MN-major: 8-key groups 1024 bytes apart, panels of 64 channels
                    // KEYS rows apart
                    const uint64_t b = smem_desc_sw128(v + s * 16 * 128, KEYS * 128, 1024);
#pragma unroll
                    for (int term = 0; term < C::kPTerms; ++term)
                        mma_f16kind_ta(tmem + C::kOCol, tmem + C::kPCol + term * (KEYS / 2) + s * 8, b,
                                       id_pv, first && s == 0 && term == 0 ? 0u : 1u);
                }
                mma_commit(bar(kPvDone));
                mma_commit(bar(kVEmpty + j % C::kVS));
            };
            auto next_qk = [&](int j) {
                if (!wait1(kKFull + j % C::kKS, j / C::kKS)) return false;
                if (j >= 2 && !wait1(kSEmpty + (j & 1), (j - 2) >> 1)) return false;
                tc_fence_after();
                qk(j);
                return true;
            };
            Walk at(w0, T, p.row_tiles);
            int piece = 0;
            bool ok = wait1(kQFull, 0) && next_qk(0);
            for (int j = 0; j < n && ok; ++j) {
                const bool first = j == 0 || at.tile == 0;
                at.next();
                const bool more = j + 1 < n, crosses = more && at.tile == 0;
                if (more && !crosses) ok = next_qk(j + 1);
                if (!ok || !wait1(kPFull, j) || !wait1(kVFull + j % C::kVS, j / C::kVS)) break;
                tc_fence_after();
                pv(j, first);
                // the next row tile's queries replace this one's once PV of its last tile ran
                if (crosses) ok = wait1(kQFull, ++piece) && next_qk(j + 1);
            }
            mma_commit(bar(kIdle));                          // every MMA issued has ended
            (void)mbar_wait_bounded(bar(kIdle), 0);
        }
        __syncwarp();
    } else {
        // =============================== softmax, partials
        const int quarter = warp & 3, part = warp >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        float* maxima = reinterpret_cast<float*>(smem + C::kOffMax);
        constexpr int KP = C::kPart;                         // keys of this thread
        constexpr int DP = D / kParts;                       // its channels of Q and O
        constexpr int DC = DP < 32 ? DP : 32;                // columns of one O load
        int pair_phase = 0;
        bool ok = true;
        // the warps of a quarter meet
        auto meet = [&]() {
            arrive(kPair + quarter);
            return wait(kPair + quarter, pair_phase++);
        };
        // x of every part of the row: the largest, or the sum
        auto share = [&](float* at, float x) {
            at[part * kRows + r] = x;
            return meet();
        };
        for (int j = 0; j < n && ok;) {
            const int64_t t = w0 + j;
            const int64_t u = t / T;                         // row tile: head, rows
            const int h = static_cast<int>(u / p.row_tiles);
            const int64_t row0 = (u - static_cast<int64_t>(h) * p.row_tiles) * kRows;
            const int j_end = min(n, j + T - static_cast<int>(t - u * T));
            // a warp whose rows all lie behind the last one only keeps step
            const bool act = row0 + 32 * quarter < R;
            const bool row_ok = row0 + r < R;
            // ---- the row tile's queries
            float rf = p.scale_log2;                         // raw S (PT: column-scaled) -> logit
            if (act) {
                const int64_t row = row0 + r;
                const int64_t b = row_ok ? row / p.G : 0;
                const int g = row_ok ? static_cast<int>(row - b * p.G) : 0;
                const __nv_bfloat16* q = p.q + (b * p.Hq + h * p.G + g) * D + part * DP;
                uint4 x[DP / 8];
#pragma unroll
                for (int c = 0; c < DP / 8; ++c) {
                    x[c] = *reinterpret_cast<const uint4*>(q + c * 8);
                    if (!row_ok) x[c] = make_uint4(0u, 0u, 0u, 0u);
                }
                auto chunk = [&](int term, int cc) {         // 16-byte piece cc of the row
                    constexpr int kPer = C::kPanelB / 16;
                    const int sw = kPer == 8 ? (cc % kPer) ^ (r & 7) : (cc % kPer) ^ ((r >> 1) & 3);
                    return reinterpret_cast<uint4*>(smem + C::kOffQ + term * C::kQB +
                                                    (cc / kPer) * (kRows * C::kPanelB) +
                                                    r * C::kPanelB + sw * 16);
                };
                if constexpr (BF16) {
#pragma unroll
                    for (int c = 0; c < DP / 8; ++c) *chunk(0, part * (DP / 8) + c) = x[c];
                } else {
                    float amax = 0.f;
#pragma unroll
                    for (int c = 0; c < DP / 8; ++c) {
                        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = unpack_bf16x2(w[i]);
                            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                    if (!share(maxima, amax)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < kParts; ++i) amax = fmaxf(amax, maxima[i * kRows + r]);
                    // the power of two that puts max |q| into [2^7, 2^8)
                    int e = 0;
                    if (amax > 0.f && amax <= 3.4e38f) {
                        frexpf(amax, &e);
                        e = min(126, max(-126, 8 - e));
                    }
                    const float up = ldexpf(1.f, e);
                    // (an infinite query, which e4m3 cannot hold, has no finite result)
                    rf = amax <= 3.4e38f ? ldexpf(1.f, -e) : CUDART_NAN_F;
                    if constexpr (!PT)
                        rf *= p.scale_log2 * p.k_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4& y = x[2 * c + i / 2];
                            const float2 f0 = unpack_bf16x2(i & 1 ? y.z : y.x);
                            const float2 f1 = unpack_bf16x2(i & 1 ? y.w : y.y);
                            uint32_t h0, h1, l0, l1;
                            e4m3_terms(f0.x * up, f0.y * up, h0, l0);
                            e4m3_terms(f1.x * up, f1.y * up, h1, l1);
                            hi[i] = h0 | (h1 << 16);
                            lo[i] = l0 | (l1 << 16);
                        }
                        const int cc = part * (DP / 16) + c;
                        *chunk(0, cc) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *chunk(1, cc) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (!meet()) {                           // every part has read the maxima
                        ok = false;
                        break;
                    }
                }
            }
            fence_proxy_async();
            arrive(kQFull);

            const uint64_t rf2 = pack_f32x2(rf, rf);
            float m = kMaxInit, l = 0.f;                     // l: times the lift if not PT
            const int j0 = j;
            for (; j < j_end; ++j) {
                const int sl = j % kScl;
                if (!wait(kSFull + (j & 1), j >> 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!act) {
                    tc_fence_before();
                    arrive(kSEmpty + (j & 1));
                    if (j > 0 && !wait(kPvDone, j - 1)) {    // (the phase before is over)
                        ok = false;
                        break;
                    }
                    arrive(kPFull);
                    if (lane == 0) mbar_arrive(bar(kSclEmpty + sl));
                    continue;
                }
                uint32_t s[KP];
                tmem_ld_n<KP>(tmem + lanes + (j & 1) * KEYS + part * KP, s);
                tmem_wait_ld();
                tc_fence_before();
                arrive(kSEmpty + (j & 1));
                if (!wait(kSclFull + sl, j / kScl)) {
                    ok = false;
                    break;
                }
                const float* scl = reinterpret_cast<const float*>(smem + C::kOffScl) + sl * 3 * 128 +
                                   part * KP;
                uint32_t bits = reinterpret_cast<const uint32_t*>(smem + C::kOffMask)[sl * 4 + part * KP / 32];
                if constexpr (KP < 32) bits = (bits >> (part * KP % 32)) & ((1u << KP) - 1u);
                // logits up to the row's factor, and the row's largest (with log2 s_v)
                if constexpr (PT) {
#pragma unroll
                    for (int i = 0; i < KP; i += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(scl + i);
                        float2 a = unpack_f32x2(mul_f32x2(
                            pack_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), pack_f32x2(f.x, f.y)));
                        s[i] = __float_as_uint(a.x);
                        s[i + 1] = __float_as_uint(a.y);
                        a = unpack_f32x2(mul_f32x2(
                            pack_f32x2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), pack_f32x2(f.z, f.w)));
                        s[i + 2] = __float_as_uint(a.x);
                        s[i + 3] = __float_as_uint(a.y);
                    }
                }
                if (bits != (KP < 32 ? (1u << (KP % 32)) - 1u : 0xffffffffu)) {
#pragma unroll
                    for (int i = 0; i < KP; ++i)
                        if (!((bits >> i) & 1u)) s[i] = __float_as_uint(-CUDART_INF_F);
                }
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                for (int i = 0; i < KP; i += 4) {
                    float2 a = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                    float2 c = make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
                    if constexpr (PT) {
                        const float4 f = *reinterpret_cast<const float4*>(scl + 256 + i);
                        a = unpack_f32x2(fma_f32x2(pack_f32x2(a.x, a.y), rf2, pack_f32x2(f.x, f.y)));
                        c = unpack_f32x2(fma_f32x2(pack_f32x2(c.x, c.y), rf2, pack_f32x2(f.z, f.w)));
                    }
                    mx[(i / 4) & 3] = fmaxf(mx[(i / 4) & 3], fmaxf(a.x, a.y));
                    mx[(i / 4 + 2) & 3] = fmaxf(mx[(i / 4 + 2) & 3], fmaxf(c.x, c.y));
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if constexpr (!PT) top *= rf;                // (the factor is positive)
                float* both = maxima + (j & 1) * kParts * kRows;
                if (!share(both, top)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kParts; ++i) top = fmaxf(top, both[i * kRows + r]);
                float alpha = 1.f;
                if (top > m + kLazy) {                       // the same in all parts
                    alpha = ex2(m - top);
                    m = top;
                    l *= alpha;
                }
                // ---- weights (not PT: the lift is part of the exponent)
                const float off = PT ? -m : C::kLiftLog2 - m;
                const uint64_t off2 = pack_f32x2(off, off);
                uint32_t hi[KP / 2], lo[BF16 ? KP / 2 : 1];
                uint64_t l2[2] = {0u, 0u};
#pragma unroll
                for (int i = 0; i < KP; i += 2) {
                    const float2 z = unpack_f32x2(fma_f32x2(
                        pack_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), rf2, off2));
                    uint64_t e2 = pack_f32x2(ex2(z.x), ex2(z.y));
                    l2[(i / 2) & 1] = add_f32x2(l2[(i / 2) & 1], e2);
                    if constexpr (PT)
                        e2 = mul_f32x2(e2, *reinterpret_cast<const uint64_t*>(scl + 128 + i));
                    const float2 w = unpack_f32x2(e2);
                    if constexpr (BF16) {
                        hi[i / 2] = pack_bf16x2(w.x, w.y);
                        const float2 f = unpack_bf16x2(hi[i / 2]);
                        lo[i / 2] = pack_bf16x2(w.x - f.x, w.y - f.y);
                    } else {
                        hi[i / 2] = pack_f16x2(w.x, w.y);
                    }
                }
                const float2 ls = unpack_f32x2(add_f32x2(l2[0], l2[1]));
                l += ls.x + ls.y;
                // O and the weights' columns are free once PV of the tile before has run
                if (j > 0) {
                    if (!wait(kPvDone, j - 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < DP / DC; ++c) {      // this part's columns of O
                        uint32_t x[DC];
                        const uint32_t at = tmem + lanes + C::kOCol + part * DP + c * DC;
                        tmem_ld_n<DC>(at, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < DC; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * alpha);
                        tmem_st_n<DC>(at, x);
                    }
                }
                const uint32_t pcol = tmem + lanes + C::kPCol + part * (KP / 2);
                tmem_st_n<KP / 2>(pcol, hi);
                if constexpr (BF16) tmem_st_n<KP / 2>(pcol + KEYS / 2, lo);
                tmem_wait_st();
                tc_fence_before();
                arrive(kPFull);
                if (lane == 0) mbar_arrive(bar(kSclEmpty + sl));
            }
            if (!ok) break;
            // ---- the piece's partial: O, m and l of its rows
            if (!wait(kPvDone, j_end - 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (act) {
                float* both = maxima + (j_end & 1) * kParts * kRows;
                if (!share(both, l)) {
                    ok = false;
                    break;
                }
                l = 0.f;
#pragma unroll
                for (int i = 0; i < kParts; ++i) l += both[i * kRows + r];
                if constexpr (!PT) l *= 1.f / C::kLift;
                const int64_t at = (static_cast<int64_t>(h) * R + row0 + r) * p.splits +
                                   (static_cast<int64_t>(blockIdx.x) - shares.first(u));
                float f = 1.f / C::kLift;
                if constexpr (!BF16 && !PT)
                    f *= p.v_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                float* dst = p.part_o + at * D + part * DP;
#pragma unroll 1
                for (int c = 0; c < DP / DC; ++c) {
                    uint32_t x[DC];
                    tmem_ld_n<DC>(tmem + lanes + C::kOCol + part * DP + c * DC, x);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < DC; i += 4)
                            *reinterpret_cast<float4*>(dst + c * DC + i) = make_float4(
                                __uint_as_float(x[i]) * f, __uint_as_float(x[i + 1]) * f,
                                __uint_as_float(x[i + 2]) * f, __uint_as_float(x[i + 3]) * f);
                    }
                }
                if (row_ok && part == 0) {
                    p.part_m[at] = m;
                    p.part_l[at] = l;
                }
                // the sums are read before a next piece's maxima go to the same place
                if (!meet()) {
                    ok = false;
                    break;
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D, bool BF16, bool PT>
cudaError_t launch_one(const PrefixAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                       cudaStream_t stream) {
    using C = Cfg<D, BF16>;
    static unsigned long long done[64] = {};
    const void* fn = reinterpret_cast<const void*>(prefix_attn_kernel<D, BF16, PT>);
    const cudaError_t e = opt_in_smem(fn, C::kSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, p.workers, kThreads, C::kSmem, stream);
    return cudaLaunchKernelEx(&cfg, prefix_attn_kernel<D, BF16, PT>, kmap, vmap, p);
}

template <int D>
cudaError_t launch_d(const PrefixAttnParams& p, const CUtensorMap& km, const CUtensorMap& vm,
                     int kv_dtype, cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16) return launch_one<D, true, false>(p, km, vm, stream);
    if (p.scale_mode == FP8KV_SCALE_PER_TOKEN_HEAD) return launch_one<D, false, true>(p, km, vm, stream);
    return launch_one<D, false, false>(p, km, vm, stream);
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixAttnParams& p, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, int D, int kv_dtype,
                               cudaStream_t stream) {
    if (D == 64) return launch_d<64>(p, kmap, vmap, kv_dtype, stream);
    if (D == 128) return launch_d<128>(p, kmap, vmap, kv_dtype, stream);
    return launch_d<256>(p, kmap, vmap, kv_dtype, stream);
}

}  // namespace fp8kv
