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
// Warps of a CTA: 8 softmax warps (a thread owns one row's half of the keys), one that issues
// the MMAs, 4 that fill K and V tiles, one that brings e4m3 pages for them.
//   * e4m3: pages arrive by bulk copies (2 KiB each at D 128) in a ring of raw tiles; their
//     codes become f16 (exactly) on the way into 128-byte swizzled tiles; q is f16 under a
//     power of two per row.  Both products are kind::f16.
//     An e4m3 MMA would need q and p in two e4m3 terms for the decode's accuracy, which costs
//     what the f16 MMA costs.
//   * weights: f16 (e4m3 cache; rounded to 2^-12 of a weight, lifted so that weights down to
//     2^-21 of the largest stay normal) or two bf16 terms (bf16 cache, 2^-16).  They go to
//     tensor memory and are the second product's A operand from there.
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
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = kSoftWarps;
constexpr int kRawWarp = kSoftWarps + 1;     // e4m3: bulk copies
constexpr int kCopyWarp = kSoftWarps + 2;    // 4 warps: tiles
constexpr int kThreads = (kCopyWarp + 4) * 32;
constexpr float kMaxInit = -1.0e30f;
constexpr float kLazy = 8.f;                 // binades a logit may pass the reference

template <int D, bool BF16>
struct Cfg {
    static constexpr int kKeys = prefix_keys(D);
    static constexpr int kPages = kKeys / kPage;
    static constexpr int kRowB = D * (BF16 ? 2 : 1);          // cached bytes of a row
    static constexpr int kChunks = kRowB / 16;                // 16-byte pieces of a row
    static constexpr int kItems = kKeys * kChunks / 128;      // pieces of a copying thread
    static constexpr int kKStages = D == 256 ? 1 : 2;         // K tiles (V: 2)
    static constexpr int kTileB = kKeys * D * 2;              // 16-bit tile in shared memory
    static constexpr int kQB = kRows * D * 2;
    static constexpr int kHalf = kKeys / 2;                   // keys of a softmax thread
    static constexpr int kPTerms = BF16 ? 2 : 1;
    static constexpr float kLift = BF16 ? 1.f : 128.f;        // w <= 2^8: below f16's 2^16
    // tensor memory: S twice, the weights (16-bit pairs), O
    static constexpr uint32_t kPCol = 2 * kKeys;
    static constexpr uint32_t kOCol = kPCol + kPTerms * kKeys / 2;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kOCol + D <= kTmemCols, "tensor memory");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kQB;
    static constexpr int kOffV = kOffK + kKStages * kTileB;
    // e4m3: K and V tiles in turn as they lie in the cache, with K's their two scale rows
    // [2][128] and the set of pages that are there
    static constexpr int kRaw = 3;
    static constexpr int kRawScl = kKeys * kRowB;
    static constexpr int kRawPages = kRawScl + 1024;
    static constexpr int kRawB = kRawPages + 128;
    static constexpr int kOffRaw = kOffV + 2 * kTileB;
    // per tile, 4 slots: key factors, value factors, log2 of the value scales
    static constexpr int kOffScl = kOffRaw + (BF16 ? 0 : kRaw * kRawB);
    static constexpr int kOffMask = kOffScl + (BF16 ? 0 : 4 * 3 * 128 * 4);
    static constexpr int kOffMax = kOffMask + 4 * 4 * 4;      // [2][2 halves][128 rows]
    static constexpr int kOffBar = kOffMax + 2 * 2 * 128 * 4;
    static constexpr int kSmem = kOffBar + 32 * 8 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

enum { kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kSFull = 8, kSEmpty = 10, kPFull = 12,
       kPvDone, kQFull, kIdle, kPair, kRawFull = kPair + 4, kRawEmpty = kRawFull + 3 };

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

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
                 : "memory");
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
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(PrefixAttnParams p) {
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
    const int64_t w0 = shares.begin(blockIdx.x), w1 = shares.begin(blockIdx.x + 1);
    if (static_cast<int64_t>(blockIdx.x) >= shares.workers) return;   // no tile for this CTA
    const int n = static_cast<int>(w1 - w0);                 // its tiles
    const int64_t R = static_cast<int64_t>(p.B) * p.G;       // rows of a head

    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), C::kTmemCols);
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kKFull + i), 4);
            mbar_init(bar(kVFull + i), 4);
            mbar_init(bar(kKEmpty + i), 1);
            mbar_init(bar(kVEmpty + i), 1);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kSEmpty + i), kSoftWarps);
        }
        mbar_init(bar(kPFull), kSoftWarps);
        mbar_init(bar(kPvDone), 1);
        mbar_init(bar(kQFull), kSoftWarps);
        mbar_init(bar(kIdle), 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar(kPair + i), 2);
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), 4);
        }
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

    if (warp >= kCopyWarp) {
        // =============================== K and V tiles
        const int lt = tid - kCopyWarp * 32;                 // 0 .. 127
        bool ok = true;
        auto wait = [&](int i, int phase) {
            return ok = ok && __all_sync(0xffffffffu, wait_or_abort(bar(i), phase & 1, abort, p.err));
        };
        auto hand_over = [&](int i) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        Walk at(w0, T, p.row_tiles);
        for (int j = 0; j < n && ok; ++j, at.next()) {
            const int key0 = at.tile * KEYS;
            uint32_t* mask = reinterpret_cast<uint32_t*>(smem + C::kOffMask) + (j & 3) * 4;
            if constexpr (BF16) {
                // asynchronous copies straight into the swizzled tile; a tile is handed over
                // once the next one's (V after K, K after V) are on their way
                const int id = fetch(at.tile, lane), st_k = j % C::kKStages;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int stages = kv ? 2 : C::kKStages, st = j % stages;
                    if (j >= stages && !wait((kv ? kVEmpty : kKEmpty) + st, (j - stages) / stages)) break;
                    const uint8_t* cache = kv ? p.v_cache : p.k_cache;
                    const uint32_t dst = smem_addr(smem + (kv ? C::kOffV : C::kOffK) + st * C::kTileB);
#pragma unroll
                    for (int i = 0; i < C::kItems; ++i) {
                        const int q = i * 128 + lt, row = q / C::kChunks, c = q % C::kChunks;
                        const int blk = __shfl_sync(0xffffffffu, id, row / kPage);
                        const bool there = blk >= 0 && key0 + row < len;
                        const uint8_t* src = cache;
                        if (there)
                            src += ((static_cast<int64_t>(blk) * p.Hkv + at.head) * kPage + row % kPage) *
                                       C::kRowB + c * 16;
                        cp_async16_or_zero(dst + (c / 8) * (KEYS * 128) + row * 128 +
                                               (((c % 8) ^ (row & 7)) << 4),
                                           src, there);
                    }
                    cp_async_commit();
                    if (kv == 0) {
                        const int blk = __shfl_sync(0xffffffffu, id, (lt / kPage) % C::kPages);
                        const uint32_t m = __ballot_sync(0xffffffffu, blk >= 0 && key0 + lt < len);
                        if (lane == 0 && lt < KEYS) mask[lt / 32] = m;
                    }
                    if (kv == 1 || j > 0) {
                        cp_async_wait<1>();
                        hand_over(kv ? kKFull + st_k : kVFull + ((j - 1) & 1));
                    }
                }
            } else {
                // codes arrive as they lie in the cache (bulk copies of the copy warp) and
                // become f16 on their way into the tile
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int i = 2 * j + kv, rs = i % C::kRaw;
                    const int stages = kv ? 2 : C::kKStages, st = j % stages;
                    if (!wait(kRawFull + rs, i / C::kRaw)) break;
                    if (j >= stages && !wait((kv ? kVEmpty : kKEmpty) + st, (j - stages) / stages)) break;
                    const uint8_t* raw = smem + C::kOffRaw + rs * C::kRawB;
                    // which of the tile's pages are there
                    const uint32_t pages = *reinterpret_cast<const uint32_t*>(raw + C::kRawPages);
                    uint8_t* dst = smem + (kv ? C::kOffV : C::kOffK) + st * C::kTileB;
#pragma unroll
                    for (int k = 0; k < C::kItems; ++k) {
                        const int q = k * 128 + lt, row = q / C::kChunks, c = q % C::kChunks;
                        uint4 x = *reinterpret_cast<const uint4*>(raw + row * C::kRowB + c * 16);
                        if (!((pages >> (row / kPage)) & 1u) || key0 + row >= len)
                            x = make_uint4(0u, 0u, 0u, 0u);
                        uint4 a, b;
                        f16x2x2_from_e4m3x4(x.x, a.x, a.y);
                        f16x2x2_from_e4m3x4(x.y, a.z, a.w);
                        f16x2x2_from_e4m3x4(x.z, b.x, b.y);
                        f16x2x2_from_e4m3x4(x.w, b.z, b.w);
                        // 16 values: two 16-byte chunks of panel c / 4; the pieces of odd
                        // panels store theirs the other way round, which keeps a row's
                        // stores apart
                        uint8_t* line = dst + (c / 4) * (KEYS * 128) + row * 128;
                        const int flip = (c >> 2) & 1, c0 = (c & 3) * 2 + flip;
                        *reinterpret_cast<uint4*>(line + ((c0 ^ (row & 7)) << 4)) = flip ? b : a;
                        *reinterpret_cast<uint4*>(line + (((c0 ^ 1) ^ (row & 7)) << 4)) = flip ? a : b;
                    }
                    if (kv == 0) {
                        const bool valid = lt < KEYS && ((pages >> (lt / kPage)) & 1u) && key0 + lt < len;
                        const uint32_t m = __ballot_sync(0xffffffffu, valid);
                        if (lane == 0 && lt < KEYS) mask[lt / 32] = m;
                        if (PT && lt < KEYS) {
                            const float* rk = reinterpret_cast<const float*>(raw + C::kRawScl);
                            const float ks = valid ? rk[lt] : 0.f, vs = valid ? rk[128 + lt] : 0.f;
                            float* scl = reinterpret_cast<float*>(smem + C::kOffScl) + (j & 3) * 3 * 128;
                            scl[lt] = ks * p.scale_log2;
                            scl[128 + lt] = vs * C::kLift;
                            scl[256 + lt] = fmaxf(__log2f(fabsf(vs)), -100.f);
                        }
                    }
                    hand_over(kv ? kVFull + st : kKFull + st);
                    if (lane == 0) mbar_arrive(bar(kRawEmpty + rs));
                }
            }
        }
        if constexpr (BF16) {
            cp_async_wait<0>();
            if (ok) hand_over(kVFull + ((n - 1) & 1));
        }
    } else if (warp == kRawWarp) {
        // =============================== e4m3: bulk copies of the pages as they lie
        if constexpr (!BF16) {
            Walk at(w0, T, p.row_tiles);
            int id = fetch(at.tile, lane), issued = 0;
            for (; issued < 2 * n; ++issued) {
                const int kv = issued & 1, rs = issued % C::kRaw;
                if (issued >= C::kRaw &&
                    !__all_sync(0xffffffffu, wait_or_abort(bar(kRawEmpty + rs),
                                                           ((issued - C::kRaw) / C::kRaw) & 1, abort, p.err)))
                    break;
                const uint32_t here = __ballot_sync(0xffffffffu, id >= 0);
                uint8_t* raw = smem + C::kOffRaw + rs * C::kRawB;
                if (lane == 0) {
                    *reinterpret_cast<uint32_t*>(raw + C::kRawPages) = here;
                    fence_proxy_async();                     // the slot was read by plain loads
                    mbar_arrive_expect_tx(bar(kRawFull + rs),
                                          __popc(here) * (kPage * C::kRowB + (PT && !kv ? 128 : 0)));
                }
                __syncwarp();
                if (id >= 0) {
                    const int64_t tile = static_cast<int64_t>(id) * p.Hkv + at.head;
                    const uint32_t dst = smem_addr(raw), b = bar(kRawFull + rs);
                    bulk_load(dst + lane * (kPage * C::kRowB),
                              (kv ? p.v_cache : p.k_cache) + tile * (kPage * C::kRowB),
                              kPage * C::kRowB, b);
                    if (PT && !kv) {
                        bulk_load(dst + C::kRawScl + lane * 64, p.k_scale_cache + tile * kPage, 64, b);
                        bulk_load(dst + C::kRawScl + 512 + lane * 64, p.v_scale_cache + tile * kPage, 64, b);
                    }
                }
                if (kv) {
                    at.next();
                    id = issued + 1 < 2 * n ? fetch(at.tile, lane) : -1;
                }
            }
            // an abort: the copies in flight land before the CTA leaves (bounded waits)
            if (*abort)
                for (int i = issued > C::kRaw ? issued - C::kRaw : 0; i < issued; ++i)
                    (void)mbar_wait_bounded(bar(kRawFull + i % C::kRaw), (i / C::kRaw) & 1);
        }
    } else if (warp == kMmaWarp) {
        // =============================== MMA issuer (one thread)
        if (lane == 0) {
            constexpr uint32_t kFmt = BF16 ? 1u : 0u;
            constexpr uint32_t id_qk = instr_desc(kFmt, kFmt, 0, 0, KEYS, kRows);
            constexpr uint32_t id_pv = instr_desc(kFmt, kFmt, 0, 1, D, kRows);
            auto wait = [&](int i, int phase) { return wait_or_abort(bar(i), phase & 1, abort, p.err); };
            auto qk = [&](int j) {
                const uint32_t k = sbase + C::kOffK + (j % C::kKStages) * C::kTileB;
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {           // 32-byte steps over D
                    const uint64_t a = smem_desc_sw128(
                        sbase + C::kOffQ + (s / 4) * (kRows * 128) + (s % 4) * 32, 16, 1024);
                    const uint64_t b = smem_desc_sw128(k + (s / 4) * (KEYS * 128) + (s % 4) * 32, 16, 1024);
                    mma_f16kind(tmem + (j & 1) * KEYS, a, b, id_qk, s > 0 ? 1u : 0u);
                }
                mma_commit(bar(kSFull + (j & 1)));
                mma_commit(bar(kKEmpty + j % C::kKStages));
            };
            auto pv = [&](int j, bool first) {
                const uint32_t v = sbase + C::kOffV + (j & 1) * C::kTileB;
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
                mma_commit(bar(kVEmpty + (j & 1)));
            };
            auto next_qk = [&](int j) {
                if (!wait(kKFull + j % C::kKStages, j / C::kKStages)) return false;
                if (j >= 2 && !wait(kSEmpty + (j & 1), (j - 2) >> 1)) return false;
                tc_fence_after();
                qk(j);
                return true;
            };
            int piece = 0;
            bool ok = wait(kQFull, 0) && next_qk(0);
            for (int j = 0; j < n && ok; ++j) {
                const int64_t t = w0 + j;
                const bool first = j == 0 || t % T == 0;
                const bool more = j + 1 < n, crosses = more && (t + 1) % T == 0;
                if (more && !crosses) ok = next_qk(j + 1);
                if (!ok || !wait(kPFull, j) || !wait(kVFull + (j & 1), j >> 1)) break;
                tc_fence_after();
                pv(j, first);
                // the next row tile's queries replace this one's once PV of its last tile ran
                if (crosses) ok = wait(kQFull, ++piece) && next_qk(j + 1);
            }
            mma_commit(bar(kIdle));                          // every MMA issued has ended
            (void)mbar_wait_bounded(bar(kIdle), 0);
        }
        __syncwarp();
    } else {
        // =============================== softmax, partials
        const int quarter = warp & 3, kh = warp >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        float* maxima = reinterpret_cast<float*>(smem + C::kOffMax);
        constexpr int KH = C::kHalf;
        int pair_phase = 0;
        bool ok = true;
        auto wait = [&](int i, int phase) {
            return __all_sync(0xffffffffu, wait_or_abort(bar(i), phase & 1, abort, p.err));
        };
        auto arrive = [&](int i) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        // the two warps of a quarter meet
        auto meet = [&]() {
            arrive(kPair + quarter);
            return wait(kPair + quarter, pair_phase++);
        };
        for (int j = 0; j < n && ok;) {
            const int64_t t = w0 + j;
            const int64_t u = t / T;                         // row tile: head, rows
            const int h = static_cast<int>(u / p.row_tiles);
            const int64_t row0 = (u - static_cast<int64_t>(h) * p.row_tiles) * kRows;
            const int j_end = min(n, j + T - static_cast<int>(t % T));
            // a warp whose rows all lie behind the last one only keeps step
            const bool act = row0 + 32 * quarter < R;
            const bool row_ok = row0 + r < R;
            // ---- the row tile's queries
            float rf = p.scale_log2;                         // raw S (PT: column-scaled) -> logit
            if (act) {
                const int64_t row = row0 + r;
                const int64_t b = row_ok ? row / p.G : 0;
                const int g = row_ok ? static_cast<int>(row - b * p.G) : 0;
                const __nv_bfloat16* q = p.q + (b * p.Hq + h * p.G + g) * D + kh * (D / 2);
                float up = 1.f;
                if constexpr (!BF16) {
                    float amax = 0.f;
#pragma unroll 4
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(q + c * 8);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = unpack_bf16x2(w[i]);
                            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                    maxima[kh * kRows + r] = amax;
                    if (!meet()) {
                        ok = false;
                        break;
                    }
                    amax = fmaxf(amax, maxima[(kh ^ 1) * kRows + r]);
                    // the power of two that puts max |q| into [2^14, 2^15): exact in f16 but
                    // for values 2^-31 and less of the largest
                    int e = 0;
                    if (amax > 0.f && amax <= 3.4e38f) {
                        frexpf(amax, &e);
                        e = min(126, max(-126, 15 - e));
                    }
                    up = ldexpf(1.f, e);
                    rf = ldexpf(1.f, -e);
                    if constexpr (!PT)
                        rf *= p.scale_log2 * p.k_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                    if (!meet()) {                           // both have read the maxima
                        ok = false;
                        break;
                    }
                }
#pragma unroll 4
                for (int c = 0; c < D / 16; ++c) {
                    uint4 x = *reinterpret_cast<const uint4*>(q + c * 8);
                    if constexpr (!BF16) {
                        uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = unpack_bf16x2(w[i]);
                            w[i] = pack_f16x2(f.x * up, f.y * up);
                        }
                        x = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (!row_ok) x = make_uint4(0u, 0u, 0u, 0u);
                    const int cc = kh * (D / 16) + c;        // 16-byte chunk of the row
                    *reinterpret_cast<uint4*>(smem + C::kOffQ + (cc / 8) * (kRows * 128) + r * 128 +
                                              (((cc % 8) ^ (r & 7)) << 4)) = x;
                }
            }
            fence_proxy_async();
            arrive(kQFull);

            float m = kMaxInit, l = 0.f;
            const int j0 = j;
            for (; j < j_end; ++j) {
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
                    continue;
                }
                float s[KH];
                {
                    uint32_t raw[KH];
#pragma unroll
                    for (int c = 0; c < KH / 32; ++c)
                        tmem_ld32(tmem + lanes + (j & 1) * KEYS + kh * KH + c * 32,
                                  *reinterpret_cast<uint32_t(*)[32]>(raw + c * 32));
                    tmem_wait_ld();
                    tc_fence_before();
                    arrive(kSEmpty + (j & 1));
#pragma unroll
                    for (int i = 0; i < KH; ++i) s[i] = __uint_as_float(raw[i]);
                }
                const float* scl = reinterpret_cast<const float*>(smem + C::kOffScl) +
                                   (j & 3) * 3 * 128 + kh * KH;
                const uint32_t* mask = reinterpret_cast<const uint32_t*>(smem + C::kOffMask) +
                                       (j & 3) * 4 + kh * (KH / 32);
                bool whole = true;
#pragma unroll
                for (int c = 0; c < KH / 32; ++c) whole = whole && mask[c] == 0xffffffffu;
                // logits up to the row's factor, and the row's largest (with log2 s_v)
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                if constexpr (PT) {
#pragma unroll
                    for (int i = 0; i < KH; i += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(scl + i);
                        s[i] *= f.x;
                        s[i + 1] *= f.y;
                        s[i + 2] *= f.z;
                        s[i + 3] *= f.w;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < KH; ++i)
                        if (!((mask[i / 32] >> (i % 32)) & 1u)) s[i] = -CUDART_INF_F;
                }
#pragma unroll
                for (int i = 0; i < KH; i += 4) {
                    if constexpr (PT) {
                        const float4 f = *reinterpret_cast<const float4*>(scl + 256 + i);
                        mx[0] = fmaxf(mx[0], fmaf(s[i], rf, f.x));
                        mx[1] = fmaxf(mx[1], fmaf(s[i + 1], rf, f.y));
                        mx[2] = fmaxf(mx[2], fmaf(s[i + 2], rf, f.z));
                        mx[3] = fmaxf(mx[3], fmaf(s[i + 3], rf, f.w));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[i + k]);
                    }
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if constexpr (!PT) top *= rf;                // (the factor is positive)
                float* both = maxima + (j & 1) * 2 * kRows;
                both[kh * kRows + r] = top;
                if (!meet()) {
                    ok = false;
                    break;
                }
                top = fmaxf(top, both[(kh ^ 1) * kRows + r]);
                float alpha = 1.f;
                if (top > m + kLazy) {                       // the same in both halves
                    alpha = ex2(m - top);
                    m = top;
                    l *= alpha;
                }
                // ---- weights
                uint32_t hi[KH / 2], lo[BF16 ? KH / 2 : 1];
                float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KH; i += 4) {
                    float w[4];
                    float4 f = make_float4(C::kLift, C::kLift, C::kLift, C::kLift);
                    if constexpr (PT) f = *reinterpret_cast<const float4*>(scl + 128 + i);
                    const float fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float e = ex2(fmaf(s[i + k], rf, -m));
                        l4[k] += e;
                        w[k] = BF16 ? e : e * fv[k];
                    }
                    if constexpr (BF16) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            hi[i / 2 + k] = pack_bf16x2(w[2 * k], w[2 * k + 1]);
                            const float2 x = unpack_bf16x2(hi[i / 2 + k]);
                            lo[i / 2 + k] = pack_bf16x2(w[2 * k] - x.x, w[2 * k + 1] - x.y);
                        }
                    } else {
                        hi[i / 2] = pack_f16x2(w[0], w[1]);
                        hi[i / 2 + 1] = pack_f16x2(w[2], w[3]);
                    }
                }
                l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
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
                    for (int c = 0; c < D / 64; ++c) {       // this half's columns of O
                        uint32_t x[32];
                        const uint32_t at = tmem + lanes + C::kOCol + kh * (D / 2) + c * 32;
                        tmem_ld32(at, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * alpha);
                        tmem_st32(at, x);
                    }
                }
                const uint32_t pcol = tmem + lanes + C::kPCol + kh * (KH / 2);
                tmem_st_n<KH / 2>(pcol, hi);
                if constexpr (BF16) tmem_st_n<KH / 2>(pcol + KEYS / 2, lo);
                tmem_wait_st();
                tc_fence_before();
                arrive(kPFull);
            }
            if (!ok) break;
            // ---- the piece's partial: O, m and l of its rows
            if (!wait(kPvDone, j_end - 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (act) {
                maxima[(j_end & 1) * 2 * kRows + kh * kRows + r] = l;
                if (!meet()) {
                    ok = false;
                    break;
                }
                l += maxima[(j_end & 1) * 2 * kRows + (kh ^ 1) * kRows + r];
                const int64_t at = (static_cast<int64_t>(h) * R + row0 + r) * p.splits +
                                   (static_cast<int64_t>(blockIdx.x) - shares.first(u));
                float f = 1.f / C::kLift;
                if constexpr (!BF16 && !PT)
                    f *= p.v_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                float* dst = p.part_o + at * D + kh * (D / 2);
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tmem + lanes + C::kOCol + kh * (D / 2) + c * 32, x);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(dst + c * 32 + i) = make_float4(
                                __uint_as_float(x[i]) * f, __uint_as_float(x[i + 1]) * f,
                                __uint_as_float(x[i + 2]) * f, __uint_as_float(x[i + 3]) * f);
                    }
                }
                if (row_ok && kh == 0) {
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
cudaError_t launch_one(const PrefixAttnParams& p, cudaStream_t stream) {
    using C = Cfg<D, BF16>;
    static unsigned long long done[64] = {};
    const void* fn = reinterpret_cast<const void*>(prefix_attn_kernel<D, BF16, PT>);
    const cudaError_t e = opt_in_smem(fn, C::kSmem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, p.workers, kThreads, C::kSmem, stream);
    return cudaLaunchKernelEx(&cfg, prefix_attn_kernel<D, BF16, PT>, p);
}

template <int D>
cudaError_t launch_d(const PrefixAttnParams& p, int kv_dtype, cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16) return launch_one<D, true, false>(p, stream);
    if (p.scale_mode == FP8KV_SCALE_PER_TOKEN_HEAD) return launch_one<D, false, true>(p, stream);
    return launch_one<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixAttnParams& p, int D, int kv_dtype,
                               cudaStream_t stream) {
    if (D == 64) return launch_d<64>(p, kv_dtype, stream);
    if (D == 128) return launch_d<128>(p, kv_dtype, stream);
    return launch_d<256>(p, kv_dtype, stream);
}

}  // namespace fp8kv
