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
// tensor pipe), the tensor pipe and the softmax beyond.  Reached: about 3000 clocks a tile of
// D 128 with per-token scales (the softmax: 5000 clocks a tile in each of its two groups, most
// of them waits for tensor memory; 47 % of the issue slots), 2200 of bf16 at D 64.  With the tails:
// 32 sequences x 8 KV heads x 4 query heads, 32768 tokens, D 128: 48.6 us; 100 x 8 x 8, 8197
// tokens, D 64, bf16: 51.5 us.  (The softmax in single values instead of pairs: 49.7 and 53.0.)
// Split: tiles of 128 rows x 128 keys (D 256: 64 keys).  The (head, row tile, key tile)
// units of the call, flattened in that order, are dealt in equal consecutive shares to one
// persistent CTA per SM; a share that crosses a row tile goes on with the next one's queries.
// A row tile's pieces go to slots of their own in the workspace.
//
// Warps of a CTA: two groups of 8 for the softmax, which take the tiles in turn, one that
// issues each product's MMAs, one that brings K (e4m3: and V) by TMA, one for scales and masks,
// 4 for V tiles.
//   * e4m3: S = Q K^T is an e4m3 MMA straight on the cached codes, q in two e4m3 terms under a
//     power of two per row (bf16's 8 bits; exact down to 2^-9 of the row's largest value,
//     beyond that to 2^-17 of it).  V's codes become f16 (exactly) on their way from where
//     bulk copies leave them into swizzled tiles, and the weights are one f16 term: rounded
//     to 2^-11 of a weight, lifted so that weights down to 2^-21 of the largest stay normal
//     (2^-13 beside per-token value scales, below).  The row's sum is of the weights before
//     that.  (Two f16 terms: load 54.9 us instead of 48.7, few 12.8 instead of 11.9; with one
//     scale, the sum of the rounded weights: few 12.5.  A bf16 result drops those bits.)
//   * bf16: q, keys and values as they are; the weights are two bf16 terms (2^-16).
//   * the weights go to tensor memory and are the second product's A operand from there.
//   * per-token V scales as in list_attn.cu: the reference m follows z + log2 s_v, so the
//     weights p s_v stay within f16 whatever the scales are.
//   * three tiles are in tensor memory: one in each group's hands, and the next one's S.
//   * references move only when a tile exceeds them by 2^8; O is rescaled in tensor memory.
//   * both groups follow the references from the tiles' maxima, so that neither waits for the
//     other's (handed over by barriers instead, with V brought by the K warp and maxima by
//     instructions: 50.1 and 58.1 us).
#include <cuda_runtime.h>
#include <math_constants.h>

#include "common.cuh"
#include "internal.h"
#include "prefix.cuh"
#include "tc.cuh"

namespace fp8kv {

namespace {

constexpr int kRows = kPrefixRows;           // query rows of a tile (MMA M)
constexpr float kMaxInit = -1.0e30f;
constexpr float kLazy = 8.f;                 // binades a logit may pass the reference
constexpr int kBuf = 3;                      // tiles in tensor memory
constexpr int kScl = kBuf + 1;               // slots of the tiles' scales and masks

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
    static constexpr int kPart = kKeys / 2;                   // keys of a softmax thread
    static constexpr int kPTerms = BF16 ? 2 : 1;
    static constexpr float kLiftLog2 = BF16 ? 0.f : 7.f;      // w <= 2^8: below f16's 2^16
    static constexpr float kLift = BF16 ? 1.f : 128.f;
    // stages: K tiles, V tiles in 16 bits, e4m3 V tiles as cached
    static constexpr int kKS = BF16 ? (D == 64 ? 3 : 2) : 3;
    static constexpr int kVS = BF16 ? (D == 256 ? 2 : 3) : 2;
    static constexpr int kRS = BF16 ? kVS : (D == 256 ? 2 : 3);
    // tensor memory: three tiles' S, each giving way to its weights (32 keys' columns hold 16 of
    // their first terms and 16 of their second ones), and O
    static constexpr uint32_t kOCol = kBuf * kKeys;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kOCol + D <= kTmemCols, "tensor memory");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kQTerms * kQB;
    static constexpr int kOffV = kOffK + kKS * kRawB;
    static constexpr int kOffRaw = kOffV + kVS * kTileB;      // (bf16: V arrives in place)
    // per tile: key factors, value factors, log2 of the value scales, which keys are there
    static constexpr int kOffScl = kOffRaw + (BF16 ? 0 : kRS * kRawB);
    static constexpr int kOffMask = kOffScl + (BF16 ? 0 : kScl * 3 * 128 * 4);
    static constexpr int kOffLv = kOffMask + kScl * 16;    // largest log2 s_v, or NaN (below)
    static constexpr int kOffPages = kOffLv + 16;             // which pages a V tile got (e4m3)
    static constexpr int kOffTop = kOffPages + 16;               // [2][groups][2 parts][128 rows]
    static constexpr int kOffRow = kOffTop + 8 * 128 * 4;     // [4 threads of a row][128]
    static constexpr int kOffBar = kOffRow + 4 * 128 * 4;
    static constexpr int kSmem = kOffBar + 64 * 8 + 1024;
    static_assert(kSmem <= 227 * 1024 - 64, "shared memory");
};

// Two groups of 8 softmax warps take the tiles in turn; then a warp that issues the first
// product's MMAs and one for the second's, one for K tiles, one for scales and masks, 4 for V tiles.
constexpr int kGroupWarps = 8;
constexpr int kSoftWarps = 2 * kGroupWarps;
constexpr int kQkWarp = kSoftWarps;
constexpr int kPvWarp = kSoftWarps + 1;
constexpr int kTmaWarp = kSoftWarps + 2;
constexpr int kSclWarp = kSoftWarps + 3;
constexpr int kVWarp = kSoftWarps + 4;
constexpr int kThreads = (kVWarp + 4) * 32;

enum { kKFull = 0, kKEmpty = 3, kRawFull = 6, kRawEmpty = 9, kVFull = 12, kVEmpty = 15, kSFull = 18,
       kPFull = 21, kPvDone = 24, kQFull = 27, kPieceDone, kIdle, kPair = kIdle + 2,
       kRow = kPair + 16, kBars = kRow + 4 };
static_assert(kBars <= 64, "barriers");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// MMAs whose descriptors differ from a base by a constant number of 16-byte units: one
// addition to a descriptor's low word, so that the issuing thread keeps ahead of the pipe (built
// anew from its address, a descriptor costs the thread more time than the MMA takes).
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t bytes) {
    return (base & 0xffffffff00000000ull) | (static_cast<uint32_t>(base) + (bytes >> 4));
}
template <bool F16, bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    if constexpr (F16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %4, 1;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %4, 1;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
            : "memory");
}
// A from tensor memory (16-bit pairs a column), B from shared memory; f16 or bf16.
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %4, 1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

// Two fp32 values -> their e4m3 codes and the codes of what those miss.
__device__ __forceinline__ void e4m3_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = e4m3x2_from_f32(a, b);
    const float2 h = unpack_f16x2(f16x2_from_e4m3x2(hi));
    lo = e4m3x2_from_f32(a - h.x, b - h.y);
}

// Two products at once.
__device__ __forceinline__ void times(uint32_t& a, uint32_t& b, uint64_t f) {
    const float2 x = unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(a), __uint_as_float(b)), f));
    a = __float_as_uint(x.x);
    b = __float_as_uint(x.y);
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

    // entry of the page table for page i of a key tile (-1: no such page), and whether it is a
    // block: looked at only when it is used, so that nothing waits for it before
    auto fetch = [&](int tile, int i) -> int {
        const int page = tile * C::kPages + i;
        if (i >= C::kPages || page >= (len + kPage - 1) / kPage) return -1;
        return p.prefix_table[page];
    };
    auto is_block = [&](int id, int tile, int i) {
        const bool ok = id >= 0 && id < p.num_blocks;
        if (!ok && i < C::kPages && tile * C::kPages + i < (len + kPage - 1) / kPage)
            report(p.err, FP8KV_ERR_BAD_INDEX);
        return ok;
    };
    Walk at(w0, T, p.row_tiles);
    // what the first tiles wait for is on its way while the CTA sets up
    int id = -1;
    if (warp >= kTmaWarp) {
        id = fetch(at.tile, lane >> (warp == kSclWarp ? 2 : 0));
    } else if (warp < kSoftWarps) {
        const int64_t row = static_cast<int64_t>(at.row_tile) * kRows + 32 * (warp & 3) + lane;
        if (row < R)
            prefetch_l2(p.q + (row / p.G * p.Hq + at.head * p.G + row % p.G) * D + (warp >> 2) * (D / 4));
    }
    if (warp == kQkWarp) tmem_alloc(smem_addr(&s_tmem), C::kTmemCols);
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar(kKFull + i), 1);
            mbar_init(bar(kKEmpty + i), 1);
            mbar_init(bar(kRawFull + i), BF16 ? 4 : 1);
            mbar_init(bar(kRawEmpty + i), 4);
            mbar_init(bar(kVFull + i), 4);
            mbar_init(bar(kVEmpty + i), 1);
        }
        for (int i = 0; i < kBuf; ++i) {
            mbar_init(bar(kSFull + i), 2);                   // the product, scales and masks
            mbar_init(bar(kPFull + i), kGroupWarps);
            mbar_init(bar(kPvDone + i), 1);
        }
        mbar_init(bar(kQFull), kSoftWarps);
        mbar_init(bar(kPieceDone), 1);
        mbar_init(bar(kIdle), 1);
        mbar_init(bar(kIdle + 1), 1);
        for (int i = 0; i < 16; ++i) mbar_init(bar(kPair + i), 2);
        for (int i = 0; i < 4; ++i) mbar_init(bar(kRow + i), 4);
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // a warp's wait for a phase, and its arrival
    auto wait = [&](int i, int phase) {
        return __all_sync(0xffffffffu, wait_or_abort(bar(i), phase & 1, abort, p.err));
    };
    auto arrive = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    if (warp >= kVWarp) {
        // =============================== V tiles for the second product.  bf16: each warp brings a
        // quarter of a tile's pages (issuing a copy takes a warp about 100 clocks, so that one
        // warp for K and V was what the tiles waited for); e4m3: each turns a quarter of its
        // codes into f16, and the warp that brings K brings them too
        const int lt = tid - kVWarp * 32, vw = warp - kVWarp;
        constexpr int kMine = C::kPages / 4;
        if (BF16 && lt == 0) prefetch_tmap(&vmap);
        Walk ahead = at;
        int issued = 0;
        // tile `issued` on its way; `here`: the pages it has
        auto issue = [&](uint32_t& here) {
            here = 0u;
            if (!BF16 || issued >= n) return true;
            const int st = issued % C::kRS, h = ahead.head;
            const bool have = is_block(id, ahead.tile, lane);
            const int64_t tile = static_cast<int64_t>(id) * p.Hkv + h;
            ahead.next();
            id = issued + 1 < n ? fetch(ahead.tile, lane) : -1;
            here = __ballot_sync(0xffffffffu, have);
            if (issued >= C::kRS && !wait(kVEmpty + st, issued / C::kRS - 1)) return false;
            const uint32_t mine = here & (((1u << kMine) - 1u) << (vw * kMine));
            if (lane == 0)
                mbar_arrive_expect_tx(bar(kRawFull + st), __popc(mine) * (kPage * C::kRowB));
            __syncwarp();
            if ((mine >> lane) & 1u)
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_3d(sbase + C::kOffV + st * C::kTileB + pn * (KEYS * 128) +
                                    lane * (kPage * 128),
                                &vmap, pn * 128, 0, static_cast<int>(tile), bar(kRawFull + st));
            ++issued;
            return true;
        };
        // tiles on their way while one is worked on: a stage is free only when the product
        // has run, which must not hold up the next tile's hand-over
        constexpr int kAhead = C::kRS - 1;
        uint32_t queue[kAhead];
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ok = ok && issue(queue[i]);
        for (int j = 0; j < n && ok; ++j, at.next()) {
            const int rs = j % C::kRS, st = j % C::kVS;
            const int left = len - at.tile * KEYS;           // keys of the tile that exist
            if (!wait(kRawFull + rs, j / C::kRS)) break;
            const uint32_t pages =
                BF16 ? queue[0] : reinterpret_cast<const uint32_t*>(smem + C::kOffPages)[rs];
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
                constexpr int kChunks = C::kRowB / 16, kLoads = KEYS * kChunks / 128;
                // every load goes before the first store, which it cannot be told apart from
                uint4 codes[kLoads];
#pragma unroll
                for (int k = 0; k < kLoads; ++k)
                    codes[k] = *reinterpret_cast<const uint4*>(raw + (k * 128 + lt) * 16);
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int q = k * 128 + lt, row = q / kChunks, c = q % kChunks;
                    uint4 x = codes[k];
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
#pragma unroll
            for (int i = 0; i + 1 < kAhead; ++i) queue[i] = queue[i + 1];
            ok = issue(queue[kAhead - 1]);
        }
        // an abort: the copies in flight land before the CTA leaves (bounded waits)
        if (BF16 && *abort)
            for (int j = max(0, issued - C::kRS); j < issued; ++j)
                (void)mbar_wait_bounded(bar(kRawFull + j % C::kRS), (j / C::kRS) & 1);
    } else if (warp == kSclWarp) {
        // =============================== scales and masks, four keys a lane
        const bool mine = lane < KEYS / 4;                   // (fetch: -1 from there on)
        int loaded = 0;
        // loads tile `at`'s, and the block ids of the one behind it
        auto load = [&](float4& ks, float4& vs, int& valid) {
            valid = is_block(id, at.tile, lane / 4) ? min(4, max(0, len - at.tile * KEYS - 4 * lane)) : 0;
            if (PT && valid > 0) {
                const int64_t row = (static_cast<int64_t>(id) * p.Hkv + at.head) * kPage + (lane & 3) * 4;
                ks = *reinterpret_cast<const float4*>(p.k_scale_cache + row);
                vs = *reinterpret_cast<const float4*>(p.v_scale_cache + row);
            }
            at.next();
            id = ++loaded < n ? fetch(at.tile, lane / 4) : -1;
        };
        float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
        int valid = 0;
        load(ks, vs, valid);
        // tile j's are there when its turn comes, and handed over once the tile before it in
        // tensor memory has its weights, which also frees the slot of tile j + 1's
        for (int j = -1; j < n; ++j) {
            if (j >= kBuf && !wait(kPFull + j % kBuf, j / kBuf - 1)) break;
            if (j >= 0) arrive(kSFull + j % kBuf);
            if (j + 1 == n) break;
            float4 ks1 = ks, vs1 = vs;
            int valid1 = 0;
            if (j + 2 < n) load(ks1, vs1, valid1);
            const int sl = (j + 1) % kScl;
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
            if constexpr (PT) {
                // value scales within 8 binades of each other: the largest one alone stands
                // for them in the reference (weights then peak at 2^-8 and more, still 13
                // binades above f16's subnormal ones); else NaN, and every key's own counts
                float top = -CUDART_INF_F, low = CUDART_INF_F;
                const float vv[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < valid) {
                        const float g = fmaxf(__log2f(fabsf(vv[i])), -100.f);
                        top = fmaxf(top, g);
                        low = fminf(low, g);
                    }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
                }
                if (lane == 0)
                    reinterpret_cast<float*>(smem + C::kOffLv)[sl] =
                        top - low <= 8.f ? top : CUDART_NAN_F;
            }
            ks = ks1;
            vs = vs1;
            valid = valid1;
        }
    } else if (warp == kTmaWarp) {
        // =============================== K tiles (tensor copies), e4m3: V tiles as cached; a lane
        // per page
        if (lane == 0) prefetch_tmap(&kmap);
        int issued = 0, v_issued = 0;
        for (int j = 0; j < n; ++j) {
            const int h = at.head;
            const bool mine = is_block(id, at.tile, lane);
            at.next();
            const int id_next = j + 1 < n ? fetch(at.tile, lane) : -1;
            const uint32_t here = __ballot_sync(0xffffffffu, mine);
            const int ks = j % C::kKS;
            const int64_t tile = static_cast<int64_t>(id) * p.Hkv + h;
            if (j >= C::kKS && !wait(kKEmpty + ks, (j - C::kKS) / C::kKS)) break;
            if (lane == 0)
                mbar_arrive_expect_tx(bar(kKFull + ks), __popc(here) * (kPage * C::kRowB));
            __syncwarp();
            if (mine)
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_3d(sbase + C::kOffK + ks * C::kRawB + pn * (KEYS * C::kPanelB) +
                                    lane * (kPage * C::kPanelB),
                                &kmap, pn * C::kPanelB, 0, static_cast<int>(tile), bar(kKFull + ks));
            ++issued;
            if constexpr (!BF16) {
                const int rs = j % C::kRS;
                if (j >= C::kRS && !wait(kRawEmpty + rs, (j - C::kRS) / C::kRS)) break;
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(smem + C::kOffPages)[rs] = here;
                    mbar_arrive_expect_tx(bar(kRawFull + rs), __popc(here) * (kPage * C::kRowB));
                }
                __syncwarp();
                if (mine)
                    bulk_load(sbase + C::kOffRaw + rs * C::kRawB + lane * (kPage * C::kRowB),
                              p.v_cache + tile * (kPage * C::kRowB), kPage * C::kRowB,
                              bar(kRawFull + rs));
                ++v_issued;
            }
            id = id_next;
        }
        // an abort: the copies in flight land before the CTA leaves (bounded waits)
        if (*abort) {
            for (int j = max(0, issued - C::kKS); j < issued; ++j)
                (void)mbar_wait_bounded(bar(kKFull + j % C::kKS), (j / C::kKS) & 1);
            for (int j = max(0, v_issued - C::kRS); j < v_issued; ++j)
                (void)mbar_wait_bounded(bar(kRawFull + j % C::kRS), (j / C::kRS) & 1);
        }
    } else if (warp == kQkWarp) {
        // =============================== MMAs of S = Q K^T.  An elected lane of the converged
        // warp issues them (from a branch that one lane takes, the same MMAs take the pipe half
        // as long again), a warp for each product: one for both spends more time on issuing
        // and waiting than the tensor pipe needs
        constexpr uint32_t kFmt = BF16 ? 1u : 0u;            // bf16; e4m3
        constexpr uint32_t idesc = instr_desc(kFmt, kFmt, 0, 0, KEYS, kRows);
        const uint64_t q0 = smem_desc(sbase + C::kOffQ, 16, 8 * C::kPanelB, C::kLayout);
        const uint64_t k0 = smem_desc(sbase + C::kOffK, 16, 8 * C::kPanelB, C::kLayout);
        int piece = 0;
        for (int j = 0; j < n; ++j, at.next()) {
            // a row tile's queries; S of tile j replaces the weights of tile j - 3
            if ((j == 0 || at.tile == 0) && !wait(kQFull, piece++)) break;
            if (!wait(kKFull + j % C::kKS, j / C::kKS)) break;
            if (j >= kBuf && !wait(kPvDone + j % kBuf, j / kBuf - 1)) break;
            tc_fence_after();
            const uint64_t k = desc_at(k0, (j % C::kKS) * C::kRawB);
            const uint32_t d = tmem + (j % kBuf) * KEYS;
            constexpr int kPer = C::kPanelB / 32;            // 32-byte steps of a panel
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < C::kRowB / 32; ++s) {
                    const uint64_t b = desc_at(k, (s / kPer) * (KEYS * C::kPanelB) + (s % kPer) * 32);
#pragma unroll
                    for (int term = 0; term < C::kQTerms; ++term) {
                        const uint64_t a = desc_at(q0, term * C::kQB + (s / kPer) * (kRows * C::kPanelB) +
                                                           (s % kPer) * 32);
                        if (s == 0 && term == 0)
                            mma_ss<BF16, false>(d, a, b, idesc);
                        else
                            mma_ss<BF16, true>(d, a, b, idesc);
                    }
                }
                mma_commit(bar(kSFull + j % kBuf));
                mma_commit(bar(kKEmpty + j % C::kKS));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(kIdle));             // every MMA issued has ended
        __syncwarp();
        (void)mbar_wait_bounded(bar(kIdle), 0);
    } else if (warp == kPvWarp) {
        // =============================== MMAs of O += P V
        constexpr uint32_t kFmt = BF16 ? 1u : 0u;            // bf16; f16
        constexpr uint32_t idesc = instr_desc(kFmt, kFmt, 0, 1, D, kRows);
        // V is MN-major: 8-key groups 1024 bytes apart, panels of 64 channels KEYS rows apart
        const uint64_t v0 = smem_desc_sw128(sbase + C::kOffV, KEYS * 128, 1024);
        for (int j = 0; j < n; ++j) {
            const bool first = j == 0 || at.tile == 0;
            at.next();
            if (!wait(kVFull + j % C::kVS, j / C::kVS) || !wait(kPFull + j % kBuf, j / kBuf)) break;
            tc_fence_after();
            const uint64_t v = desc_at(v0, (j % C::kVS) * C::kTileB);
            const uint32_t a0 = tmem + (j % kBuf) * KEYS, d = tmem + C::kOCol;
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < KEYS / 16; ++s) {        // 16 keys a step
                    const uint64_t b = desc_at(v, s * 16 * 128);
                    const uint32_t a = a0 + (s / 2) * 32 + (s % 2) * 8;
                    if (s == 0 && first)
                        mma_ts<false>(d, a, b, idesc);
                    else
                        mma_ts<true>(d, a, b, idesc);
                    if constexpr (C::kPTerms == 2) mma_ts<true>(d, a + 16, b, idesc);
                }
                mma_commit(bar(kPvDone + j % kBuf));
                mma_commit(bar(kVEmpty + j % C::kVS));
                if (j + 1 == n || at.tile == 0) mma_commit(bar(kPieceDone));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(kIdle + 1));
        __syncwarp();
        (void)mbar_wait_bounded(bar(kIdle + 1), 0);
    } else {
        // =============================== softmax, partials
        // Group j % 2 takes tile j: while one turns logits into weights, the other finds its
        // tile's maxima, so that the tensor pipe always has a product to run.
        const int quarter = warp & 3, part = (warp >> 2) & 1, group = warp >> 3;
        const int fourth = warp >> 2;                        // which of a row's four threads
        const int r = 32 * quarter + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
        float* const rows4 = reinterpret_cast<float*>(smem + C::kOffRow) + r;
        constexpr int KP = C::kPart;                         // keys of this thread
        constexpr int DP = D / 4;                            // its channels of Q and of a partial
        constexpr int DC = DP < 32 ? DP : 32;                // columns of one O load
        int row_phase = 0, piece = 0;
        bool ok = true;
        // x of the row's four threads to all of them
        auto share = [&](float x) {
            rows4[fourth * kRows] = x;
            arrive(kRow + quarter);
            return wait(kRow + quarter, row_phase++);
        };
        for (int j = 0; j < n && ok; ++piece) {
            const int h = at.head;
            const int64_t row0 = static_cast<int64_t>(at.row_tile) * kRows;
            const int j_end = min(n, j + T - at.tile);
            const bool starts = at.tile == 0;                // the row tile's first piece
            // a warp whose rows all lie behind the last one only keeps step
            const bool act = row0 + 32 * quarter < R;
            const bool row_ok = row0 + r < R;
            // ---- the row tile's queries
            float rf = p.scale_log2;                         // raw S (PT: column-scaled) -> logit
            if (act) {
                const int64_t row = row0 + r;
                const int64_t b = row_ok ? row / p.G : 0;
                const int g = row_ok ? static_cast<int>(row - b * p.G) : 0;
                const __nv_bfloat16* q = p.q + (b * p.Hq + h * p.G + g) * D + fourth * DP;
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
                    for (int c = 0; c < DP / 8; ++c) *chunk(0, fourth * (DP / 8) + c) = x[c];
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
                    if (!share(amax)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) amax = fmaxf(amax, rows4[i * kRows]);
                    // the power of two that puts max |q| into [2^7, 2^8)
                    int e = 0;
                    if (amax > 0.f && amax <= 3.4e38f) {
                        frexpf(amax, &e);
                        e = min(126, max(-126, 8 - e));
                    }
                    float up = ldexpf(1.f, e);
                    // (an infinite query, which e4m3 cannot hold, has no finite result)
                    rf = amax <= 3.4e38f ? ldexpf(1.f, -e) : CUDART_NAN_F;
                    if constexpr (!PT) {
                        rf *= p.scale_log2 * p.k_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                        // The factor stays above zero, so that the largest S is the largest
                        // logit and a masked -inf stays one: the sign of a key scale goes to
                        // the query's terms, and where the factor is zero (a zero scale, or a
                        // product below fp32) the terms are, so that every logit is.
                        if (rf < 0.f) {
                            rf = -rf;
                            up = -up;
                        } else if (rf == 0.f) {
                            rf = 1.f;
                            up = 0.f;
                        }
                    }
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
                        const int cc = fourth * (DP / 16) + c;
                        *chunk(0, cc) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *chunk(1, cc) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            fence_proxy_async();
            arrive(kQFull);

            float m = kMaxInit, l = 0.f;                     // l: times the lift if not PT
            const int j0 = j;
            // The row's reference behind tile t of the other group, whose maxima both groups see:
            // every thread follows it from maximum to maximum, so that no group waits for
            // what the other makes of them.
            auto tops_of = [&](int t) {
                return reinterpret_cast<float*>(smem + C::kOffTop) +
                       (t & 3) * 2 * kRows + r;
            };
            // Their barriers and places alternate too: tile t + 4's maxima need tile t + 1's
            // weights, before which their group has seen tile t's.
            auto pair = [&](int t) { return kPair + (t & 3) * 4 + quarter; };
            auto behind = [&](int t, float& ref) {
                if (!wait(pair(t), t >> 2)) return false;
                const float top = fmaxf(tops_of(t)[0], tops_of(t)[kRows]);
                ref = top > m + kLazy ? top : m;
                return true;
            };
            for (j += (j & 1) != group; j < j_end; j += 2) {
                const int buf = j % kBuf;
                if (!wait(kSFull + buf, j / kBuf)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!act) {
                    if (lane == 0) mbar_arrive(bar(pair(j)));
                    tc_fence_before();
                    arrive(kPFull + buf);
                    continue;
                }
                const float* scl = reinterpret_cast<const float*>(smem + C::kOffScl) + j % kScl * 3 * 128 +
                                   part * KP;
                const uint32_t* bits =
                    reinterpret_cast<const uint32_t*>(smem + C::kOffMask) + j % kScl * 4 + part * (KP / 32);
                const uint32_t scol = tmem + lanes + buf * KEYS + part * KP;
                // ---- logits up to the row's factor (where columns are scaled or masked they go
                //      back to tensor memory), and the row's largest (with log2 s_v)
                float lv = 0.f, top = -CUDART_INF_F;
                if constexpr (PT) lv = reinterpret_cast<const float*>(smem + C::kOffLv)[j % kScl];
                uint32_t all = 0xffffffffu;
#pragma unroll
                for (int c = 0; c < KP / 32; ++c) all &= bits[c];
                if (!PT && all == 0xffffffffu) {
                    float mx = -CUDART_INF_F;
#pragma unroll
                    for (int c = 0; c < KP / 32; ++c) mx = fmaxf(mx, tmem_max32(scol + c * 32));
                    top = mx * rf;
                } else {
#pragma unroll 1
                    for (int c = 0; c < KP / 32; ++c) {
                        uint32_t s[32];
                        tmem_ld32(scol + c * 32, s);
                        tmem_wait_ld();
                        if constexpr (PT) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scl + c * 32 + i);
                                times(s[i], s[i + 1], f.x);
                                times(s[i + 2], s[i + 3], f.y);
                            }
                        }
                        const uint32_t there = bits[c];
                        if (there != 0xffffffffu) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((there >> i) & 1u)) s[i] = __float_as_uint(-CUDART_INF_F);
                        }
                        tmem_st32(scol + c * 32, s);
                        float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                        if (!PT || lv == lv) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2)
                                mx[(i / 2) & 3] = fmaxf(mx[(i / 2) & 3], fmaxf(__uint_as_float(s[i]),
                                                                               __uint_as_float(s[i + 1])));
                            top = fmaxf(top, fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), rf, lv));
                        } else {                             // value scales far apart
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                mx[i & 3] = fmaxf(mx[i & 3],
                                                  fmaf(__uint_as_float(s[i]), rf, scl[256 + c * 32 + i]));
                            top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                        }
                    }
                }
                tops_of(j)[part * kRows] = top;
                arrive(pair(j));
                // ---- the reference, as the tile before left it, moved if need be
                float before = m;                            // (m: behind this group's last tile)
                if ((j > j0 && !behind(j - 1, before)) || !wait(pair(j), j >> 2)) {
                    ok = false;
                    break;
                }
                top = fmaxf(tops_of(j)[0], tops_of(j)[kRows]);
                const float now = top > before + kLazy ? top : before;   // the same in both parts
                if (now != m) {
                    l *= ex2(m - now);
                    m = now;
                }
                if (j > j0 && __any_sync(0xffffffffu, now != before)) {
                    // O holds the tiles before once PV of the last of them has run
                    if (!wait(kPvDone + (j - 1) % kBuf, (j - 1) / kBuf)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float alpha = ex2(before - now);
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {       // this part's columns
                        uint32_t x[32];
                        const uint32_t o = tmem + lanes + C::kOCol + part * (D / 2) + c * 32;
                        tmem_ld32(o, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * alpha);
                        tmem_st32(o, x);
                    }
                }
                // ---- weights, in their logits' place (not PT: the lift is part of the exponent)
                const float off = PT ? -m : C::kLiftLog2 - m;
                const uint64_t rf2 = pack_f32x2(rf, rf), off2 = pack_f32x2(off, off);
                uint64_t l2[2] = {0ull, 0ull};
                tmem_wait_st();
#pragma unroll 1
                for (int c = 0; c < KP / 32; ++c) {
                    uint32_t s[32], hi[16], lo[16];
                    tmem_ld32(scol + c * 32, s);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float w[4];
                        ulonglong2 f = make_ulonglong2(0ull, 0ull);
                        if constexpr (PT) f = *reinterpret_cast<const ulonglong2*>(scl + 128 + c * 32 + i);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 z = unpack_f32x2(fma_f32x2(
                                pack_f32x2(__uint_as_float(s[i + 2 * k]), __uint_as_float(s[i + 2 * k + 1])),
                                rf2, off2));
                            const uint64_t e = pack_f32x2(ex2(z.x), ex2(z.y));
                            l2[k] = add_f32x2(l2[k], e);
                            const float2 y = unpack_f32x2(PT ? mul_f32x2(e, k ? f.y : f.x) : e);
                            w[2 * k] = y.x;
                            w[2 * k + 1] = y.y;
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if constexpr (BF16) {
                                hi[i / 2 + k] = pack_bf16x2(w[2 * k], w[2 * k + 1]);
                                const float2 y = unpack_bf16x2(hi[i / 2 + k]);
                                lo[i / 2 + k] = pack_bf16x2(w[2 * k] - y.x, w[2 * k + 1] - y.y);
                            } else {
                                hi[i / 2 + k] = pack_f16x2(w[2 * k], w[2 * k + 1]);
                            }
                        }
                    }
                    tmem_st16(scol + c * 32, hi);
                    if constexpr (BF16) tmem_st16(scol + c * 32 + 16, lo);
                }
                const float2 la = unpack_f32x2(l2[0]), lb = unpack_f32x2(l2[1]);
                l += (la.x + la.y) + (lb.x + lb.y);
                tmem_wait_st();
                tc_fence_before();
                arrive(kPFull + buf);
            }
            if (!ok) break;
            j = j_end;
            // ---- the piece's partial: O, m and l of its rows
            if (!wait(kPieceDone, piece)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (act) {
                float last = m;
                if (((j_end - 1) & 1) != group && !behind(j_end - 1, last)) {
                    ok = false;
                    break;
                }
                if (!share(l * ex2(m - last))) {
                    ok = false;
                    break;
                }
                l = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) l += rows4[i * kRows];
                if constexpr (!PT) l *= 1.f / C::kLift;
                // which piece of its row tile
                const int64_t nth =
                    starts ? 0
                           : static_cast<int64_t>(blockIdx.x) -
                                 shares.first(static_cast<int64_t>(h) * p.row_tiles + at.row_tile);
                const int64_t slot = (static_cast<int64_t>(h) * R + row0 + r) * p.splits + nth;
                float f = 1.f / C::kLift;
                if constexpr (!BF16 && !PT)
                    f *= p.v_scale[p.scale_mode == FP8KV_SCALE_PER_HEAD ? h : 0];
                float* dst = p.part_o + slot * D + fourth * DP;
#pragma unroll 1
                for (int c = 0; c < DP / DC; ++c) {
                    uint32_t x[DC];
                    tmem_ld_n<DC>(tmem + lanes + C::kOCol + fourth * DP + c * DC, x);
                    tmem_wait_ld();
                    if (row_ok) {
#pragma unroll
                        for (int i = 0; i < DC; i += 8) {    // whole sectors
                            Bytes32 y;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                y.w[k] = __float_as_uint(__uint_as_float(x[i + k]) * f);
                            store32(dst + c * DC + i, y);
                        }
                    }
                }
                if (row_ok && fourth == 0) {
                    p.part_m[slot] = last;
                    p.part_l[slot] = l;
                }
                // the row's four have read the sums before a next piece's go to their place
                arrive(kRow + quarter);
                if (!wait(kRow + quarter, row_phase++)) {
                    ok = false;
                    break;
                }
            }
            tc_fence_before();
            at.tile = 0;                                     // the next row tile
            if (++at.row_tile == p.row_tiles) {
                at.row_tile = 0;
                ++at.head;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kQkWarp) {
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
