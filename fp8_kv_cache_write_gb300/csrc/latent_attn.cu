// latent_attn.cu -- attention of one (or a few) new tokens over the paged latent
// cache, absorbed form: every head reads the same row x_t = [c_t (L) | k_t (64)] of
// a cached token, as its key (all W = L + 64 values) and, its first L values, as
// its value.
//
//     z_t = softmax_scale * q . x_t,   out = sum_t softmax(z)_t c_t
//
// for every row (query token s, head h) of sequence b over keys
// t <= context_len - S + s.  Because all heads share the row, the S * H query rows
// of a sequence form one matrix and both contractions are matrix products.
//
// Both products run with the CACHE as the M operand (tcgen05, fp32 in TMEM):
//     S^T [keys x rows]  = X [keys x W]  . Q^T          (X K-major)
//     O^T [L x rows]    += C^T [L x keys] . P^T         (C MN-major, the same bytes)
// so a tile of keys is staged once by TMA, straight from the pages, and serves both;
// the row count is the N of the instruction (16, 32 or 64: no padding to 128 rows
// for few heads), and O^T for 64 rows and L = 512 takes 4 x 64 columns of tensor
// memory instead of all 512.  The price is that the softmax's keys lie across TMEM
// lanes: a thread owns one key, and a row's maximum is a reduction over 128 threads.
// It is taken only when a vote says that some column's reference has to move, and the
// row sums stay per thread until the end.
//
// e4m3 cache: codes enter the tensor core as they are.  Q (bf16) is taken as two
// e4m3 terms after an exact power-of-two scaling per row: hi has bf16's first 4
// significant bits, lo the other 4, so the pair is bf16's value exactly down to
// 2^-17 of the row's largest.  The terms are extra ROWS of the N operand (2N <= 128
// columns, added by the softmax), which costs less than a second pass over the
// keys.  P is two terms too, two k-steps into the same accumulator: e4m3 (4 significant
// bits) and, of what that misses, e5m2 (3 more: 2^-8 of the weight, as a second e4m3
// term's worst case is 2^-9, but down to 2^-17 where that ends at 2^-10, so that many
// weak keys beside a strong one keep their share: with two e4m3 terms a quarter of a
// row's mass could be lost).  A third term would not fit beside 64 rows of Q.  bf16
// cache: bf16 Q, P as two bf16 terms (2^-16 of a weight), 64-key tiles of the same size
// in bytes.  Up to 32 rows the terms are columns of one product, whose results are added
// at the end; 64 rows take a second run of k-steps, and the second terms lie in the
// tile's own rotary panel, which only S reads.
//
// Per-token scales s_t (e4m3): the logit takes s_t, and the weight of a CODE is
// p_t s_t = 2^(z_t + log2 s_t - m): the running reference m is of that sum, so the
// weights stay in e4m3's range whatever the scales, and the row sum adds the weight
// divided by s_t again.  A row whose scale is below 2^-100 (a row of zeros has 0) is all
// zeros as a value; its weight is that of a scale of 2^-40, which leaves the reference to
// the rows that count and the sum in fp32's range.
//
// Split: workers of `groups` CTAs (one per group of at most 64 rows) take consecutive
// shares of all (sequence, key tile) pairs; a sequence cut between workers leaves fp32
// partials (O, m, l) that a second kernel joins.  The groups of a worker read the same
// tiles at about the same time, so the second read hits L2.
//
// Roles of a CTA (one per SM): 8 softmax warps, 2 that issue the tensor copies, one that
// issues the MMAs.  Two stages of a tile's rows alternate; S of a tile runs while the
// softmax works on the one before.
//
// What bounds it.  Few rows (N 16, 32): HBM; a 72 KiB tile takes 3150 to 3400 cycles of
// the 3140 that the copy rate allows.  64 rows: a cycle of latencies, not the pipe (31 %
// active): the MMAs of a 128-key tile take 1220 (S) + 1800 (PV) cycles, its period without
// a move is 4100, because a stage is refilled only after its PV (1800 cycles until the rows
// are there) and the softmax (1700) stands between S and PV; a third stage does not fit
// beside Q.  A move of a reference adds 1600.  Around the loop every call pays some 9000
// cycles until the first S (queries, first tile), 7000 to write 64 rows out, and the merge
// (7 to 8 us, where sequences are cut).
// Measured (8 x 18k-22k keys, us a call): e4m3 with per-token scales, 128 heads 71 (625
// TFLOP/s), 64: 51, 32: 42, 16: 33; with one scale, 128 heads: 67; bf16, 128 heads 97,
// 64: 63, 32: 52, 16: 48; 32 x 1k-32k keys, 2 x 16 rows, bf16: 81 (4.3 TB/s).
// Tried and dropped (each against the kernel of its time): S chunk by chunk as its copies
// land (the pipe idles between short runs: 84 against 72 us), 16-byte lane copies instead
// of tensor copies (no change), PV in two runs with S between (72 against 68 us), three
// copying warps (no change), a merge of 512 threads a row (13 -> 29 us), bf16 in groups of
// 32 rows at most with 64 and 128 heads (70 and 117 us against 63 and 97).
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace fp8kv {

namespace {

constexpr int kRope = kLatentRope;
constexpr int kParts = 2;                    // softmax warps per TMEM lane quarter: a key's
                                             // columns in two halves
constexpr int kSoftWarps = 4 * kParts;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kLoadWarps = 2;                // each issues half of every tile's pages
constexpr int kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kRopeSlotBytes = 8192;         // e4m3: the shared keys of a tile
constexpr int kMiscBytes = 3 * 1024;
constexpr int kSmemLimit = 227 * 1024;
constexpr uint32_t kTmemAll = 512;
constexpr uint32_t kSCol = 256;              // S^T buffers from here, O^T from column 0
constexpr float kMinScale = 0x1p-100f, kZeroRowScale = 0x1p-40f;
// A column's reference goes down to this far below its highest, its floor: a tile that
// lies deeper moves it there and no further, and a tile behind it that weighs more moves
// it up again.  Keys under what the floor resolves weigh less than 2^-54 of the largest.
// The sums then hold up to 2^40 times larger values: weights up to 2^8.5 over the smallest
// scale so far, of 2^24 keys, stay in fp32's range with kSumRoom + log2(scale) binades to
// go down, so rows with scales below 2^-54 leave less.
constexpr float kDeepest = 40.f, kSumRoom = 94.f;

template <int N, bool BF16>
struct Cfg {
    static constexpr int kElem = BF16 ? 2 : 1;
    static constexpr int kKeys = BF16 ? 64 : 128;        // keys of a tile
    static constexpr int kPages = kKeys / kPage;
    static constexpr int kQRows = BF16 ? N : 2 * N;      // columns of an S^T buffer
    // bf16: the second terms of the weights are columns of their own
    static constexpr bool kPairs = BF16 && N <= 32;
    static constexpr int kOCols = kPairs ? 2 * N : N;    // columns of a chunk of O^T
    static constexpr int kQBytes = kQRows * (512 + kRope) * kElem;
    // P^T, MN-major: a row of 64 values per key, of which the first kOCols are used
    static constexpr int kPRow = 64 * kElem;
    static constexpr int kPTerm = kKeys * kPRow;
    static constexpr int kPBytes = BF16 ? kPTerm : 2 * kPTerm;
    // two stages of a tile's rows, in groups of 8 keys: [group][128-byte panel][8][128].
    // bf16 rows are whole panels, L / 64 and one of the shared key; e4m3 rows are L / 128
    // panels, and the shared keys (64 bytes) lie apart, [keys][64], in two slots or, with
    // 64 columns, in the one that fits
    static constexpr int kStageBytes = kKeys * (512 + (BF16 ? kRope : 0)) * kElem;
    static constexpr int kRopeSlots =
        BF16 ? 0
        : 2 * kStageBytes + 2 * kRopeSlotBytes + kPBytes + kQBytes + kMiscBytes <= kSmemLimit ? 2
                                                                                             : 1;
    static constexpr int kOffRope = 2 * kStageBytes;
    static constexpr int kOffP = kOffRope + kRopeSlots * kRopeSlotBytes;
    static constexpr int kOffQ = kOffP + kPBytes;
    static constexpr int kOffMisc = kOffQ + kQBytes;
    static constexpr int kSmem = kOffMisc + kMiscBytes;
    // The weights of an e4m3 cache have little range, 448 down to steps of 2^-16 (of the
    // second term), so the reference of a column follows its tiles both ways (O and the
    // sums are rescaled in fp32): a column starts with its first tile's largest weight at
    // 2^kLift; where a weight would pass 2^kLimit (< 448) the tile's largest becomes
    // 2^kHigh, so that ordinary tiles stay in range below an outlier; where a tile's
    // largest falls under 2^kLow (behind a key that dwarfs the others) it becomes 2^kLift,
    // or what it is at the column's floor (kDeepest).
    // kLow is set by what 127 weak keys beside a strong one may lose in all: each is off
    // by 2^-14 at most, together 2^-8 of a largest weight of 2.  A move costs some 1600
    // cycles; 8 x 18k-22k keys, 128 heads, per-token scales: kLow 1: 72 us, 0: 71, -1: 70,
    // -2: 69.  bf16 weights have fp32's range, and only move up.
    static constexpr float kLimit = BF16 ? 8.f : 8.5f;
    static constexpr float kHigh = BF16 ? 0.f : 7.f;
    static constexpr float kLift = BF16 ? 0.f : 4.f;
    static constexpr float kLow = 1.f;
    static_assert(kSmem <= kSmemLimit, "shared memory");
    static_assert(4 * kOCols <= kSCol, "tensor memory of O");
    static_assert(kOCols <= 64, "a row of P");
};

// misc region
struct Misc {
    uint64_t f[32], nm[32];      // pairs of columns: logit factors, running references
                                 // m (negated)
    int last[64];                // last key position the column sees
    float red[4][64];            // per-warp column maxima / sums
    float delta[64], alpha[64];  // a move of the reference: by how much, O's factor
    float top[64];               // the column's highest reference; -inf: it has none yet
    float low[kParts][4];        // per warp: log2 of the smallest scale so far
    uint32_t under[2][kSoftWarps];   // per tile parity and warp: columns all under 2^kLow
    uint32_t quiet[kParts];      // a half's columns that no tile moves down: see the move
    uint64_t full[2], empty[2], rope_empty;
    uint64_t s_full[2], s_empty[2], p_full, pv_done, q_full, idle;
    int64_t first_tile, num_tiles;   // this worker's share, in its first sequence's tiles
    int b0;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc region");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bounded wait that also gives up as soon as another thread raised `abort`.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         int32_t* err) {
    const uint32_t a = smem_addr(bar);
    if (mbar_try_wait(a, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(a, parity)) return true;
        if ((i & 63u) == 0u) {
            if (*abort_flag) return false;
            if (global_ns() - t0 > kWaitBudgetNs) {
                *abort_flag = 1;
                report(err, FP8KV_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// One look at a barrier's phase, without the suspended wait of try_wait.
__device__ __forceinline__ bool test_bar(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Barrier of the softmax warps; true if any thread's predicate holds.  Every
// softmax thread reaches it the same number of times.
__device__ __forceinline__ bool soft_any(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "n"(kSoftThreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Largest of the warp's values (NaN only where all are).
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float warp_min(float x) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// soft_any among the four warps (one a quarter) that hold one half of the columns.
__device__ __forceinline__ bool half_any(int part, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %3, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "n"(kSoftThreads / kParts), "r"(2 + part)
        : "memory");
    return r != 0;
}

// Column reduction over a warp: every lane holds N <= 32 columns of its own key;
// the 32 / N lanes from l * 32 / N on end with column l of the whole warp in v[0].
template <int N, typename Op>
__device__ __forceinline__ void reduce_columns(float (&v)[N], int lane, Op op) {
    int n = N;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
        if (n > 1) {
            const int half = n / 2;
            const bool upper = (lane & step) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < half) {
                    const float keep = upper ? v[i + half] : v[i];
                    const float send = upper ? v[i] : v[i + half];
                    v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, step));
                }
            n = half;
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], step));
        }
    }
}

// Two values (|x| <= 448) -> their e4m3 codes (hi) and the codes of what hi misses
// (lo), by way of f16: its rounding, 2^-11 of the value, is below lo's, and the
// difference is exact there.  lo is e4m3 (a query's 4 further bits, exactly) or e5m2 (a
// weight's: 3 bits, and seven binades more below).
template <__nv_fp8_interpretation_t LO>
__device__ __forceinline__ void split_e4m3x2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 x = __floats2half2_rn(a, b);
    hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 h = __half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3));
    lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(x, h)), __NV_SATFINITE, LO);
}

// No NaN among 16 e4m3 codes, no NaN or infinity among 8 bf16 values.
template <bool BF16>
__device__ __forceinline__ bool all_finite(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t hit = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        hit |= BF16 ? __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u)
                    : __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
    return hit == 0u;
}

__device__ __forceinline__ int swz128(int r, int cc) { return r * 128 + ((cc ^ (r & 7)) << 4); }
__device__ __forceinline__ int swz64(int r, int cc) {
    return r * 64 + ((cc ^ ((r >> 1) & 3)) << 4);
}

// Keys of sequence b that exist in its page table.
__device__ __forceinline__ int context_of(const LatentAttnParams& p, int b) {
    const int ctx = p.context_lens[b];
    const int most = p.max_blocks_per_seq * kPage;
    return ctx < 0 ? 0 : (ctx > most ? most : ctx);
}

// The partition.  A worker that crosses into another sequence pays for the end of one
// segment and the start of the next (its queries, the first reference, its output), the
// time of several tiles.  So the shares are equal not in tiles but in units: between the
// tiles of two sequences lie `gap` units without work, the price of that crossing.
// (Equal counts of tiles left the crossing workers running 59 us where the others ended
// after 43.)
struct Partition {
    int64_t units;               // of the launch
    int64_t workers;             // that get work: at most one per tile
    int gap;
};
// `tiles` and the number of sequences that have some
template <int N, int KEYS>
__device__ __forceinline__ Partition partition_of(const LatentAttnParams& p, int64_t tiles,
                                                  int sequences) {
    Partition pt;
    pt.workers = tiles < p.workers ? tiles : p.workers;
    // a crossing costs about 17000 cycles with 64 columns, 9000 with fewer; a tile 3800
    // or 3200.  Small shares leave less to trade.
    constexpr int kGap = N == 64 ? 5 : 3;
    const int64_t half = pt.workers > 0 ? tiles / pt.workers / 2 : 0;
    pt.gap = half < kGap ? static_cast<int>(half) : kGap;
    pt.units = tiles + (sequences > 0 ? static_cast<int64_t>(sequences - 1) * pt.gap : 0);
    return pt;
}

// The segments of a worker's share, in order: sequence b, its tiles [t0, t0 + n).
// Every role walks the same list.
template <int KEYS>
struct Segments {
    const LatentAttnParams& p;
    int b;
    int64_t off, left;
    int ctx, n;
    __device__ __forceinline__ Segments(const LatentAttnParams& p_, const Misc& m)
        : p(p_), b(m.b0), off(m.first_tile), left(m.num_tiles), ctx(0), n(0) {}
    __device__ __forceinline__ bool next() {
        if (n > 0) {
            ++b;
            off = 0;
        }
        while (left > 0 && b < p.B) {
            ctx = context_of(p, b);
            const int64_t nt = (ctx + KEYS - 1) / KEYS;
            if (nt - off > 0) {
                n = static_cast<int>(nt - off < left ? nt - off : left);
                left -= n;
                return true;
            }
            ++b;
            off = 0;
        }
        return false;
    }
    __device__ __forceinline__ int tile0() const { return static_cast<int>(off); }
    __device__ __forceinline__ bool whole() const {
        return off == 0 && n == (ctx + KEYS - 1) / KEYS;
    }
};

template <int N, bool BF16, bool PT>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap latent_map,
                       const __grid_constant__ CUtensorMap rope_map, LatentAttnParams p) {
    using C = Cfg<N, BF16>;
    constexpr int kKeys = C::kKeys;
    extern __shared__ __align__(1024) uint8_t smem[];    // 128-byte swizzle: 1024-byte atoms
    Misc& ms = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int worker = blockIdx.x / p.groups, group = blockIdx.x - worker * p.groups;
    const int chunks = p.L / 128;            // M 128 products of O^T
    // 128-byte panels of a row in a stage, bytes of 8 keys
    const int panels = chunks * C::kElem + (BF16 ? 1 : 0);
    const uint32_t group_bytes = panels * 1024;
    volatile int* abort_flag = &ms.abort;

    if (tid == 0) {
        mbar_init(smem_addr(&ms.rope_empty), 1);
        for (int i = 0; i < 2; ++i) {
            // every copying warp announces the rows' bytes and (e4m3) the shared keys'
            mbar_init(smem_addr(&ms.full[i]), kLoadWarps * (BF16 ? 1 : 2));
            mbar_init(smem_addr(&ms.empty[i]), 1);
            mbar_init(smem_addr(&ms.s_full[i]), 1);
            mbar_init(smem_addr(&ms.s_empty[i]), kSoftThreads);
        }
        mbar_init(smem_addr(&ms.p_full), kSoftThreads);
        mbar_init(smem_addr(&ms.pv_done), 1);
        mbar_init(smem_addr(&ms.q_full), kSoftThreads);
        mbar_init(smem_addr(&ms.idle), 1);
        ms.abort = 0;
        mbar_init_fence();
        prefetch_tmap(&latent_map);
        prefetch_tmap(&rope_map);
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&ms.tmem), kTmemAll);
    pdl_wait();                              // inputs of earlier kernels are visible
    pdl_trigger();
    if (warp == 0) {                         // this worker's share
        int64_t total = 0;
        int nseq = 0;
        for (int b = lane; b < p.B; b += 32) {
            const int nt = (context_of(p, b) + kKeys - 1) / kKeys;
            total += nt;
            nseq += nt > 0;
        }
        total = warp_sum(total);
        nseq = static_cast<int>(warp_sum(static_cast<int64_t>(nseq)));
        const Partition pt = partition_of<N, kKeys>(p, total, nseq);
        int64_t ulo = 0, uhi = 0;            // the worker's units
        if (worker < pt.workers) {
            ulo = worker * pt.units / pt.workers;
            uhi = (worker + 1) * pt.units / pt.workers;
        }
        // its tiles [lo, hi): those behind as many units; b0: the sequence of tile lo,
        // `at` the tiles in front of that sequence
        int64_t lo = 0, hi = 0, units = 0, tiles = 0, at = 0;
        int b0 = p.B;
        for (int base = 0; base < p.B && ulo < uhi; base += 32) {
            const int b = base + lane;
            const int64_t nt = b < p.B ? (context_of(p, b) + kKeys - 1) / kKeys : 0;
            const int64_t nu = nt > 0 ? nt + pt.gap : 0;
            int64_t it = nt, iu = nu;        // inclusive sums
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t yt = __shfl_up_sync(0xffffffffu, it, o);
                const int64_t yu = __shfl_up_sync(0xffffffffu, iu, o);
                if (lane >= o) {
                    it += yt;
                    iu += yu;
                }
            }
            const int64_t start = units + iu - nu;                   // unit of its first tile
            const int64_t clo = ulo <= start ? 0 : (ulo - start < nt ? ulo - start : nt);
            const int64_t chi = uhi <= start ? 0 : (uhi - start < nt ? uhi - start : nt);
            lo += warp_sum(clo);
            hi += warp_sum(chi);
            // the first sequence with a tile of the share
            const unsigned hit = __ballot_sync(0xffffffffu, chi > clo);
            if (b0 == p.B && hit) {
                const int src = __ffs(hit) - 1;
                b0 = base + src;
                at = tiles + __shfl_sync(0xffffffffu, it - nt, src);
            }
            units += __shfl_sync(0xffffffffu, iu, 31);
            tiles += __shfl_sync(0xffffffffu, it, 31);
        }
        if (lane == 0) {
            ms.b0 = b0;
            ms.first_tile = hi > lo ? lo - at : 0;
            ms.num_tiles = hi - lo;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    const int row0 = group * p.rows_per_group;
    const int nrows = min(p.rows_per_group, p.S * p.H - row0);

    if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ------------------------------------------------ loaders: a warp walks the tiles
        // converged (lane = page of a tile), one elected lane issues the tensor copies
        // of every second page: half a page (8 keys, all panels) each
        // The two stages hold too little to cover HBM's latency, so a tile's pages are
        // asked into L2 kAhead tiles before their copies.
        constexpr int kHalf = C::kPages / kLoadWarps;
        constexpr int kAhead = 2;
        const int first = warp - kSoftWarps;             // pages first, first + 2, ...
        const uint32_t page_bytes = kPage * (p.L + kRope) * C::kElem;
        int tile = 0;                                    // tiles begun
        int in_tile = 0;                                 // parts of the last one issued
        bool ok = true;
        Segments<kKeys> sg(p, ms);
        while (ok && sg.next()) {
            const int32_t* bt = p.block_table + static_cast<int64_t>(sg.b) * p.max_blocks_per_seq;
            const int pages = (sg.ctx + kPage - 1) / kPage;
            // whether tile j has a page for this lane: told by its number, as any value of
            // the table may be an id
            auto has_page = [&](int j) {
                return lane < C::kPages && j < sg.n &&
                       (sg.tile0() + j) * C::kPages + lane < pages;
            };
            auto block_of = [&](int j) {
                return has_page(j) ? bt[(sg.tile0() + j) * C::kPages + lane] : -1;
            };
            int next[kAhead + 1];            // pages of the tiles behind the current one
#pragma unroll
            for (int i = 0; i <= kAhead; ++i) next[i] = block_of(i);
            for (int j = 0; j < sg.n && ok; ++j) {
                const int blk = next[0];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) next[i] = next[i + 1];
                next[kAhead] = block_of(j + kAhead + 1);
                if (next[kAhead - 1] >= 0 && next[kAhead - 1] < p.num_blocks &&
                    (lane & 1) == first)
                    bulk_prefetch_l2(p.cache + static_cast<int64_t>(next[kAhead - 1]) * page_bytes,
                                     page_bytes);
                bool have = has_page(j);
                if (have && (blk < 0 || blk >= p.num_blocks)) {
                    report(p.err, FP8KV_ERR_BAD_INDEX);
                    have = false;            // skipped: its keys get no weight
                }
                const unsigned mask =
                    __ballot_sync(0xffffffffu, have) & (0x55555555u << first);
                const int n = __popc(mask);
                int pb[kHalf];
#pragma unroll
                for (int i = 0; i < kHalf; ++i)
                    pb[i] = __shfl_sync(0xffffffffu, blk, kLoadWarps * i + first);
                const int st = tile & 1;
                const uint32_t bar = smem_addr(&ms.full[st]);
                ++tile;
                in_tile = 0;
                if (tile > 2)
                    ok = __all_sync(0xffffffffu, wait_bar(&ms.empty[st], ((tile - 3) >> 1) & 1,
                                                          abort_flag, p.err));
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, n * (2 * group_bytes));
                    const uint32_t dst = sbase + st * C::kStageBytes;
#pragma unroll
                    for (int i = 0; i < kHalf; ++i) {
                        const int pg = kLoadWarps * i + first;
                        if ((mask >> pg) & 1u) {
                            tma_load_4d(dst + (2 * pg) * group_bytes, &latent_map, 0, 0, 0, pb[i],
                                        bar);
                            tma_load_4d(dst + (2 * pg + 1) * group_bytes, &latent_map, 0, 8, 0,
                                        pb[i], bar);
                        }
                    }
                }
                __syncwarp();
                ++in_tile;
                if constexpr (!BF16) {
                    // The shared keys last.  Of two slots the tile's own is free (PV of the
                    // tile before last has run); a single one when S of the previous tile
                    // has begun, and the rows' copies must not wait for that.
                    if (C::kRopeSlots == 1 && tile > 1)
                        ok = __all_sync(0xffffffffu, wait_bar(&ms.rope_empty, (tile - 2) & 1,
                                                              abort_flag, p.err));
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar, n * (kPage * kRope));
                        const uint32_t dst =
                            sbase + C::kOffRope + (C::kRopeSlots == 2 ? st * kRopeSlotBytes : 0);
#pragma unroll
                        for (int i = 0; i < kHalf; ++i) {
                            const int pg = kLoadWarps * i + first;
                            if ((mask >> pg) & 1u)
                                tma_load_3d(dst + pg * (kPage * kRope), &rope_map, p.L, 0, pb[i],
                                            bar);
                        }
                    }
                    __syncwarp();
                    ++in_tile;
                }
            }
        }
        // Copies still in flight land before the CTA can leave: whole tiles complete
        // their stage's phase; a tile that an abort cut short is completed by arrivals
        // without bytes.
        if (*abort_flag && lane == 0) {
            if (tile > 0)
                for (; in_tile < (BF16 ? 1 : 2); ++in_tile)
                    mbar_arrive(smem_addr(&ms.full[(tile - 1) & 1]));
            for (int t = tile > 2 ? tile - 2 : 0; t < tile; ++t)
                (void)mbar_wait_bounded(smem_addr(&ms.full[t & 1]), (t >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ MMA issuer: the warp walks the
        // tiles converged, one elected lane issues a product whole, its descriptors a
        // base plus constants.  (The pipe hides nothing between two issuing blocks:
        // looking at barriers chunk by chunk cost more than the MMAs, 5550 instead of
        // 3200 cycles a tile of 128 keys and 64 rows.)
        constexpr uint32_t kFmt = BF16 ? 1u : 0u;
        constexpr uint32_t id_s = instr_desc(kFmt, kFmt, 0, 0, C::kQRows, kKeys);
        // of a weight's first term, and (e4m3) of its second, e5m2
        constexpr uint32_t id_o = instr_desc(kFmt, kFmt, 1, 1, C::kOCols, 128);
        constexpr uint32_t id_o2 = instr_desc(0, 1, 1, 1, N, 128);
        auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
            if constexpr (BF16)
                mma_f16kind(d, a, b, id, acc ? 1u : 0u);
            else
                mma_f8f6f4(d, a, b, id, acc ? 1u : 0u);
        };
        // descriptors of the regions' starts; an offset adds its 16-byte units (smem
        // addresses stay below the field's 2^18 bytes)
        const uint64_t dx = smem_desc_sw128(sbase, 16, group_bytes);           // X as S's A
        const uint64_t dv = smem_desc_sw128(sbase, 1024, group_bytes);         // X as O's A
        const uint32_t group_units = group_bytes / 16;
        const uint64_t dq = smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
        const uint64_t dr = smem_desc(sbase + C::kOffRope, 16, 8 * kRope, kLayoutSw64);
        const uint64_t drq = smem_desc(sbase + C::kOffQ + C::kQRows * p.L, 16, 8 * kRope,
                                       kLayoutSw64);
        const uint64_t dp = smem_desc(sbase + C::kOffP, 16, 8 * C::kPRow,
                                      BF16 ? kLayoutSw128 : kLayoutSw64);
        // S^T of a tile into its buffer, panel by panel of the rows (e4m3: behind the
        // shared keys' own 64-byte panel)
        auto issue_s = [&](int t) {
            const uint32_t d = tmem + kSCol + (t & 1) * C::kQRows;
            uint64_t a = dx + static_cast<uint32_t>((t & 1) * (C::kStageBytes / 16));
            uint64_t b = dq;
            const uint64_t r =
                dr + static_cast<uint32_t>(C::kRopeSlots == 2 ? (t & 1) * (kRopeSlotBytes / 16) : 0);
            if (elect_one()) {
                if constexpr (!BF16) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma(d, r + k * 2, drq + k * 2, id_s, k > 0);
                    if constexpr (C::kRopeSlots == 1) mma_commit(smem_addr(&ms.rope_empty));
                }
#pragma unroll 1
                for (int pn = 0; pn < panels; ++pn) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma(d, a + k * 2, b + k * 2, id_s, !BF16 || pn > 0 || k > 0);
                    a += 1024 / 16;
                    b += C::kQRows * 8;
                }
                mma_commit(smem_addr(&ms.s_full[t & 1]));
            }
            __syncwarp();
        };
        // O^T += C^T P^T of a tile
        auto issue_o = [&](int t, bool first) {
            uint64_t a = dv + static_cast<uint32_t>((t & 1) * (C::kStageBytes / 16));
            const uint64_t dp2 =             // bf16, 64 rows: second terms in the rotary panel
                dx + static_cast<uint32_t>((t & 1) * (C::kStageBytes / 16) +
                                           chunks * C::kElem * (1024 / 16));
            uint32_t d = tmem;
            if (elect_one()) {
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    constexpr int kSteps = kKeys * C::kElem / 32;      // 4: k-steps of a term
                    // 32 (e4m3) or 16 (bf16) keys a step
                    constexpr int kKeyStep = 32 / C::kElem;
#pragma unroll
                    for (int k = 0; k < (C::kPairs ? 1 : 2) * kSteps; ++k) {
                        const int kk = k % kSteps;
                        uint64_t b = dp + kk * (kKeyStep * C::kPRow / 16);
                        if (k >= kSteps)
                            b = BF16 ? dp2 + kk * (kKeyStep / 8) * group_units
                                     : b + C::kPTerm / 16;
                        mma(d, a + kk * (kKeyStep / 8) * group_units, b,
                            BF16 || k < kSteps ? id_o : id_o2, !first || k > 0);
                    }
                    a += C::kElem * (1024 / 16);
                    d += C::kOCols;
                }
                mma_commit(smem_addr(&ms.empty[t & 1]));
                mma_commit(smem_addr(&ms.pv_done));
            }
            __syncwarp();
        };
        // S of the next tile and PV of the current one are issued in the order in
        // which their operands arrive: a late tile must not hold back a ready P, whose
        // product frees the slots of the tile after it.
        int tile = 0, seg = 0;
        bool ok = true;
        Segments<kKeys> sg(p, ms);
        while (ok && sg.next()) {
            ok = __all_sync(0xffffffffu, wait_bar(&ms.q_full, seg & 1, abort_flag, p.err));
            ++seg;
            tc_fence_after();
            int js = 0, jo = 0;                          // next S, next PV
            unsigned long long idle_since = 0;
            uint32_t looks = 0;
            while (ok && jo < sg.n) {
                // one look: lane 1 at the S buffer, lane 2 at P, the others at the tile
                const int t = tile + js;
                uint64_t* bar = lane == 1 ? &ms.s_empty[t & 1] : lane == 2 ? &ms.p_full
                                                                           : &ms.full[t & 1];
                const int parity = lane == 1 ? (t >> 1) - 1 : lane == 2 ? tile + jo : t >> 1;
                const unsigned seen =
                    __ballot_sync(0xffffffffu, test_bar(bar, parity & 1) || (lane == 1 && t < 2));
                if (js < sg.n && js <= jo + 1 && (seen & 3u) == 3u) {
                    tc_fence_after();
                    issue_s(t);
                    ++js;
                    idle_since = 0;
                } else if (jo < js && (seen & 4u)) {
                    tc_fence_after();
                    issue_o(tile + jo, jo == 0);
                    ++jo;
                    idle_since = 0;
                } else if ((++looks & 63u) == 0u) {
                    bool late = false;
                    const unsigned long long now = global_ns();
                    if (idle_since == 0) {
                        idle_since = now;
                    } else if (now - idle_since > kWaitBudgetNs) {
                        late = true;
                        *abort_flag = 1;
                        report(p.err, FP8KV_ERR_TIMEOUT);
                    }
                    ok = __all_sync(0xffffffffu, !late && *abort_flag == 0);
                }
            }
            tile += sg.n;
        }
        // every issued MMA finishes before tensor memory is released
        if (elect_one()) mma_commit(smem_addr(&ms.idle));
        __syncwarp();
        (void)mbar_wait_bounded(smem_addr(&ms.idle), 0);
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax: a thread owns one key
        // and one half of the columns.  M 128: TMEM lane = key; M 64 (bf16): 16 keys in
        // the first lanes of each quarter
        constexpr int NC = N / kParts;
        constexpr int kW = NC;                           // columns of one TMEM access
        const int quarter = warp & 3, part = warp >> 2, n0 = part * NC;
        const int key = 16 * (BF16 ? 1 : 2) * quarter + (BF16 ? lane & 15 : lane);
        const bool owner = !BF16 || lane < 16;
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        const float kconst = BF16 || PT ? 1.f : p.scale[0];
        constexpr float kInf = __builtin_huge_valf();
        int tile = 0;
        bool ok = true;
        Segments<kKeys> sg(p, ms);
        while (ok && sg.next()) {
            // ---- Q operand and the columns' constants: 256 / N neighbouring threads share
            // a row, every load in flight before the first is used (they queue behind the
            // first tiles' copies: in batches of three this took 17000 cycles)
            {
                constexpr int kShare = kSoftThreads / N;             // threads of a row
                constexpr int kPieces = (72 + kShare - 1) / kShare;  // 16-byte pieces of each
                const int n = tid / kShare, first = tid % kShare;
                const int pieces = (p.L + kRope) / 8;
                const __nv_bfloat16* q =
                    p.q + (static_cast<int64_t>(sg.b) * p.S * p.H + row0 + n) * (p.L + kRope);
                uint8_t* qs = smem + C::kOffQ;
                uint4 x[kPieces];
#pragma unroll
                for (int u = 0; u < kPieces; ++u) {
                    x[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (n < nrows && first + u * kShare < pieces)
                        x[u] = *reinterpret_cast<const uint4*>(q + (first + u * kShare) * 8);
                }
                float f = p.scale_log2 * kconst, mul = 1.f;
                if constexpr (!BF16) {
                    uint32_t amax = 0u;      // bits of max |q|, two at a time: ordered like it
#pragma unroll
                    for (int u = 0; u < kPieces; ++u) {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) amax = __vmaxu2(amax, w[e] & 0x7fff7fffu);
                    }
                    amax = max(amax >> 16, amax & 0xffffu);
#pragma unroll
                    for (int o = kShare / 2; o > 0; o >>= 1)
                        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (amax >= 0x7f80u) {
                        f = __int_as_float(0x7fffffff);  // inf or NaN in q: the row is NaN
                    } else if (amax != 0u) {
                        // 2^e: max |q| into [128, 256); exact, undone in f
                        int e = 134 - static_cast<int>(amax >> 7);
                        e = e > 120 ? 120 : e;
                        mul = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                        f *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    }
                }
#pragma unroll
                for (int u = 0; u < kPieces; ++u) {
                    const int pc = first + u * kShare;   // values [8 pc, 8 pc + 8)
                    if (pc >= pieces) break;
                    if constexpr (BF16) {                // panels of 64 values
                        *reinterpret_cast<uint4*>(qs + (pc >> 3) * (N * 128) + swz128(n, pc & 7)) =
                            x[u];
                    } else {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            split_e4m3x2<__NV_E4M3>(bf16_bits_to_float(w[e] & 0xffffu) * mul,
                                                    __uint_as_float(w[e] & 0xffff0000u) * mul,
                                                    hi[e], lo[e]);
                        const int rel = pc - p.L / 8;    // >= 0: the rotary panel
                        const int o0 = (rel >= 0 ? C::kQRows * p.L + swz64(n, rel >> 1)
                                                 : (pc >> 4) * (C::kQRows * 128) +
                                                       swz128(n, (pc & 15) >> 1)) +
                                       (pc & 1) * 8;
                        const int o1 = o0 + N * (rel >= 0 ? 64 : 128);
                        *reinterpret_cast<uint2*>(qs + o0) =
                            make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                        *reinterpret_cast<uint2*>(qs + o1) =
                            make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
                    }
                }
                if (first == 0) {
                    reinterpret_cast<float*>(ms.f)[n] = f;
                    reinterpret_cast<float*>(ms.nm)[n] = 0.f;
                    // columns beyond the group's rows (q = 0) see everything
                    ms.last[n] = n < nrows ? sg.ctx - p.S + (row0 + n) / p.H : 0x7fffffff;
                }
            }
            if (tid < kParts) ms.quiet[tid] = 0u;
            bool unset = true;               // some column of the half has no reference yet
            fence_proxy_async();             // generic writes -> tensor core reads
            mbar_arrive(smem_addr(&ms.q_full));
            soft_any(false);                 // f, nm, last, quiet visible

            // this key's page and scale, loaded a tile (the page: two) ahead
            const int32_t* bt = p.block_table + static_cast<int64_t>(sg.b) * p.max_blocks_per_seq;
            auto block_of = [&](int j) {
                const int pos = (sg.tile0() + j) * kKeys + key;
                const int blk = owner && j < sg.n && pos < sg.ctx ? bt[pos / kPage] : -1;
                return blk < p.num_blocks ? blk : -1;    // no page: the key has no weight
            };
            auto scale_of = [&](int blk) {
                return PT && blk >= 0 ? p.scale_cache[static_cast<int64_t>(blk) * kPage + key % kPage]
                                      : 1.f;
            };
            int blk0 = block_of(0), blk1 = block_of(1);
            float ks_next = scale_of(blk0);
            float ls_next = 0.f, rs_next = 1.f, ls_low = 0.f;
            auto code_scale = [&](float s) {             // log2 and 1 / of a row's scale
                if constexpr (PT) {
                    const float se = s >= kMinScale ? s : kZeroRowScale;   // NaN: finite here
                    ls_next = __log2f(se);
                    rs_next = __fdividef(1.f, se);
                    ls_low = fminf(ls_low, ls_next);
                }
            };
            code_scale(ks_next);

            uint64_t l[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) l[i] = 0ull;
            for (int j = 0; j < sg.n; ++j, ++tile) {
                const bool here = blk0 >= 0;
                const float ks = ks_next, ls = ls_next, rs = rs_next;
                blk0 = blk1;
                blk1 = block_of(j + 2);
                ks_next = scale_of(blk0);
                const int buf = tile & 1;
                {
                    const bool w = wait_bar(&ms.s_full[buf], (tile >> 1) & 1, abort_flag, p.err);
                    ok = __all_sync(0xffffffffu, w && ok);
                }
                tc_fence_after();
                // ---- raw logits of this key, this half's columns, in pairs
                uint64_t d[NC / 2];
                const uint32_t sa = tmem + lane_addr + kSCol + buf * C::kQRows + n0;
                {
                    uint32_t a[kW];
                    tmem_ld_n<kW>(sa, a);
                    if constexpr (!BF16) {
                        uint32_t b[kW];
                        tmem_ld_n<kW>(sa + N, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < NC / 2; ++i)
                            d[i] = add_f32x2(pack_f32x2(__uint_as_float(a[2 * i]),
                                                        __uint_as_float(a[2 * i + 1])),
                                             pack_f32x2(__uint_as_float(b[2 * i]),
                                                        __uint_as_float(b[2 * i + 1])));
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < NC / 2; ++i)
                            d[i] = pack_f32x2(__uint_as_float(a[2 * i]),
                                              __uint_as_float(a[2 * i + 1]));
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_addr(&ms.s_empty[buf]));

                // ---- d = log2 weight against the running reference
                const int pos = (sg.tile0() + j) * kKeys + key;
                const uint64_t ks2 = pack_f32x2(ks, ks), ls2 = pack_f32x2(ls, ls),
                               rs2 = pack_f32x2(rs, rs);
                const ulonglong2* f4 = reinterpret_cast<const ulonglong2*>(ms.f + n0 / 2);
                const ulonglong2* nm4 = reinterpret_cast<const ulonglong2*>(ms.nm + n0 / 2);
                // the first query token sees keys up to ctx - S; only the tiles behind
                // that, and tiles with skipped pages, need the masks
                const bool open = __all_sync(0xffffffffu, !owner || (here && pos <= sg.ctx - p.S));
                float most = -kInf;
                float most2 = -kInf;
#pragma unroll
                for (int i = 0; i < NC / 4; ++i) {
                    const ulonglong2 f = f4[i], nm = nm4[i];
                    if constexpr (PT) {
                        d[2 * i] = fma_f32x2(mul_f32x2(d[2 * i], ks2), f.x, add_f32x2(ls2, nm.x));
                        d[2 * i + 1] =
                            fma_f32x2(mul_f32x2(d[2 * i + 1], ks2), f.y, add_f32x2(ls2, nm.y));
                    } else {
                        d[2 * i] = fma_f32x2(d[2 * i], f.x, nm.x);
                        d[2 * i + 1] = fma_f32x2(d[2 * i + 1], f.y, nm.y);
                    }
                    const float2 x = unpack_f32x2(d[2 * i]), y = unpack_f32x2(d[2 * i + 1]);
                    most = fmaxf(most, fmaxf(x.x, x.y));
                    most2 = fmaxf(most2, fmaxf(y.x, y.y));
                }
                most = fmaxf(most, most2);
                if (BF16 && !owner) {        // TMEM lanes that hold no key
                    most = -kInf;
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) d[i] = pack_f32x2(-kInf, -kInf);
                } else if (!open) {
                    most = -kInf;
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) {
                        float2 x = unpack_f32x2(d[i]);
                        if (!here || pos > ms.last[n0 + 2 * i]) x.x = -kInf;
                        if (!here || pos > ms.last[n0 + 2 * i + 1]) x.y = -kInf;
                        most = fmaxf(most, fmaxf(x.x, x.y));
                        d[i] = pack_f32x2(x.x, x.y);
                    }
                }
                const bool need = most > C::kLimit || unset;
                if constexpr (!BF16) {       // this key's columns under 2^kLow, bit i = column i
                    uint32_t under = 0u;
                    const uint64_t low2 = pack_f32x2(-C::kLow, -C::kLow);
#pragma unroll
                    for (int i = NC / 2 - 1; i >= 0; --i) {
                        const float2 x = unpack_f32x2(add_f32x2(d[i], low2));
                        under = __funnelshift_l(__float_as_uint(x.y), under, 1);   // sign bits
                        under = __funnelshift_l(__float_as_uint(x.x), under, 1);
                    }
                    under = __reduce_and_sync(0xffffffffu, under);
                    if (lane == 0) ms.under[buf][warp] = under;
                }
                // a half's columns are its own: its four warps decide and move alone
                bool move = half_any(part, need || !ok);
                if constexpr (!BF16) {       // a column under it in all four quarters
                    constexpr uint32_t kAll = NC == 32 ? 0xffffffffu : (1u << (NC & 31)) - 1u;
                    const uint4 u = *reinterpret_cast<const uint4*>(&ms.under[buf][4 * part]);
                    move = move || (u.x & u.y & u.z & u.w & ~ms.quiet[part] & kAll) != 0u;
                }
                if (move) {
                    // ---- move references: column maxima over the tile's keys
                    float mx_lane = -kInf;               // lane i: column n0 + i
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) {
                        const float2 x = unpack_f32x2(d[i]);
                        const float a = warp_max(x.x), b = warp_max(x.y);
                        if (lane == 2 * i) mx_lane = a;
                        if (lane == 2 * i + 1) mx_lane = b;
                    }
                    if (lane < NC) ms.red[quarter][n0 + lane] = mx_lane;
                    if constexpr (PT) {
                        const float low = warp_min(ls_low);
                        if (lane == 0) ms.low[part][quarter] = low;
                    }
                    if (half_any(part, !ok)) {
                        ok = false;
                        break;
                    }
                    bool missing = false;
                    if (quarter == 0 && lane < NC) {
                        const int n = n0 + lane;
                        const float mx = fmaxf(fmaxf(ms.red[0][n], ms.red[1][n]),
                                               fmaxf(ms.red[2][n], ms.red[3][n]));
                        const float top = j == 0 ? -kInf : ms.top[n];
                        const bool was = top > -kInf;
                        const bool any = mx > -kInf;
                        const float ref = -reinterpret_cast<float*>(ms.nm)[n];
                        float delta = 0.f, alpha = 1.f, deepest = kDeepest;
                        if constexpr (PT) {
                            const float4 low = *reinterpret_cast<const float4*>(ms.low[part]);
                            const float room =
                                kSumRoom + fminf(fminf(low.x, low.y), fminf(low.z, low.w));
                            deepest = fmaxf(fminf(deepest, room), 0.f);
                        }
                        if (any) {
                            // up: with the one that has to, columns close behind
                            if (!was)
                                delta = mx - C::kLift;
                            else if (mx > C::kLimit - 1.f)
                                delta = mx - C::kHigh;
                            else if (!BF16 && mx < C::kLow)      // down, to the floor at most
                                delta = fminf(fmaxf(mx - C::kLift, top - deepest - ref), 0.f);
                            if (was) alpha = ex2(-delta);
                        }
                        ms.top[n] = any ? fmaxf(top, ref + delta) : top;
                        if constexpr (!BF16) {
                            constexpr unsigned kLanes =
                                NC == 32 ? 0xffffffffu : (1u << (NC & 31)) - 1u;
                            // on its floor (but for a rounding), or past the last key that
                            // the column sees: nothing below is to be followed
                            const bool hush = ref + delta < top - (deepest - 1.f) ||
                                              ms.last[n] < (sg.tile0() + j) * kKeys;
                            const unsigned q = __ballot_sync(kLanes, hush);
                            if (lane == 0) ms.quiet[part] = q;
                        }
                        ms.delta[n] = -delta;
                        ms.alpha[n] = alpha;
                        reinterpret_cast<float*>(ms.nm)[n] = -(ref + delta);
                        missing = !was && !any;
                    }
                    unset = half_any(part, missing);
                    const uint64_t* dl2 = reinterpret_cast<const uint64_t*>(ms.delta + n0);
                    const uint64_t* al2 = reinterpret_cast<const uint64_t*>(ms.alpha + n0);
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) {
                        d[i] = add_f32x2(d[i], dl2[i]);
                        l[i] = mul_f32x2(l[i], al2[i]);
                    }
                    // O's columns that moved (few: a column moves a handful of times)
                    unsigned moved =
                        __ballot_sync(0xffffffffu, lane < NC && ms.alpha[n0 + lane % NC] != 1.f);
                    if (j > 0 && moved) {
                        const bool w = wait_bar(&ms.pv_done, (tile - 1) & 1, abort_flag, p.err);
                        ok = __all_sync(0xffffffffu, w && ok);
                        tc_fence_after();
                        for (; moved; moved &= moved - 1) {
                            const int n = n0 + __ffs(moved) - 1;
                            const float a = ms.alpha[n];
                            const uint32_t oa = tmem + lane_addr + n;
                            constexpr int kTerms = C::kOCols / N;
                            uint32_t o[4 * kTerms];
#pragma unroll
                            for (int c = 0; c < 4 * kTerms; ++c)
                                if (c < chunks * kTerms) o[c] = tmem_ld1(oa + c * N);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 4 * kTerms; ++c)
                                if (c < chunks * kTerms)
                                    tmem_st1(oa + c * N,
                                             __float_as_uint(__uint_as_float(o[c]) * a));
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    // red, delta and alpha are written again only behind the next vote
                }

                // ---- weights, row sums, P operand
                uint32_t hi[NC * C::kElem / 4], lo[NC * C::kElem / 4];
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    const float2 x = unpack_f32x2(d[i]);
                    const float a = ex2(x.x), b = ex2(x.y);
                    if constexpr (PT)
                        l[i] = fma_f32x2(pack_f32x2(a, b), rs2, l[i]);
                    else
                        l[i] = add_f32x2(pack_f32x2(a, b), l[i]);
                    if constexpr (BF16) {
                        hi[i] = pack_bf16x2(a, b);
                        const float2 h = unpack_bf16x2(hi[i]);
                        lo[i] = pack_bf16x2(a - h.x, b - h.y);
                    } else {
                        uint32_t ch, cl;
                        split_e4m3x2<__NV_E5M2>(a, b, ch, cl);
                        if (i & 1) {
                            hi[i >> 1] |= ch << 16;
                            lo[i >> 1] |= cl << 16;
                        } else {
                            hi[i >> 1] = ch;
                            lo[i >> 1] = cl;
                        }
                    }
                }
                // the P buffer is free once PV of the previous tile has run
                if (tile > 0) {
                    const bool w = wait_bar(&ms.pv_done, (tile - 1) & 1, abort_flag, p.err);
                    ok = __all_sync(0xffffffffu, w) && ok;
                }
                if (owner && ok) {
                    uint8_t* ps = smem + C::kOffP;
                    constexpr int kBytes = NC * C::kElem;          // of this key's half row
                    if constexpr (kBytes >= 16) {
#pragma unroll
                        for (int c = 0; c < kBytes / 16; ++c) {
                            const int cc = part * (kBytes / 16) + c;
                            const int at = BF16 ? swz128(key, cc) : swz64(key, cc);
                            *reinterpret_cast<uint4*>(ps + at) =
                                make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                            uint8_t* second =
                                C::kPairs ? ps + swz128(key, cc + N / 8)
                                : BF16    ? smem + buf * C::kStageBytes + (key >> 3) * group_bytes +
                                             chunks * (C::kElem * 1024) + swz128(key & 7, cc)
                                          : ps + C::kPTerm + at;
                            *reinterpret_cast<uint4*>(second) =
                                make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                        }
                    } else {                             // e4m3, N 16: 8 bytes each
                        const int at = swz64(key, 0) + part * 8;
                        *reinterpret_cast<uint2*>(ps + at) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(ps + C::kPTerm + at) = make_uint2(lo[0], lo[1]);
                    }
                    // A key without weight: its bytes (never written, or of no page) could be
                    // NaN, and 0 * NaN would reach every output.  One of the last S tokens
                    // has no weight in the queries before it: what of it is not finite goes
                    // too, as a query that does see it has a logit, and so all its values,
                    // that are not finite either (but for a logit of -inf, weight 0).
                    // A row without a scale is cleared as well.
                    const bool clear = !here || (PT && ks < kMinScale);
                    if (clear || pos > sg.ctx - p.S) {
                        if (!clear)          // (complete: S has read the tile)
                            (void)wait_bar(&ms.full[buf], (tile >> 1) & 1, abort_flag, p.err);
                        for (int c = part; c < chunks; c += kParts) {
                            uint8_t* xs = smem + buf * C::kStageBytes + (key >> 3) * group_bytes +
                                          c * (C::kElem * 1024) + (key & 7) * 128;
#pragma unroll
                            for (int pn = 0; pn < C::kElem; ++pn)
#pragma unroll
                                for (int cc = 0; cc < 8; ++cc) {
                                    uint4* x = reinterpret_cast<uint4*>(xs + pn * 1024 + cc * 16);
                                    if (clear || !all_finite<BF16>(*x))
                                        *x = make_uint4(0u, 0u, 0u, 0u);
                                }
                        }
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                mbar_arrive(smem_addr(&ms.p_full));
                code_scale(ks_next);
            }
            if (!ok) *abort_flag = 1;
            if (soft_any(!ok)) break;

            // ---- the segment's end: row sums over all keys, O out of tensor memory
            {
                float v[NC];
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    const float2 x = unpack_f32x2(l[i]);
                    v[2 * i] = x.x;
                    v[2 * i + 1] = x.y;
                }
                reduce_columns<NC>(v, lane, [](float a, float b) { return a + b; });
                ms.red[quarter][n0 + lane / (32 / NC)] = v[0];
            }
            ok = wait_bar(&ms.pv_done, (tile - 1) & 1, abort_flag, p.err) && ok;
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool direct = sg.whole();
            // a partial's slot: 0 for the worker's first segment, 1 for its last
            const int64_t slot =
                (2 * static_cast<int64_t>(worker) + (sg.b == ms.b0 ? 0 : 1)) * p.groups + group;
            if (tid < N) {
                const float sum = (ms.red[0][tid] + ms.red[1][tid]) +
                                  (ms.red[2][tid] + ms.red[3][tid]);
                if (direct) {
                    ms.alpha[tid] = sum != 0.f ? 1.f / sum : 0.f;
                } else {
                    ms.alpha[tid] = 1.f;
                    if (tid < nrows) {
                        p.ws_m[slot * N + tid] = -reinterpret_cast<float*>(ms.nm)[tid];
                        p.ws_l[slot * N + tid] = sum;
                    }
                }
            }
            soft_any(false);
            // rows n0, n0 + 1, ..: L values apart in the output and in a partial
            const int rows = min(NC, nrows - n0);
            const float4* al4 = reinterpret_cast<const float4*>(ms.alpha + n0);
            auto store = [&](auto* to, auto as) {
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    uint32_t o[kW];
                    tmem_ld_n<kW>(tmem + lane_addr + c * C::kOCols + n0, o);
                    if constexpr (C::kPairs) {           // the second terms' columns
                        uint32_t o2[kW];
                        tmem_ld_n<kW>(tmem + lane_addr + c * C::kOCols + N + n0, o2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kW; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(o2[i]));
                    } else {
                        tmem_wait_ld();
                    }
                    auto* at = to + c * 128 + 32 * quarter + lane;
#pragma unroll
                    for (int i = 0; i < NC / 4; ++i) {
                        const float4 a4 = al4[i];
                        const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u, at += p.L)
                            // a row that saw nothing has sum 0: zeros, whatever its O holds
                            if (4 * i + u < rows)
                                *at = as(a[u] != 0.f ? __uint_as_float(o[4 * i + u]) * kconst * a[u]
                                                     : 0.f);
                    }
                }
            };
            const int64_t first_row = static_cast<int64_t>(sg.b) * p.S * p.H + row0 + n0;
            if (!direct)
                store(p.ws_o + (slot * N + n0) * p.L, [](float x) { return x; });
            else if (p.out_bf16)
                store(static_cast<__nv_bfloat16*>(p.out) + first_row * p.L,
                      [](float x) { return __float2bfloat16_rn(x); });
            else
                store(static_cast<float*>(p.out) + first_row * p.L, [](float x) { return x; });
            tc_fence_before();               // O is drained: the next segment may start it anew
            soft_any(false);                 // f, nm, red, alpha are free again
        }
        if (!ok) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemAll);
    }
}

// Joins the partials of sequences cut between workers: out = sum_i O_i 2^(m_i - M) /
// sum_i l_i 2^(m_i - M), M the largest m_i; sequences without keys get zero rows.
// Sequences of one worker were written by the attention kernel.  A warp holds 128
// values of a row, 4 a lane; its lanes weigh 32 partials at once, then read them 8 at
// a time.
template <int N, int KEYS>
__global__ void __launch_bounds__(128) latent_merge_kernel(LatentAttnParams p) {
    const int b = blockIdx.y;
    const int per_row = p.L / 4;
    const int row = blockIdx.x * (128 / per_row) + threadIdx.x / per_row;
    const int dim = (threadIdx.x % per_row) * 4;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    int64_t before = 0, total = 0;           // tiles in front of the sequence, of all
    int64_t seqs = 0;                        // sequences that have some, (before << 32) + all
    for (int i = lane; i < p.B; i += 32) {
        const int64_t nt = (context_of(p, i) + KEYS - 1) / KEYS;
        total += nt;
        seqs += nt > 0;
        if (i < b) {
            before += nt;
            seqs += static_cast<int64_t>(nt > 0) << 32;
        }
    }
    before = warp_sum(before);
    total = warp_sum(total);
    seqs = warp_sum(seqs);
    const int64_t mine = (context_of(p, b) + KEYS - 1) / KEYS;
    if (row >= p.S * p.H) return;            // whole warps
    const int64_t at = (static_cast<int64_t>(b) * p.S * p.H + row) * p.L + dim;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine > 0) {
        const Partition pt = partition_of<N, KEYS>(p, total, static_cast<int>(seqs & 0xffffffff));
        const int64_t tile0 = before + (seqs >> 32) * pt.gap;        // its first tile's unit
        const int w0 = static_cast<int>(((tile0 + 1) * pt.workers - 1) / pt.units);
        const int parts =
            static_cast<int>(((tile0 + mine) * pt.workers - 1) / pt.units) - w0 + 1;
        if (parts == 1) return;              // written whole
        const int g = row / p.rows_per_group, n = row - g * p.rows_per_group;
        // slot 0 if the sequence is the first worker's first: nothing before the gap
        const int first = w0 * pt.units / pt.workers >= tile0 - pt.gap ? 0 : 1;
        constexpr float kInf = __builtin_huge_valf();
        float m = -kInf, l = 0.f;
        for (int base = 0; base < parts; base += 32) {
            const int i = base + lane;
            const int64_t slot =
                ((2 * static_cast<int64_t>(w0 + i) + (i == 0 ? first : 0)) * p.groups + g) * N + n;
            float li = 0.f, mi = -kInf;
            if (i < parts) {
                li = p.ws_l[slot];
                mi = li != 0.f ? p.ws_m[slot] : -kInf;   // a part in which the row saw nothing
            }
            float mc = fmaxf(m, mi);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, s));
            const float a = mi > -kInf ? exp2f(mi - mc) : 0.f;
            const float old = m > -kInf ? exp2f(m - mc) : 0.f;
            m = mc;
            float lc = li != 0.f ? li * a : 0.f;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) lc += __shfl_xor_sync(0xffffffffu, lc, s);
            l = l * old + lc;
            o.x *= old;
            o.y *= old;
            o.z *= old;
            o.w *= old;
            const int here = min(32, parts - base);
            for (int k = 0; k < here; k += 8) {
                float4 x[8];
                float ak[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    ak[u] = __shfl_sync(0xffffffffu, a, (k + u) & 31);
                    const int64_t sk = __shfl_sync(0xffffffffu, slot, (k + u) & 31);
                    x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k + u < here)
                        x[u] = *reinterpret_cast<const float4*>(p.ws_o + sk * p.L + dim);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (k + u >= here || ak[u] == 0.f) continue;
                    o.x = fmaf(x[u].x, ak[u], o.x);
                    o.y = fmaf(x[u].y, ak[u], o.y);
                    o.z = fmaf(x[u].z, ak[u], o.z);
                    o.w = fmaf(x[u].w, ak[u], o.w);
                }
            }
        }
        const float r = l != 0.f ? 1.f / l : 0.f;
        o.x *= r;
        o.y *= r;
        o.z *= r;
        o.w *= r;
    }
    if (p.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
}

template <int N, bool BF16, bool PT>
cudaError_t launch(const LatentAttnParams& p, const CUtensorMap& lm, const CUtensorMap& rm,
                   cudaStream_t stream) {
    using C = Cfg<N, BF16>;
    auto kern = latent_attn_kernel<N, BF16, PT>;
    static unsigned long long attr_done[64] = {};
    cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(kern), C::kSmem, attr_done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(attr, static_cast<int64_t>(p.workers) * p.groups, kThreads,
                                        C::kSmem, stream);
    e = cudaLaunchKernelEx(&cfg, kern, lm, rm, p);
    if (e != cudaSuccess) return e;
    const int rows = 128 / (p.L / 4);
    cfg = pdl_config(attr, 1, 128, 0, stream);
    cfg.gridDim = dim3(static_cast<unsigned>((p.S * p.H + rows - 1) / rows),
                       static_cast<unsigned>(p.B));
    return cudaLaunchKernelEx(&cfg, latent_merge_kernel<N, C::kKeys>, p);
}

template <bool BF16, bool PT>
cudaError_t launch_columns(const LatentAttnParams& p, int n, const CUtensorMap& lm,
                           const CUtensorMap& rm, cudaStream_t s) {
    return n == 16   ? launch<16, BF16, PT>(p, lm, rm, s)
           : n == 32 ? launch<32, BF16, PT>(p, lm, rm, s)
                     : launch<64, BF16, PT>(p, lm, rm, s);
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnParams& p, int columns, int kv_dtype,
                               const CUtensorMap& latent_map, const CUtensorMap& rope_map,
                               cudaStream_t stream) {
    if (kv_dtype == FP8KV_KV_BF16)
        return launch_columns<true, false>(p, columns, latent_map, rope_map, stream);
    if (p.mode == FP8KV_SCALE_PER_TOKEN_HEAD)
        return launch_columns<false, true>(p, columns, latent_map, rope_map, stream);
    return launch_columns<false, false>(p, columns, latent_map, rope_map, stream);
}

}  // namespace fp8kv
