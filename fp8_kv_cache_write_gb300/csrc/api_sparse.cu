// api_sparse.cu -- the extern "C" boundary of the calls that read part of a cache: page
// bounds, page selection, attention over the pages taken, and attention behind a shared
// prefix with its plan.  Every check runs before the first launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp8kv.h"
#include "internal.h"
#include "prefix.cuh"

namespace {

using namespace fp8kv;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_d(int D) { return D == 64 || D == 128 || D == 256; }

// Positions of a sequence fit 32 bits, a page behind the last included.
constexpr int kMaxPages = (1 << 27) - 32;
// Entries of a list: counted in 31 bits, a CTA's stride behind the last included.
constexpr int kMaxBudget = 1 << 30;
// Largest grid, in blocks or cluster ranks.
constexpr int64_t kMaxGrid = (int64_t{1} << 31) - 1;

int check_cache(int kv_dtype, int scale_mode) {
    if (kv_dtype != FP8KV_KV_E4M3 && kv_dtype != FP8KV_KV_BF16) return FP8KV_ERR_INVALID;
    if (kv_dtype == FP8KV_KV_E4M3 &&
        (scale_mode < FP8KV_SCALE_PER_TENSOR || scale_mode > FP8KV_SCALE_PER_TOKEN_HEAD))
        return FP8KV_ERR_INVALID;
    return FP8KV_OK;
}

// The scale array the mode reads is there; a page's per-token scales are read 16 bytes at a time.
bool have_scale(int kv_dtype, int mode, const float* scale, const float* scale_cache) {
    if (kv_dtype != FP8KV_KV_E4M3) return true;
    if (mode == FP8KV_SCALE_PER_TOKEN_HEAD) return scale_cache != nullptr && aligned(scale_cache, 16);
    return scale != nullptr && aligned(scale, 4);
}

int status(cudaError_t e) { return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA; }

// Workspace of the page selection: a 32-bit key a page and head.  False: more (sequence, head)
// pairs or pages than its grids and 32-bit indexes hold.
bool select_bytes(int B, int Hkv, int max_blocks, size_t* bytes) {
    const int64_t units = static_cast<int64_t>(B) * Hkv;
    if (max_blocks > kMaxPages || units > kMaxGrid / (max_blocks / 512 + 1)) return false;
    *bytes = static_cast<size_t>(units) * static_cast<size_t>(max_blocks) * 4;
    return true;
}

// How the prefix part of a call is dealt: one persistent CTA per SM, or one per tile where
// there are fewer; a row's partials in splits slots of the workspace.
struct PrefixPlan {
    int row_tiles, workers;
    int64_t units, splits;
    size_t rows, bytes;
};

PrefixPlan prefix_plan(int B, int Hq, int Hkv, int D, int prefix_pages) {
    PrefixPlan pl{};
    const int64_t R = static_cast<int64_t>(B) * (Hq / Hkv);
    const int per_tile = prefix_keys(D) / FP8KV_PAGE_SIZE;
    const int64_t tiles = (static_cast<int64_t>(prefix_pages) + per_tile - 1) / per_tile;
    pl.row_tiles = static_cast<int>((R + kPrefixRows - 1) / kPrefixRows);
    pl.units = static_cast<int64_t>(pl.row_tiles) * Hkv;
    const int64_t sms = sm_count();
    pl.workers = static_cast<int>(tiles < 1 || pl.units < 1 ? 1
                                  : tiles > sms / pl.units ? sms
                                                           : pl.units * tiles);
    pl.splits = prefix_splits(pl.units < 1 ? 1 : pl.units, pl.workers);
    pl.rows = static_cast<size_t>(R) * Hkv * pl.splits;
    pl.bytes = pl.rows * (static_cast<size_t>(D) + 2) * sizeof(float);
    return pl;
}

// Sizes the prefix call takes: rows of a head and row tiles within 32 bits, the tail's grid
// (two groups of query heads a KV head, clusters of 8) within a launch's, a CTA's share of the
// (row tile, key tile) pairs within 31 bits.
bool prefix_sizes(int B, int Hq, int Hkv, int prefix_pages, int max_blocks) {
    const int64_t rows = static_cast<int64_t>(B) * Hq;
    return rows <= (int64_t{1} << 26) && Hq / Hkv <= 16 && prefix_pages <= kMaxPages &&
           max_blocks <= kMaxPages &&
           (rows / kPrefixRows + Hkv) <= (int64_t{1} << 36) / (prefix_pages / 4 + 1);
}

// Tensor map over a cache's tiles [num_blocks * Hkv][16][row_bytes]: boxes of 16 rows x 128
// bytes (64-byte rows: whole), swizzled as wide as the box.
bool tile_map(const void* base, int row_bytes, int64_t tiles, CUtensorMap* out) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(row_bytes);
    const cuuint64_t dims[3] = {row, FP8KV_PAGE_SIZE, static_cast<cuuint64_t>(tiles)};
    const cuuint64_t strides[2] = {row, row * FP8KV_PAGE_SIZE};
    const cuuint32_t box[3] = {row_bytes == 64 ? 64u : 128u, FP8KV_PAGE_SIZE, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int fp8kv_kv_page_bounds(const void* k_cache, int kv_dtype, int scale_mode, const float* k_scale,
                         const float* k_scale_cache, const int32_t* block_table,
                         int max_blocks_per_seq, const int32_t* context_lens, int B, int Hkv,
                         int D, int64_t num_blocks, int new_tokens, void* bounds,
                         float* bounds_scale, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (B < 0 || Hkv <= 0 || max_blocks_per_seq < 0 || num_blocks < 0 || new_tokens < 0)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D)) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1) return FP8KV_ERR_INVALID;
    if (max_blocks_per_seq > kMaxPages || num_blocks >= (int64_t{1} << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (!k_cache || !block_table || !context_lens || !bounds || !bounds_scale)
        return FP8KV_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(bounds_scale, 4) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, k_scale, k_scale_cache)) return FP8KV_ERR_INVALID;
    PageBoundsParams p{};
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.block_table = block_table;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.B = B;
    p.Hkv = Hkv;
    p.num_blocks = num_blocks;
    p.new_tokens = new_tokens;
    // new_tokens positions reach over at most this many pages, wherever they start
    const int64_t touched = (static_cast<int64_t>(new_tokens) + FP8KV_PAGE_SIZE - 2) /
                                FP8KV_PAGE_SIZE + 1;
    p.pages_per_seq = static_cast<unsigned>(
        new_tokens == 0 || touched > max_blocks_per_seq ? max_blocks_per_seq : touched);
    // (sequence, page, head) items are counted in 31 bits
    if (static_cast<int64_t>(B) * Hkv > kMaxGrid / p.pages_per_seq) return FP8KV_ERR_UNSUPPORTED;
    p.k_scale = k_scale;
    p.k_scale_cache = k_scale_cache;
    p.mode = scale_mode;
    p.bounds = static_cast<int8_t*>(bounds);
    p.bounds_scale = bounds_scale;
    p.err = err_flag;
    return status(launch_page_bounds(p, D, kv_dtype, static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_kv_page_select_workspace_bytes(int B, int Hkv, int max_blocks_per_seq, size_t* bytes) {
    if (B < 0 || Hkv <= 0 || max_blocks_per_seq < 0 || !bytes) return FP8KV_ERR_INVALID;
    return select_bytes(B, Hkv, max_blocks_per_seq, bytes) ? FP8KV_OK : FP8KV_ERR_UNSUPPORTED;
}

int fp8kv_kv_page_select(const void* q, const void* bounds, const float* bounds_scale,
                         const int32_t* block_table, int max_blocks_per_seq,
                         const int32_t* context_lens, int B, int Hq, int Hkv, int D,
                         int64_t num_blocks, int budget, int sink, int recent, void* workspace,
                         size_t workspace_bytes, int32_t* pages, int32_t* counts,
                         int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq < 0 || num_blocks < 0)
        return FP8KV_ERR_INVALID;
    if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D) || Hq / Hkv > 16) return FP8KV_ERR_UNSUPPORTED;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1) return FP8KV_ERR_INVALID;
    size_t need = 0;
    if (num_blocks >= (int64_t{1} << 31) || budget > kMaxBudget ||
        !select_bytes(B, Hkv, max_blocks_per_seq, &need))
        return FP8KV_ERR_UNSUPPORTED;
    if (!q || !bounds || !bounds_scale || !block_table || !context_lens || !pages || !counts)
        return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(bounds_scale, 4) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(pages, 4) ||
        !aligned(counts, 4))
        return FP8KV_ERR_INVALID;
    if (!workspace || workspace_bytes < need) return FP8KV_ERR_WORKSPACE;
    if (!aligned(workspace, 4)) return FP8KV_ERR_INVALID;
    PageSelectParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.bounds = static_cast<const int8_t*>(bounds);
    p.bounds_scale = bounds_scale;
    p.block_table = block_table;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.num_blocks = num_blocks;
    p.budget = budget;
    p.sink = sink;
    p.recent = recent;
    p.pages = pages;
    p.counts = counts;
    p.keys = static_cast<uint32_t*>(workspace);
    p.err = err_flag;
    return status(launch_page_select(p, D, static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_sparse_decode_attn(const void* q, const void* k_cache, const void* v_cache,
                             int kv_dtype, int scale_mode, const float* k_scale,
                             const float* v_scale, const float* k_scale_cache,
                             const float* v_scale_cache, const int32_t* block_table,
                             int max_blocks_per_seq, const int32_t* context_lens,
                             const int32_t* pages, const int32_t* counts, int budget, int B,
                             int Hq, int Hkv, int D, int64_t num_blocks, float softmax_scale,
                             void* out, int out_dtype, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq < 0 ||
        num_blocks < 0 || budget < 1)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D) || Hq / Hkv > 16) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (out_dtype != FP8KV_OUT_F32 && out_dtype != FP8KV_OUT_BF16) return FP8KV_ERR_INVALID;
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!(softmax_scale > 0.f) || !std::isfinite(scale_log2)) return FP8KV_ERR_INVALID;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1) return FP8KV_ERR_INVALID;
    // (two groups of 8 query heads at most, clusters of 8)
    if (max_blocks_per_seq > kMaxPages || num_blocks >= (int64_t{1} << 31) ||
        budget > kMaxBudget || static_cast<int64_t>(B) * Hkv > kMaxGrid / 16)
        return FP8KV_ERR_UNSUPPORTED;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !pages || !out)
        return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(pages, 4) ||
        !aligned(counts, 4))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, k_scale, k_scale_cache) ||
        !have_scale(kv_dtype, scale_mode, v_scale, v_scale_cache))
        return FP8KV_ERR_INVALID;
    ListAttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_scale_cache = k_scale_cache;
    p.v_scale_cache = v_scale_cache;
    p.scale_mode = scale_mode;
    p.block_table = block_table;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale_log2;
    p.pages = pages;
    p.counts = counts;
    p.budget = budget;
    p.out = out;
    p.out_bf16 = out_dtype == FP8KV_OUT_BF16;
    p.err = err_flag;
    return status(launch_list_attn(p, D, kv_dtype, static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_prefix_attn_plan(int B, int Hq, int Hkv, int D, int prefix_pages, int* workers_out,
                           size_t* workspace_bytes_out) {
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || prefix_pages < 0)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D) || !prefix_sizes(B, Hq, Hkv, prefix_pages, 0)) return FP8KV_ERR_UNSUPPORTED;
    const PrefixPlan pl = prefix_plan(B, Hq, Hkv, D, prefix_pages);
    if (workers_out) *workers_out = pl.workers;
    if (workspace_bytes_out) *workspace_bytes_out = pl.bytes;
    return FP8KV_OK;
}

int fp8kv_prefix_decode_attn(const void* q, const void* k_cache, const void* v_cache,
                             int kv_dtype, int scale_mode, const float* k_scale,
                             const float* v_scale, const float* k_scale_cache,
                             const float* v_scale_cache, const int32_t* prefix_table,
                             int prefix_pages, const int32_t* prefix_len,
                             const int32_t* block_table, int max_blocks_per_seq,
                             const int32_t* context_lens, int B, int Hq, int Hkv, int D,
                             int64_t num_blocks, float softmax_scale, void* workspace,
                             size_t workspace_bytes, void* out, int out_dtype, int32_t* err_flag,
                             void* cuda_stream) {
    clear_warning();
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq < 0 ||
        num_blocks < 0 || prefix_pages < 0)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D) || !prefix_sizes(B, Hq, Hkv, prefix_pages, max_blocks_per_seq))
        return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (out_dtype != FP8KV_OUT_F32 && out_dtype != FP8KV_OUT_BF16) return FP8KV_ERR_INVALID;
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!(softmax_scale > 0.f) || !std::isfinite(scale_log2)) return FP8KV_ERR_INVALID;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1 || prefix_pages < 1) return FP8KV_ERR_INVALID;
    // (block, head) tiles are a 32-bit coordinate of the tensor copies
    if (num_blocks > kMaxGrid / Hkv) return FP8KV_ERR_UNSUPPORTED;
    if (!q || !k_cache || !v_cache || !prefix_table || !prefix_len || !block_table ||
        !context_lens || !out)
        return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(prefix_table, 4) || !aligned(prefix_len, 4) || !aligned(block_table, 4) ||
        !aligned(context_lens, 4))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, k_scale, k_scale_cache) ||
        !have_scale(kv_dtype, scale_mode, v_scale, v_scale_cache))
        return FP8KV_ERR_INVALID;
    const PrefixPlan pl = prefix_plan(B, Hq, Hkv, D, prefix_pages);
    if (!workspace || workspace_bytes < pl.bytes) return FP8KV_ERR_WORKSPACE;
    if (!aligned(workspace, 32)) return FP8KV_ERR_INVALID;   // (partials are stored 32 bytes at a time)
    const int row_bytes = D * (kv_dtype == FP8KV_KV_BF16 ? 2 : 1);
    CUtensorMap km;
    if (!tile_map(k_cache, row_bytes, num_blocks * Hkv, &km)) return FP8KV_ERR_CUDA;
    CUtensorMap vm = km;                                     // (e4m3 values come by plain bulk copies)
    if (kv_dtype == FP8KV_KV_BF16 && !tile_map(v_cache, row_bytes, num_blocks * Hkv, &vm))
        return FP8KV_ERR_CUDA;
    float* const part_o = static_cast<float*>(workspace);
    float* const part_m = part_o + pl.rows * D;
    PrefixAttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_scale_cache = k_scale_cache;
    p.v_scale_cache = v_scale_cache;
    p.scale_mode = scale_mode;
    p.prefix_table = prefix_table;
    p.prefix_pages = prefix_pages;
    p.prefix_len = prefix_len;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale_log2;
    p.row_tiles = pl.row_tiles;
    p.units = pl.units;
    p.workers = pl.workers;
    p.splits = static_cast<int>(pl.splits);
    p.part_o = part_o;
    p.part_m = part_m;
    p.part_l = part_m + pl.rows;
    p.err = err_flag;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (const int st = status(launch_prefix_attn(p, km, vm, D, kv_dtype, stream))) return st;
    ListAttnParams a{};
    a.q = p.q;
    a.k_cache = p.k_cache;
    a.v_cache = p.v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_scale_cache = k_scale_cache;
    a.v_scale_cache = v_scale_cache;
    a.scale_mode = scale_mode;
    a.block_table = block_table;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = p.G;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale_log2;
    a.pre_o = p.part_o;
    a.pre_m = p.part_m;
    a.pre_l = p.part_l;
    a.splits = p.splits;
    a.prefix_len = prefix_len;
    a.prefix_pages = prefix_pages;
    a.row_tiles = p.row_tiles;
    a.units = p.units;
    a.workers = p.workers;
    a.out = out;
    a.out_bf16 = out_dtype == FP8KV_OUT_BF16;
    a.err = err_flag;
    return status(launch_list_attn(a, D, kv_dtype, stream));
}

}  // extern "C"
