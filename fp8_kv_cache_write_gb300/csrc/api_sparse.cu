// api_sparse.cu -- the extern "C" boundary of the calls that read part of a cache: page
// bounds, page selection and attention over the pages taken.  Every check runs before the
// first launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp8kv.h"
#include "internal.h"

namespace {

using namespace fp8kv;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_d(int D) { return D == 64 || D == 128 || D == 256; }

// Positions of a sequence fit 32 bits, a page behind the last included.
constexpr int kMaxPages = (1 << 27) - 32;
// Largest grid, in blocks or cluster ranks.
constexpr int64_t kMaxGrid = (int64_t{1} << 31) - 1;

int check_cache(int kv_dtype, int scale_mode) {
    if (kv_dtype != FP8KV_KV_E4M3 && kv_dtype != FP8KV_KV_BF16) return FP8KV_ERR_INVALID;
    if (kv_dtype == FP8KV_KV_E4M3 &&
        (scale_mode < FP8KV_SCALE_PER_TENSOR || scale_mode > FP8KV_SCALE_PER_TOKEN_HEAD))
        return FP8KV_ERR_INVALID;
    return FP8KV_OK;
}

// The scale array the mode reads is there.
bool have_scale(int kv_dtype, int mode, const float* scale, const float* scale_cache) {
    if (kv_dtype != FP8KV_KV_E4M3) return true;
    const float* s = mode == FP8KV_SCALE_PER_TOKEN_HEAD ? scale_cache : scale;
    return s != nullptr && aligned(s, 4);
}

int status(cudaError_t e) { return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA; }

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
    p.pages_per_seq = new_tokens == 0 || touched > max_blocks_per_seq ? max_blocks_per_seq
                                                                      : touched;
    // the grid has a warp for each of these
    if (static_cast<int64_t>(B) * Hkv > kMaxGrid / p.pages_per_seq) return FP8KV_ERR_UNSUPPORTED;
    p.k_scale = k_scale;
    p.k_scale_cache = k_scale_cache;
    p.mode = scale_mode;
    p.bounds = static_cast<int8_t*>(bounds);
    p.bounds_scale = bounds_scale;
    p.err = err_flag;
    return status(launch_page_bounds(p, D, kv_dtype, static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_kv_page_select(const void* q, const void* bounds, const float* bounds_scale,
                         const int32_t* block_table, int max_blocks_per_seq,
                         const int32_t* context_lens, int B, int Hq, int Hkv, int D,
                         int64_t num_blocks, int budget, int sink, int recent, int32_t* pages,
                         int32_t* counts, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq < 0 || num_blocks < 0)
        return FP8KV_ERR_INVALID;
    if (budget < 1 || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
        return FP8KV_ERR_INVALID;
    if (!valid_d(D) || Hq / Hkv > 16) return FP8KV_ERR_UNSUPPORTED;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1) return FP8KV_ERR_INVALID;
    if (max_blocks_per_seq > kSelectRanks * kSelectMaxKeys || num_blocks >= (int64_t{1} << 31) ||
        static_cast<int64_t>(B) * Hkv > kMaxGrid / kSelectRanks)
        return FP8KV_ERR_UNSUPPORTED;
    if (!q || !bounds || !bounds_scale || !block_table || !context_lens || !pages || !counts)
        return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(bounds_scale, 4) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(pages, 4) ||
        !aligned(counts, 4))
        return FP8KV_ERR_INVALID;
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
        budget > (1 << 30) || static_cast<int64_t>(B) * Hkv > kMaxGrid / 16)
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

}  // extern "C"
