// api_latent.cu -- the extern "C" boundary of the rotary cache writes, the cache
// reads and the latent cache: host-side validation, the latent attention's plan and
// its tensor maps.  Every check runs before the first launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp8kv.h"
#include "internal.h"

namespace {

using namespace fp8kv;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_d(int D) { return D == 64 || D == 128 || D == 256; }
bool valid_l(int L) { return L == 128 || L == 256 || L == 512; }

// Largest grid the row counts may ask for (blocks of at least one row each).
constexpr int64_t kMaxRows = int64_t{1} << 30;
// Longest page table of a sequence: the attention's 32-bit positions go up to two tiles of
// 128 keys behind the last, rounded up.
constexpr int kMaxPages = (1 << 27) - 32;

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

// Strides of [T][H][64] rows: multiples of 8, and no two rows overlap, be tokens outside
// heads in memory or heads outside tokens.
bool rows_apart(int64_t T, int64_t H, int64_t token, int64_t head) {
    if ((T > 1 && token % 8 != 0) || (H > 1 && head % 8 != 0)) return false;
    if (T > 1 && token < kLatentRope) return false;
    if (H > 1 && head < kLatentRope) return false;
    return T <= 1 || H <= 1 || token >= (H - 1) * head + kLatentRope ||
           head >= (T - 1) * token + kLatentRope;
}

int status(cudaError_t e) { return e == cudaSuccess ? FP8KV_OK : FP8KV_ERR_CUDA; }

// Sizes that the latent attention takes.
bool attn_sizes(int B, int S, int H, int max_blocks) {
    return B <= 65535 && H <= 65535 && S <= 65535 && static_cast<int64_t>(S) * H <= 65536 &&
           max_blocks <= kMaxPages;
}

struct LatentPlan {
    int columns, groups, rows_per_group;
    int64_t workers;
    size_t bytes;
};

// Rows of a sequence (S * H) go to ceil(rows / 64) equal groups; a worker is one
// CTA per group, and there are as many workers as fill the SMs once.
LatentPlan latent_plan(int B, int S, int H, int L, int max_blocks, int num_splits) {
    LatentPlan pl{};
    const int64_t rows = static_cast<int64_t>(S) * H;
    pl.groups = static_cast<int>((rows + 63) / 64);
    if (pl.groups < 1) pl.groups = 1;
    pl.rows_per_group = static_cast<int>((rows + pl.groups - 1) / pl.groups);
    pl.columns = pl.rows_per_group <= 16 ? 16 : pl.rows_per_group <= 32 ? 32 : 64;
    const int64_t tiles = static_cast<int64_t>(B) * ((static_cast<int64_t>(max_blocks) + 3) / 4);
    int64_t n = num_splits > 0 ? num_splits : sm_count() / pl.groups;
    if (n > tiles) n = tiles;
    if (n > 1024) n = 1024;
    if (n < 1) n = 1;
    pl.workers = n;
    pl.bytes = static_cast<size_t>(2) * n * pl.groups * pl.columns *
               (static_cast<size_t>(L) + 2) * sizeof(float);
    return pl;
}

// Tensor maps over latent rows [num_blocks][16][row_bytes].
//   panels > 0: boxes of 8 rows x `panels` 128-byte panels (the row's first panels),
//     copied panel by panel ([panel][8][128], 128-byte swizzle)
//   panels 0: boxes of 16 rows x 64 bytes (64-byte swizzle)
bool latent_map(const void* base, int row_bytes, int64_t num_blocks, int panels,
                CUtensorMap* out) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t row = static_cast<cuuint64_t>(row_bytes),
                     blocks = static_cast<cuuint64_t>(num_blocks);
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r;
    if (panels > 0) {
        const cuuint64_t dims[4] = {128, FP8KV_PAGE_SIZE, static_cast<cuuint64_t>(panels), blocks};
        const cuuint64_t strides[3] = {row, 128, row * FP8KV_PAGE_SIZE};
        const cuuint32_t boxes[4] = {128, 8, static_cast<cuuint32_t>(panels), 1};
        r = fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, boxes,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        const cuuint64_t dims[3] = {row, FP8KV_PAGE_SIZE, blocks};
        const cuuint64_t strides[2] = {row, row * FP8KV_PAGE_SIZE};
        const cuuint32_t boxes[3] = {64, FP8KV_PAGE_SIZE, 1};
        r = fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, boxes,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int fp8kv_rope_freqs(int rotary_dim, double base, int scaling, double factor,
                     double original_context, double low, double high, int64_t* freqs,
                     float* mscale) {
    clear_warning();
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || !freqs || !mscale) return FP8KV_ERR_INVALID;
    if (scaling < FP8KV_ROPE_NONE || scaling > FP8KV_ROPE_BANDS) return FP8KV_ERR_INVALID;
    if (!(base > 1.0) || !std::isfinite(base)) return FP8KV_ERR_INVALID;
    if (scaling != FP8KV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return FP8KV_ERR_INVALID;
    if (scaling == FP8KV_ROPE_NTK && rotary_dim < 4) return FP8KV_ERR_INVALID;
    const bool bands = scaling == FP8KV_ROPE_YARN || scaling == FP8KV_ROPE_BANDS;
    if (bands && (!(original_context > 0.0) || !std::isfinite(original_context) || !(low > 0.0) ||
                  !(high > low) || !std::isfinite(high)))
        return FP8KV_ERR_INVALID;
    const double pi2 = 6.283185307179586476925286766559;
    const int pairs = rotary_dim / 2;
    if (scaling == FP8KV_ROPE_NTK)
        base *= std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
    // YaRN: pairs that turn `high` times or more over the original context keep their
    // frequency, those that turn `low` times or fewer are interpolated, a linear ramp
    // over the pair index in between
    double ramp0 = 0.0, ramp1 = 1.0;
    if (scaling == FP8KV_ROPE_YARN) {
        const auto pair_of = [&](double turns) {
            return rotary_dim * std::log(original_context / (turns * pi2)) / (2.0 * std::log(base));
        };
        ramp0 = std::floor(pair_of(high));
        ramp1 = std::ceil(pair_of(low));
        ramp0 = ramp0 < 0.0 ? 0.0 : ramp0;
        ramp1 = ramp1 > rotary_dim - 1 ? rotary_dim - 1 : ramp1;
        if (ramp1 <= ramp0) ramp1 = ramp0 + 0.001;
    }
    for (int i = 0; i < pairs; ++i) {
        double t = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == FP8KV_ROPE_LINEAR) {
            t /= factor;
        } else if (scaling == FP8KV_ROPE_YARN) {
            double w = (i - ramp0) / (ramp1 - ramp0);
            w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
            t = t / factor * w + t * (1.0 - w);
        } else if (scaling == FP8KV_ROPE_BANDS) {
            const double turns = original_context * t / pi2;    // over the original context
            if (turns < low) {
                t /= factor;
            } else if (turns <= high) {
                const double w = (turns - low) / (high - low);
                t = (1.0 - w) * t / factor + w * t;
            }
        }
        freqs[i] = static_cast<int64_t>(std::llround(std::ldexp(t / pi2, 64)));
    }
    *mscale = scaling == FP8KV_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return FP8KV_OK;
}

int fp8kv_rope_kv_cache_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, const int64_t* positions,
                              const int64_t* slot_mapping, const int64_t* rope_freqs,
                              int rotary_dim, int interleaved, float mscale, int64_t T, int Hq,
                              int Hkv, int D, void* q_out, int64_t q_out_stride, void* k_cache,
                              void* v_cache, int64_t num_blocks, int kv_dtype, int scale_mode,
                              const float* k_scale, const float* v_scale, float* k_scale_cache,
                              float* v_scale_cache, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (T < 0 || Hq < 0 || Hkv <= 0 || num_blocks < 0 || !(mscale == mscale))
        return FP8KV_ERR_INVALID;
    if (!valid_d(D)) return FP8KV_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > D) return FP8KV_ERR_INVALID;
    if (rotary_dim % 16 != 0) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (Hq > 65535 || Hkv > 65535) return FP8KV_ERR_UNSUPPORTED;
    if (T > kMaxRows / (Hq + 2 * static_cast<int64_t>(Hkv))) return FP8KV_ERR_UNSUPPORTED;
    if (T == 0) return FP8KV_OK;
    if (!k || !v || !positions || !slot_mapping || !rope_freqs || !k_cache || !v_cache ||
        (Hq > 0 && (!q || !q_out)))
        return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(positions, 8) ||
        !aligned(slot_mapping, 8) || !aligned(rope_freqs, 8))
        return FP8KV_ERR_INVALID;
    const int64_t qrow = static_cast<int64_t>(Hq) * D, krow = static_cast<int64_t>(Hkv) * D;
    if (T > 1 && ((Hq > 0 && (q_stride < qrow || q_out_stride < qrow)) || k_stride < krow ||
                  v_stride < krow))
        return FP8KV_ERR_INVALID;
    if (T > 1 && (q_stride % 8 || q_out_stride % 8 || k_stride % 8 || v_stride % 8))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, k_scale, k_scale_cache) ||
        !have_scale(kv_dtype, scale_mode, v_scale, v_scale_cache))
        return FP8KV_ERR_INVALID;
    RopeWriteParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.freqs = rope_freqs;
    p.rotary_dim = rotary_dim;
    p.mscale = mscale;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.q_out_stride = q_out_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.num_blocks = num_blocks;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_scale_cache = k_scale_cache;
    p.v_scale_cache = v_scale_cache;
    p.kv_bf16 = kv_dtype == FP8KV_KV_BF16;
    p.mode = scale_mode;
    p.err = err_flag;
    return status(launch_rope_kv_cache_write(p, D, interleaved != 0,
                                             static_cast<cudaStream_t>(cuda_stream), sm_count()));
}

int fp8kv_kv_cache_read(const void* k_cache, const void* v_cache, int64_t num_blocks,
                        int kv_dtype, int scale_mode, const float* k_scale, const float* v_scale,
                        const float* k_scale_cache, const float* v_scale_cache,
                        const int64_t* slot_mapping, int64_t T, int Hkv, int D, void* k_out,
                        void* v_out, int out_dtype, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (T < 0 || Hkv <= 0 || num_blocks < 0) return FP8KV_ERR_INVALID;
    if (!valid_d(D)) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (out_dtype != FP8KV_OUT_F32 && out_dtype != FP8KV_OUT_BF16) return FP8KV_ERR_INVALID;
    if (T > kMaxRows / Hkv) return FP8KV_ERR_UNSUPPORTED;
    if (T == 0) return FP8KV_OK;
    if (!k_cache || !v_cache || !slot_mapping || !k_out || !v_out) return FP8KV_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || !aligned(slot_mapping, 8))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, k_scale, k_scale_cache) ||
        !have_scale(kv_dtype, scale_mode, v_scale, v_scale_cache))
        return FP8KV_ERR_INVALID;
    ReadParams p{};
    p.cache[0] = static_cast<const uint8_t*>(k_cache);
    p.cache[1] = static_cast<const uint8_t*>(v_cache);
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.scale_cache[0] = k_scale_cache;
    p.scale_cache[1] = v_scale_cache;
    p.mode = scale_mode;
    p.num_blocks = num_blocks;
    p.slot_mapping = slot_mapping;
    p.T = T;
    p.H = Hkv;
    p.err = err_flag;
    return status(launch_cache_read(p, 2, D, kv_dtype, out_dtype == FP8KV_OUT_F32,
                                    static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_latent_cache_write(const void* c, int64_t c_stride, const void* k_pe,
                             int64_t k_pe_stride, const int64_t* positions,
                             const int64_t* rope_freqs, int interleaved, float mscale,
                             const int64_t* slot_mapping, int64_t T, int L, void* cache,
                             int64_t num_blocks, int kv_dtype, int scale_mode, const float* scale,
                             float* scale_cache, const void* q_pe, int64_t q_stride,
                             int64_t q_head_stride, void* q_pe_out, int64_t q_out_stride,
                             int64_t q_out_head_stride, int H, int32_t* err_flag,
                             void* cuda_stream) {
    clear_warning();
    if (T < 0 || H < 0 || num_blocks < 0 || !(mscale == mscale)) return FP8KV_ERR_INVALID;
    if (!valid_l(L)) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if ((positions == nullptr) != (rope_freqs == nullptr)) return FP8KV_ERR_INVALID;
    if ((q_pe == nullptr) != (q_pe_out == nullptr) || (q_pe != nullptr && H == 0))
        return FP8KV_ERR_INVALID;
    if (H > 65535 || T > kMaxRows / (H + 1)) return FP8KV_ERR_UNSUPPORTED;
    if (T == 0) return FP8KV_OK;
    if (!c || !k_pe || !slot_mapping || !cache) return FP8KV_ERR_INVALID;
    if (!aligned(c, 16) || !aligned(k_pe, 16) || !aligned(cache, 16) || !aligned(q_pe, 16) ||
        !aligned(q_pe_out, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 8) ||
        !aligned(rope_freqs, 8))
        return FP8KV_ERR_INVALID;
    if (T > 1 && (c_stride < L || k_pe_stride < kLatentRope || c_stride % 8 || k_pe_stride % 8))
        return FP8KV_ERR_INVALID;
    if (q_pe != nullptr) {
        if (!rows_apart(T, H, q_stride, q_head_stride) ||
            !rows_apart(T, H, q_out_stride, q_out_head_stride))
            return FP8KV_ERR_INVALID;
    }
    if (!have_scale(kv_dtype, scale_mode, scale, scale_cache)) return FP8KV_ERR_INVALID;
    LatentWriteParams p{};
    p.c = static_cast<const __nv_bfloat16*>(c);
    p.k_pe = static_cast<const __nv_bfloat16*>(k_pe);
    p.c_stride = c_stride;
    p.k_pe_stride = k_pe_stride;
    p.positions = positions;
    p.freqs = rope_freqs;
    p.mscale = mscale;
    p.slot_mapping = slot_mapping;
    p.T = T;
    p.L = L;
    p.cache = static_cast<uint8_t*>(cache);
    p.num_blocks = num_blocks;
    p.kv_bf16 = kv_dtype == FP8KV_KV_BF16;
    p.mode = scale_mode;
    p.scale = scale;
    p.scale_cache = scale_cache;
    p.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
    p.q_stride = q_stride;
    p.q_head_stride = q_head_stride;
    p.q_out = static_cast<__nv_bfloat16*>(q_pe_out);
    p.q_out_stride = q_out_stride;
    p.q_out_head_stride = q_out_head_stride;
    p.H = H;
    p.err = err_flag;
    return status(launch_latent_cache_write(p, interleaved != 0,
                                            static_cast<cudaStream_t>(cuda_stream), sm_count()));
}

int fp8kv_latent_cache_read(const void* cache, int64_t num_blocks, int kv_dtype, int scale_mode,
                            const float* scale, const float* scale_cache,
                            const int64_t* slot_mapping, int64_t T, int L, void* out,
                            int out_dtype, int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (T < 0 || num_blocks < 0) return FP8KV_ERR_INVALID;
    if (!valid_l(L)) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (out_dtype != FP8KV_OUT_F32 && out_dtype != FP8KV_OUT_BF16) return FP8KV_ERR_INVALID;
    if (T > kMaxRows) return FP8KV_ERR_UNSUPPORTED;
    if (T == 0) return FP8KV_OK;
    if (!cache || !slot_mapping || !out) return FP8KV_ERR_INVALID;
    if (!aligned(cache, 16) || !aligned(out, 16) || !aligned(slot_mapping, 8))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, scale, scale_cache)) return FP8KV_ERR_INVALID;
    ReadParams p{};
    p.cache[0] = static_cast<const uint8_t*>(cache);
    p.out[0] = out;
    p.scale[0] = scale;
    p.scale_cache[0] = scale_cache;
    p.mode = scale_mode;
    p.num_blocks = num_blocks;
    p.slot_mapping = slot_mapping;
    p.T = T;
    p.H = 1;
    p.err = err_flag;
    return status(launch_cache_read(p, 1, L + kLatentRope, kv_dtype, out_dtype == FP8KV_OUT_F32,
                                    static_cast<cudaStream_t>(cuda_stream)));
}

int fp8kv_latent_attn_plan(int B, int S, int H, int L, int max_blocks_per_seq, int num_splits,
                           int* num_splits_out, size_t* workspace_bytes_out) {
    if (B < 0 || S <= 0 || H <= 0 || max_blocks_per_seq < 0 || num_splits < 0)
        return FP8KV_ERR_INVALID;
    if (!valid_l(L) || !attn_sizes(B, S, H, max_blocks_per_seq)) return FP8KV_ERR_UNSUPPORTED;
    const LatentPlan pl = latent_plan(B, S, H, L, max_blocks_per_seq, num_splits);
    if (num_splits_out) *num_splits_out = static_cast<int>(pl.workers);
    if (workspace_bytes_out) *workspace_bytes_out = pl.bytes;
    return FP8KV_OK;
}

int fp8kv_latent_decode_attn(const void* q, const void* cache, int kv_dtype, int scale_mode,
                             const float* scale, const float* scale_cache,
                             const int32_t* block_table, int max_blocks_per_seq,
                             const int32_t* context_lens, int B, int S, int H, int L,
                             int64_t num_blocks, float softmax_scale, int num_splits,
                             void* workspace, size_t workspace_bytes, void* out, int out_dtype,
                             int32_t* err_flag, void* cuda_stream) {
    clear_warning();
    if (B < 0 || S <= 0 || H <= 0 || num_splits < 0 || max_blocks_per_seq < 0 || num_blocks < 0)
        return FP8KV_ERR_INVALID;
    if (!valid_l(L)) return FP8KV_ERR_UNSUPPORTED;
    if (const int st = check_cache(kv_dtype, scale_mode)) return st;
    if (out_dtype != FP8KV_OUT_F32 && out_dtype != FP8KV_OUT_BF16) return FP8KV_ERR_INVALID;
    // a NaN scale means nothing, a zero or negative one is not a softmax over q . k,
    // an infinite one (also in binades, as the kernel takes it) has no finite logits
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!(softmax_scale > 0.f) || !std::isfinite(scale_log2)) return FP8KV_ERR_INVALID;
    if (B == 0) return FP8KV_OK;
    if (max_blocks_per_seq < 1 || num_blocks < 1) return FP8KV_ERR_INVALID;
    if (!attn_sizes(B, S, H, max_blocks_per_seq) || num_blocks >= (int64_t{1} << 31))
        return FP8KV_ERR_UNSUPPORTED;
    if (!q || !cache || !block_table || !context_lens || !out) return FP8KV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(context_lens, 4))
        return FP8KV_ERR_INVALID;
    if (!have_scale(kv_dtype, scale_mode, scale, scale_cache)) return FP8KV_ERR_INVALID;
    const LatentPlan pl = latent_plan(B, S, H, L, max_blocks_per_seq, num_splits);
    if (!workspace || workspace_bytes < pl.bytes) return FP8KV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FP8KV_ERR_INVALID;
    // bf16 rows are panels throughout; e4m3's shared key is half a panel, with a map
    // of its own
    const bool bf16 = kv_dtype == FP8KV_KV_BF16;
    const int row_bytes = (L + kLatentRope) * (bf16 ? 2 : 1);
    CUtensorMap lm, rm;
    if (!latent_map(cache, row_bytes, num_blocks, bf16 ? row_bytes / 128 : L / 128, &lm) ||
        (!bf16 && !latent_map(cache, row_bytes, num_blocks, 0, &rm)))
        return FP8KV_ERR_CUDA;
    if (bf16) rm = lm;
    LatentAttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.scale = scale;
    p.scale_cache = scale_cache;
    p.block_table = block_table;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.B = B;
    p.S = S;
    p.H = H;
    p.L = L;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale_log2;
    p.mode = scale_mode;
    p.groups = pl.groups;
    p.rows_per_group = pl.rows_per_group;
    p.workers = static_cast<int>(pl.workers);
    const size_t slots = static_cast<size_t>(2) * pl.workers * pl.groups * pl.columns;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_m = p.ws_o + slots * L;
    p.ws_l = p.ws_m + slots;
    p.out = out;
    p.out_bf16 = out_dtype == FP8KV_OUT_BF16;
    p.err = err_flag;
    return status(launch_latent_attn(p, pl.columns, kv_dtype, lm, rm,
                                     static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
