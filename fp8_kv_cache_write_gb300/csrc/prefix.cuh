// prefix.cuh -- how a shared prefix's (row tile, key tile) units are dealt to CTAs: what
// prefix_attn.cu computes by and list_attn.cu finds the pieces of a row by.
#pragma once

#include <stdint.h>

namespace fp8kv {

constexpr int kPrefixRows = 128;             // query rows of a tile

// Keys of a tile: 128, or 64 where a tile of 128 would not leave room for two.
__host__ __device__ constexpr int prefix_keys(int D) { return D == 256 ? 64 : 128; }

// `units` row tiles of `tiles` key tiles each, flattened, in `workers` equal shares: worker w
// takes [w W / n, (w + 1) W / n).  Pieces of a unit go to consecutive workers.
struct PrefixShares {
    int tiles;
    int64_t total, workers;
    __host__ __device__ PrefixShares(int len, int keys, int64_t units, int64_t grid) {
        tiles = len > 0 ? (len - 1) / keys + 1 : 0;
        total = units * tiles;
        workers = total < grid ? total : grid;
    }
    __host__ __device__ int64_t begin(int64_t w) const {
        return workers > 0 ? w * total / workers : 0;
    }
    // the worker that holds tile t
    __host__ __device__ int64_t holder(int64_t t) const { return ((t + 1) * workers - 1) / total; }
    // first worker and number of pieces of unit u (tiles > 0)
    __host__ __device__ int64_t first(int64_t u) const { return holder(u * tiles); }
    __host__ __device__ int pieces(int64_t u) const {
        return static_cast<int>(holder((u + 1) * tiles - 1) - first(u)) + 1;
    }
};

// Pieces a unit can have at most: a unit's tiles span at most ceil(n / units) share borders.
__host__ __device__ constexpr int64_t prefix_splits(int64_t units, int64_t grid) {
    return (grid + units - 1) / units + 1;
}

}  // namespace fp8kv
