// rope.cuh -- rotary positions in registers: exact angles from 64-bit fixed-point
// frequencies, and the rotation of the 16 values one lane owns.
#pragma once

#include "common.cuh"

namespace fp8kv {

// A row's first `rotary_dim` values form rotary_dim / 2 pairs; pair i turns by
// position * theta_i.  The table holds F_i = 2^64 theta_i / 2 pi (turns per
// position in 2^-64ths), so the low 64 bits of position * F_i are the angle's
// fraction of a turn: whole turns drop out of the product by themselves, and the
// only error is that of F_i (from doubles: 2^-52 of it) times the position, under 2^-30
// turns at position 2^24 and 2^-14 at 2^40.  fp32 angles would be off by 2^-24 of the
// angle itself, a radian at position 2^24.  The fraction's top 32 bits, taken signed,
// are an angle in [-1/2, 1/2) turns; in fp32 that is exact to 2^-26 turns.
__device__ __forceinline__ float2 rope_cos_sin(int64_t position, int64_t freq) {
    const uint64_t turns = static_cast<uint64_t>(position) * static_cast<uint64_t>(freq);
    const float t = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(t, &s, &c);                    // of pi * t = 2 pi * turns
    return make_float2(c, s);
}

// One lane's 16 values of a row: two groups of 8, at element offsets a and b.
//   rotated, half layout   [8u, 8u + 8) and their partners [rd/2 + 8u, ...)
//   rotated, interleaved   [16u, 16u + 16): pairs of neighbours
//   behind the rotated part, both layouts: [16u, 16u + 16)
// so a rotated lane u always holds pairs 8u .. 8u + 7.
struct RopeUnit {
    int a, b;
    bool turns;
};

template <bool INTERLEAVED>
__device__ __forceinline__ RopeUnit rope_unit(int u, int rotary_dim) {
    RopeUnit r;
    r.turns = u < rotary_dim / 16;
    if (!INTERLEAVED && r.turns) {
        r.a = 8 * u;
        r.b = rotary_dim / 2 + 8 * u;
    } else {
        r.a = 16 * u;
        r.b = 16 * u + 8;
    }
    return r;
}

// Cosines and sines of a lane's 8 pairs, two pairs to a register pair.
struct RopeAngles {
    uint64_t c[4], s[4], ns[4];              // ns = -s
    __device__ __forceinline__ void set(int e, float2 a, float2 b) {   // pairs 2e, 2e + 1
        c[e] = pack_f32x2(a.x, b.x);
        s[e] = pack_f32x2(a.y, b.y);
        ns[e] = pack_f32x2(-a.y, -b.y);
    }
};

// Turns the pairs of f (group a in f[0..8), group b in f[8..16)); any magnitude is
// already folded into the angles.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_turn(float (&f)[16], const RopeAngles& an) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float& x0 = INTERLEAVED ? f[4 * e] : f[2 * e];
        float& y0 = INTERLEAVED ? f[4 * e + 1] : f[8 + 2 * e];
        float& x1 = INTERLEAVED ? f[4 * e + 2] : f[2 * e + 1];
        float& y1 = INTERLEAVED ? f[4 * e + 3] : f[8 + 2 * e + 1];
        const uint64_t x = pack_f32x2(x0, x1), y = pack_f32x2(y0, y1);
        const float2 tx = unpack_f32x2(fma_f32x2(y, an.ns[e], mul_f32x2(x, an.c[e])));
        const float2 ty = unpack_f32x2(fma_f32x2(x, an.s[e], mul_f32x2(y, an.c[e])));
        x0 = tx.x;
        x1 = tx.y;
        y0 = ty.x;
        y1 = ty.y;
    }
}

// cos and sin of the 8 pairs of unit lane % U at `position`, for a warp of
// 32 / U rows with the same position: each of the rows' lanes computes a share
// and the shares meet in shuffles.  Every lane of the warp calls it.
template <int U>
__device__ __forceinline__ void rope_share(RopeAngles& an, int64_t position,
                                           const int64_t* freqs, int rotary_dim, float mscale,
                                           int lane) {
    constexpr int kRows = 32 / U;
    constexpr int kEach = kRows >= 8 ? 1 : 8 / kRows;
    const int u = lane % U, g = lane / U;
    float2 mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        mine[i] = make_float2(1.f, 0.f);
        const int e = g * kEach + i;
        if (u < rotary_dim / 16 && e < 8) {
            mine[i] = rope_cos_sin(position, freqs[8 * u + e]);
            mine[i].x *= mscale;
            mine[i].y *= mscale;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float2 m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int src = (e + i) / kEach * U + u;
            m[i].x = __shfl_sync(0xffffffffu, mine[(e + i) % kEach].x, src);
            m[i].y = __shfl_sync(0xffffffffu, mine[(e + i) % kEach].y, src);
        }
        an.set(e / 2, m[0], m[1]);
    }
}

__device__ __forceinline__ void unpack_bf16x8(uint4 x, float* f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_bits_to_float(w[i] & 0xffffu);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// e4m3 codes of fp32(f / s) for a lane's 16 values: group a in codes[0..1], group
// b in codes[2..3].  Values the certified multiplies reject take the IEEE divide
// (e4m3_codes_by_multiply); a zero scale gives code 0.  (Exact quotients by two remainder
// steps, no pair ever redone, need fewer instructions but in one dependent chain: the
// rotary write of 32768 tokens 123 -> 135 us, the latent write 35.5 -> 34.1.)
__device__ __forceinline__ void e4m3_codes16(const float (&f)[16], float s, uint32_t (&codes)[4]) {
    codes[0] = codes[1] = codes[2] = codes[3] = 0u;
    if (s == 0.0f) return;
    const uint32_t redo = e4m3_codes_by_multiply(f, s, codes);
    if (redo) {
#pragma unroll
        for (int i = 0; i < 8; ++i)          // constant register indexes
            if ((redo >> i) & 1u) {
                const uint32_t c = e4m3x2_by_divide(f[2 * i], f[2 * i + 1], s);
                codes[i >> 1] = (i & 1) ? (codes[i >> 1] & 0x0000ffffu) | (c << 16)
                                        : (codes[i >> 1] & 0xffff0000u) | c;
            }
    }
}

}  // namespace fp8kv
