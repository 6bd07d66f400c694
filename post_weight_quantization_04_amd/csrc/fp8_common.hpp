// Shared device helpers of the 8-bit operators (e4m3 values, one float32 scale
// per block of 128): element loads of the three input types, the block scale
// and the conversion to e4m3.
#pragma once

#include "common.hpp"

namespace gptq {

typedef __bf16 bf16_t;
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef int int8v __attribute__((ext_vector_type(8)));

constexpr int kF8Block = 128;                  // channels (and weight rows) per scale
constexpr float kF8Max = 448.0f;               // largest e4m3 value
constexpr uint32_t kF8FloorBits = 0x0F800000u; // 2^-96: peak assumed for a block of (near) zeros,
                                               // so that its scale and the scale's reciprocal stay finite

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(half_t v) { return (float)v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return (float)v; }

// v[0..8) = p[0..8) as float32, zeros from index `valid` on.  kVec: p is
// 16-byte aligned and valid is 8 or <= 0.  Otherwise p has its type's
// alignment, which global memory's wide loads take as well (a little slower),
// and eight values are loaded at once all the same: 10026 rows of 2018 float32
// normed in 22.7 us, 73 us element by element; only a row's last few values go
// one by one.  kOnce: the data is not kept in the caches (nontemporal).
template <typename T, bool kVec, bool kOnce = false>
__device__ __forceinline__ void load8(float (&v)[8], const T* __restrict__ p, int64_t valid) {
    constexpr int kPieces = (int)sizeof(T) / 2;
    T raw[8];
    if (valid >= 8) {
        if (kVec) {
            const uint4v* src = reinterpret_cast<const uint4v*>(p);
            uint4v* dst = reinterpret_cast<uint4v*>(raw);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) dst[i] = kOnce ? __builtin_nontemporal_load(src + i) : src[i];
        } else {
            __builtin_memcpy(raw, p, sizeof(raw));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = (T)0.0f;
        if (!kVec)
            for (int e = 0; e < (int)valid; ++e) {
                const T x = p[e];
#pragma unroll
                for (int k = 0; k < 8; ++k) raw[k] = k == e ? x : raw[k];
            }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(raw[e]);
}

// p[0..8) = v[0..8) rounded to T (nearest even), only the first `valid`.
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* __restrict__ p, const float (&v)[8], int64_t valid) {
    constexpr int kPieces = (int)sizeof(T) / 2;
    T raw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) raw[e] = (T)v[e];
    if (valid >= 8) {
        if (kVec) {
            const uint4v* src = reinterpret_cast<const uint4v*>(raw);
            uint4v* dst = reinterpret_cast<uint4v*>(p);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) dst[i] = src[i];
        } else {
            __builtin_memcpy(p, raw, sizeof(raw));
        }
    } else if (!kVec) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < valid) p[e] = raw[e];
    }
}

// |v| as bits: they order like the values, with infinity above every finite
// value and NaN above infinity, so an unsigned maximum carries both along.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t peak8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(v[e]));
    return m;
}

// Maximum over the 16 lanes of a DPP row, in every lane of it.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // row_ror:8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));  // row_ror:4
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));  // row_ror:2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));  // row_ror:1
    return v;
}

// Scale of a block with the given peak: max(peak, 2^-96) / 448.  A block that
// holds an infinity or a NaN gets an infinite or NaN scale, so that every
// value of it stands for NaN.
__device__ __forceinline__ float f8_scale(uint32_t peak_bits) {
    return __builtin_bit_cast(float, max(peak_bits, kF8FloorBits)) / kF8Max;
}

// Four e4m3 codes of v * inv, nearest even.  |v| * inv is at most
// 448 (1 + 2^-22), far below 464 where rounding would leave the format.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

__device__ __forceinline__ uint2v f8_pack8(const float (&v)[8], float inv) {
    uint2v r;
    r.x = f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    r.y = f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    return r;
}

}  // namespace gptq
