// Shared device helpers of the attention kernels: MFMA on the two 16-bit types,
// transposed reads from LDS, the online softmax.
#pragma once

#include "fp8_common.hpp"

namespace gptq {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896f;
constexpr float kLowest = -__FLT_MAX__;  // a row's maximum before its first key

// Vector types and MFMA of the two input types.  Operands as in common.hpp;
// 16x16x16: A[i][k] from lane i + 16 kg with k = 4 kg .. 4 kg + 3.
template <typename T>
struct Mat;
template <>
struct Mat<half_t> {
    typedef half8 v8;
    typedef half4 v4;
    static __device__ __forceinline__ float4v mfma16(v8 a, v8 b, float4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float4v mfma16h(v4 a, v4 b, float4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float16v mfma32(v8 a, v8 b, float16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mat<bf16_t> {
    typedef bf16x8 v8;
    typedef bf16x4 v4;
    static __device__ __forceinline__ float4v mfma16(v8 a, v8 b, float4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float4v mfma16h(v4 a, v4 b, float4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4v, a), __builtin_bit_cast(short4v, b),
                                                         c, 0, 0, 0);
    }
    static __device__ __forceinline__ float16v mfma32(v8 a, v8 b, float16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// Four rows by sixteen columns of 16-bit values, turned: lane i of sixteen points
// at columns 4 (i % 4) .. of row i / 4 and receives column i of the four rows.
typedef __attribute__((address_space(3))) short4v lds_short4;
template <typename T>
__device__ __forceinline__ typename Mat<T>::v4 read_turned(const uint8_t* p) {
    return __builtin_bit_cast(typename Mat<T>::v4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)p));
}

// Where chunk c (sixteen bytes) of row r lies in its row of LDS, kDp values long.
// Keys are read by rows: sixteen lanes, sixteen rows, one chunk.  Values are read
// turned: eight rows of two chunks at a time.  Either way the sixteen chunks
// cover all banks.
template <int kDp>
__device__ __forceinline__ int key_place(int r, int c) {
    return c ^ (kDp == 128 ? r % 16 : r / 2 % 8);
}
template <int kDp>
__device__ __forceinline__ int value_place(int r, int c) {
    return c ^ (kDp == 128 ? r % 8 * 2 : r / 2 % 4 * 2);
}

typedef __attribute__((address_space(3))) void lds_void;

// Values of the other half of the wave (lane ^ 32) beside one's own.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float add_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// exp2 of the hardware (one unit in the last place, results below 2^-126 are
// zero: such weights are below half a unit of any sum they join).
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// -m * c for the exponent fma(s, c, .), kept finite so that a masked score of
// -infinity stays one.
__device__ __forceinline__ float exponent_offset(float m, float c) { return fminf(-m * c, __FLT_MAX__); }

// exponent_offset is rounded: the largest exponent of a row comes out as what that left
// over in place of zero.  It multiplies all of the row's weights alike and goes out with
// the division, as long as they stay within their type and the row's maximum where it is.
// Up to exponents of 2^14 it is at most 2^-11, less than a score of that size is rounded
// by; at 2^33 it is hundreds.
constexpr float kFarExponent = 0x1p14f;

// Weights go into the second product as 16-bit numbers.  float16 has full steps from
// 2^-14 and nothing below 2^-25, but goes up to 2^15.99: its weights are raised by 2^15,
// or, beside a maximum that may lag behind by kLag, by as much less; sums and parts
// with them, so that the division takes it out again.  (Without it a long flat tail 17
// nats below one key lost up to all of its weight in the product and none in the sum.)
constexpr float kLag = 4.0f;
template <typename T>
__device__ constexpr float raised(float lag) {
    return __is_same(T, half_t) ? 15.0f - lag : 0.0f;
}

}  // namespace gptq
