// Shared device helpers of the products with packed few-bit weights: loads of a
// lane's run of 32 codes, its conversion to 16-bit whole numbers q - z, and the
// epilogue.
#pragma once

#include "attention_common.hpp"
#include "kernels.hpp"

namespace gptq {

constexpr int kPmBlock = 128;              // codes of a row that a step takes
constexpr uint32_t kPmOut = 0x80000000u;   // an offset past every buffer: the load returns zero

struct PmArgs {
    PackedProduct c;
    int nw, ng, nb;                          // words and groups of a row, blocks of 128
    uint32_t group, group_mul, group_shift;  // the group's size (a whole row for 0), and division by it
    int vec;                                 // rows of x start 16-byte aligned and hold whole chunks of eight
    int y32;                                 // results, bias and residual in float32, else in x's type
    unsigned mt, nt;                         // tiles along the weight rows and the tokens
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t pm_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// Group of column k; columns behind the last belong to the last.
__device__ __forceinline__ uint32_t group_of(const PmArgs& a, uint32_t k) {
    k = min(k, (uint32_t)a.c.K - 1u);
    const uint32_t t = __umulhi(a.group_mul, k);
    return a.group_shift ? (t + ((k - t) >> 1)) >> (a.group_shift - 1) : k;
}

// The words of 32 codes at byte offset off + base of a buffer.  (The range check is
// each word's own, so a run that passes the matrix's end brings what is left of
// it and zeros.)
template <int kBits>
__device__ __forceinline__ void load_run(uint32_t (&w)[kBits], __amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t base) {
    if constexpr (kBits >= 4) {
        const uint4v v = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(r, off, base, 0));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    constexpr int kRest = kBits % 4, kAt = kBits / 4 * 4;
    if constexpr (kBits == 8) {
        const uint4v v = __builtin_bit_cast(uint4v, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, base, 0));
        w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
    } else if constexpr (kRest == 3) {
        typedef uint32_t uint3v __attribute__((ext_vector_type(3)));
        const uint3v v = __builtin_bit_cast(uint3v, __builtin_amdgcn_raw_buffer_load_b96(r, off + 4 * kAt, base, 0));
        w[kAt] = v.x, w[kAt + 1] = v.y, w[kAt + 2] = v.z;
    } else if constexpr (kRest == 2) {
        const uint2v v = __builtin_bit_cast(uint2v, __builtin_amdgcn_raw_buffer_load_b64(r, off + 4 * kAt, base, 0));
        w[kAt] = v.x, w[kAt + 1] = v.y;
    } else if constexpr (kRest == 1) {
        w[kAt] = __builtin_amdgcn_raw_buffer_load_b32(r, off + 4 * kAt, base, 0);
    }
}

// Codes 2 i and 2 i + 1 of a run as q - z, in one word.  Both are at most 255, so
// the differences are exact in either type.
//
// float16: under the exponent of 1024 the ten fraction bits are a whole number.  A
// pair's bytes go to both halves of a word (one byte permutation, from any byte
// of the run), a mask leaves the first code in the lower half and the second in
// the upper one, each where it stands in its bytes, and one packed fma takes 1024,
// the position and z out again: three instructions a pair.  Codes of six or seven
// bits do not fit beside each other and are shifted first.
// bfloat16, which has no packed arithmetic: by way of float32.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename T, int kBits>
struct Zero;

template <int kBits>
struct Zero<half_t, kBits> {
    half_t z;
    uint32_t exponent;  // in a vector register: two literals do not fit one instruction
    __device__ __forceinline__ explicit Zero(int zero) {
        z = (half_t)(float)zero;
        exponent = 0x64006400u;
        asm("" : "+v"(exponent));
    }
    // 1024 + c 2^kLow, 1024 + d 2^kHigh -> c - z, d - z
    template <int kLow, int kHigh>
    __device__ __forceinline__ uint32_t out(uint32_t pair) const {
        const half2v v = __builtin_bit_cast(half2v, pair | exponent);
        if constexpr (kLow == 0 && kHigh == 0) return __builtin_bit_cast(uint32_t, v + ((half2v)(half_t)-1024.0f - (half2v)z));
        constexpr float kL = 1.0f / (1 << kLow), kH = 1.0f / (1 << kHigh);
        const half2v mul = {(half_t)kL, (half_t)kH}, one = {(half_t)(-1024.0f * kL), (half_t)(-1024.0f * kH)};
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, mul, one - (half2v)z));
    }
    template <int kI>
    __device__ __forceinline__ uint32_t pair(const uint32_t (&w)[kBits]) const {
        constexpr int kBit = 2 * kI * kBits, kWord = kBit / 32, kByte = kBit % 32 / 8, kIn = kBit % 8;
        constexpr uint32_t kMask = (1u << kBits) - 1u;
        if constexpr (kBits == 8) {
            return out<0, 0>(__builtin_amdgcn_perm(0u, w[kWord], kByte == 0 ? 0x0C010C00u : 0x0C030C02u));
        } else if constexpr (kIn + 2 * kBits <= 10 && kByte + (kIn + 2 * kBits > 8) <= 3) {
            constexpr uint32_t kSel = kIn + 2 * kBits > 8 ? (uint32_t)((kByte + 1) << 8 | kByte) * 0x10001u
                                                          : 0x0C000C00u | (uint32_t)kByte * 0x10001u;
            return out<kIn, kIn + kBits>(__builtin_amdgcn_perm(0u, w[kWord], kSel) & (kMask << kIn | kMask << (kIn + kBits) << 16));
        } else {
            constexpr int kShift = kBit % 32;
            uint32_t u = w[kWord] >> kShift;
            if constexpr (kShift + 2 * kBits > 32) u = __builtin_amdgcn_alignbit(w[kWord + 1], w[kWord], kShift);
            if constexpr (2 * kBits <= 10) {
                return out<0, kBits>(__builtin_amdgcn_perm(0u, u, 0x01000100u) & (kMask | kMask << kBits << 16));
            } else {
                return out<0, 0>(__builtin_amdgcn_perm(u >> kBits, u, 0x05040100u) & (kMask * 0x10001u));
            }
        }
    }
};

template <int kBits>
struct Zero<bf16_t, kBits> {
    float z;
    __device__ __forceinline__ explicit Zero(int zero) { z = (float)zero; }
    template <int kI>
    __device__ __forceinline__ uint32_t pair(const uint32_t (&w)[kBits]) const {
        constexpr int kBit = 2 * kI * kBits, kWord = kBit / 32, kShift = kBit % 32;
        constexpr uint32_t kMask = (1u << kBits) - 1u;
        float lo, hi;
        if constexpr (kBits == 4 || kBits == 8) {
            // (a byte of eight converts in one instruction)
            const uint32_t even = kBits == 4 ? w[kWord] & 0x0F0F0F0Fu : w[kWord];
            const uint32_t odd = kBits == 4 ? w[kWord] >> 4 & 0x0F0F0F0Fu : w[kWord];
            lo = (float)(even >> kShift & 0xFFu);
            hi = (float)(odd >> (kBits == 4 ? kShift : kShift + 8) & 0xFFu);
        } else {
            uint32_t u = w[kWord] >> kShift;
            if constexpr (kShift + 2 * kBits > 32) u = __builtin_amdgcn_alignbit(w[kWord + 1], w[kWord], kShift);
            lo = (float)(u & kMask);
            hi = (float)(u >> kBits & kMask);
        }
        return __builtin_bit_cast(uint32_t, (bf16x2){(bf16_t)(lo - z), (bf16_t)(hi - z)});
    }
};

typedef uint32_t frag_t __attribute__((ext_vector_type(4)));  // eight 16-bit values

template <typename T, int kBits, int kE>
__device__ __forceinline__ frag_t codes8(const uint32_t (&w)[kBits], const Zero<T, kBits>& z) {
    return (frag_t){z.template pair<4 * kE>(w), z.template pair<4 * kE + 1>(w), z.template pair<4 * kE + 2>(w),
                    z.template pair<4 * kE + 3>(w)};
}

// The four fragments of a run.  zb: the zero of its last sixteen codes.
template <typename T, int kBits>
__device__ __forceinline__ void codes32(frag_t (&f)[4], const uint32_t (&w)[kBits], int za, int zb) {
    const Zero<T, kBits> a(za), b(zb);
    f[0] = codes8<T, kBits, 0>(w, a);
    f[1] = codes8<T, kBits, 1>(w, a);
    f[2] = codes8<T, kBits, 2>(w, b);
    f[3] = codes8<T, kBits, 3>(w, b);
}

// Loads of what belongs to sixteen weight rows give four neighbouring lanes to a
// row: the address unit takes sixteen lanes at a time, and asks once for what
// neighbours read of one line (16 requests an instruction; 64 with the lanes in
// the order of the MFMA's operands, which held the products' tiles up longer
// than anything else).  from_row hands a value to the operand's lane: row l16, k
// group kg or, for what is the row's, any.
__device__ __forceinline__ uint32_t from_row(uint32_t v, int place) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * place, (int)v);
}

// A lane of k group kg holds columns 32 kg + 8 e .. of a block of 128 as f[e].
// Turned, f[e] holds columns 32 e + 8 kg: the four lanes of a row exchange
// fragments as a 4 x 4 transpose, halves of the wave first, then halves of those.
__device__ __forceinline__ void turn_blocks(frag_t (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4] = {f[0][i], f[1][i], f[2][i], f[3][i]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto r = __builtin_amdgcn_permlane32_swap(v[e], v[e + 2], false, false);
            v[e] = (uint32_t)r[0], v[e + 2] = (uint32_t)r[1];
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const auto r = __builtin_amdgcn_permlane16_swap(v[e], v[e + 1], false, false);
            v[e] = (uint32_t)r[0], v[e + 1] = (uint32_t)r[1];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e][i] = v[e];
    }
}

// Where chunk c (sixteen bytes) of token row r lies in its row of 256 bytes of
// LDS: c ^ pm_swizzle(r).  LDS serves sixteen lanes at a time: eight rows of one k
// group (0-3, 12-15) with the other eight (4-11) of the next, whose chunk differs
// by 4 (codes by runs) or by 1 (turned).  The swizzle is a permutation that
// takes the bits 0 and 1 of r, which leave rows 4-11 among themselves, to the
// bits 2 and 0, so that the sixteen chunks differ either way.
__host__ __device__ constexpr int pm_swizzle(int r) {
    return (r & 1) << 2 | (r >> 1 & 1) | (r >> 2 & 1) << 1 | (r & 8);
}

__device__ __forceinline__ void pm_copy16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off, uint32_t base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, base, 0, 0);
}

// x whose rows start at any element: the words around eight columns, and the columns
// out of them a step later.  (As eight elements, or as sixteen bytes of any alignment
// under a condition, each load was waited for on its own: 3000 x 1001 -> 2000 87 us.)
// The buffer begins at the word that holds the first element and ends with the one that
// holds the last.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t pm_words_rsrc(const T* x, uint32_t elements, uint32_t& first) {
    first = (uint32_t)(reinterpret_cast<uintptr_t>(x) / 2 % 2);
    return pm_rsrc(x - first, (2 * (first + elements) + 3) & ~3u);
}
struct PmWords {
    uint4v w;
    uint32_t next;
};
__device__ __forceinline__ PmWords pm_words(__amdgpu_buffer_rsrc_t r, uint32_t element, uint32_t base) {
    const uint32_t at = 2 * element & ~3u;
    PmWords p;
    p.w = __builtin_amdgcn_raw_buffer_load_b128(r, at, base, 0);
    p.next = __builtin_amdgcn_raw_buffer_load_b32(r, at + 16, base, 0);
    return p;
}
// left: columns of the row from the first of these on, what follows them as zeros
__device__ __forceinline__ frag_t pm_columns(const PmWords& p, uint32_t element, int left) {
    const uint32_t by = element % 2 * 16;
    uint4v f;
    f[0] = __builtin_amdgcn_alignbit(p.w[1], p.w[0], by);
    f[1] = __builtin_amdgcn_alignbit(p.w[2], p.w[1], by);
    f[2] = __builtin_amdgcn_alignbit(p.w[3], p.w[2], by);
    f[3] = __builtin_amdgcn_alignbit(p.next, p.w[3], by);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = left >= 2 * i + 2 ? f[i] : left == 2 * i + 1 ? f[i] & 0xffffu : 0u;
    return __builtin_bit_cast(frag_t, f);
}

// v Phi(v), within 2^-20 of itself down to -13 (where float32 ends).  1 + erf(v / sqrt 2)
// would lose a negative v's value: 4% at -5, all of it from -5.6 on.  So the part of
// Phi beyond |v| is taken as it is,
//   h = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) g(a),  a = |v|,
// with g, which falls from 1/2 like 1 / a, as a polynomial of degree 8 in 1 / (1 + 0.3 a)
// (fitted by least squares to g's own size: 2^-24 of it), and what the square and its
// product with log2 e / 2 are rounded by put back by a factor.
__device__ __forceinline__ float gelu(float v) {
    const float a = fminf(fabsf(v), 15.0f);  // beyond, h is zero
    const float u = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
    float g = 3.84254903e-2f;
    g = fmaf(g, u, -1.69395193e-1f);
    g = fmaf(g, u, 2.29132429e-1f);
    g = fmaf(g, u, -7.70454779e-2f);
    g = fmaf(g, u, 1.42906785e-1f);
    g = fmaf(g, u, 9.45259184e-2f);
    g = fmaf(g, u, 1.21960498e-1f);
    g = fmaf(g, u, 1.19482085e-1f);
    g = fmaf(g, u, 7.49559513e-6f);
    constexpr float kHalf = (float)(0.5 * 1.4426950408889634), kRest = (float)(0.5 * 1.4426950408889634 - (double)kHalf);
    const float sq = a * a, t = sq * kHalf;
    const float more = fmaf(fmaf(a, a, -sq), kHalf, fmaf(sq, kRest, fmaf(sq, kHalf, -t)));
    const float h = g * exp2_fast(-t) * fmaf(more, -0.69314718f, 1.0f);
    return v * (v < 0.0f ? h : 1.0f - h);
}

// v / (1 + exp(-v)).  exact, for float32 results (to -87, where the exponential ends):
// as v / (1 + e) or v e / (1 + e) with e = exp(-|v|), whose exponent's rounding is put back
// by a factor, and one step of Newton's on the reciprocal.  Sixteen bits do not show the
// 2^-17 that a plain reciprocal and the fast exponential are off (8192 x 4096 -> 11008
// 745 us, 772 with the steps of float32, 735 without activation).
__device__ __forceinline__ float silu(float v, bool exact) {
    if (!exact) return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    constexpr float kLog = (float)1.4426950408889634, kRest = (float)(1.4426950408889634 - (double)kLog);
    const float a = fminf(fabsf(v), 128.0f), t = a * kLog;  // (beyond, e is zero)
    const float e = exp2_fast(-t) * fmaf(fmaf(a, kRest, fmaf(a, kLog, -t)), -0.69314718f, 1.0f);
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
    const float q = fmaf(fmaf(-d, r, 1.0f), r, r);
    return v * (v < 0.0f ? e * q : q);
}

__device__ __forceinline__ float activated(float v, int activation, bool exact) {
    if (activation == 1) return v < 0.0f ? 0.0f : v;  // keeps NaN
    if (activation == 2) return silu(v, exact);
    if (activation == 3) return gelu(v);
    return v;
}

}  // namespace gptq
