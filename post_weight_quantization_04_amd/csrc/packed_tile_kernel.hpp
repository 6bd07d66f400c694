// The kernel of products with packed few-bit weights for many tokens.
#pragma once

#include "packed_tile.hpp"

namespace gptq {

namespace {

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

// kTT tokens by kTR weight rows a workgroup, kWT x kWR waves.  A block of 128
// columns of x is a stage of LDS, copied from memory without passing registers
// one block ahead, one barrier a block (kVec; else, where rows of x are not
// aligned or end inside a chunk, by way of registers).  A wave loads the codes of
// its own rows into registers, a block ahead, and converts them there once a
// block: they then meet all of its tokens.
template <typename T, int kBits, bool kFine, bool kVec, int kTT, int kTR, int kWT, int kWR, int kPerCu>
__global__ __launch_bounds__(kWT* kWR* kWave, kWT* kWR / 4 * kPerCu) void packed_tile_kernel(PmArgs a) {
    constexpr int kWaves = kWT * kWR, kMt = kTT / kWT / 16, kNt = kTR / kWR / 16;
    constexpr int kCopies = kTT / 4 / kWaves;  // of four token rows, a wave and stage
    static_assert(kTT % (4 * kWaves) == 0, "whole copies");
    constexpr int kBytes = kTT * 2 * kPmBlock;
    // separate arrays: the compiler then knows that a read of one does not wait for copies into another
    __shared__ __align__(16) uint8_t lds0[kBytes];
    __shared__ __align__(16) uint8_t lds1[kBytes];
    typedef typename Mat<T>::v8 v8;

    const PackedProduct& c = a.c;
    const int tid = threadIdx.x, lane = tid % kWave, w = wave_id(), l16 = lane % 16, kg = lane / 16;
    const int wt = w / kWR, wr = w % kWR;
    unsigned mi, ni;
    xcd_tile_of(blockIdx.x, a.mt, a.nt, mi, ni);
    const int64_t r0 = (int64_t)mi * kTR, t0 = (int64_t)ni * kTT;
    const int rows = (int)min(c.M - r0, (int64_t)kTR), toks = (int)min(c.n - t0, (int64_t)kTT);
    const int nb = a.nb;
    const bool ragged = c.K % kPmBlock != 0;
    const T* x = static_cast<const T*>(c.x) + t0 * c.ldx;

    const __amdgpu_buffer_rsrc_t rw = pm_rsrc(c.packed + r0 * a.nw, (uint32_t)rows * (uint32_t)a.nw * 4u);
    const __amdgpu_buffer_rsrc_t rs = pm_rsrc(c.scales + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    const __amdgpu_buffer_rsrc_t rz = pm_rsrc(c.zeros + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    const __amdgpu_buffer_rsrc_t rx = pm_rsrc(x, (uint32_t)(((toks - 1) * c.ldx + c.K) * 2));

    // Sources of this lane's copies: four rows an instruction; every fourth
    // instruction has the same swizzle.  Rows past the last lie past the end of the
    // buffer (a row's stride covers what is read of it), and load zero.
    const int copy_row = 4 * kCopies * w + lane / 16;
    uint32_t xo[4];
    int xc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = copy_row + 4 * i;
        xc[i] = 8 * ((lane % 16) ^ pm_swizzle(r % 16));
        xo[i] = 2 * ((uint32_t)r * (uint32_t)c.ldx + (uint32_t)xc[i]);
    }
    auto copy = [&](uint8_t* st, int b) {
        const int k0 = min(b, nb - 1) * kPmBlock;  // past the last block, that one again, never used
        const bool tail = ragged && b >= nb - 1;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            uint8_t* to = st + 1024 * (kCopies * w + i);
            if (kVec) {
                const uint32_t off = tail && k0 + xc[i % 4] >= c.K ? kPmOut : xo[i % 4];
                pm_copy16(rx, to, off, (uint32_t)(2 * k0) + (uint32_t)(i / 4) * 32u * (uint32_t)c.ldx);
            } else {
                const int r = copy_row + 4 * i, k = k0 + xc[i % 4];
                const T* p = x + r * c.ldx + k;
                T v[8] = {};
                if (r < toks) {
                    if (k + 8 <= c.K) __builtin_memcpy(v, p, 16);
                    else
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (k + e < c.K) v[e] = p[e];
                }
                __builtin_memcpy(to + 16 * lane, v, 16);
            }
        }
    };

    // This lane's rows: 16 j + l16 of the wave's.
    uint32_t wo[kNt], so[kNt];
#pragma unroll
    for (int j = 0; j < kNt; ++j) {
        const uint32_t r = (uint32_t)((wr * kNt + j) * 16 + l16);
        wo[j] = 4u * (r * (uint32_t)a.nw + (uint32_t)(kg * kBits));
        so[j] = 4u * r * (uint32_t)a.ng;
    }
    constexpr int kZeros = kFine ? 2 : 1;
    uint32_t words[kNt][kBits];
    int zs[kNt][kZeros];
    float ss[kNt];  // of groups of whole blocks
    auto load = [&](int b) {
        b = min(b, nb - 1);
        const bool tail = ragged && b == nb - 1;
        const uint32_t k0 = (uint32_t)b * kPmBlock, base = (uint32_t)b * (16u * kBits);
#pragma unroll
        for (int j = 0; j < kNt; ++j) load_run<kBits>(words[j], rw, wo[j], base, tail);
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            if (kFine) {
#pragma unroll
                for (int h = 0; h < kZeros; ++h)
                    zs[j][h] = (int)__builtin_amdgcn_raw_buffer_load_b32(rz, so[j] + 4 * group_of(a, k0 + 32 * kg + 16 * h), 0, 0);
            } else {
                const uint32_t at = 4 * group_of(a, k0);
                zs[j][0] = (int)__builtin_amdgcn_raw_buffer_load_b32(rz, so[j], at, 0);
                ss[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, so[j], at, 0));
            }
        }
    };

    float4v acc[kMt][kNt];
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int j = 0; j < kNt; ++j) acc[i][j] = (float4v){};

    const int place = l16 * 2 * kPmBlock;
    auto tokens = [&](const uint8_t* st, int i, int e) {
        const int chunk = kFine ? 4 * e + kg : 4 * kg + e;
        return *reinterpret_cast<const v8*>(st + ((wt * kMt + i) * 16 * 2 * kPmBlock + place + 16 * (chunk ^ pm_swizzle(l16))));
    };
    auto step = [&](uint8_t* st, uint8_t* nx, int b) {
        frag_t f[kNt][4];
        float s[kNt];
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            codes32<T, kBits>(f[j], words[j], zs[j][0], zs[j][kZeros - 1]);
            if (kFine) turn_blocks(f[j]);
            s[j] = ss[j];
        }
        // this block has landed for all waves, and all are done with the one before
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load(b + 1);
        copy(nx, b + 1);
        if (!kFine) {
#pragma unroll
            for (int i = 0; i < kMt; ++i) {
                v8 xf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) xf[e] = tokens(st, i, e);
#pragma unroll
                for (int j = 0; j < kNt; ++j) {
                    float4v p = {};
#pragma unroll
                    for (int e = 0; e < 4; ++e) p = Mat<T>::mfma16(xf[e], __builtin_bit_cast(v8, f[j][e]), p);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[v], s[j], acc[i][j][v]);
                }
                __builtin_amdgcn_sched_barrier(0);  // left alone, the scheduler reads every fragment first and spills
            }
        } else {
            // 32 columns at a time, or twice sixteen (the others as zeros)
            const bool halves = a.group % 32 != 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float sa[kNt], sb[kNt];
                const uint32_t ga = 4 * group_of(a, (uint32_t)(b * kPmBlock + 32 * e)), gb = 4 * group_of(a, (uint32_t)(b * kPmBlock + 32 * e + 16));
#pragma unroll
                for (int j = 0; j < kNt; ++j) {
                    sa[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, so[j], ga, 0));
                    sb[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, so[j], gb, 0));
                }
#pragma unroll
                for (int i = 0; i < kMt; ++i) {
                    const v8 xf = tokens(st, i, e);
                    const v8 xa = halves && kg >= 2 ? (v8){} : xf, xb = kg >= 2 ? xf : (v8){};
#pragma unroll
                    for (int j = 0; j < kNt; ++j) {
                        const v8 wf = __builtin_bit_cast(v8, f[j][e]);
                        const float4v p = Mat<T>::mfma16(xa, wf, (float4v){});
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[v], sa[j], acc[i][j][v]);
                        if (halves) {
                            const float4v q = Mat<T>::mfma16(xb, wf, (float4v){});
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(q[v], sb[j], acc[i][j][v]);
                        }
                    }
                }
            }
        }
    };
    if (nb > 0) {
        load(0);
        copy(lds0, 0);
        for (int b = 0; b < nb; b += 2) {
            step(lds0, lds1, b);
            if (b + 1 == nb) break;
            step(lds1, lds0, b + 1);
        }
    }
    // copies still in flight would land in memory that the epilogue uses
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    // A lane holds four tokens of one weight row.  A wave turns sixteen tokens at
    // a time in LDS of its own; then a lane has eight neighbouring rows of a token.
    constexpr int kRun = 16 * kNt, kPitch = kRun + 4;
    static_assert(kWaves * 16 * kPitch * 4 <= kBytes, "the lines of every wave");
    float* lines = reinterpret_cast<float*>(lds0) + w * 16 * kPitch;
    const int64_t o0 = r0 + wr * kRun;
#pragma unroll
    for (int i = 0; i < kMt; ++i) {
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) lines[(4 * kg + v) * kPitch + 16 * j + l16] = acc[i][j][v];
        __builtin_amdgcn_wave_barrier();
        for (int q = lane; q < 2 * kRun; q += kWave) {
            const int line = q / (kRun / 8), at = q % (kRun / 8) * 8;
            const int64_t t = t0 + (wt * kMt + i) * 16 + line, o = o0 + at, left = c.M - o;
            if (t >= c.n || left <= 0) continue;
            float y[8], e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = lines[line * kPitch + at + k];
            if (c.bias) {
                if (a.y32) load8<float, false>(e, static_cast<const float*>(c.bias) + o, left);
                else load8<T, false>(e, static_cast<const T*>(c.bias) + o, left);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] += e[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = activated(y[k], c.activation);
            if (c.residual) {
                if (a.y32) load8<float, false>(e, static_cast<const float*>(c.residual) + t * c.ldr + o, left);
                else load8<T, false>(e, static_cast<const T*>(c.residual) + t * c.ldr + o, left);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] += e[k];
            }
            if (a.y32) store8<float, false>(static_cast<float*>(c.y) + t * c.ldy + o, y, left);
            else store8<T, false>(static_cast<T*>(c.y) + t * c.ldy + o, y, left);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int kBits, bool kFine, bool kVec, int kTT, int kTR, int kWT, int kWR, int kPerCu>
hipError_t tile_go(PmArgs a, hipStream_t s) {
    const TimedLaunch t(K_PACKED_MATMUL, s);
    a.mt = (unsigned)((a.c.M + kTR - 1) / kTR);
    a.nt = (unsigned)((a.c.n + kTT - 1) / kTT);
    GPTQ_LAUNCH(t, (packed_tile_kernel<T, kBits, kFine, kVec, kTT, kTR, kWT, kWR, kPerCu>), dim3(a.mt * a.nt), dim3(kWT * kWR * kWave), 0, s, a);
    return hipGetLastError();
}

}  // namespace

template <typename T, int kBits>
hipError_t launch_packed_tile(const PmArgs& a, bool fine, hipStream_t s) {
    const bool vec = a.c.K % 8 == 0 && a.c.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(a.c.x) % 16 == 0;
    if (fine) return vec ? tile_go<T, kBits, true, true, 128, 128, 2, 2, 2>(a, s) : tile_go<T, kBits, true, false, 128, 128, 2, 2, 2>(a, s);
    if (!vec) return tile_go<T, kBits, false, false, 128, 128, 2, 2, 2>(a, s);
    const int64_t big = ((a.c.M + 255) / 256) * ((a.c.n + 255) / 256), mid = ((a.c.M + 127) / 128) * ((a.c.n + 127) / 128);
    const int64_t cus = device_cu_count();
    if (cus <= 0) return hipErrorInvalidDevice;
    if (big >= cus) return tile_go<T, kBits, false, true, 256, 256, 2, 4, 1>(a, s);
    if (mid >= cus) return tile_go<T, kBits, false, true, 128, 128, 2, 2, 2>(a, s);
    return tile_go<T, kBits, false, true, 64, 64, 2, 2, 2>(a, s);
}

}  // namespace gptq
