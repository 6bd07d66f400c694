// The kernel of products with packed few-bit weights for many tokens.
#pragma once

#include <type_traits>

#include "packed_tile.hpp"

namespace gptq {

namespace {

// Bias, activation and residual of eight neighbouring rows of token t, and their store.
template <typename T>
__device__ __forceinline__ void pm_finish(const PmArgs& a, const float* sums, int64_t t, int64_t o) {
    const PackedProduct& c = a.c;
    const int64_t left = c.M - o;
    if (t >= c.n || left <= 0) return;
    float y[8], e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = sums[k];
    if (c.bias) {
        if (a.y32) load8<float, false>(e, static_cast<const float*>(c.bias) + o, left);
        else load8<T, false>(e, static_cast<const T*>(c.bias) + o, left);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] += e[k];
    }
    // (one branch for all eight, whose steps then lie beside one another: a branch each
    // takes 777 x 1000 -> 1363 with bias and GELU from 12.9 to 15.0 us, 8192 x 4096 ->
    // 11008 with SiLU from 745 to 803)
    if (c.activation == 3) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = gelu(y[k]);
    } else if (c.activation == 2 && a.y32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = silu(y[k], true);
    } else if (c.activation == 2) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = silu(y[k], false);
    } else if (c.activation) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = activated(y[k], 1, false);
    }
    if (c.residual) {
        if (a.y32) load8<float, false>(e, static_cast<const float*>(c.residual) + t * c.ldr + o, left);
        else load8<T, false>(e, static_cast<const T*>(c.residual) + t * c.ldr + o, left);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] += e[k];
    }
    if (a.y32) store8<float, false>(static_cast<float*>(c.y) + t * c.ldy + o, y, left);
    else store8<T, false>(static_cast<T*>(c.y) + t * c.ldy + o, y, left);
}

// kTT tokens by kTR weight rows a workgroup, whose waves share the rows: each
// wave loads the codes of its own into registers, converts them there once a
// block and has them meet all of the tokens.  A block of 128 columns of x is a
// stage of LDS, four of which are a ring: copied from memory without passing
// registers three blocks ahead, one barrier a block (kVec; else, where rows of x
// are not aligned or end inside a chunk, by way of registers).
//
// Tokens and rows lie this way round because copies are what the tile waits for:
// with waves two by four over 256 x 192, which copies twice the x for the same
// products, 8192 x 4096 -> 11008 took 881 us, 616 of them without the copies.
//
// 8192 x 4096 -> 11008, 4 bits: 733 us, 1008 TFLOP/s (745 with SiLU; bfloat16, whose
// conversion goes by way of float32, 812); up to 780 by the clocks the card holds; a dense
// float16 product by the library takes 714.  4.4 VALU instructions an MFMA (conversions 2
// to 3, scaling 1) take as many cycles as the MFMA itself (busy in 43%): a tile of more
// tokens would convert less often but its sums do not fit the registers.
//
// A tile that has a CU to itself takes 0.9 us a block whatever its size: each step
// is a chain of reads, conversions and products.  So small products have kGroups
// such groups of waves in a workgroup, which take turns with the blocks and add
// their sums at the end.
template <typename T, int kBits, bool kFine, bool kVec, int kTT, int kTR, int kWaves, int kPerCu, int kRing, int kGroups>
__global__ __launch_bounds__(kGroups* kWaves* kWave, kGroups* kWaves / 4 * kPerCu) void packed_tile_kernel(PmArgs a) {
    constexpr int kMt = kTT / 16, kNt = kTR / kWaves / 16;
    constexpr int kCopies = kTT / 4 / kWaves;  // of four token rows, a wave and stage
    static_assert(kRing == 1 || kRing == 4, "steps come in fours");
    static_assert(kTT % (4 * kWaves) == 0 && kTR % (16 * kWaves) == 0, "whole copies and rows");
    constexpr int kBytes = kTT * 2 * kPmBlock;
    // separate arrays: the compiler then knows that a read of one does not wait for copies into another
    __shared__ __align__(16) uint8_t lds0[kGroups * kBytes];
    __shared__ __align__(16) uint8_t lds1[kGroups * kBytes];
    __shared__ __align__(16) uint8_t lds2[kGroups * kBytes];
    __shared__ __align__(16) uint8_t lds3[kGroups * kBytes];
    typedef typename Mat<T>::v8 v8;

    const PackedProduct& c = a.c;
    const int tid = threadIdx.x, lane = tid % kWave, l16 = lane % 16, kg = lane / 16;
    const int set = kGroups > 1 ? wave_id() / kWaves : 0, w = wave_id() - set * kWaves, base = set * kBytes;
    unsigned mi, ni;
    xcd_tile_of(blockIdx.x, a.mt, a.nt, mi, ni);
    const int64_t r0 = (int64_t)mi * kTR, t0 = (int64_t)ni * kTT;
    const int rows = (int)min(c.M - r0, (int64_t)kTR), toks = (int)min(c.n - t0, (int64_t)kTT);
    const int nb = a.nb;
    const T* x = static_cast<const T*>(c.x) + t0 * c.ldx;

    const __amdgpu_buffer_rsrc_t rw = pm_rsrc(c.packed + r0 * a.nw, (uint32_t)rows * (uint32_t)a.nw * 4u);
    const __amdgpu_buffer_rsrc_t rs = pm_rsrc(c.scales + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    const __amdgpu_buffer_rsrc_t rz = pm_rsrc(c.zeros + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    uint32_t first = 0;
    const uint32_t elements = (uint32_t)((toks - 1) * c.ldx + c.K);
    const __amdgpu_buffer_rsrc_t rx = kVec ? pm_rsrc(x, 2 * elements) : pm_words_rsrc(x, elements, first);

    // Sources of this lane's copies: four rows an instruction; every fourth
    // instruction has the same swizzle.  Rows past the last lie past the end of the
    // buffer (a row's stride covers what is read of it), and load zero; so do
    // chunks past the last column, since what follows it is not the row's.
    const int copy_row = 4 * kCopies * w + lane / 16;
    uint32_t xo[kCopies];
    int xk[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = copy_row + 4 * i;
        xk[i] = 8 * ((lane % 16) ^ pm_swizzle(r % 16));
        xo[i] = (kVec ? 2 : 1) * ((uint32_t)r * (uint32_t)c.ldx + (uint32_t)xk[i]) + first;
    }
    // (steps count the group's blocks: every kGroups-th)
    PmWords held[kVec ? 1 : kCopies];  // by way of registers: what goes to LDS a step after it was asked for
    auto copy = [&](uint8_t* st, int step) {
        const int b = step * kGroups + set, left = (int)c.K - b * kPmBlock;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            if (kVec) pm_copy16(rx, st + (base + 1024 * (kCopies * w + i)), xk[i] < left ? xo[i] : kPmOut, (uint32_t)(2 * b * kPmBlock));
            else held[i] = pm_words(rx, xo[i], (uint32_t)(2 * b * kPmBlock));
        }
    };
    auto put = [&](uint8_t* st, int step) {
        const int left = (int)c.K - (step * kGroups + set) * kPmBlock;
#pragma unroll
        for (int i = 0; i < kCopies && !kVec; ++i)
            *reinterpret_cast<frag_t*>(st + (base + 1024 * (kCopies * w + i) + 16 * lane)) = pm_columns(held[i], xo[i], left - xk[i]);
    };

    // The wave's rows, 16 j + l16 for this lane; scales and zeros come by way of row 16 j + lane / 4.
    const uint32_t r = (uint32_t)(w * kNt * 16 + lane / 4);
    const uint32_t wo = 4u * ((uint32_t)(w * kNt * 16 + l16) * (uint32_t)a.nw + (uint32_t)(kg * kBits)), so = 4u * r * (uint32_t)a.ng;
    const uint32_t w16 = 64u * (uint32_t)a.nw, s16 = 64u * (uint32_t)a.ng;  // sixteen rows on
    // The codes of the next kRing blocks (one where registers are short).
    uint32_t words[kRing][kNt][kBits];
    auto load = [&](int step, int slot) {
        const int b = step * kGroups + set;
#pragma unroll
        for (int j = 0; j < kNt; ++j) load_run<kBits>(words[slot][j], rw, wo, (uint32_t)b * (16u * kBits) + (uint32_t)j * w16);
    };
    // Scales and zeros of four blocks, one a lane of the row's four (groups of
    // whole blocks; of finer ones, those of a run of 32 codes of one block a lane,
    // two halves of it).
    constexpr int kZeros = kFine ? 2 : 1;
    uint32_t ss[kNt][kZeros], zs[kNt][kZeros];
    auto load_grids = [&](int step) {
        const int b = step * kGroups + set;
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            if (kFine) {
#pragma unroll
                for (int h = 0; h < kZeros; ++h) {
                    const uint32_t at = so + 4 * group_of(a, (uint32_t)(b * kPmBlock + 32 * (lane % 4) + 16 * h));
                    zs[j][h] = __builtin_amdgcn_raw_buffer_load_b32(rz, at, (uint32_t)j * s16, 0);
                    ss[j][h] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, (uint32_t)j * s16, 0);
                }
            } else {
                const uint32_t at = so + 4 * group_of(a, (uint32_t)((b + lane % 4 * kGroups) * kPmBlock));
                zs[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rz, at, (uint32_t)j * s16, 0);
                ss[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, (uint32_t)j * s16, 0);
            }
        }
    };

    float4v acc[kMt][kNt];
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int j = 0; j < kNt; ++j) acc[i][j] = (float4v){};

    const int place = base + l16 * 2 * kPmBlock;
    auto tokens = [&](const uint8_t* st, int i, int e) {
        const int chunk = kFine ? 4 * e + kg : 4 * kg + e;
        return *reinterpret_cast<const v8*>(st + (i * 16 * 2 * kPmBlock + place + 16 * (chunk ^ pm_swizzle(l16))));
    };
    // Block b, the i4-th of four, from stage st; the block three on goes to `to`,
    // which all waves were done with at this step's barrier (kVec; otherwise the one
    // two on goes to the stage `before` that, and the one three on to registers).
    auto step = [&](uint8_t* st, uint8_t* before, uint8_t* to, int b, int i4) {
        // (this block's copies; behind them are the next two blocks' and, with a ring
        // of codes, two blocks of those, an instruction or two a run)
        if (kVec) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * kCopies + (kRing > 1 ? 2 * kNt : 0)) : "memory");
        else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        frag_t f[kNt][4];
        if (!kFine) {
            // A token tile's fragments are read while the one before is multiplied,
            // and its products scaled while the next one is.
            float s[kNt];
            v8 xf[2][4];
            float4v late[kNt];
#pragma unroll
            for (int e = 0; e < 4; ++e) xf[0][e] = tokens(st, 0, e);
#pragma unroll
            for (int i = 0; i < kMt; ++i) {
                if (i + 1 < kMt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) xf[(i + 1) % 2][e] = tokens(st, i + 1, e);
                }
                float4v p[kNt];
                if (i == 0) {
                    // the codes become fragments beside the first products
#pragma unroll
                    for (int j = 0; j < kNt; ++j) {
                        const int z = (int)from_row(zs[j][0], 4 * l16 + i4);
                        s[j] = __builtin_bit_cast(float, from_row(ss[j][0], 4 * l16 + i4));
                        codes32<T, kBits>(f[j], words[i4 % kRing][j], z, z);
                        p[j] = (float4v){};
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[j] = Mat<T>::mfma16(xf[0][e], __builtin_bit_cast(v8, f[j][e]), p[j]);
                    }
                } else {
                    if (i == 1) {
                        // (the codes first: they are waited for with the copies before these)
                        load(b + kRing, i4 % kRing);
                        if (i4 == 3) load_grids(b + 1);
                        put(before, b + 2);
                        copy(to, b + 3);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < kNt; ++j)
                            p[j] = Mat<T>::mfma16(xf[i % 2][e], __builtin_bit_cast(v8, f[j][e]), e == 0 ? (float4v){} : p[j]);
#pragma unroll
                    for (int j = 0; j < kNt; ++j)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i - 1][j][v] = fmaf(late[j][v], s[j], acc[i - 1][j][v]);
                }
#pragma unroll
                for (int j = 0; j < kNt; ++j) late[j] = p[j];
                __builtin_amdgcn_sched_barrier(0);  // left alone, the scheduler reads every fragment first and spills
            }
#pragma unroll
            for (int j = 0; j < kNt; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[kMt - 1][j][v] = fmaf(late[j][v], s[j], acc[kMt - 1][j][v]);
        } else {
#pragma unroll
            for (int j = 0; j < kNt; ++j) {
                codes32<T, kBits>(f[j], words[i4 % kRing][j], (int)from_row(zs[j][0], 4 * l16 + kg), (int)from_row(zs[j][kZeros - 1], 4 * l16 + kg));
                turn_blocks(f[j]);
            }
            float sa[4][kNt], sb[4][kNt];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < kNt; ++j) {
                    sa[e][j] = __builtin_bit_cast(float, from_row(ss[j][0], 4 * l16 + e));
                    sb[e][j] = __builtin_bit_cast(float, from_row(ss[j][kZeros - 1], 4 * l16 + e));
                }
            load(b + kRing, i4 % kRing);
            load_grids(b + 1);
            put(before, b + 2);
            copy(to, b + 3);
            // 32 columns at a time, or twice sixteen (the others as zeros): one branch
            // around all of it, since between the products each would be waited for
            // (500 tokens of 2048 x 2048 in groups of 32 48 us, so 28)
            auto products = [&](auto halved) {
                constexpr bool kHalves = decltype(halved)::value;
                // as above: the next fragments read, these multiplied, the products before scaled
                v8 xf[2];
                float4v pa[2][kNt], pb[2][kNt];
                xf[0] = tokens(st, 0, 0);
                auto scale = [&](int q) {
                    const int e = q / kMt, i = q % kMt;
#pragma unroll
                    for (int j = 0; j < kNt; ++j)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            acc[i][j][v] = fmaf(pa[q % 2][j][v], sa[e][j], acc[i][j][v]);
                            if (kHalves) acc[i][j][v] = fmaf(pb[q % 2][j][v], sb[e][j], acc[i][j][v]);
                        }
                };
#pragma unroll
                for (int q = 0; q < 4 * kMt; ++q) {
                    if (q + 1 < 4 * kMt) xf[(q + 1) % 2] = tokens(st, (q + 1) % kMt, (q + 1) / kMt);
                    const v8 x = xf[q % 2], xa = kHalves && kg >= 2 ? (v8){} : x, xb = kg >= 2 ? x : (v8){};
#pragma unroll
                    for (int j = 0; j < kNt; ++j) {
                        const v8 wf = __builtin_bit_cast(v8, f[j][q / kMt]);
                        pa[q % 2][j] = Mat<T>::mfma16(xa, wf, (float4v){});
                        if (kHalves) pb[q % 2][j] = Mat<T>::mfma16(xb, wf, (float4v){});
                    }
                    if (q > 0) scale(q - 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
                scale(4 * kMt - 1);
            };
            if (a.group % 32 != 0) products(std::true_type{});
            else products(std::false_type{});
        }
    };
    if (nb > 0) {
        // (in the order that the waits count on: the compiler may not move them past one another)
        auto in_order = [] { asm volatile("" ::: "memory"); };
        constexpr int kFirst = kRing > 1 ? kRing - 2 : 1;
#pragma unroll
        for (int b = 0; b < kFirst; ++b) load(b, b);
        load_grids(0);
        in_order();
        copy(lds0, 0);
        put(lds0, 0);
        in_order();
        if (kRing > 1) load(kFirst, kFirst);
        copy(lds1, 1);
        put(lds1, 1);
        in_order();
        if (kRing > 1) load(kFirst + 1, kFirst + 1);
        copy(lds2, 2);
        // Four steps without a branch between them (the compiler would move the
        // scaling of products past it and keep them all in registers).  Blocks past
        // the last have x of zeros.
        for (int b = 0; b * kGroups < nb; b += 4) {
            step(lds0, lds2, lds3, b, 0);
            step(lds1, lds3, lds0, b + 1, 1);
            step(lds2, lds0, lds1, b + 2, 2);
            step(lds3, lds1, lds2, b + 3, 3);
        }
    }
    // copies still in flight would land in memory that the epilogue uses
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    if (kGroups > 1) {
        // the groups' sums, added in group order
        constexpr int kOne = kWaves * kMt * kNt * 4 * kWave;
        static_assert(4 * (kGroups - 1) * kOne <= kGroups * kBytes, "the sums in a stage");
        float* sums = reinterpret_cast<float*>(lds2);
        auto at = [&](int g, int i, int j, int v) -> float& { return sums[(g - 1) * kOne + (((w * kMt + i) * kNt + j) * 4 + v) * kWave + lane]; };
        if (set > 0) {
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) at(set, i, j, v) = acc[i][j][v];
        }
        __syncthreads();
        if (set > 0) return;
#pragma unroll
        for (int g = 1; g < kGroups; ++g)
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] += at(g, i, j, v);
    }
    // A lane holds four tokens of one weight row.  A wave turns sixteen tokens at
    // a time in LDS of its own; then a lane has eight neighbouring rows of a token.
    constexpr int kRun = 16 * kNt, kPitch = kRun + 4;
    constexpr int kHalf = kWaves / 2;
    static_assert(kHalf * 16 * kPitch * 4 <= kGroups * kBytes, "the lines of every wave");
    float* lines = reinterpret_cast<float*>(w < kHalf ? lds0 : lds1) + w % kHalf * 16 * kPitch;
    const int64_t o0 = r0 + w * kRun;
#pragma unroll
    for (int i = 0; i < kMt; ++i) {
#pragma unroll
        for (int j = 0; j < kNt; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) lines[(4 * kg + v) * kPitch + 16 * j + l16] = acc[i][j][v];
        __builtin_amdgcn_wave_barrier();
        for (int q = lane; q < 2 * kRun; q += kWave) {
            pm_finish<T>(a, lines + q / (kRun / 8) * kPitch + q % (kRun / 8) * 8, t0 + 16 * i + q / (kRun / 8), o0 + q % (kRun / 8) * 8);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int kBits, bool kFine, bool kVec, int kTT, int kTR, int kWaves, int kPerCu, int kRing, int kGroups>
hipError_t tile_go(PmArgs a, hipStream_t s) {
    const TimedLaunch t(K_PACKED_MATMUL, s);
    a.mt = (unsigned)((a.c.M + kTR - 1) / kTR);
    a.nt = (unsigned)((a.c.n + kTT - 1) / kTT);
    GPTQ_LAUNCH(t, (packed_tile_kernel<T, kBits, kFine, kVec, kTT, kTR, kWaves, kPerCu, kRing, kGroups>), dim3(a.mt * a.nt), dim3(kGroups * kWaves * kWave), 0, s, a);
    return hipGetLastError();
}

}  // namespace

template <typename T, int kBits>
hipError_t launch_packed_tile(const PmArgs& a, int kernel, bool fine, hipStream_t s) {
    // (fine groups of unaligned rows have one tile, and never come with another)
    if (!a.vec && fine) return tile_go<T, kBits, true, false, 64, 128, 4, 2, 1, 1>(a, s);
    if (kernel == kPm32x64) {
        if (!a.vec) return tile_go<T, kBits, false, false, 32, 64, 4, 1, 1, 4>(a, s);
        return fine ? tile_go<T, kBits, true, true, 32, 64, 4, 1, 1, 4>(a, s) : tile_go<T, kBits, false, true, 32, 64, 4, 1, 4, 4>(a, s);
    }
    if (!a.vec) return tile_go<T, kBits, false, false, 64, 128, 4, 2, 1, 1>(a, s);
    if (fine) return tile_go<T, kBits, true, true, 64, 128, 4, 2, 4, 1>(a, s);
    if (kernel == kPm64x128) return tile_go<T, kBits, false, true, 64, 128, 4, 2, 4, 1>(a, s);
    return tile_go<T, kBits, false, true, 128, 384, 8, 1, 1, 1>(a, s);
}

}  // namespace gptq
