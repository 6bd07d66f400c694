// The kernel of products with packed few-bit weights for few tokens.
#pragma once

#include "packed_tile.hpp"

namespace gptq {

namespace {

// ---------------------------------------------------------------------------
// Few tokens: sixteen weight rows and 4 kQuads tokens a workgroup, whose waves
// share the blocks of 128 columns and work on their own, without barriers.  A
// wave loads a block's codes into registers and copies its piece of x to LDS of
// its own, two blocks ahead; codes are turned, since x read in the order of the
// columns takes all banks, and so that small groups come out alone.  (x in
// registers straight from memory asks for 64 pieces of sixteen bytes an
// instruction: 24 tokens of 11008 x 4096 in 23.8 us.)  The waves' sums meet in
// LDS, added in wave order.
//
// One token of 4096 x 4096, 4 bits: 4.8 us, 1.8 TB/s, of which 3 are the launch and
// the first loads (bfloat16 5.5); 1 x 4096 -> 11008 9.4; 24 x 11008 -> 4096 13.6, bfloat16
// 14.9, 1.6 TB/s, bound by the conversions, which every 32 tokens repeat, and their waits.
// ---------------------------------------------------------------------------
template <typename T, int kBits, bool kFine, bool kVec, int kWaves, int kQuads>
__global__ __launch_bounds__(kWaves* kWave) void packed_few_kernel(PmArgs a) {
    constexpr int kTn = (kQuads + 3) / 4;
    constexpr int kScales = kFine ? 2 : 1;  // of a lane: of a run of 32 codes, halves of it
    constexpr int kPart = kTn * 4096;       // a wave's part of a stage
    __shared__ __align__(16) uint8_t lds0[kWaves * kPart];
    __shared__ __align__(16) uint8_t lds1[kWaves * kPart];
    __shared__ float sums[kWaves][kTn][4][kWave];
    typedef typename Mat<T>::v8 v8;
    const PackedProduct& c = a.c;
    const int tid = threadIdx.x, lane = tid % kWave, w = wave_id(), l16 = lane % 16, kg = lane / 16;
    const int64_t r0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (4 * kQuads);
    const int rows = (int)min(c.M - r0, (int64_t)16), toks = (int)min(c.n - t0, (int64_t)(4 * kQuads));
    const int nb = a.nb;
    const T* x = static_cast<const T*>(c.x) + t0 * c.ldx;
    const __amdgpu_buffer_rsrc_t rw = pm_rsrc(c.packed + r0 * a.nw, (uint32_t)rows * (uint32_t)a.nw * 4u);
    const __amdgpu_buffer_rsrc_t rs = pm_rsrc(c.scales + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    const __amdgpu_buffer_rsrc_t rz = pm_rsrc(c.zeros + r0 * a.ng, (uint32_t)rows * (uint32_t)a.ng * 4u);
    uint32_t first = 0;
    const uint32_t elements = (uint32_t)((toks - 1) * c.ldx + c.K);
    const __amdgpu_buffer_rsrc_t rx = kVec ? pm_rsrc(x, 2 * elements) : pm_words_rsrc(x, elements, first);
    const uint32_t wo = 4u * ((uint32_t)(lane / 4) * (uint32_t)a.nw + (uint32_t)(lane % 4 * kBits));
    const uint32_t so = 4u * (uint32_t)(lane / 4) * (uint32_t)a.ng;
    uint32_t xo[kQuads];
    auto chunk_of = [&](int i) { return (lane % 16) ^ pm_swizzle((4 * i + lane / 16) % 16); };
#pragma unroll
    for (int i = 0; i < kQuads; ++i) xo[i] = (kVec ? 2 : 1) * ((uint32_t)(4 * i + lane / 16) * (uint32_t)c.ldx + 8u * (uint32_t)chunk_of(i)) + first;

    struct Block {
        uint32_t w[kBits], s[kScales], z[2];
        PmWords x[kVec ? 1 : kQuads];
        int left;
    };
    auto load = [&](Block& g, uint8_t* st, int b) {
        b = min(b, nb - 1);  // past the last block, that one again, never used
        const uint32_t k0 = (uint32_t)b * kPmBlock;
        load_run<kBits>(g.w, rw, wo, (uint32_t)b * (16u * kBits));
        if (kFine) {
#pragma unroll
            for (int h = 0; h < kScales; ++h) {
                const uint32_t at = so + 4 * group_of(a, k0 + 32 * (lane % 4) + 16 * h);
                g.z[h] = __builtin_amdgcn_raw_buffer_load_b32(rz, at, 0, 0);
                g.s[h] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
            }
        } else {
            const uint32_t at = 4 * group_of(a, k0);
            g.z[0] = __builtin_amdgcn_raw_buffer_load_b32(rz, so, at, 0);
            g.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, so, at, 0);
        }
        const int left = g.left = (int)(c.K - k0);  // what follows the last column is not the row's
        if (kVec) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i)
                pm_copy16(rx, st + (w * kPart + 1024 * i), 8 * chunk_of(i) < left ? xo[i] : kPmOut, 2 * k0);
        } else {
#pragma unroll
            for (int i = 0; i < kQuads; ++i) g.x[i] = pm_words(rx, xo[i], 2 * k0);
        }
    };
    float4v acc[kTn];
#pragma unroll
    for (int j = 0; j < kTn; ++j) acc[j] = (float4v){};
    auto use = [&](const Block& g, uint8_t* st) {
        if (!kVec) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i)
                *reinterpret_cast<frag_t*>(st + (w * kPart + 1024 * i + 16 * lane)) = pm_columns(g.x[i], xo[i], g.left - 8 * chunk_of(i));
        }
        uint32_t mine[kBits];
        frag_t f[4];
#pragma unroll
        for (int q = 0; q < kBits; ++q) mine[q] = from_row(g.w[q], 4 * l16 + kg);
        const int z = (int)from_row(g.z[0], 4 * l16 + (kFine ? kg : 0));
        codes32<T, kBits>(f, mine, z, kFine ? (int)from_row(g.z[1], 4 * l16 + kg) : z);
        turn_blocks(f);
        float s[kFine ? 8 : 1];
#pragma unroll
        for (int h = 0; h < (kFine ? 8 : 1); ++h) s[h] = __builtin_bit_cast(float, from_row(g.s[h % kScales], 4 * l16 + h / 2));
#pragma unroll
        for (int j = 0; j < kTn; ++j) {
            v8 xf[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                xf[e] = *reinterpret_cast<const v8*>(st + (w * kPart + (16 * j + l16) * 2 * kPmBlock + 16 * ((4 * e + kg) ^ pm_swizzle(l16))));
            if (!kFine) {
                float4v p = {};
#pragma unroll
                for (int e = 0; e < 4; ++e) p = Mat<T>::mfma16(xf[e], __builtin_bit_cast(v8, f[e]), p);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(p[v], s[0], acc[j][v]);
            } else {
                // sixteen columns at a time, the others as zeros (of both: an infinity times zero would be NaN)
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const frag_t half = kg / 2 == h % 2 ? f[h / 2] : (frag_t){};
                    const v8 xh = kg / 2 == h % 2 ? xf[h / 2] : (v8){};
                    const float4v p = Mat<T>::mfma16(xh, __builtin_bit_cast(v8, half), (float4v){});
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(p[v], s[h], acc[j][v]);
                }
            }
        }
    };
    const int mine = w < nb ? (nb - w + kWaves - 1) / kWaves : 0;
    if (mine > 0) {
        Block g0, g1;
        load(g0, lds0, w);
        load(g1, lds1, w + kWaves);
        auto go = [&](Block& g, uint8_t* st, int i) {
            use(g, st);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before it is copied over
            load(g, st, w + (i + 2) * kWaves);
        };
        int i = 0;
        for (; i + 2 <= mine; i += 2) {
            go(g0, lds0, i);
            go(g1, lds1, i + 1);
        }
        if (i < mine) use(g0, lds0);
    }
#pragma unroll
    for (int j = 0; j < kTn; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) sums[w][j][v][lane] = acc[j][v];
    __syncthreads();
    // value i of the 256 kTn: token tile, register, lane
    for (int i = tid; i < 256 * kTn; i += kWaves * kWave) {
        const int j = i / 256, v = i / kWave % 4, l = i % kWave;
        float y = 0.0f;
#pragma unroll
        for (int ww = 0; ww < kWaves; ++ww) y += sums[ww][j][v][l];
        const int64_t t = t0 + 16 * j + 4 * (l / 16) + v, o = r0 + l % 16;
        if (t >= c.n || o >= c.M) continue;
        if (a.y32) {
            if (c.bias) y += static_cast<const float*>(c.bias)[o];
            y = activated(y, c.activation, true);
            if (c.residual) y += static_cast<const float*>(c.residual)[t * c.ldr + o];
            static_cast<float*>(c.y)[t * c.ldy + o] = y;
        } else {
            if (c.bias) y += to_f32(static_cast<const T*>(c.bias)[o]);
            y = activated(y, c.activation, false);
            if (c.residual) y += to_f32(static_cast<const T*>(c.residual)[t * c.ldr + o]);
            static_cast<T*>(c.y)[t * c.ldy + o] = (T)y;
        }
    }
}

template <typename T, int kBits, bool kFine, bool kVec, int kWaves, int kQuads>
hipError_t few_go(const PmArgs& a, hipStream_t s) {
    const TimedLaunch t(K_PACKED_MATMUL, s);
    const dim3 grid((unsigned)((a.c.M + 15) / 16), (unsigned)((a.c.n + 4 * kQuads - 1) / (4 * kQuads)));
    GPTQ_LAUNCH(t, (packed_few_kernel<T, kBits, kFine, kVec, kWaves, kQuads>), grid, dim3(kWaves * kWave), 0, s, a);
    return hipGetLastError();
}

template <typename T, int kBits, bool kFine>
hipError_t few_launch(const PmArgs& a, hipStream_t s) {
    if (!a.vec) return a.c.n <= 4 ? few_go<T, kBits, kFine, false, 8, 1>(a, s) : few_go<T, kBits, kFine, false, 8, 8>(a, s);
    if (a.c.n <= 4) return few_go<T, kBits, kFine, true, 8, 1>(a, s);
    if (a.c.n <= 16) return few_go<T, kBits, kFine, true, 8, 4>(a, s);
    return few_go<T, kBits, kFine, true, 8, 8>(a, s);
}

}  // namespace

template <typename T, int kBits>
hipError_t launch_packed_few(const PmArgs& a, bool fine, hipStream_t s) {
    return fine ? few_launch<T, kBits, true>(a, s) : few_launch<T, kBits, false>(a, s);
}

}  // namespace gptq
