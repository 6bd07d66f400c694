// Product with packed few-bit weights, bias, activation and residual:
//   y[t, o] = act( sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[t, k] + b[o] ) + r[t, o]
// The differences q - z are whole numbers that both 16-bit types hold, so MFMA
// forms their products with x exactly and sums them in float32; a group's sum
// (or a part of it) times its scale is added in float32.  The scale is never
// multiplied into 16-bit weights, which would round each of them.
//
// Tokens are the rows of the MFMA's result and weight rows its columns: a lane's
// values belong to one weight row, so that scale and zero are one value a lane.
//
// This file: few tokens, and which kernel a product is sent to.
#include <algorithm>

#include "packed_common.hpp"
#include "packed_tile.hpp"

namespace gptq {

namespace {

// ---------------------------------------------------------------------------
// Few tokens: sixteen weight rows and 16 kTn tokens a workgroup, whose waves
// share the blocks of 128 columns and work on their own, without barriers.  A
// lane loads a run of 32 codes of its row (64 neighbouring bytes for the four
// lanes of a row at four bits), and of x what stands beside one MFMA step, 64
// neighbouring bytes of a token, which is why the codes are turned: read by runs,
// x would come in 64 pieces of 16 bytes.  Two blocks are in flight a wave.  The
// waves' sums meet in LDS, added in wave order.
// ---------------------------------------------------------------------------
template <typename T, int kBits, bool kFine, int kWaves, int kTn>
__global__ __launch_bounds__(kWaves* kWave) void packed_few_kernel(PmArgs a) {
    constexpr int kScales = kFine ? 8 : 1;  // of a block
    __shared__ float sums[kWaves][kTn][4][kWave];
    typedef typename Mat<T>::v8 v8;
    const PackedProduct& c = a.c;
    const int tid = threadIdx.x, lane = tid % kWave, w = wave_id(), l16 = lane % 16, kg = lane / 16;
    const int64_t r0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * kTn);
    const int rows = (int)min(c.M - r0, (int64_t)16);
    const int row = min(l16, rows - 1);
    const __amdgpu_buffer_rsrc_t rw = pm_rsrc(c.packed + r0 * a.nw, (uint32_t)rows * (uint32_t)a.nw * 4u);
    const uint32_t wo = 4u * ((uint32_t)row * (uint32_t)a.nw + (uint32_t)(kg * kBits));
    const float* scales = c.scales + (r0 + row) * a.ng;
    const int32_t* zeros = c.zeros + (r0 + row) * a.ng;
    const T* x[kTn];
#pragma unroll
    for (int j = 0; j < kTn; ++j)
        x[j] = static_cast<const T*>(c.x) + min(t0 + 16 * j + l16, c.n - 1) * c.ldx + 8 * kg;
    const int nb = a.nb;
    const bool ragged = c.K % kPmBlock != 0;

    struct Block {
        uint32_t w[kBits];
        v8 x[kTn][4];
        float s[kScales];
        int z[2];
    };
    auto load = [&](Block& g, int b) {
        b = min(b, nb - 1);  // past the last block, that one again, never used
        const bool tail = ragged && b == nb - 1;
        const uint32_t k0 = (uint32_t)b * kPmBlock;
        load_run<kBits>(g.w, rw, wo, (uint32_t)b * (16u * kBits), tail);
        if (kFine) {
            g.z[0] = zeros[group_of(a, k0 + 32 * kg)];
            g.z[1] = zeros[group_of(a, k0 + 32 * kg + 16)];
#pragma unroll
            for (int i = 0; i < kScales; ++i) g.s[i] = scales[group_of(a, k0 + 16 * i)];
        } else {
            const uint32_t at = group_of(a, k0);
            g.z[0] = g.z[1] = zeros[at];
            g.s[0] = scales[at];
        }
#pragma unroll
        for (int j = 0; j < kTn; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const T* p = x[j] + (k0 + 32 * e);
                if (!tail) {
                    __builtin_memcpy(&g.x[j][e], p, 16);
                } else {
                    const int left = (int)c.K - (int)(k0 + 32 * e + 8 * kg);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g.x[j][e][i] = i < left ? p[i] : (T)0.0f;
                }
            }
    };
    float4v acc[kTn];
#pragma unroll
    for (int j = 0; j < kTn; ++j) acc[j] = (float4v){};
    auto use = [&](const Block& g) {
        frag_t f[4];
        codes32<T, kBits>(f, g.w, g.z[0], g.z[1]);
        turn_blocks(f);
#pragma unroll
        for (int j = 0; j < kTn; ++j) {
            if (!kFine) {
                float4v p = {};
#pragma unroll
                for (int e = 0; e < 4; ++e) p = Mat<T>::mfma16(g.x[j][e], __builtin_bit_cast(v8, f[e]), p);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(p[v], g.s[0], acc[j][v]);
            } else {
                // sixteen columns at a time: the others' codes as zeros
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const frag_t half = kg / 2 == h % 2 ? f[h / 2] : (frag_t){};
                    const v8 xh = kg / 2 == h % 2 ? g.x[j][h / 2] : (v8){};  // an infinity times zero would be NaN
                    const float4v p = Mat<T>::mfma16(xh, __builtin_bit_cast(v8, half), (float4v){});
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(p[v], g.s[h], acc[j][v]);
                }
            }
        }
    };
    const int mine = w < nb ? (nb - w + kWaves - 1) / kWaves : 0;
    if (mine > 0) {
        Block g0, g1;
        load(g0, w);
        load(g1, w + kWaves);
        int i = 0;
        for (; i + 2 <= mine; i += 2) {
            use(g0);
            load(g0, w + (i + 2) * kWaves);
            use(g1);
            load(g1, w + (i + 3) * kWaves);
        }
        if (i < mine) use(g0);
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
            y = activated(y, c.activation);
            if (c.residual) y += static_cast<const float*>(c.residual)[t * c.ldr + o];
            static_cast<float*>(c.y)[t * c.ldy + o] = y;
        } else {
            if (c.bias) y += to_f32(static_cast<const T*>(c.bias)[o]);
            y = activated(y, c.activation);
            if (c.residual) y += to_f32(static_cast<const T*>(c.residual)[t * c.ldr + o]);
            static_cast<T*>(c.y)[t * c.ldy + o] = (T)y;
        }
    }
}

template <typename T, int kBits, bool kFine, int kWaves, int kTn>
hipError_t few_go(const PmArgs& a, hipStream_t s) {
    const TimedLaunch t(K_PACKED_MATMUL, s);
    const dim3 grid((unsigned)((a.c.M + 15) / 16), (unsigned)((a.c.n + 16 * kTn - 1) / (16 * kTn)));
    GPTQ_LAUNCH(t, (packed_few_kernel<T, kBits, kFine, kWaves, kTn>), grid, dim3(kWaves * kWave), 0, s, a);
    return hipGetLastError();
}

template <typename T, int kBits, bool kFine>
hipError_t few_launch(const PmArgs& a, hipStream_t s) {
    if (a.c.n <= 16) return few_go<T, kBits, kFine, 8, 1>(a, s);
    return few_go<T, kBits, kFine, 8, 2>(a, s);
}

constexpr int64_t kPmFewTokens = 32;  // the few-token kernel up to here

template <typename T, int kBits>
hipError_t bits_go(const PmArgs& a, hipStream_t s) {
    const bool fine = a.group % kPmBlock != 0 && a.ng > 1;
    if (a.c.n <= kPmFewTokens) return fine ? few_launch<T, kBits, true>(a, s) : few_launch<T, kBits, false>(a, s);
    return launch_packed_tile<T, kBits>(a, fine, s);
}

template <typename T>
hipError_t typed_go(const PmArgs& a, hipStream_t s) {
    switch (a.c.bits) {
        case 2: return bits_go<T, 2>(a, s);
        case 3: return bits_go<T, 3>(a, s);
        case 4: return bits_go<T, 4>(a, s);
        case 5: return bits_go<T, 5>(a, s);
        case 6: return bits_go<T, 6>(a, s);
        case 7: return bits_go<T, 7>(a, s);
        default: return bits_go<T, 8>(a, s);
    }
}

}  // namespace

hipError_t launch_packed_matmul(const PackedProduct& c, int x_dtype, int y_dtype, hipStream_t s) {
    PmArgs a = {};
    a.c = c;
    a.nw = (int)((c.K * c.bits + 31) / 32);
    a.ng = (int)(c.group && c.K ? c.K / c.group : 1);
    a.nb = (int)((c.K + kPmBlock - 1) / kPmBlock);
    a.group = (uint32_t)std::max<int64_t>(c.group ? c.group : c.K, 1);
    while (((uint64_t)1 << a.group_shift) < a.group) ++a.group_shift;
    a.group_mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << a.group_shift) - a.group)) / a.group + 1);
    a.y32 = y_dtype == 1;
    return x_dtype == 0 ? typed_go<half_t>(a, s) : typed_go<bf16_t>(a, s);
}

}  // namespace gptq
