// Writers of the 8-bit format: weights (one scale per 128 x 128 block),
// activations (one scale per token and 128 channels) and the root-mean-square
// norm with the residual's addition, whose output is written in that format.
//
// A block's scale is s = max(peak, 2^-96) / 448 with peak its largest
// magnitude, and its codes are e4m3(fl32(x fl32(1/s))), nearest even.  Every
// kernel reads its input once, holds it in registers between the peak and the
// conversion, and is bound by HBM.
#include "fp8_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

constexpr int kQThreads = kF8RowsThreads;

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// ---------------------------------------------------------------------------
// weights: one workgroup per 128 x 128 block; thread t holds columns
// 8 (t % 16) .. +8 of rows t / 16 + 64 i.  The codes are stored nontemporally
// (a layer is quantized once and read much later): 11008 x 4096 float16 in
// 22.0 us, 6150 GB/s, where a large copy reaches 5230.  Timed together: 24.4 us,
// 32.1 with plain stores; 512 and 256 threads 24.7 and 26.6 us, at 128 x 248
// bfloat16 3.4 and 4.3 us against 3.2.
// ---------------------------------------------------------------------------
constexpr int kWThreads = kF8WeightThreads;
constexpr int kWRows = 128 * 16 / kWThreads;  // rows a thread

template <typename T, bool kVec>
__global__ __launch_bounds__(kWThreads) void f8_weight_kernel(const T* __restrict__ W, int64_t M, int64_t K, int64_t ldw,
                                                              uint8_t* __restrict__ q, int64_t ldq,
                                                              float* __restrict__ scales, int64_t lds, unsigned nb) {
    __shared__ uint32_t peaks[kWThreads / kWave];
    const int tid = threadIdx.x;
    const int64_t bi = blockIdx.x / nb, bj = blockIdx.x % nb;
    const int64_t row0 = bi * kF8Block, col = bj * kF8Block + 8 * (tid % 16);
    float v[kWRows][8];
#pragma unroll
    for (int i = 0; i < kWRows; ++i) {
        const int64_t r = row0 + tid / 16 + kWThreads / 16 * i;
        load8<T, kVec>(v[i], W + r * ldw + col, r < M ? K - col : 0);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kWRows; ++i) m = max(m, peak8(v[i]));
    m = row16_max(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
    if (tid % kWave == 0) peaks[tid / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWThreads / kWave; ++w) m = max(m, peaks[w]);
    const float s = f8_scale(m), inv = 1.0f / s;
    if (tid == 0) scales[bi * lds + bj] = s;
#pragma unroll
    for (int i = 0; i < kWRows; ++i) {
        const int64_t r = row0 + tid / 16 + kWThreads / 16 * i;
        if (r < M) __builtin_nontemporal_store(f8_pack8(v[i], inv), reinterpret_cast<uint2v*>(q + r * ldq + col));
    }
}

// ---------------------------------------------------------------------------
// activations, token-major: sixteen lanes per (token, block), eight channels
// a lane.  X is loaded nontemporally.  16384 x 4096 float16 in 38.3 us, 5310
// GB/s, the rate of a large copy; two, four or eight blocks a lane, their loads
// in flight together, 39.0, 41.5 and 42.3 us.
// ---------------------------------------------------------------------------
template <typename T, bool kVec>
__global__ __launch_bounds__(kQThreads) void f8_rows_kernel(const T* __restrict__ X, unsigned blocks, int64_t d,
                                                            int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scales, int64_t lds, unsigned nb) {
    const int tid = threadIdx.x;
    const unsigned id = blockIdx.x * (kQThreads / 16) + tid / 16;
    if (id >= blocks) return;  // sixteen lanes, a whole DPP row, together
    const int64_t row = id / nb, blk = id % nb, c = blk * kF8Block + 8 * (tid % 16);
    float v[8];
    load8<T, kVec, true>(v, X + row * ldx + c, d - c);
    const float s = f8_scale(row16_max(peak8(v))), inv = 1.0f / s;
    *reinterpret_cast<uint2v*>(q + row * ldq + c) = f8_pack8(v, inv);
    if (tid % 16 == 0) scales[blk * lds + row] = s;
}

// ---------------------------------------------------------------------------
// activations, channel-major: one workgroup per 128 channels x kCmTokens
// tokens; thread t holds channels 4 (t / kCmEights) + i (i < 4) of tokens
// 8 (t % kCmEights) .. +8.  The peaks meet in LDS, and the codes turn there: a
// thread's four channels of a token are one 32-bit word, stored where the
// lanes of a wave write 64 distinct banks, read back as 32 bytes of a token.
// X is loaded nontemporally.  4096 x 16384 float16 in 36.9 us, 5520 GB/s, past
// the rate of a large copy; 128 tokens a workgroup 44.2 us (49.2 with X kept in
// the caches), or tokens before channels in the order of the workgroups 46 us.
// ---------------------------------------------------------------------------
constexpr int kCmTokens = 64;
constexpr int kCmEights = kCmTokens / 8;
constexpr int kCmThreads = 32 * kCmEights;
static_assert(kCmThreads == kF8ColumnsThreads && kCmTokens == 64, "the entry point's limit");

// word of (token, four channels): rows of 33 words
__device__ __forceinline__ int cm_word(int token, int quad) { return token * (kF8Block / 4 + 1) + quad; }

template <typename T, bool kVec>
__global__ __launch_bounds__(kCmThreads) void f8_columns_kernel(const T* __restrict__ X, int64_t n, int64_t d,
                                                                int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ scales, int64_t lds, unsigned nb) {
    constexpr int kWaves = kCmThreads / kWave;
    __shared__ uint32_t peaks[kWaves][kCmTokens];
    __shared__ uint32_t codes[kCmTokens * (kF8Block / 4 + 1)];
    const int tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
    const int64_t blk = blockIdx.x % nb, t0 = (int64_t)(blockIdx.x / nb) * kCmTokens;
    const int64_t t = t0 + 8 * (tid % kCmEights), c0 = blk * kF8Block + 4 * (tid / kCmEights);
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) load8<T, kVec, true>(v[i], X + (c0 + i) * ldx + t, c0 + i < d ? n - t : 0);
    uint32_t m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = max(max(abs_bits(v[0][e]), abs_bits(v[1][e])), max(abs_bits(v[2][e]), abs_bits(v[3][e])));
#pragma unroll
        for (int o = kCmEights; o < kWave; o <<= 1) m[e] = max(m[e], (uint32_t)__shfl_xor((int)m[e], o, kWave));
    }
    if (lane < kCmEights) {
#pragma unroll
        for (int e = 0; e < 8; ++e) peaks[w][8 * lane + e] = m[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int tt = 8 * (tid % kCmEights) + e;
        uint32_t p = 0;
#pragma unroll
        for (int g = 0; g < kWaves; ++g) p = max(p, peaks[g][tt]);
        const float s = f8_scale(p), inv = 1.0f / s;
        if (tid < kCmEights && t + e < n) scales[blk * lds + t + e] = s;
        codes[cm_word(tt, tid / kCmEights)] = f8_pack4(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv);
    }
    __syncthreads();
    const int64_t tok = t0 + tid / 4;
    if (tok >= n) return;
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = codes[cm_word(tid / 4, 8 * (tid % 4) + e)];
    uint4v* dst = reinterpret_cast<uint4v*>(q + tok * ldq + blk * kF8Block + 32 * (tid % 4));
    dst[0] = (uint4v){r[0], r[1], r[2], r[3]};
    dst[1] = (uint4v){r[4], r[5], r[6], r[7]};
}

// ---------------------------------------------------------------------------
// root-mean-square norm: h = x + r, y = h / sqrt(mean h^2 + eps) * gain
//
// kThreads threads per row, chunks of eight channels: chunk c = t + kThreads j,
// so that sixteen neighbouring lanes hold one block of 128.  kJ chunks a
// thread stay in registers between the sum and the conversion; kJ = 0 is the
// form for rows past that, which reads x and r a second time (and writes h
// only then, so that h may overwrite x or r).  Bound by HBM: 16384 x 4096
// bfloat16 with a residual in 89.7 us, 5260 GB/s, the rate of a large copy.
// ---------------------------------------------------------------------------
template <typename T>
struct NormArgs {
    const T* x;
    const T* r;     // or null
    T* sum;         // or null
    const T* gain;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldr, ldo, ldq, lds, n;
    int d, chunks;  // chunks = 16 ceil(d / 128)
    float eps;
};

template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float* part, int tid) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    if (kThreads == kWave) return v;
    if (tid % kWave == 0) part[tid / kWave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) s += part[w];
    __syncthreads();
    return s;
}

template <typename T, bool kVec>
__device__ __forceinline__ void norm_load(float (&h)[8], const T* x, const T* r, int c, int d) {
    load8<T, kVec>(h, x + 8 * c, d - 8 * c);
    if (r) {
        float b[8];
        load8<T, kVec>(b, r + 8 * c, d - 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += b[e];
    }
}

__device__ __forceinline__ float sum_squares(const float (&h)[8], float by) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = h[e] * by;
        s += v * v;
    }
    return s;
}

// Squares of values above 2^64 leave float32: such a row's sum is formed again
// with every value scaled by 2^-80 (exact, and eps is then far below the last
// bit).  A row that holds an infinity or a NaN keeps it.
constexpr float kSmall = 0x1p-80f;

template <typename T>
__device__ __forceinline__ void norm_chunk_out(const NormArgs<T>& a, float (&h)[8], const float (&g)[8], float inv,
                                               int64_t row, int c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = h[e] * inv * g[e];
    const float s = f8_scale(row16_max(peak8(h)));
    if (c < a.chunks) {
        *reinterpret_cast<uint2v*>(a.q + row * a.ldq + 8 * c) = f8_pack8(h, 1.0f / s);
        if (c % 16 == 0) a.scales[(int64_t)(c / 16) * a.lds + row] = s;
    }
}

template <typename T, int kThreads, int kRows, int kJ, bool kVec>
__global__ __launch_bounds__(kThreads* kRows) void f8_rms_norm_kernel(NormArgs<T> a) {
    static_assert(kThreads * kRows <= kF8NormThreads, "the entry point's limit");
    __shared__ float part[kThreads / kWave];
    const int tid = threadIdx.x % kThreads;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kThreads;
    if (row >= a.n) return;  // whole waves: kThreads is a multiple of 64, and one row per workgroup where it is more
    const T* x = a.x + row * a.ldx;
    const T* r = a.r ? a.r + row * a.ldr : nullptr;
    T* sum = a.sum ? a.sum + row * a.ldo : nullptr;
    if (kJ > 0) {
        float h[kJ > 0 ? kJ : 1][8], g[kJ > 0 ? kJ : 1][8];
#pragma unroll
        for (int j = 0; j < kJ; ++j) norm_load<T, kVec>(h[j], x, r, tid + kThreads * j, a.d);
#pragma unroll
        for (int j = 0; j < kJ; ++j) load8<T, kVec>(g[j], a.gain + 8 * (tid + kThreads * j), a.d - 8 * (tid + kThreads * j));
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            if (sum) store8<T, kVec>(sum + 8 * (tid + kThreads * j), h[j], a.d - 8 * (tid + kThreads * j));
            ss += sum_squares(h[j], 1.0f);
        }
        ss = row_sum<kThreads>(ss, part, tid);
        float inv = 1.0f / sqrtf(ss / (float)a.d + a.eps);
        if (!(ss < INFINITY)) {
            float s2 = 0.0f;
#pragma unroll
            for (int j = 0; j < kJ; ++j) s2 += sum_squares(h[j], kSmall);
            s2 = row_sum<kThreads>(s2, part, tid);
            inv = kSmall / sqrtf(s2 / (float)a.d);
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) norm_chunk_out(a, h[j], g[j], inv, row, tid + kThreads * j);
    } else {
        float ss = 0.0f;
        for (int c = tid; c < a.chunks; c += kThreads) {
            float h[8];
            norm_load<T, kVec>(h, x, r, c, a.d);
            ss += sum_squares(h, 1.0f);
        }
        ss = row_sum<kThreads>(ss, part, tid);
        float inv = 1.0f / sqrtf(ss / (float)a.d + a.eps);
        if (!(ss < INFINITY)) {
            float s2 = 0.0f;
            for (int c = tid; c < a.chunks; c += kThreads) {
                float h[8];
                norm_load<T, kVec>(h, x, r, c, a.d);
                s2 += sum_squares(h, kSmall);
            }
            s2 = row_sum<kThreads>(s2, part, tid);
            inv = kSmall / sqrtf(s2 / (float)a.d);
        }
        // chunks is a multiple of 16, so the sixteen lanes of a block run the loop together
        for (int c = tid; c < a.chunks; c += kThreads) {
            float h[8], g[8];
            norm_load<T, kVec>(h, x, r, c, a.d);
            load8<T, kVec>(g, a.gain + 8 * c, a.d - 8 * c);
            if (sum) store8<T, kVec>(sum + 8 * c, h, a.d - 8 * c);
            norm_chunk_out(a, h, g, inv, row, c);
        }
    }
}

template <typename T, bool kVec>
hipError_t norm_launch(const NormArgs<T>& a, TimedLaunch t, hipStream_t s) {
    const unsigned n = (unsigned)a.n;
    if (a.chunks <= 64) GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 64, 4, 1, kVec>), dim3((n + 3) / 4), dim3(256), 0, s, a);
    else if (a.chunks <= 256) GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 256, 1, 1, kVec>), dim3(n), dim3(256), 0, s, a);
    else if (a.chunks <= 512) GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 256, 1, 2, kVec>), dim3(n), dim3(256), 0, s, a);
    else if (a.chunks <= 1024) GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 512, 1, 2, kVec>), dim3(n), dim3(512), 0, s, a);
    else if (a.chunks <= 2048) GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 512, 1, 4, kVec>), dim3(n), dim3(512), 0, s, a);
    else GPTQ_LAUNCH(t, (f8_rms_norm_kernel<T, 512, 1, 0, kVec>), dim3(n), dim3(512), 0, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t norm_typed(const RmsNormCall& c, hipStream_t s) {
    NormArgs<T> a;
    a.x = static_cast<const T*>(c.x);
    a.r = static_cast<const T*>(c.residual);
    a.sum = static_cast<T*>(c.sum_out);
    a.gain = static_cast<const T*>(c.gain);
    a.q = c.q;
    a.scales = c.scales;
    a.ldx = c.ldx;
    a.ldr = c.ldr;
    a.ldo = c.ldo;
    a.ldq = c.ldq;
    a.lds = c.lds;
    a.n = c.n;
    a.d = (int)c.d;
    a.chunks = (int)((c.d + kF8Block - 1) / kF8Block) * (kF8Block / 8);
    a.eps = (float)c.eps;
    const bool vec = c.d % 8 == 0 && aligned16(c.x) && aligned16(c.gain) && c.ldx * sizeof(T) % 16 == 0 &&
                     (!c.residual || (aligned16(c.residual) && c.ldr * sizeof(T) % 16 == 0)) &&
                     (!c.sum_out || (aligned16(c.sum_out) && c.ldo * sizeof(T) % 16 == 0));
    TimedLaunch t(K_F8_NORM, s);
    return vec ? norm_launch<T, true>(a, t, s) : norm_launch<T, false>(a, t, s);
}

template <typename T>
hipError_t weight_typed(const void* W, int64_t M, int64_t K, int64_t ldw, uint8_t* q, int64_t ldq, float* scales,
                        int64_t lds, hipStream_t s) {
    const T* w = static_cast<const T*>(W);
    const unsigned nb = (unsigned)((K + kF8Block - 1) / kF8Block), rb = (unsigned)((M + kF8Block - 1) / kF8Block);
    TimedLaunch t(K_F8_WEIGHT, s);
    if (aligned16(W) && K % 8 == 0 && ldw * sizeof(T) % 16 == 0)
        GPTQ_LAUNCH(t, (f8_weight_kernel<T, true>), dim3(nb * rb), dim3(kWThreads), 0, s, w, M, K, ldw, q, ldq, scales, lds, nb);
    else
        GPTQ_LAUNCH(t, (f8_weight_kernel<T, false>), dim3(nb * rb), dim3(kWThreads), 0, s, w, M, K, ldw, q, ldq, scales, lds, nb);
    return hipGetLastError();
}

template <typename T>
hipError_t rows_typed(const void* X, int64_t n, int64_t d, int64_t ldx, uint8_t* q, int64_t ldq, float* scales,
                      int64_t lds, hipStream_t s) {
    const T* x = static_cast<const T*>(X);
    const unsigned nb = (unsigned)((d + kF8Block - 1) / kF8Block), blocks = (unsigned)n * nb;
    constexpr unsigned kPer = kQThreads / 16;
    const dim3 grid((blocks + kPer - 1) / kPer);
    TimedLaunch t(K_F8_ROWS, s);
    if (aligned16(X) && d % 8 == 0 && ldx * sizeof(T) % 16 == 0)
        GPTQ_LAUNCH(t, (f8_rows_kernel<T, true>), grid, dim3(kQThreads), 0, s, x, blocks, d, ldx, q, ldq, scales, lds, nb);
    else
        GPTQ_LAUNCH(t, (f8_rows_kernel<T, false>), grid, dim3(kQThreads), 0, s, x, blocks, d, ldx, q, ldq, scales, lds, nb);
    return hipGetLastError();
}

template <typename T>
hipError_t columns_typed(const void* X, int64_t n, int64_t d, int64_t ldx, uint8_t* q, int64_t ldq, float* scales,
                         int64_t lds, hipStream_t s) {
    const T* x = static_cast<const T*>(X);
    const unsigned nb = (unsigned)((d + kF8Block - 1) / kF8Block), nt = (unsigned)((n + kCmTokens - 1) / kCmTokens);
    TimedLaunch t(K_F8_COLUMNS, s);
    if (aligned16(X) && n % 8 == 0 && ldx * sizeof(T) % 16 == 0)
        GPTQ_LAUNCH(t, (f8_columns_kernel<T, true>), dim3(nb * nt), dim3(kCmThreads), 0, s, x, n, d, ldx, q, ldq, scales, lds, nb);
    else
        GPTQ_LAUNCH(t, (f8_columns_kernel<T, false>), dim3(nb * nt), dim3(kCmThreads), 0, s, x, n, d, ldx, q, ldq, scales, lds, nb);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_weight(const void* W, int dtype, int64_t M, int64_t K, int64_t ldw, uint8_t* q, int64_t ldq,
                            float* scales, int64_t lds, hipStream_t s) {
    if (dtype == 0) return weight_typed<half_t>(W, M, K, ldw, q, ldq, scales, lds, s);
    if (dtype == 1) return weight_typed<float>(W, M, K, ldw, q, ldq, scales, lds, s);
    return weight_typed<bf16_t>(W, M, K, ldw, q, ldq, scales, lds, s);
}

hipError_t launch_f8_activations(const void* X, int dtype, int64_t n, int64_t d, int64_t ldx, int channel_major,
                                 uint8_t* q, int64_t ldq, float* scales, int64_t lds, hipStream_t s) {
    if (channel_major) {
        if (dtype == 0) return columns_typed<half_t>(X, n, d, ldx, q, ldq, scales, lds, s);
        if (dtype == 1) return columns_typed<float>(X, n, d, ldx, q, ldq, scales, lds, s);
        return columns_typed<bf16_t>(X, n, d, ldx, q, ldq, scales, lds, s);
    }
    if (dtype == 0) return rows_typed<half_t>(X, n, d, ldx, q, ldq, scales, lds, s);
    if (dtype == 1) return rows_typed<float>(X, n, d, ldx, q, ldq, scales, lds, s);
    return rows_typed<bf16_t>(X, n, d, ldx, q, ldq, scales, lds, s);
}

hipError_t launch_f8_rms_norm(const RmsNormCall& c, int dtype, hipStream_t s) {
    if (dtype == 0) return norm_typed<half_t>(c, s);
    if (dtype == 1) return norm_typed<float>(c, s);
    return norm_typed<bf16_t>(c, s);
}

}  // namespace gptq
