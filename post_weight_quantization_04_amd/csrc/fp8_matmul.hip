// Products of 8-bit operands: Y = act(X W^T) over e4m3 values with a scale per
// token and 128 channels (X) and per 128 x 128 block (W), and the gated
// feed-forward projections silu(X G^T) * (X U^T) with their result written in
// 8 bits again.
//
//   y[t, o] = sum_b xs[b, t] ws[o / 128, b] sum_{k in block b} xq[t, k] wq[o, k]
//
// The inner sum over a block of 128 runs on MFMA from zero; its result times
// the product of the two scales is added to the float32 accumulators.
//
// Two kinds of MFMA form the inner sum.  The e4m3 one (16x16x128) adds each
// lane's eight neighbouring k with 13 bits below the largest of the eight
// products and cuts the rest (measured: beside a product of 2^16, one of 2^3
// stays and one of 2^2 is lost), which leaves results about 2e-5 of their norm
// from exact.  The float16 one (four 16x16x32, the values converted in
// registers, every product exact) stays within 1e-7 at half the rate.  float16
// and bfloat16 outputs, whose last bit is 5e-4 and 4e-3, come from the e4m3
// MFMA in the tile kernel; float32 outputs and the gated block, whose scales
// are float32, from the float16 one, and so does everything the few-token
// kernel computes, which HBM bounds either way.
#include <algorithm>

#include "fp8_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

constexpr uint32_t kF8Out = 0x80000000u;  // an offset past every buffer: the load returns zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// An MFMA operand of 128 k as stored (e4m3) and as four float16 operands.
struct Halves {
    half8 h[4];
};

typedef _Float16 half2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ Halves to_halves(int8v v) {
    Halves r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        union {
            half2 p[4];
            half8 v;
        } u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            u.p[2 * j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + j], 1.0f, false);
            u.p[2 * j + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + j], 1.0f, true);
        }
        r.h[i] = u.v;
    }
    return r;
}

__device__ __forceinline__ float4v block_product(const Halves& a, const Halves& b) {
    float4v c = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.h[i], b.h[i], c, 0, 0, 0);
    return c;
}

// D = A B + C over 128 e4m3 values of k.  Lane l holds 32 consecutive k of row
// (A) or column (B) l % 16, the k group l / 16; result lane l holds
// C[4 (l / 16) + v][l % 16].  Both operands are loaded by the same map, so the
// sum does not depend on the order of k inside a group.
__device__ __forceinline__ float4v block_product(int8v a, int8v b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, (float4v){}, 0, 0, 0, 0, 0, 0);
}

template <bool kHalf>
struct Operand {
    typedef int8v type;
    static __device__ __forceinline__ type of(int8v v) { return v; }
};
template <>
struct Operand<true> {
    typedef Halves type;
    static __device__ __forceinline__ type of(int8v v) { return to_halves(v); }
};

__device__ __forceinline__ float relu_if(float y, int relu) { return relu && y < 0.0f ? 0.0f : y; }  // keeps NaN

// silu(g) u = g u / (1 + exp(-g)); exp overflows to infinity for g below -88,
// where the result is -0.  The hardware's reciprocal (one unit in the last
// place) takes the place of the division's ten instructions (8320 channels, k 72,
// 4671 tokens: 54.0 us for 61.6); 2^-64 keeps it a normal number.
__device__ __forceinline__ float gated(float g, float u) {
    return g * (__builtin_amdgcn_rcpf((1.0f + __expf(-g)) * 0x1p-64f) * 0x1p-64f) * u;
}

// Where chunk c of row r goes in the row's 128 bytes of LDS: c ^ f8_swizzle(r).
// A fragment read takes 16 bytes a lane, row l % 16, and LDS serves it sixteen
// lanes at a time: eight rows of one k group (0-3, 12-15) with the other eight
// (4-11) of the next, then the reverse (measured).  The next group's chunk is
// the same one with bit 1 flipped, so rows 4-11 repeat the others' values and
// the sixteen lanes take sixteen different chunks of two rows' 256 bytes.
__host__ __device__ constexpr int f8_swizzle(int r) { return (r / 2 % 2) | (r / 8 % 2) * 6; }

typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off, uint32_t base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, base, 0, 0);
}
__device__ __forceinline__ void copy4(__amdgpu_buffer_rsrc_t r, float* lds, uint32_t off, uint32_t base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, off, base, 0, 0);
}

// The fragment of sixteen rows at byte `at` of an LDS array that lane (l16, kg)
// holds: chunks 2 kg and 2 kg + 1 of row l16, which lie at at0 and at1 of the
// sixteen rows.  (The offsets are summed before they meet the array: the
// compiler tells arrays apart through a few steps of address arithmetic only,
// and where it cannot, a read waits for every copy in flight.)
__device__ __forceinline__ int8v f8_fragment(const uint8_t* lds, int at, int at0, int at1) {
    union {
        uint4v h[2];
        int8v v;
    } u;
    u.h[0] = *reinterpret_cast<const uint4v*>(lds + (at + at0));
    u.h[1] = *reinterpret_cast<const uint4v*>(lds + (at + at1));
    return u.v;
}

struct MmArgs {
    const uint8_t* wq[2];
    const float* ws[2];
    const uint8_t* xq;
    const float* xs;
    void* y;
    int64_t ldw, ldws, ldx, ldxs, ldy, M, n;
    int nb, channel_major, relu;
};

// ---------------------------------------------------------------------------
// Few tokens, and small products of more: sixteen weight rows and 16 kTn tokens
// a workgroup, so that the weights are read once for every 32 tokens.  The waves
// share the blocks of k and work on their own, without barriers: a wave copies
// its next two blocks to its own part of LDS (eight rows of 128 bytes
// an instruction; loads into registers would ask for 64 separate pieces of 16
// bytes, since neighbouring lanes of a fragment hold different rows, and the
// address unit bounds them: 16 us at 24 tokens of 11008 x 4096).  The waves'
// sums meet in LDS, added in wave order.  kOctets: rows of tokens that are
// copied, in eights (the others' columns are computed from whatever lies there
// and never stored).  Three or four blocks ahead: no faster (24 tokens of 11008 x
// 4096: 10.8 us, 11.2 and 10.7).
// ---------------------------------------------------------------------------
template <typename T, int kWaves, int kOctets, int kMats>
__global__ __launch_bounds__(kWaves* kWave) void f8_few_kernel(MmArgs a) {
    constexpr int kTn = (kOctets + 1) / 2;
    constexpr int kLoads = 2 * kMats + kOctets + kTn + kMats;  // vector memory instructions a block
    constexpr int kPart = 2048 * (kMats + kTn);                // a wave's part of a stage
    static_assert(kLoads < 64, "the wait counts to 63");
    static_assert(kMats * kTn * 1024 <= kPart, "the sums meet in the first stage");
    __shared__ __align__(16) uint8_t stage0[kWaves * kPart];
    __shared__ __align__(16) uint8_t stage1[kWaves * kPart];
    const int tid = threadIdx.x, lane = tid % kWave, w = wave_id();
    const int64_t r0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * kTn);
    const int rows = (int)min(a.M - r0, (int64_t)16), toks = (int)min(a.n - t0, (int64_t)(16 * kTn));
    const int nb = a.nb, l16 = lane % 16, kg = lane / 16;
    const uint32_t wbytes = (uint32_t)((rows - 1) * a.ldw + nb * kF8Block);
    const __amdgpu_buffer_rsrc_t rw = f8_rsrc(a.wq[0] + r0 * a.ldw, wbytes);
    const __amdgpu_buffer_rsrc_t ru = kMats == 2 ? f8_rsrc(a.wq[1] + r0 * a.ldw, wbytes) : rw;
    const __amdgpu_buffer_rsrc_t rx = f8_rsrc(a.xq + t0 * a.ldx, (uint32_t)((toks - 1) * a.ldx + nb * kF8Block));
    const __amdgpu_buffer_rsrc_t rws = f8_rsrc(a.ws[0] + (r0 / kF8Block) * a.ldws, (uint32_t)(4 * nb));
    const __amdgpu_buffer_rsrc_t rus =
        kMats == 2 ? f8_rsrc(a.ws[1] + (r0 / kF8Block) * a.ldws, (uint32_t)(4 * nb)) : rws;

    uint32_t ao[2], bo[kOctets], so[kTn];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + lane / 8;
        ao[i] = r < rows ? (uint32_t)(r * a.ldw + 16 * ((lane % 8) ^ f8_swizzle(r))) : kF8Out;
    }
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        const int r = 8 * i + lane / 8;
        bo[i] = r < toks ? (uint32_t)(r * a.ldx + 16 * ((lane % 8) ^ f8_swizzle(r))) : kF8Out;
    }
#pragma unroll
    for (int j = 0; j < kTn; ++j) so[j] = 16 * j + l16 < toks ? (uint32_t)(4 * (16 * j + l16)) : kF8Out;
    const int at0 = l16 * kF8Block + 16 * ((2 * kg) ^ f8_swizzle(l16));
    const int at1 = l16 * kF8Block + 16 * ((2 * kg + 1) ^ f8_swizzle(l16));

    float4v acc[kMats][kTn];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int j = 0; j < kTn; ++j) acc[m][j] = (float4v){};

    // the wave's i-th block; workgroups start at different ones, so that they
    // do not all ask for the same lines of X at once
    const int shift = nb > 0 ? (int)(blockIdx.x * 5u % (unsigned)nb) : 0;
    const int mine = w < nb ? (nb - w + kWaves - 1) / kWaves : 0;
    float xs[2][kTn], ws[2][kMats];
    auto copy = [&](uint8_t* stage, float (&x)[kTn], float (&s)[kMats], int i) {
        int b = w + min(i, mine - 1) * kWaves + shift;  // past the wave's last block, that one again, never used
        b = b >= nb ? b - nb : b;
        const uint32_t ko = (uint32_t)(b * kF8Block);
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c) copy16(m ? ru : rw, stage + (w * kPart + 2048 * m + 1024 * c), ao[c], ko);
#pragma unroll
        for (int c = 0; c < kOctets; ++c) copy16(rx, stage + (w * kPart + 2048 * kMats + 1024 * c), bo[c], ko);
        const __amdgpu_buffer_rsrc_t rs = f8_rsrc(a.xs + b * a.ldxs + t0, (uint32_t)(4 * toks));
#pragma unroll
        for (int j = 0; j < kTn; ++j) x[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, so[j], 0, 0));
        s[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rws, 4 * b, 0, 0));
        if (kMats == 2) s[kMats - 1] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rus, 4 * b, 0, 0));
    };
    auto step = [&](uint8_t* stage, float (&x)[kTn], float (&s)[kMats], int i) {
        // (the next step's scales, multiplied here, would wait for every load in flight)
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        int8v av[kMats], bv[kTn];
#pragma unroll
        for (int m = 0; m < kMats; ++m) av[m] = f8_fragment(stage, w * kPart + 2048 * m, at0, at1);
#pragma unroll
        for (int j = 0; j < kTn; ++j) bv[j] = f8_fragment(stage, w * kPart + 2048 * (kMats + j), at0, at1);
        float sc[kMats][kTn];
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
            for (int j = 0; j < kTn; ++j) sc[m][j] = x[j] * s[m];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before it is copied over
        copy(stage, x, s, i + 2);
        Halves bh[kTn];
#pragma unroll
        for (int j = 0; j < kTn; ++j) bh[j] = to_halves(bv[j]);
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            const Halves ah = to_halves(av[m]);
#pragma unroll
            for (int j = 0; j < kTn; ++j) {
                const float4v q = block_product(ah, bh[j]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[m][j][v] = fmaf(q[v], sc[m][j], acc[m][j][v]);
            }
        }
    };
    if (mine > 0) {
        copy(stage0, xs[0], ws[0], 0);
        copy(stage1, xs[1], ws[1], 1);
        int i = 0;
        for (; i + 2 <= mine; i += 2) {
            step(stage0, xs[0], ws[0], i);
            step(stage1, xs[1], ws[1], i + 1);
        }
        if (i < mine) step(stage0, xs[0], ws[0], i);
    }
    // every copy has landed before the memory is used for the sums
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    float* part = reinterpret_cast<float*>(stage0);  // [kWaves][kMats kTn][4][kWave]
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int j = 0; j < kTn; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) part[((w * kMats * kTn + m * kTn + j) * 4 + v) * kWave + lane] = acc[m][j][v];
    __syncthreads();
    // value i of the 256 kTn: token tile, register, lane
#pragma unroll
    for (int i = tid; i < 256 * kTn; i += kWaves * kWave) {
        const int j = i / 256, v = (i / kWave) % 4, l = i % kWave;
        float sum[kMats];
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            sum[m] = 0.0f;
#pragma unroll
            for (int ww = 0; ww < kWaves; ++ww) sum[m] += part[((ww * kMats * kTn + m * kTn + j) * 4 + v) * kWave + l];
        }
        const int t = 16 * j + l % 16, r = 4 * (l / 16) + v;
        if (t < toks && r < rows) {
            const float y = kMats == 2 ? gated(sum[0], sum[kMats - 1]) : relu_if(sum[0], a.relu);
            T* o = static_cast<T*>(a.y);
            if (a.channel_major) o[(r0 + r) * a.ldy + t0 + t] = (T)y;
            else o[(t0 + t) * a.ldy + r0 + r] = (T)y;
        }
    }
}

template <typename T, int kWaves, int kOctets, int kMats>
hipError_t few_go(const MmArgs& a, TimedLaunch t, hipStream_t s) {
    constexpr int kTn = (kOctets + 1) / 2;
    const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)((a.n + 16 * kTn - 1) / (16 * kTn)));
    GPTQ_LAUNCH(t, (f8_few_kernel<T, kWaves, kOctets, kMats>), grid, dim3(kWaves * kWave), 0, s, a);
    return hipGetLastError();
}

// Workgroups of the few-token kernel.
int64_t f8_few_groups(int64_t n, int64_t M) { return ((M + 15) / 16) * ((n + 31) / 32); }

// Eight waves share k where a workgroup has a CU to itself and blocks enough
// for them, four otherwise (two or three workgroups a CU then hide each other's
// ends): 11008 x 4096 weights, 24 tokens, 10.8 against 11.9 us; 4096 x 11008,
// one token, 9.8 against 9.5 us, 24 tokens 14.4 against 11.7 us; both
// projections of the gated block, one token, 22.2 against 18.9 us.
template <typename T, int kOctets, int kMats>
hipError_t few_waves(const MmArgs& a, TimedLaunch t, hipStream_t s) {
    if (f8_few_groups(a.n, a.M) <= device_cu_count() && a.nb >= 16) return few_go<T, 8, kOctets, kMats>(a, t, s);
    return few_go<T, 4, kOctets, kMats>(a, t, s);
}

template <typename T, int kMats>
hipError_t few_launch(const MmArgs& a, TimedLaunch t, hipStream_t s) {
    if (a.n <= 8) return few_waves<T, 1, kMats>(a, t, s);
    if (a.n <= 16) return few_waves<T, 2, kMats>(a, t, s);
    if (a.n <= 24) return few_waves<T, 3, kMats>(a, t, s);
    return few_waves<T, 4, kMats>(a, t, s);
}

// ---------------------------------------------------------------------------
// Many tokens: a workgroup computes kTM weight rows by kTN tokens, its waves
// (kWM x kWN) a rectangle each; kSplit groups of such waves share k, each with
// stages of its own, and add their sums at the end.  One block of k (128 bytes a
// row) of both operands is a stage; stages are copied from memory to LDS without
// passing registers, kStages - 1 ahead of the one in use, one barrier a stage.
//
// Bound by MFMA: 16384 x 11008 -> 4096 in 589 us, 2510 TFLOP/s (e4m3 MFMA, 63 %
// of the cycles busy); float32 8192 x 11008 -> 4096 in 538 us, 1370 TFLOP/s, and
// the gated block 8192 x 4096 -> 11008 in 1130 us, 1310 TFLOP/s (float16 MFMA,
// 52 % busy: the conversions and the scaling take the other cycles).  Four waves
// of twice the size in place of eight read less of LDS, and lose: 8192 x 11008
// -> 4096, 256 x 128 394 us against 338, 256 x 256 1130 against 297.
//
// A copy instruction of a wave places 64 x 16 bytes one after the other: eight
// rows of 128 bytes.  The chunk c of row r is put at c ^ f8_swizzle(r): each lane
// chooses its source accordingly.
//
// The gated form stages gate rows and the same up rows, and every wave holds
// both projections of its channels.  With 128 of each the workgroup holds whole
// blocks of the result, which it writes in 8 bits; smaller tiles store float32.
// ---------------------------------------------------------------------------
struct TileArgs {
    MmArgs m;
    uint8_t* q;  // gated: the 8-bit result
    float* qs;
    int64_t ldq, ldqs;
    unsigned mt, nt;  // tiles along the weight rows and the tokens
};

constexpr int kXcd = 8;
constexpr unsigned kBand = 8;  // tiles of weight rows that share their tokens before the next tokens

// Workgroup id -> tile.  Workgroups go to the eight XCDs in turn; each XCD gets
// a run of tiles, in bands of kBand tile rows, tokens outermost in a band, so
// that the tiles it works on at a time share rows in its own L2.
__device__ __forceinline__ void f8_tile_of(unsigned id, unsigned mt, unsigned nt, unsigned& mi, unsigned& ni) {
    const unsigned tiles = mt * nt, per = tiles / kXcd, rest = tiles % kXcd;
    const unsigned x = id % kXcd, i = id / kXcd;
    const unsigned t = x * per + min(x, rest) + i;
    const unsigned band = t / (kBand * nt), in = t % (kBand * nt);
    const unsigned rows = min(kBand, mt - band * kBand);
    mi = band * kBand + in % rows;
    ni = in / rows;
}

template <typename T, int kTM, int kTN, int kWM, int kWN, int kStages, int kSplit, bool kGated, bool kHalf, bool kChannels, bool kEarly, bool kCarry>
__global__ __launch_bounds__(kSplit* kWM* kWN* kWave) void f8_tile_kernel(TileArgs a) {
    constexpr int kWaves = kWM * kWN, kThreads = kWaves * kWave;  // of one group
    constexpr int kMt = kTM / kWM / 16, kNt = kTN / kWN / 16;
    constexpr int kAi = kTM / 8 / kWaves, kBi = kTN / 8 / kWaves;  // copy instructions of a wave and stage
    constexpr int kLoads = kAi + kBi + 1;                          // and one for the token scales
    static_assert(kTM % (8 * kWaves) == 0 && kTN % (8 * kWaves) == 0 && kTN % 64 == 0, "whole copies");
    static_assert(kTN / 64 <= kWaves && kWaves % (kTN / 64) == 0, "every wave copies one run of scales");
    constexpr bool kPack = kGated && kTM == 256;  // whole blocks of channels of both matrices, written in 8 bits
    static_assert(!kGated || kPack || kF8Block % (kTM / 2) == 0, "channels of one block");
    static_assert(kMt >= 2 && kNt >= 2, "tiles of a wave");
    constexpr int kABytes = kTM * kF8Block, kBBytes = kTN * kF8Block, kBytes = kABytes + kBBytes + 4 * kTN;
    // separate arrays: the compiler then knows that a read of one does not wait for copies into another
    __shared__ __align__(16) uint8_t lds0[kSplit * kBytes];
    __shared__ __align__(16) uint8_t lds1[kSplit * kBytes];
    __shared__ __align__(16) uint8_t lds2[kStages > 2 ? kSplit * kBytes : 16];
    static_assert(kStages == 2 || kStages == 3, "stages");
    static_assert(kSplit == 1 || !kPack, "whole blocks are not split");

    const MmArgs& m = a.m;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int group = kSplit > 1 ? wave_id() / kWaves : 0, w = wave_id() - group * kWaves;
    const int base = kSplit > 1 ? group * kBytes : 0;  // of the group's part of a stage
    const int wm = w / kWN, wn = w % kWN, l16 = lane % 16, kg = lane / 16;
    unsigned mi, ni;
    f8_tile_of(blockIdx.x, a.mt, a.nt, mi, ni);
    constexpr int kRows = kGated ? kTM / 2 : kTM;  // rows of one matrix
    const int64_t m0 = (int64_t)mi * kRows, t0 = (int64_t)ni * kTN;
    const int rows = (int)min(m.M - m0, (int64_t)kRows), toks = (int)min(m.n - t0, (int64_t)kTN);
    // the group's blocks of k: every kSplit-th, as many steps for every group
    const int nb = m.nb, steps = (nb + kSplit - 1) / kSplit;

    const __amdgpu_buffer_rsrc_t rw = f8_rsrc(m.wq[0] + m0 * m.ldw, (uint32_t)((rows - 1) * m.ldw + nb * kF8Block));
    const __amdgpu_buffer_rsrc_t ru =
        kGated ? f8_rsrc(m.wq[1] + m0 * m.ldw, (uint32_t)((rows - 1) * m.ldw + nb * kF8Block)) : rw;
    const __amdgpu_buffer_rsrc_t rx = f8_rsrc(m.xq + t0 * m.ldx, (uint32_t)((toks - 1) * m.ldx + nb * kF8Block));

    // Sources of this lane's copies: wave w copies rows 8 kAi w .. of A and 8 kBi
    // w .. of B, eight an instruction.  Every second instruction has the same
    // swizzle, so the first two offsets lead to all.  Rows past the last need no
    // test: a row's stride covers what is read of it, so they lie past the end
    // of the buffer, and load zero.
    auto source = [&](int r, int64_t ld) { return (uint32_t)(r * ld + 16 * ((lane % 8) ^ f8_swizzle(r))); };
    const int ar = 8 * kAi * w % kRows + lane / 8, br = 8 * kBi * w + lane / 8;
    const uint32_t ao[2] = {source(ar, m.ldw), source(ar + 8, m.ldw)};
    const uint32_t bo[2] = {source(br, m.ldx), source(br + 8, m.ldx)};
    auto advance = [](uint32_t off, int64_t ld, int c) {
        uint32_t by = (uint32_t)(16 * (c / 2) * ld);
        if (!kCarry) asm volatile("" : "+s"(by));  // added where it is used: kept over the loop, the sums cost registers
        return c < 2 ? off : off + by;
    };
    const int sr = 64 * (w % (kTN / 64));  // this wave's run of token scales
    const uint32_t so = sr + lane < toks ? (uint32_t)(4 * (sr + lane)) : kF8Out;
    const bool up = kGated && w >= kWaves / 2;  // rows of the up matrix (whole waves)

    // copy c of the wave's kLoads into stage st: the block of step i (past the last block, that one again, counted zero)
    auto copy = [&](uint8_t* st, int i, int c) {
        const int b = min(i * kSplit + group, nb - 1);
        const uint32_t ko = (uint32_t)(b * kF8Block);
        if (c < kAi) copy16(up ? ru : rw, st + (base + 1024 * (kAi * w + c)), advance(ao[c % 2], m.ldw, c), ko);
        else if (c < kAi + kBi) copy16(rx, st + (base + kABytes + 1024 * (kBi * w + c - kAi)), advance(bo[(c - kAi) & 1], m.ldx, c - kAi), ko);
        else {
            const __amdgpu_buffer_rsrc_t rs = f8_rsrc(m.xs + b * m.ldxs + t0, (uint32_t)(4 * toks));
            copy4(rs, reinterpret_cast<float*>(st + (base + kABytes + kBBytes + 4 * sr)), so, 0);
        }
    };

    float4v acc[kMt][kNt];
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int j = 0; j < kNt; ++j) acc[i][j] = (float4v){};

    constexpr int kWaveRows = kTM / kWM;
    // weight scales: a wave's rows lie in one block of 128 of each matrix
    const int64_t ob = (kGated ? m0 : m0 + wm * kWaveRows) / kF8Block;
    const bool live = kGated || m0 + wm * kWaveRows < m.M;
    const float* wsr = m.ws[0] + (live ? ob : 0) * m.ldws;
    const float* usr = kGated ? m.ws[1] + ob * m.ldws : nullptr;

    auto row_of = [&](int i) {  // first row of the wave's m-tile i in the stage
        if (!kGated) return wm * kWaveRows + 16 * i;
        return i < kMt / 2 ? wm * (kRows / kWM) + 16 * i : kRows + wm * (kRows / kWM) + 16 * (i - kMt / 2);
    };
    const int at0 = base + l16 * kF8Block + 16 * ((2 * kg) ^ f8_swizzle(l16));
    const int at1 = base + l16 * kF8Block + 16 * ((2 * kg + 1) ^ f8_swizzle(l16));
    auto rows_fragment = [&](const uint8_t* st, int i) { return f8_fragment(st, row_of(i) * kF8Block, at0, at1); };
    auto toks_fragment = [&](const uint8_t* st, int j) {
        return f8_fragment(st, kABytes + (wn * kNt + j) * 16 * kF8Block, at0, at1);
    };

    // What a step starts with, read from its stage while the step before ends:
    // the token fragments, the first weight fragment (kEarly; otherwise as the
    // step begins, for want of registers) and the token scales.
    constexpr int kMats = kGated ? 2 : 1;
    typedef typename Operand<kHalf>::type op_t;
    op_t bf[kNt];
    int8v raw;
    float sx[kNt];
    auto read_scales = [&](const uint8_t* st) {
#pragma unroll
        for (int j = 0; j < kNt; ++j)
            sx[j] = *reinterpret_cast<const float*>(st + (base + kABytes + kBBytes + 4 * ((wn * kNt + j) * 16 + l16)));
    };
    // products that are still to be scaled and added: two MFMAs old when that
    // happens, the last two of a step in the next one (kCarry)
    float4v late[2];
    float late_s[2] = {0.0f, 0.0f};
    late[0] = late[1] = (float4v){};
    auto add = [&](float4v& to, const float4v& p, float s) {
#pragma unroll
        for (int v = 0; v < 4; ++v) to[v] = fmaf(p[v], s, to[v]);
    };

    constexpr int kPerTile = 2;  // copies issued with the barrier and with each m-tile after it, all before the last
    constexpr int kPre = kPerTile;
    constexpr int kAhead = kStages - 1;

    // One block of k, from stage st.  Copies go to the block kAhead later, whose
    // stage `to` was free at the last barrier.  Before the last m-tile, with
    // every fragment of st in registers, the waves meet: the next stage `nx`
    // has landed for all of them, and st may be copied over.
    auto step = [&](uint8_t* st, uint8_t* nx, uint8_t* to, int b, float sw, float su) {
        float sc[kMats][kNt];
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            sc[0][j] = sx[j] * sw;
            if (kGated) sc[kMats - 1][j] = sx[j] * su;
        }
        int8v nraw[kEarly ? kNt : 1];
        if (!kEarly) {
            raw = rows_fragment(st, 0);
#pragma unroll
            for (int j = 0; j < kNt; ++j) bf[j] = Operand<kHalf>::of(toks_fragment(st, j));
        }
#pragma unroll
        for (int i = 0; i < kMt; ++i) {
            const op_t af = Operand<kHalf>::of(raw);
            if (i + 1 < kMt) {
                raw = rows_fragment(st, i + 1);
                constexpr int kLast = kMt - 2;
#pragma unroll
                for (int c = 0; c < kLoads; ++c)
                    if (c >= kPre && (i == kLast ? c >= kPre + i * kPerTile
                                                 : c >= kPre + i * kPerTile && c < kPre + (i + 1) * kPerTile))
                        copy(to, b + kAhead, c);
            } else {
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * kLoads) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int j = 0; kEarly && j < kNt; ++j) nraw[kEarly ? j : 0] = toks_fragment(nx, j);
                if (kEarly) raw = rows_fragment(nx, 0);
                read_scales(nx);
#pragma unroll
                for (int c = 0; c < kPre; ++c) copy(st, b + 1 + kAhead, c);
            }
#pragma unroll
            for (int j = 0; j < kNt; ++j) {
                const float4v p = block_product(af, bf[j]);
                const int g = kGated && i >= kMt / 2 ? kMats - 1 : 0;
                const int q = i * kNt + j;
                // the one two back: of this step or, for its first two, of the step before
                if (kCarry || q >= 2)
                    add(q >= 2 ? acc[(q - 2) / kNt][(q - 2) % kNt] : acc[kMt - 1][kNt - 2 + q], late[q % 2], late_s[q % 2]);
                late[q % 2] = p;
                late_s[q % 2] = sc[g][j];
                if (kEarly && i == kMt - 1) bf[j] = Operand<kHalf>::of(nraw[kEarly ? j : 0]);
            }
            __builtin_amdgcn_sched_barrier(0);  // left alone, the scheduler reads every fragment first and spills
        }
        if (!kCarry) {
            add(acc[kMt - 1][kNt - 2], late[0], late_s[0]);
            add(acc[kMt - 1][kNt - 1], late[1], late_s[1]);
        }
    };
    if (nb > 0) {
        // the weight scales of kMany steps at a time, one a lane (the first ones
        // ahead of the copies: loads return in order)
        constexpr int kMany = 64 / kStages * kStages;
        int wl, ul;
        auto load_scales = [&](int i0) {
            const int at = (i0 + lane) * kSplit + group;
            wl = __builtin_bit_cast(int, at < nb ? wsr[at] : 0.0f);
            ul = kGated ? __builtin_bit_cast(int, at < nb ? usr[at] : 0.0f) : 0;
        };
        load_scales(0);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
#pragma unroll
            for (int c = 0; c < kLoads; ++c) copy(d == 0 ? lds0 : lds1, d, c);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        uint8_t* const last = kStages == 2 ? lds1 : lds2;
#pragma unroll
        for (int j = 0; j < kNt; ++j) bf[j] = Operand<kHalf>::of(toks_fragment(lds0, j));
        raw = rows_fragment(lds0, 0);
        read_scales(lds0);
#pragma unroll
        for (int c = 0; c < kPre; ++c) copy(last, kAhead, c);

        for (int i0 = 0; i0 < steps; i0 += kMany) {
            const int run = min(kMany, steps - i0);
            if (i0 > 0) load_scales(i0);
            auto go = [&](uint8_t* st, uint8_t* nx, uint8_t* to, int i) {
                step(st, nx, to, i0 + i, __builtin_bit_cast(float, __builtin_amdgcn_readlane(wl, i)),
                     kGated ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(ul, i)) : 0.0f);
            };
            uint8_t* const after1 = kStages > 2 ? lds2 : lds0;
            int i = 0;
            if constexpr (!kCarry && kStages == 2) {
                // (an odd step of its own, as below, was compiled with many registers spilled)
                for (; i < run; i += 2) {
                    go(lds0, lds1, last, i);
                    if (i + 1 == run) break;
                    go(lds1, after1, lds0, i + 1);
                }
                continue;
            }
            // no branch between the steps of the loop: the compiler would move
            // the scaling of products past it and keep them all in registers
            for (; i + kStages <= run; i += kStages) {
                go(lds0, lds1, last, i);
                go(lds1, after1, lds0, i + 1);
                if (kStages > 2) go(lds2, lds0, lds1, i + 2);
            }
            if (i < run) go(lds0, lds1, last, i);
            if (kStages > 2 && i + 1 < run) go(lds1, after1, lds0, i + 1);
        }
        if (kCarry) {
            add(acc[kMt - 1][kNt - 2], late[0], late_s[0]);
            add(acc[kMt - 1][kNt - 1], late[1], late_s[1]);
        }
    }
    // copies still in flight would land in memory that the epilogue (or the
    // next workgroup) uses
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    if (kSplit > 1) {
        // the groups' sums, added in group order
        constexpr int kOne = kWaves * kMt * kNt * 4 * kWave;
        static_assert(kSplit == 1 || 4 * (kSplit - 1) * kOne <= kSplit * kBytes, "the sums in the second stages");
        float* sums = reinterpret_cast<float*>(lds1);
        auto at = [&](int g, int i, int j, int v) -> float& {
            return sums[(g - 1) * kOne + (((w * kMt + i) * kNt + j) * 4 + v) * kWave + lane];
        };
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) at(group, i, j, v) = acc[i][j][v];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < kSplit; ++g)
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] += at(g, i, j, v);
    }
    if (kPack) {
        uint32_t* peaks = reinterpret_cast<uint32_t*>(lds1);  // [kWM][kTN]
        uint32_t* codes = reinterpret_cast<uint32_t*>(lds0);  // [kTN][kCodePitch]
        constexpr int kCodePitch = kF8Block / 4 + 1;
        static_assert(4 * kTN * kCodePitch <= kABytes + kBBytes && 4 * kWM * kTN <= kABytes, "epilogue's LDS");
        uint32_t pk[kNt];
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            pk[j] = 0;
#pragma unroll
            for (int i = 0; i < kMt / 2; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    acc[i][j][v] = gated(acc[i][j][v], acc[i + kMt / 2][j][v]);
                    pk[j] = max(pk[j], abs_bits(acc[i][j][v]));
                }
            pk[j] = max(pk[j], (uint32_t)__shfl_xor((int)pk[j], 16, kWave));
            pk[j] = max(pk[j], (uint32_t)__shfl_xor((int)pk[j], 32, kWave));
            if (kg == 0) peaks[wm * kTN + (wn * kNt + j) * 16 + l16] = pk[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
            const int t = (wn * kNt + j) * 16 + l16;
            uint32_t p = 0;
#pragma unroll
            for (int g = 0; g < kWM; ++g) p = max(p, peaks[g * kTN + t]);
            const float s = f8_scale(p), inv = 1.0f / s;
            if (wm == 0 && kg == 0 && t < toks) a.qs[(int64_t)mi * a.ldqs + t0 + t] = s;
#pragma unroll
            for (int i = 0; i < kMt / 2; ++i)
                codes[t * kCodePitch + (wm * (kRows / kWM) + 16 * i) / 4 + kg] =
                    f8_pack4(acc[i][j][0] * inv, acc[i][j][1] * inv, acc[i][j][2] * inv, acc[i][j][3] * inv);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTN * 8 / kThreads; ++i) {
            const int t = (i * kThreads + tid) / 8, c = 4 * (tid % 8);
            const uint32_t* r = codes + t * kCodePitch + c;
            if (t < toks)
                *reinterpret_cast<uint4v*>(a.q + (t0 + t) * a.ldq + m0 + 4 * c) = (uint4v){r[0], r[1], r[2], r[3]};
        }
        return;
    }
    // A lane holds four neighbouring channels of one token.  A wave turns sixteen
    // lines of Y at a time (a line: one token's channels, or one channel's tokens)
    // in LDS of its own and stores whole runs of them.  (For channel-major Y the
    // MFMA's operands could change places, a lane then holding four tokens of a
    // channel: it needs four token scales a product, for which the largest tile
    // has no registers: float32 8192 x 4096 -> 4096 282 us, so 220.  Smaller
    // tiles take the same time either way.)
    if (kGated) {
#pragma unroll
        for (int i = 0; i < kMt / 2; ++i)
#pragma unroll
            for (int j = 0; j < kNt; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = gated(acc[i][j][v], acc[i + kMt / 2][j][v]);
    }
    constexpr int kMo = kGated ? kMt / 2 : kMt, kOutRows = kRows / kWM;  // of a wave
    constexpr int kRun = kChannels ? 16 * kNt : 16 * kMo, kOuter = kChannels ? kMo : kNt, kInner = kChannels ? kNt : kMo;
    constexpr int kPitch = kRun * (int)sizeof(T) + 16, kVec = 16 / (int)sizeof(T);
    // (float32 lines of the largest tile need both stages; in the split form a
    // slower wave may still read its sums from the second)
    constexpr bool kBoth = kWaves * 16 * kPitch > kBytes;
    static_assert(kPack || !kBoth || (kSplit == 1 && kWaves / 2 * 16 * kPitch <= kBytes), "the lines of every wave");
    uint8_t* lines = kBoth && w >= kWaves / 2 ? lds1 + (w - kWaves / 2) * 16 * kPitch : lds0 + w * 16 * kPitch;
    T* y = static_cast<T*>(m.y);
    const int first = kChannels ? wn * kRun : wm * kRun;           // of the run, within the tile
    const int left = (kChannels ? toks : rows) - first;            // of the run, within Y
    const int64_t start = (kChannels ? t0 : m0) + first;
#pragma unroll
    for (int o = 0; o < kOuter; ++o) {
#pragma unroll
        for (int k = 0; k < kInner; ++k) {
            const float4v& v = acc[kChannels ? o : k][kChannels ? k : o];
            struct alignas(4 * sizeof(T)) { T e[4]; } out;
#pragma unroll
            for (int e = 0; e < 4; ++e) out.e[e] = (T)relu_if(v[e], m.relu);
            if (kChannels) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<T*>(lines + (4 * kg + e) * kPitch + (16 * k + l16) * sizeof(T)) = out.e[e];
            } else {
                *reinterpret_cast<decltype(out)*>(lines + l16 * kPitch + (16 * k + 4 * kg) * sizeof(T)) = out;
            }
        }
        __builtin_amdgcn_wave_barrier();
        const int line0 = kChannels ? wm * kOutRows + 16 * o : (wn * kNt + o) * 16;
        const int count = (kChannels ? rows : toks) - line0;       // lines within Y
        T* base = y + ((kChannels ? m0 : t0) + line0) * m.ldy + start;
        // (16 bytes at a time; Y's lines need no more than their type's alignment)
        constexpr int kPer = kRun / kVec;
#pragma unroll
        for (int q = 0; q < 16 * kPer / kWave; ++q) {
            const int line = (q * kWave + lane) / kPer, at = (q * kWave + lane) % kPer * kVec;
            const uint4v v = *reinterpret_cast<const uint4v*>(lines + line * kPitch + at * sizeof(T));
            if (line >= count) continue;
            T* o = base + line * m.ldy + at;
            if (at + kVec <= left) __builtin_memcpy(o, &v, 16);
            else {
                T e[kVec];
                __builtin_memcpy(e, &v, 16);
#pragma unroll
                for (int k = 0; k < kVec - 1; ++k)
                    if (at + k < left) o[k] = e[k];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int kTM, int kTN, int kWM, int kWN, int kStages, bool kGated, bool kHalf, int kSplit = 1, bool kEarly = true, bool kCarry = true>
hipError_t tile_launch(TileArgs a, TimedLaunch t, hipStream_t s) {
    constexpr int kRows = kGated ? kTM / 2 : kTM;
    a.mt = (unsigned)((a.m.M + kRows - 1) / kRows);
    a.nt = (unsigned)((a.m.n + kTN - 1) / kTN);
    const dim3 grid(a.mt * a.nt), block(kSplit * kWM * kWN * kWave);
    if (!kGated && a.m.channel_major)
        GPTQ_LAUNCH(t, (f8_tile_kernel<T, kTM, kTN, kWM, kWN, kStages, kSplit, kGated, kHalf, !kGated, kEarly, kCarry>), grid, block, 0, s, a);
    else
        GPTQ_LAUNCH(t, (f8_tile_kernel<T, kTM, kTN, kWM, kWN, kStages, kSplit, kGated, kHalf, false, kEarly, kCarry>), grid, block, 0, s, a);
    return hipGetLastError();
}

constexpr int64_t kFewTokens = 32;  // the few-token kernel always, up to here

// Which kernel and tile, by estimated time: rounds of tiles over the CUs, each
// with a part of its own (its first copies, its epilogue) and one for a block of
// k, in us with every CU at work (the time to write Y is the same for all and
// left out):
//                   256 x 256   256 x 128   128 x 128   128 x 64*  64 x 64, three a CU  two   one*
//   e4m3 MFMA       1.3 + 1.8   1.5 + 1.05  1.7 + 0.58  2.6 + 0.33  1.4 + 0.5   2.2 + 0.41  2.5 + 0.2
//   float16 MFMA    0.4 + 3.0   0.5 + 1.8               2.6 + 0.55  1.4 + 1.3   2.2 + 0.76  2.5 + 0.35
// (*: two groups of waves share k).  The parts fit whole times over many sizes;
// they do not split one launch's time (256 x 128, 2048 tokens, 4096 rows: 8.7 us
// at one block, 14.8 at 8, 33.8 at 32, 62.4 at 64, Y included).  The few-token
// kernel, which runs workgroups of sixteen rows by 32 tokens and reads the
// weights again for each 32: 1.3 us, 0.002 a workgroup and, a block, 0.07 and
// 0.0003 a workgroup.  Measured, 4096 x 4096 weights, e4m3: 256
// tokens 10.7 us in 64 x 64 tiles (13.4 in one group), 13.4 in 128 x 64, 29 in
// 256 x 128; 512 tokens 14.6 in 128 x 64, 16.5 in 64 x 64; 1024 tokens 22 in 128
// x 128, 28 in 128 x 64, 31 in 256 x 128; 4096 tokens 59 in 256 x 256 (float32
// 107), 76 in 256 x 128 (float32 119), 112 in 64 x 64.  14919 tokens, k 1024, 1280
// rows: 36 us in 256 x 256, 35 in 256 x 128, 37 in 128 x 128, 46 in 64 x 64
// (float32 63, 60, -, 66).  The few-token kernel against 64 x 64 tiles: 512 rows,
// k 4096, 100 tokens 5.4 against 8.1 us (float32 13.6); 1363 rows, 200 tokens
// 12.0 against 10.4 (15.2); 5376 rows, 64 tokens 12.0 against 9.6 (14.4).
enum F8Kernel { kFew, k64Split, k64, k128x64Split, k128, k256x128, k256 };
const char* const kF8KernelNames[] = {"few tokens", "64 x 64, k in two groups", "64 x 64", "128 x 64, k in two groups", "128 x 128",
                                      "256 x 128", "256 x 256"};

F8Kernel f8_matmul_choice(int64_t M, int64_t n, int nb, bool half, int64_t cus) {
    if (n <= kFewTokens) return kFew;
    auto rounds = [&](int64_t tm, int64_t tn, int64_t each) {
        return (((M + tm - 1) / tm) * ((n + tn - 1) / tn) + cus * each - 1) / (cus * each);
    };
    const bool one = rounds(64, 64, 1) == 1, two = rounds(64, 64, 2) == 1;
    auto cost = [&](int64_t rounds, double own, double block) { return rounds * (own + block * nb); };
    const double groups = (double)f8_few_groups(n, M);
    // (its grid's second dimension, 32 tokens each, holds less than 2^16)
    const double few = n > ((int64_t)1 << 20) ? 1e30 : 1.3 + 0.002 * groups + (0.07 + 0.0003 * groups) * nb;
    double t[] = {few, one ? cost(1, 2.5, 0.2) : 1e30, two ? cost(1, 2.2, 0.41) : cost(rounds(64, 64, 3), 1.4, 0.5),
                  cost(rounds(128, 64, 1), 2.6, 0.33), cost(rounds(128, 128, 1), 1.7, 0.58),
                  cost(rounds(256, 128, 1), 1.5, 1.05), cost(rounds(256, 256, 1), 1.3, 1.8)};
    if (half) {
        t[k64Split] = one ? cost(1, 2.5, 0.35) : 1e30;
        t[k64] = two ? cost(1, 2.2, 0.76) : cost(rounds(64, 64, 3), 1.4, 1.3);
        t[k128x64Split] = cost(rounds(128, 64, 1), 2.6, 0.55);
        t[k128] = 1e30;
        t[k256x128] = cost(rounds(256, 128, 1), 0.5, 1.8);
        t[k256] = cost(rounds(256, 256, 1), 0.4, 3.0);
    }
    if (one) t[k64] = 1e30;
    return (F8Kernel)(std::min_element(t, t + 7) - t);
}

template <typename T, bool kHalf>
hipError_t matmul_typed(const MmArgs& m, hipStream_t s) {
    TimedLaunch t(K_F8_MATMUL, s);
    const int64_t cus = m.n <= kFewTokens ? 1 : device_cu_count();
    if (cus <= 0) return hipErrorInvalidDevice;
    TileArgs a = {};
    a.m = m;
    switch (f8_matmul_choice(m.M, m.n, m.nb, kHalf, cus)) {
        case kFew: return few_launch<T, 1>(m, t, s);
        case k64Split: return tile_launch<T, 64, 64, 2, 2, 3, false, kHalf, 2>(a, t, s);
        case k64: return tile_launch<T, 64, 64, 2, 2, 3, false, kHalf>(a, t, s);
        case k128x64Split: return tile_launch<T, 128, 64, 2, 2, 3, false, kHalf, 2>(a, t, s);
        case k128:
            if constexpr (!kHalf) return tile_launch<T, 128, 128, 4, 2, 3, false, false>(a, t, s);
            break;
        case k256x128: return tile_launch<T, 256, 128, 4, 2, kHalf ? 2 : 3, false, kHalf>(a, t, s);
        case k256: return tile_launch<T, 256, 256, 2, 4, 2, false, kHalf, 1, !kHalf, !kHalf>(a, t, s);
    }
    return hipErrorInvalidValue;
}

// Up to here the gated block may leave its products in float32: few tokens, or
// tiles of 128 channels by 64 tokens that leave half of 256 CUs idle.  The
// workspace's size goes by this rule, so it knows neither k nor the device; the
// choice below, which does, may still take one kernel.
constexpr int64_t kGatedTiles = 128;
bool f8_gated_in_two(int64_t n, int64_t M) {
    return n <= kFewTokens || ((M + kF8Block - 1) / kF8Block) * ((n + 63) / 64) <= kGatedTiles;
}

}  // namespace

hipError_t launch_f8_matmul(const F8Product& c, int y_dtype, hipStream_t s) {
    MmArgs a = {{c.wq[0], nullptr}, {c.ws[0], nullptr}, c.xq, c.xs, c.y, c.ldw, c.ldws, c.ldx, c.ldxs, c.ldy, c.M, c.n,
                (int)((c.K + kF8Block - 1) / kF8Block), c.channel_major, c.relu};
    if (y_dtype == 0) return matmul_typed<half_t, false>(a, s);
    if (y_dtype == 1) return matmul_typed<float, true>(a, s);
    return matmul_typed<bf16_t, false>(a, s);
}

size_t f8_gated_workspace_bytes(int64_t n, int64_t d_ff) {
    if (!f8_gated_in_two(n, d_ff)) return 0;
    return (size_t)(n * ((d_ff + kF8Block - 1) / kF8Block) * kF8Block) * sizeof(float);
}

namespace {

enum F8GatedKernel { kGatedFew, kGated32, kGated64, kGated128x64, kGated128x128, kGated128x256 };
const char* const kF8GatedNames[] = {"few tokens, then the quantizer", "32 channels x 64, k in two groups, then the quantizer",
                                     "64 channels x 64, k in two groups, then the quantizer", "128 channels x 64",
                                     "128 channels x 128", "128 channels x 256"};

// In one kernel: tiles of 128 channels, which are whole blocks of the result,
// 64, 128 or 256 tokens wide.  At 256 a wave converts fewer values for its
// products (192 an m-tile for four token tiles of twice the rows, against 128),
// but holds no registers for fragments ahead.  In two: a kernel that leaves the
// products in float32, the few-token one or tiles of 64 or 32 channels by 64
// tokens in two groups of waves, and the activations' quantizer.
//
// The choice goes by estimated time, as for the product: rounds of tiles over
// the CUs, each with a part of its own (start, epilogue) and one for a block of
// k; the forms in two parts 2 us more.  Measured, 11008 channels, k 4096: 64
// tokens 35.5 us in one kernel, 26.6 in 64-channel tiles, 33.6 in 32-channel
// ones, 38.6 with the few-token kernel; 128 tokens 40 in one kernel; 1024 tokens
// 208, 174 and 204 for 64, 128 and 256 tokens wide; 4096 tokens 776, 640 and
// 616.  1408 channels, k 4096, 100 tokens: 33.8, 22.0, 17.1 and 12.9 with the
// few-token kernel; 200 tokens 34.1, 22.4, 18.4 and 18.1.  8320 channels, k
// 128, 4671 tokens: 91, 65 and 50 us for 64, 128 and 256 tokens wide.
F8GatedKernel f8_gated_choice(int64_t M, int64_t n, int nb, int64_t cus) {
    if (n <= kFewTokens) return kGatedFew;
    auto cost = [&](int64_t channels, int64_t tokens, double own, double block) {
        const int64_t tiles = ((M + channels - 1) / channels) * ((n + tokens - 1) / tokens);
        return ((tiles + cus - 1) / cus) * (own + block * nb);
    };
    double t[] = {1e30, 1e30, 1e30, cost(128, 64, 4.0, 0.97), cost(128, 128, 4.9, 1.73), cost(128, 256, 7.0, 3.1)};
    if (f8_gated_in_two(n, M)) {
        const double groups = (double)f8_few_groups(n, M);
        const double two[] = {3.4 + 0.0032 * groups + (0.08 + 0.00037 * groups) * nb, cost(32, 64, 4.0, 0.32),
                              cost(64, 64, 5.0, 0.47)};
        for (int i = 0; i < 3; ++i) t[i] = two[i] + 2.0;
        const double one = std::min(t[3], std::min(t[4], t[5]));
        for (int i = 0; i < 3; ++i)
            if (!(t[i] < one)) t[i] = 1e30;
    }
    return (F8GatedKernel)(std::min_element(t, t + 6) - t);
}

}  // namespace

const char* f8_matmul_kernel_name(int64_t M, int64_t K, int64_t n, int y_dtype, int64_t cus) {
    return kF8KernelNames[f8_matmul_choice(M, n, (int)((K + kF8Block - 1) / kF8Block), y_dtype == 1, cus)];
}

const char* f8_gated_kernel_name(int64_t M, int64_t K, int64_t n, int64_t cus) {
    return kF8GatedNames[f8_gated_choice(M, n, (int)((K + kF8Block - 1) / kF8Block), cus)];
}

hipError_t launch_f8_gated(const F8Product& c, uint8_t* q, int64_t ldq, float* scales, int64_t lds, void* ws,
                           hipStream_t s) {
    const int64_t cus = device_cu_count();
    if (cus <= 0) return hipErrorInvalidDevice;
    const int nb = (int)((c.K + kF8Block - 1) / kF8Block);
    const F8GatedKernel kernel = f8_gated_choice(c.M, c.n, nb, cus);
    const bool two = kernel <= kGated64;
    const int64_t ldh = (c.M + kF8Block - 1) / kF8Block * kF8Block;
    TileArgs t = {};
    t.m = {{c.wq[0], c.wq[1]}, {c.ws[0], c.ws[1]}, c.xq, c.xs, two ? ws : nullptr, c.ldw, c.ldws, c.ldx, c.ldxs,
           two ? ldh : 0, c.M, c.n, nb, 0, 0};
    t.q = q;
    t.qs = scales;
    t.ldq = ldq;
    t.ldqs = lds;
    const TimedLaunch k(K_F8_GATED, s);
    hipError_t e = hipErrorInvalidValue;
    switch (kernel) {
        case kGatedFew: e = few_launch<float, 2>(t.m, k, s); break;
        case kGated32: e = tile_launch<float, 64, 64, 2, 2, 3, true, true, 2>(t, k, s); break;
        case kGated64: e = tile_launch<float, 128, 64, 2, 2, 3, true, true, 2>(t, k, s); break;
        case kGated128x64: return tile_launch<float, 256, 64, 4, 2, 3, true, true>(t, k, s);
        case kGated128x128: return tile_launch<float, 256, 128, 4, 2, 2, true, true>(t, k, s);
        case kGated128x256: return tile_launch<float, 256, 256, 2, 4, 2, true, true, 1, false, false>(t, k, s);
    }
    if (e != hipSuccess) return e;
    return launch_f8_activations(ws, 1, c.n, c.M, ldh, 0, q, ldq, scales, lds, s);
}

}  // namespace gptq
