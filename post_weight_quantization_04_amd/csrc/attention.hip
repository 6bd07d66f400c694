// Attention over whole prompts, several sequences packed one behind the other:
//   y[i, h] = sum_j p_ij v[j, h'],  p_ij = softmax over j of scale q[i, h] . k[j, h']
// with a running maximum and sum per row, so that scores never leave the
// registers.
//
// The query heads that share a key head are rows of one tile: row r stands for
// token r / rows_per_token and head r % rows_per_token, so that a key is read
// once for all of them and short prompts fill a tile.  A wave has 32 rows, as
// columns of S^T = K Q^T and of O^T = V^T P^T (MFMA 32x32x16): a lane's scores,
// maximum, sum and outputs belong to one row, the two halves of the wave hold
// alternate runs of four keys of it, and P^T leaves the first product in the
// layout that the second takes.  Keys and values come 64 at a time, copied
// straight to LDS one tile ahead, one barrier a tile; values are read turned.
//
// Bound by MFMA and the softmax's arithmetic in turn: 8192 causal tokens, 32 heads of
// 128 over 8, float16 553 to 590 us by the clocks the card holds (994 to 930 TFLOP/s),
// bfloat16 521 to 566; MFMA is busy in 49% of the cycles, VALU in 43%, and two waves a SIMD
// do not lay one over the other.  Heads of 96 take 516 us and of 80 499, as 128 with zeros;
// of 64 310.
// Four waves a workgroup: two (keys copied twice as often) and eight (more waiting at
// the barrier) are slower, and so is one loop for whole and masked tiles, which spills
// (731 us).  77 tokens 9.3 us: a chain of two tiles of keys, a launch and the stores.
#include "attention_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer: the load returns zero
constexpr int kTileKeys = 64;

struct AttArgs {
    AttentionCall c;
    int rows;         // query heads of a key head in a tile (at most 16): rows per token
    int head_groups;  // tiles that share a key head
    int tokens;       // of a tile
    unsigned units, tiles;
    float c2;         // scale log2 e
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t att_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
}

// First token of sequence s (of n: the end of the last), whatever stands there.
__device__ __forceinline__ int64_t start_of(const AttArgs& a, int64_t s) {
    if (!a.c.starts) return s == 0 ? 0 : a.c.n;
    return min(max((int64_t)a.c.starts[s], (int64_t)0), a.c.n);
}

// The sequence that a tile belongs to: tiles of sequence s are those from
// start / tokens + s on, which leaves room for its last, partly filled one.  (64
// sequences are looked at a time; the wave's lanes one each.)
__device__ __forceinline__ int64_t sequence_of(const AttArgs& a, int64_t tile) {
    const int lane = threadIdx.x % kWave;
    int64_t lo = 0, range = a.c.n_seqs;
    for (;;) {
        const int64_t stride = (range + kWave - 1) / kWave, s = lo + lane * stride;
        const bool below = s < lo + range && (uint32_t)start_of(a, s) / (uint32_t)a.tokens + s <= tile;
        const int count = __builtin_popcountll(__ballot(below));
        lo += max(count - 1, 0) * stride;
        if (stride == 1) return lo;
        range = min(stride, a.c.n_seqs - lo);
    }
}

// Bits 15 and 31: whether the two 16-bit values of a word are infinite or NaN, that is,
// have an exponent of ones, which the addition carries out of.
template <typename T>
__device__ __forceinline__ uint32_t odd_pair(uint32_t two) {
    constexpr uint32_t kExponent = __is_same(T, half_t) ? 0x7C007C00u : 0x7F807F80u, kOne = __is_same(T, half_t) ? 0x04000400u : 0x00800080u;
    return (two & kExponent) + kOne;
}

struct Plain {
    static constexpr bool value = false;
};
struct Masked {
    static constexpr bool value = true;
};

template <typename T, int kDp, int kWaves, bool kCausal>
__global__ __launch_bounds__(kWaves* kWave, 2) void attention_kernel(AttArgs a) {
    constexpr int kChunks = kDp / 8, kRowsEach = kWave / kChunks;  // of a row; rows a copy instruction takes
    constexpr int kCopies = kTileKeys / kRowsEach / kWaves;        // instructions a wave, keys or values
    constexpr int kTile = kTileKeys * kDp * 2;                     // bytes
    static_assert(kTileKeys % (kRowsEach * kWaves) == 0, "whole copies");
    // separate arrays: the compiler then knows that a read of one does not wait for copies into another
    __shared__ __align__(16) uint8_t lds0[2 * kTile];
    __shared__ __align__(16) uint8_t lds1[2 * kTile];
    __shared__ int again[kWaves];
    typedef typename Mat<T>::v8 v8;
    typedef typename Mat<T>::v4 v4;

    const AttentionCall& c = a.c;
    const int lane = threadIdx.x % kWave, w = wave_id(), l32 = lane % 32, l16 = lane % 16, kg = lane / 32;
    // longest rows first; a unit's tiles follow one another by `units`, so that, of
    // a multiple of eight units, each stays on one XCD, whose L2 keeps its keys
    const unsigned unit = blockIdx.x % a.units;
    const int64_t tile = a.tiles - 1 - blockIdx.x / a.units;
    const int64_t seq = sequence_of(a, tile);
    const int64_t first = start_of(a, seq);
    const int64_t len = start_of(a, seq + 1) - first;
    const int64_t t0 = (tile - ((uint32_t)first / (uint32_t)a.tokens + seq)) * a.tokens;  // within the sequence
    if (t0 < 0 || t0 >= len) return;
    const int64_t hk = unit / a.head_groups;
    const int group = (int)(c.heads / c.kv_heads);
    const int h0 = (int)(hk * group + unit % a.head_groups * 16);
    const int rows = min(a.rows, (int)((hk + 1) * group) - h0);

    const int r = 32 * w + l32;
    const int64_t token = t0 + r / a.rows;  // of this lane's row
    const int head = r % a.rows;
    const bool live = r / a.rows < a.tokens && token < len && head < rows;
    const int limit = (int)(kCausal ? min(token + 1, len) : len);  // keys that the row sees
    const int wave_last = (int)(kCausal ? min(t0 + (32 * w + 31) / a.rows + 1, len) : len);
    const int keys_end = (int)(kCausal ? min(t0 + a.tokens, len) : len);
    const int full = (int)((kCausal ? min(t0 + 1, len) : len) / kTileKeys);  // tiles that every row sees whole
    const int tiles = (keys_end + kTileKeys - 1) / kTileKeys;

    const T* keys = static_cast<const T*>(c.k) + first * c.ldk[0] + hk * c.ldk[1];
    const T* values = static_cast<const T*>(c.v) + first * c.ldv[0] + hk * c.ldv[1];

    // This lane's pieces of the copies: row of the tile, and where in it.
    uint32_t ko[kCopies], vo[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int row = kRowsEach * (kCopies * w + i) + lane / kChunks;
        const int ck = 8 * key_place<kDp>(row, lane % kChunks), cv = 8 * value_place<kDp>(row, lane % kChunks);
        ko[i] = ck < c.d ? 2 * (uint32_t)(row * c.ldk[0] + ck) : kOut;
        vo[i] = cv < c.d ? 2 * (uint32_t)(row * c.ldv[0] + cv) : kOut;
    }
    // Rows past the sequence lie past the buffer's end, and load zero.
    auto copy = [&](uint8_t* st, int i) {
        const int64_t k0 = (int64_t)i * kTileKeys;
        const int64_t left = max(min(len - k0, (int64_t)kTileKeys), (int64_t)0);
        const __amdgpu_buffer_rsrc_t rk = att_rsrc(keys + k0 * c.ldk[0], (uint32_t)(left * c.ldk[0] * 2));
        const __amdgpu_buffer_rsrc_t rv = att_rsrc(values + k0 * c.ldv[0], (uint32_t)(left * c.ldv[0] * 2));
#pragma unroll
        for (int e = 0; e < kCopies; ++e) {
            copy16(rk, st + (1024 * (kCopies * w + e)), ko[e]);
            copy16(rv, st + (kTile + 1024 * (kCopies * w + e)), vo[e]);
        }
    };

    copy(lds0, 0);
    // (every lane loads, from a row that is there: under a condition each load would
    // be waited for before the next)
    const T* qrow = static_cast<const T*>(c.q) + (first + min(token, len - 1)) * c.ldq[0] + (h0 + min(head, rows - 1)) * c.ldq[1];
    v8 qf[kDp / 16];
#pragma unroll
    for (int e = 0; e < kDp / 16; ++e) qf[e] = *reinterpret_cast<const v8*>(qrow + (16 * e + 8 * kg < c.d ? 16 * e + 8 * kg : 0));
#pragma unroll
    for (int e = 0; e < kDp / 16; ++e) qf[e] = (live & (16 * e + 8 * kg < c.d)) ? qf[e] : (v8){};

    float16v acc[kDp / 32];
#pragma unroll
    for (int i = 0; i < kDp / 32; ++i) acc[i] = (float16v){};
    constexpr float kRaised = raised<T>(kLag);
    float m = kLowest, l = 0.0f, off = 0.0f;
    bool far = false;  // the row's exponents have passed kFarExponent

    // exact: rows that went far have their maximum taken from the scores themselves
    auto compute = [&](const uint8_t* st, int k0, auto masked, auto exact) {
        constexpr bool kMasked = decltype(masked)::value, kExact = decltype(exact)::value;
        float16v s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = (float16v){};
#pragma unroll
            for (int e = 0; e < kDp / 16; ++e) {
                const int row = 32 * t + l32;
                const v8 kf = *reinterpret_cast<const v8*>(st + (row * 2 * kDp + 16 * key_place<kDp>(row, 2 * e + kg)));
                s[t] = Mat<T>::mfma32(kf, qf[e], s[t]);
            }
        }
        uint64_t odd = 0;  // keys of the tile whose values hold an infinity or a NaN
        if (kMasked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int v = 0; v < 16; ++v) s[t][v] = k0 + 32 * t + acc32_row(v, lane) < limit ? s[t][v] : -__builtin_inff();
            uint32_t bad = 0;
#pragma unroll
            for (int e = 0; e < kChunks; ++e) {
                const uint4v x = *reinterpret_cast<const uint4v*>(st + (kTile + lane * 2 * kDp + 16 * e));
                bad |= odd_pair<T>(x.x) | odd_pair<T>(x.y) | odd_pair<T>(x.z) | odd_pair<T>(x.w);
            }
            odd = __ballot((bad & 0x80008000u) != 0);
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) top = fmaxf(top, s[t][v]);
        top = max_halves(top);
        // The maximum moves only when the row's weights would pass 2^kLag (raised), which
        // both types hold with all of their bits: most tiles leave the sums as they are.
        // (Each row by itself: its bits do not depend on its neighbours.)
        const bool moves = (top - m) * a.c2 > kLag;
        if (__any(moves)) {
            top = moves ? top : m;
            const float keep = exp2_fast((m - top) * a.c2);
            m = top;
            off = exponent_offset(m, a.c2) + kRaised;
            if (!kExact) far |= fabsf(off) > kFarExponent;
            l *= keep;
#pragma unroll
            for (int i = 0; i < kDp / 32; ++i) acc[i] *= keep;
        }
        const float base = kExact && far ? m : 0.0f, rest = kExact && far ? kRaised : off;
        auto weight_of = [&](float score) { return exp2_fast(fmaf(kExact ? score - base : score, a.c2, rest)); };
        if (kMasked) {
            // The infinities and NaN of values, times their weights, where the row sees
            // the key.  Below they count as zeros: a weight of zero would make NaN of them.
            for (uint64_t left = odd; left; left &= left - 1) {
                const int key = __builtin_ctzll(left), at = key / 32 * 16 + key % 32 / 8 * 4 + key % 4;
                float mine = 0.0f;
#pragma unroll
                for (int v = 0; v < 32; ++v) mine = v == at ? s[v / 16][v % 16] : mine;
                const float weight = weight_of(__shfl(mine, l32 + key / 4 % 2 * 32, kWave));
                const bool seen = k0 + key < limit;
                const uint8_t* row = st + (kTile + key * 2 * kDp + 8 * kg);
#pragma unroll
                for (int i = 0; i < kDp / 32; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const v4 x = *reinterpret_cast<const v4*>(row + 16 * value_place<kDp>(key, 4 * i + g));
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float y = fmaf(weight, to_f32(x[v]), acc[i][4 * g + v]);
                            acc[i][4 * g + v] = (seen & !__builtin_isfinite(to_f32(x[v]))) ? y : acc[i][4 * g + v];
                        }
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < kTileKeys / 16; ++j) {
            v8 p;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const float e = weight_of(s[j / 2][j % 2 * 8 + v]);
                // (the weight rounded to sixteen bits, which puts outputs 2.3e-4 to 2.7e-4 of
                // their norm off in float16 where their own rounding is 2.0e-4, and 1.96e-3 and
                // 1.58e-3 in bfloat16; a second product of what the rounding leaves out takes
                // 8192 tokens from 561 to 752 us, bfloat16 from 528 to 730)
                l += e;
                p[v] = (T)e;
            }
#pragma unroll
            for (int i = 0; i < kDp / 32; ++i) {
                const int row = 16 * j + 4 * kg + l16 / 4, chunk = 4 * i + l32 / 16 * 2 + l16 % 4 / 2;
                union {
                    v4 h[2];
                    v8 v;
                    uint32_t u[4];
                } vf;
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    vf.h[g] = read_turned<T>(st + (kTile + (row + 8 * g) * 2 * kDp + 16 * value_place<kDp>(row + 8 * g, chunk) + 8 * (l16 % 2)));
                if (kMasked && odd) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) vf.u[g] &= ~((odd_pair<T>(vf.u[g]) >> 15 & 0x10001u) * 0xFFFFu);
                }
                acc[i] = Mat<T>::mfma32(vf.v, p, acc[i]);
            }
        }
    };
    auto step = [&](uint8_t* st, uint8_t* nx, int i, auto masked, auto exact) {
        // this tile has landed for all waves, and all are done with the one before
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (i + 1 < tiles) copy(nx, i + 1);
        if (!decltype(masked)::value || i * kTileKeys < wave_last) compute(st, i * kTileKeys, masked, exact);
    };
    auto finish = [&] {
        l = add_halves(l);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* out = static_cast<T*>(c.out) + (first + token) * c.ldo[0] + (h0 + head) * c.ldo[1];
        // A lane holds every other run of four values of its row; the halves of the
        // wave exchange runs, so that each stores sixteen bytes.
#pragma unroll
        for (int i = 0; i < kDp / 32; ++i)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                union {
                    v4 h;
                    uint32_t u[2];
                } x, y;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    x.h[v] = (T)(acc[i][8 * g + v] * inv);
                    y.h[v] = (T)(acc[i][8 * g + 4 + v] * inv);
                }
                union {
                    uint32_t u[4];
                    uint4v v;
                } o;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const auto sw = __builtin_amdgcn_permlane32_swap(x.u[v], y.u[v], false, false);
                    o.u[v] = (uint32_t)sw[0];
                    o.u[2 + v] = (uint32_t)sw[1];
                }
                const int d = 32 * i + 16 * g + 8 * kg;
                if (live && d < c.d) *reinterpret_cast<uint4v*>(out + d) = o.v;
            }
    };
    // (a loop for each kind of tile: in one loop they would hold their addresses at the same time, and spill)
    int i = 0;
    for (; i + 2 <= full; i += 2) {
        step(lds0, lds1, i, Plain{}, Plain{});
        step(lds1, lds0, i + 1, Plain{}, Plain{});
    }
    if (i < full) {
        step(lds0, lds1, i, Plain{}, Plain{});
        if (++i < tiles) step(lds1, lds0, i++, Masked{}, Plain{});
    }
    for (; i < tiles; i += 2) {
        step(lds0, lds1, i, Masked{}, Plain{});
        if (i + 1 == tiles) break;
        step(lds1, lds0, i + 1, Masked{}, Plain{});
    }
    finish();

    // Rows whose exponents went far (see kFarExponent) are computed once more, with a
    // subtraction a score that the loops above do without (a subtraction there takes 2 to
    // 9% of all calls, a branch around it spills).  The workgroup's other rows get the
    // same bits again.
    const int mine = __any(far & live);
    if (lane == 0) again[w] = mine;
    __syncthreads();
    int any = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) any |= again[i];
    if (!any) return;
    m = kLowest, l = 0.0f, off = 0.0f;
#pragma unroll
    for (int i = 0; i < kDp / 32; ++i) acc[i] = (float16v){};
    copy(lds0, 0);
    for (i = 0; i < tiles; i += 2) {
        step(lds0, lds1, i, Masked{}, Masked{});
        if (i + 1 == tiles) break;
        step(lds1, lds0, i + 1, Masked{}, Masked{});
    }
    finish();
}

template <typename T, int kDp>
hipError_t attention_go(AttArgs a, hipStream_t s) {
    constexpr int kWaves = 4;
    a.tokens = 32 * kWaves / a.rows;
    a.tiles = (unsigned)(a.c.n / a.tokens + a.c.n_seqs);
    const dim3 grid(a.tiles * a.units), block(kWaves * kWave);
    const TimedLaunch t(K_ATTENTION, s);
    if (a.c.causal) GPTQ_LAUNCH(t, (attention_kernel<T, kDp, kWaves, true>), grid, block, 0, s, a);
    else GPTQ_LAUNCH(t, (attention_kernel<T, kDp, kWaves, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttentionCall& c, int dtype, hipStream_t s) {
    AttArgs a = {};
    a.c = c;
    const int64_t group = c.heads / c.kv_heads;
    a.rows = (int)(group < kHeadRows ? group : kHeadRows);
    a.head_groups = (int)((group + kHeadRows - 1) / kHeadRows);
    a.units = (unsigned)(c.kv_heads * a.head_groups);
    a.c2 = c.scale * kLog2e;
    if (c.d <= 64) return dtype == 0 ? attention_go<half_t, 64>(a, s) : attention_go<bf16_t, 64>(a, s);
    return dtype == 0 ? attention_go<half_t, 128>(a, s) : attention_go<bf16_t, 128>(a, s);
}

}  // namespace gptq
