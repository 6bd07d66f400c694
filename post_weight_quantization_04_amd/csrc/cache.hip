// Paged cache of keys and values: the store of new tokens, and the attention of
// one new token of each sequence over its pages,
//   y[b, h] = sum_{j < length[b]} p_j V[b, j, h'],  p = softmax over j of scale q[b, h] . K[b, j, h'].
#include <algorithm>

#include "attention_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

// One thread copies sixteen bytes of a key row and of the value row beside it: 8192
// tokens of 8 heads of 128 10 to 11.5 us, 5.8 to 6.6 TB/s of reads and writes, bound by
// HBM and its caches; 24 tokens 3 us, a launch.
__global__ __launch_bounds__(256) void cache_store_kernel(CacheStoreCall c, int chunks) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = id / chunks, e = id % chunks * 8;
    if (row >= c.n * c.kv_heads) return;
    const int64_t t = row / c.kv_heads, h = row % c.kv_heads;
    const int64_t slot = c.slots[t];
    if (slot < 0 || slot >= c.cache.pages * c.cache.page_size) return;
    const int64_t page = slot / c.cache.page_size, r = slot % c.cache.page_size;
    const CacheView& v = c.cache;
    *reinterpret_cast<uint4v*>(static_cast<uint16_t*>(v.keys) + page * v.ldk[0] + h * v.ldk[1] + r * v.ldk[2] + e) =
        *reinterpret_cast<const uint4v*>(static_cast<const uint16_t*>(c.k) + t * c.ldk[0] + h * c.ldk[1] + e);
    *reinterpret_cast<uint4v*>(static_cast<uint16_t*>(v.values) + page * v.ldv[0] + h * v.ldv[1] + r * v.ldv[2] + e) =
        *reinterpret_cast<const uint4v*>(static_cast<const uint16_t*>(c.v) + t * c.ldv[0] + h * c.ldv[1] + e);
}

// ---------------------------------------------------------------------------
// Attention over the cache.  A unit is a sequence's key head with up to sixteen
// of the query heads that share it: they are the columns of S^T = K Q^T and of
// O^T = V^T P^T, so a lane's scores, maximum and sum belong to one query row, and
// P^T leaves the first product in the layout that the second takes.  A unit's
// keys are cut into steps; a workgroup's waves take a tile of kKeys keys each of
// a step, copy it to LDS of their own two tiles ahead (buffers of memory lie in
// flight, which is what HBM wants) and work without barriers.  At the end of a
// unit the waves' results are joined in LDS.
//
// Long sequences (kSplit): all steps of all units, in order, are shared equally
// among the workgroups, whatever the lengths, so that a batch of unequal
// sequences ends at one time.  A workgroup that computes a part of a unit leaves
// (maximum, sum, O) in the workspace: slot 2 w for a part that begins inside the
// unit, 2 w + 1 for one that begins with it.  cached_join_kernel adds the parts
// in order.
//
// Bound by HBM for long tables: 131072 tokens of 8 key heads of 128 103 us and 8 for the
// join (5.2 TB/s over the first), 48 sequences of up to 8192 172 to 178 us and 10 (4.9);
// 64 x 500 tokens 24.6 (5.3).  Short ones by the chain of lengths, pages, keys, launch:
// 333 tokens 8.7 us.
// ---------------------------------------------------------------------------
struct CachedArgs {
    CachedAttentionCall c;
    int rows;          // query heads of a unit
    int head_groups;   // units per key head
    uint32_t page_mul, page_shift;  // division by the page size
    float c2;          // scale log2 e
    float* parts;
    int64_t workers;   // at most
};

// Floats of a part: O [rows][dp], then each row's maximum, then its sum, up to a multiple
// of four, since O is read and written as sixteen bytes.
__host__ __device__ constexpr int64_t part_floats(int64_t rows, int64_t dp) { return (rows * (dp + 2) + 3) / 4 * 4; }

__device__ const uint32_t kZeroRow[64] = {};  // 256 bytes: what keys that are none are read from

__device__ __forceinline__ uint32_t page_of(const CachedArgs& a, uint32_t pos) {
    const uint32_t t = __umulhi(a.page_mul, pos);
    return a.page_shift ? (t + ((pos - t) >> 1)) >> (a.page_shift - 1) : pos;
}

__device__ __forceinline__ uint32_t cached_length(const CachedArgs& a, int64_t b) {
    const int64_t n = a.c.lengths[b];
    return (uint32_t)min(max(n, (int64_t)0), a.c.max_pages * a.c.cache.page_size);
}

// Workgroups among which `all` steps are shared: two steps each at least, since a part
// costs the join about as much.
__device__ __forceinline__ int64_t cached_workers(int64_t most, int64_t all) { return min(most, (all + 1) / 2); }

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) {
        const int64_t u = __shfl_up(v, o, kWave);
        v += lane >= o ? u : 0;
    }
    return v;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Steps of all sequences, of one unit each.
__device__ __forceinline__ int64_t count_steps(const CachedArgs& a, uint32_t per) {
    int64_t sum = 0;
    for (int64_t b = threadIdx.x % kWave; b < a.c.n_seqs; b += kWave) sum += (cached_length(a, b) + (uint64_t)per - 1) / per;
    return uniform64(__shfl(wave_scan(sum), kWave - 1, kWave));
}

// The sequence b that holds step `at` < all, and the steps `before` it (a unit's).
// (False, and every loop over sequences ends, also where lengths change meanwhile.)
__device__ __forceinline__ bool find_step(const CachedArgs& a, uint32_t per, int64_t units, int64_t at, int64_t& b, int64_t& before) {
    const int lane = threadIdx.x % kWave;
    before = 0;
    for (b = 0; b < a.c.n_seqs; b += kWave) {
        const int64_t mine = b + lane < a.c.n_seqs ? (cached_length(a, b + lane) + (uint64_t)per - 1) / per : 0;
        const int64_t sum = wave_scan(mine);
        const uint64_t past = __ballot((before + sum) * units > at);
        if (past) {
            const int in = __builtin_ctzll(past);
            before += uniform64(__shfl(sum - mine, in, kWave));
            b += in;
            return true;
        }
        before += uniform64(__shfl(sum, kWave - 1, kWave));
    }
    return false;
}

// Memory to LDS without registers in between, a wave's lanes one behind the
// other from `lds` on.  The pages of a cache lie further apart than a buffer
// load's 32-bit offsets reach, and the compiler takes the global form for one
// that may read LDS: it would wait for all copies in flight at every LDS read.
// As assembly (without outputs, so no register is pending) it leaves the waits
// to the code that copies.  M0, which the compiler reserves, is used by nothing
// else in these kernels.
__device__ __forceinline__ void copy_row_piece(const void* p, const void* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(p) : "memory");
}
__device__ __forceinline__ void copy_word(const void* p, const void* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(p) : "memory");
}

// Weights go into the second product in two parts, so that what their rounding to sixteen
// bits leaves out counts too: 1.5 2^-21 of each in float16 and 1.5 2^-15 in bfloat16 are lost,
// and the outputs are as exact as their own rounding (1 x 333 tokens in float16: 2.12e-4 of the
// norm off 64 bits, 2.57e-4 with one part; 131072 in bfloat16 1.66e-3 and 2.16e-3).
// HBM hides most of it: 131072 tokens 106.2 -> 107.3 us, 48 sequences 183 as before, but
// 333 tokens 8.4 -> 8.7 and 900 tokens 13.4 -> 14.3.  (Weights of 32 bits on the float32
// MFMA: 333 tokens 11.7, 900 tokens 22.4, 48 sequences 204.)
// The first part is that of a little less than the weight: the second one is then never
// zero or below, and an infinite value times both remains that infinity.
template <typename T>
constexpr float kMost = 1.0f - (__is_same(T, half_t) ? 0x1p-10f : 0x1p-7f);

template <typename T, int kDp, int kWaves, bool kSplit>
__global__ __launch_bounds__(kWaves* kWave, 2) void cached_kernel(CachedArgs a) {
    constexpr int kChunks = kDp / 8;                 // of a row
    constexpr int kCopies = 4;                       // instructions for a tile of keys
    constexpr int kRowsEach = kWave / kChunks;       // rows an instruction copies
    constexpr int kKeys = kCopies * kRowsEach;       // of a tile
    constexpr int kStep = kWaves * kKeys;
    constexpr int kTile = 1024 * kCopies;            // bytes of a tile of keys or of values
    __shared__ __align__(16) uint8_t lds0[kWaves * 2 * kTile];
    __shared__ __align__(16) uint8_t lds1[kWaves * 2 * kTile];
    __shared__ __align__(16) int32_t pages[2][kWaves][kWave];
    __shared__ float tops[kWaves][16], sums[kWaves][16];
    typedef typename Mat<T>::v8 v8;
    typedef typename Mat<T>::v4 v4;

    const CachedAttentionCall& c = a.c;
    const int tid = threadIdx.x, lane = tid % kWave, w = wave_id(), l16 = lane % 16, kg = lane / 16;
    const int64_t units = c.kv_heads * a.head_groups;  // of a sequence
    const int group = (int)(c.heads / c.kv_heads);

    int64_t b, unit, step, left;  // the first unit, the step in it, and how many steps are this workgroup's
    if (kSplit) {
        const int64_t all = count_steps(a, kStep) * units;
        const int64_t workers = cached_workers(a.workers, all);
        if (blockIdx.x >= workers) return;
        const int64_t from = (int64_t)blockIdx.x * all / workers, to = ((int64_t)blockIdx.x + 1) * all / workers;
        left = to - from;
        int64_t before;
        if (!find_step(a, kStep, units, from, b, before)) return;
        const int64_t steps = max((int64_t)((cached_length(a, b) + (uint64_t)kStep - 1) / kStep), (int64_t)1);
        unit = min((from - before * units) / steps, units - 1);
        step = (from - before * units) % steps;
    } else {
        b = blockIdx.x / units;
        unit = blockIdx.x % units;
        step = 0;
        left = 1;
    }

    const int chunk = lane % kChunks;
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(kZeroRow) + 16 * chunk;
    for (; left > 0; ++unit) {
        if (kSplit && unit == units) {
            unit = 0;
            do ++b;
            while (b < c.n_seqs && cached_length(a, b) == 0);
            if (b >= c.n_seqs) return;
        }
        const uint32_t length = __builtin_amdgcn_readfirstlane(cached_length(a, b));
        const int64_t steps = ((uint64_t)length + kStep - 1) / kStep;
        const int64_t last = kSplit ? min(steps, step + left) : steps;
        const int64_t hk = unit / a.head_groups;
        const int h0 = (int)(hk * group + unit % a.head_groups * 16);
        const int rows = min(a.rows, (int)((hk + 1) * group) - h0);
        const bool whole = step == 0 && last == steps;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (step == 0);

        // (every lane loads, from a row that is there: under a condition each load would
        // be waited for before the next)
        const T* qrow = static_cast<const T*>(c.q) + b * c.ldq[0] + (h0 + min(l16, rows - 1)) * c.ldq[1];
        v8 qf[kDp / 32];
#pragma unroll
        for (int s = 0; s < kDp / 32; ++s) qf[s] = *reinterpret_cast<const v8*>(qrow + (32 * s + 8 * kg < c.d ? 32 * s + 8 * kg : 0));
#pragma unroll
        for (int s = 0; s < kDp / 32; ++s) qf[s] = ((l16 < rows) & (32 * s + 8 * kg < c.d)) ? qf[s] : (v8){};
        const T* keys = static_cast<const T*>(c.cache.keys) + hk * c.cache.ldk[1];
        const T* values = static_cast<const T*>(c.cache.values) + hk * c.cache.ldv[1];
        const int32_t* table = c.table + b * c.ldt;

        // The pages of the tile at k0, a word a key (lanes past the tile repeat it).
        auto copy_pages = [&](int32_t* to, uint32_t k0) {
            const uint32_t pos = k0 + (uint32_t)(lane % kKeys);
            copy_word(table + (pos < length ? page_of(a, pos) : 0u), to);
        };
        // The tile itself; true if a key of it is on a page outside the cache.
        auto copy = [&](uint8_t* st, const int32_t* pages, uint32_t k0) {
            bool odd = false;
            uint32_t pg[kCopies];
#pragma unroll
            for (int i = 0; i < kCopies; ++i) pg[i] = (uint32_t)pages[kRowsEach * i + lane / kChunks];
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r = kRowsEach * i + lane / kChunks;
                const uint32_t pos = k0 + (uint32_t)r, page = pg[i];
                const bool in = page < (uint32_t)c.cache.pages, ok = (pos < length) & in;
                odd |= (pos < length) & !in;
                const uint32_t row = pos - page_of(a, pos) * (uint32_t)c.cache.page_size;
                const int ck = 8 * key_place<kDp>(r, chunk), cv = 8 * value_place<kDp>(r, chunk);
                const uint8_t* kp = reinterpret_cast<const uint8_t*>(keys + ck) +
                                    2 * ((uint64_t)page * (uint32_t)c.cache.ldk[0] + (uint64_t)row * (uint32_t)c.cache.ldk[2]);
                const uint8_t* vp = reinterpret_cast<const uint8_t*>(values + cv) +
                                    2 * ((uint64_t)page * (uint32_t)c.cache.ldv[0] + (uint64_t)row * (uint32_t)c.cache.ldv[2]);
                asm("" : "+v"(kp), "+v"(vp));  // selected from, not branched around
                kp = (ok & (ck < c.d)) ? kp : zero;
                vp = (ok & (cv < c.d)) ? vp : zero;
                copy_row_piece(kp, st + (w * 2 * kTile + 1024 * i));
                copy_row_piece(vp, st + (w * 2 * kTile + kTile + 1024 * i));
            }
            return __any(odd);
        };

        float4v acc[kDp / 16];
#pragma unroll
        for (int i = 0; i < kDp / 16; ++i) acc[i] = (float4v){};
        float m = kLowest, l = 0.0f;

        auto compute = [&](const uint8_t* st, uint32_t k0, bool odd) {
            constexpr int kTiles = kKeys / 16;
            float4v s[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                s[t] = (float4v){};
#pragma unroll
                for (int e = 0; e < kDp / 32; ++e) {
                    const int r = 16 * t + l16;
                    const v8 kf = *reinterpret_cast<const v8*>(st + (w * 2 * kTile + r * 2 * kDp + 16 * key_place<kDp>(r, 4 * e + kg)));
                    s[t] = Mat<T>::mfma16(kf, qf[e], s[t]);
                }
            }
            if (k0 + kKeys > length || odd) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint32_t pos = k0 + (uint32_t)(16 * t + 4 * kg + v);
                        bool ok = pos < length;
                        if (ok && odd) ok = (uint32_t)table[page_of(a, pos)] < (uint32_t)c.cache.pages;
                        s[t][v] = ok ? s[t][v] : -__builtin_inff();
                    }
            }
            float top = m;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v) top = fmaxf(top, s[t][v]);
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            const float keep = exp2_fast((m - top) * a.c2);
            m = top;
            l *= keep;
#pragma unroll
            for (int i = 0; i < kDp / 16; ++i) acc[i] *= keep;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                v4 p, rest;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float e = exp2_fast(fmaf(s[t][v] - top, a.c2, raised<T>(0.0f)));
                    l += e;
                    p[v] = (T)(e * kMost<T>);
                    rest[v] = (T)(e - to_f32(p[v]));
                }
                const int r = 16 * t + 4 * kg + l16 / 4;
#pragma unroll
                for (int i = 0; i < kDp / 16; ++i) {
                    const v4 vf = read_turned<T>(st + (w * 2 * kTile + kTile + r * 2 * kDp +
                                                       16 * value_place<kDp>(r, 2 * i + l16 % 4 / 2) + 8 * (l16 % 2)));
                    acc[i] = Mat<T>::mfma16h(vf, p, acc[i]);
                    acc[i] = Mat<T>::mfma16h(vf, rest, acc[i]);
                }
            }
        };

        if (step < last) {
            constexpr int kLoads = 2 * kCopies;
            const int count = (int)(last - step);
            uint32_t at = (uint32_t)step * kStep + (uint32_t)(w * kKeys);  // this wave's tile of the step in work
            copy_pages(pages[0][w], at);
            copy_pages(pages[1][w], at + kStep);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            bool odd0 = copy(lds0, pages[0][w], at);
            copy_pages(pages[0][w], at + 2 * kStep);
            bool odd1 = copy(lds1, pages[1][w], at + kStep);
            // One tile from `st`, whose memory then takes the tile two steps on
            // (past the last step: positions past the length, or steps of
            // another workgroup, copied and never used).  In flight at its
            // start, in order: this tile, the next but one's pages, the next tile.
            auto go = [&](uint8_t* st, bool& odd, int32_t* mine, int32_t* next) {
                copy_pages(next, at + 3 * kStep);
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads + 1) : "memory");
                compute(st, at, odd);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                odd = copy(st, mine, at + 2 * kStep);
                at += kStep;
            };
            int i = 0;
            for (; i + 2 <= count; i += 2) {
                go(lds0, odd0, pages[0][w], pages[1][w]);
                go(lds1, odd1, pages[1][w], pages[0][w]);
            }
            if (i < count) go(lds0, odd0, pages[0][w], pages[1][w]);
        }

        // the waves' results
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __syncthreads();
        l += __shfl_xor(l, 16, kWave);
        l += __shfl_xor(l, 32, kWave);
        float* o = reinterpret_cast<float*>(lds0);  // [kWaves][16][kDp], sixteen bytes at c ^ row
        if (kg == 0) {
            tops[w][l16] = m;
            sums[w][l16] = l;
        }
#pragma unroll
        for (int i = 0; i < kDp / 16; ++i)
            *reinterpret_cast<float4v*>(o + ((w * 16 + l16) * kDp + 4 * ((4 * i + kg) ^ l16))) = acc[i];
        __syncthreads();
        for (int id = tid; id < rows * kChunks; id += kWaves * kWave) {
            const int r = id / kChunks, e = id % kChunks * 8;
            float top = tops[0][r];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) top = fmaxf(top, tops[i][r]);
            float sum = 0.0f, y[8] = {};
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const float f = exp2_fast((tops[i][r] - top) * a.c2);
                sum = fmaf(sums[i][r], f, sum);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4v v = *reinterpret_cast<const float4v*>(o + ((i * 16 + r) * kDp + 4 * ((e / 4 + j) ^ r)));
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[4 * j + k] = fmaf(v[k], f, y[4 * j + k]);
                }
            }
            if (!kSplit || whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (e < c.d) {
                    v8 out;
#pragma unroll
                    for (int k = 0; k < 8; ++k) out[k] = (T)(y[k] * inv);
                    *reinterpret_cast<v8*>(static_cast<T*>(c.out) + b * c.ldo[0] + (h0 + r) * c.ldo[1] + e) = out;
                }
            } else {
                float* part = a.parts + slot * part_floats(a.rows, kDp);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<float4v*>(part + (r * kDp + e + 4 * j)) = (float4v){y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]};
                if (e == 0) {
                    part[a.rows * kDp + r] = top;
                    part[a.rows * (kDp + 1) + r] = sum;
                }
            }
        }
        __syncthreads();
        left -= kSplit ? last - step : 1;
        step = 0;
    }
}

// Adds the parts of the units that several workgroups computed, each unit in the
// workgroup that has the number of the second of them: no more workgroups than there
// were, however many units.  Threads of eight outputs each, in groups that take turns
// with the parts, and the groups' results added in their order.  (One thread for all
// parts of its outputs, one workgroup a unit: 313 parts in 45 us; these 9.)  Zeros for
// sequences without tokens besides.
constexpr int kJoinThreads = 1024;
template <typename T, int kDp>
__global__ __launch_bounds__(kJoinThreads) void cached_join_kernel(CachedArgs a, uint32_t per_step) {
    typedef typename Mat<T>::v8 v8;
    constexpr int kChunks = kDp / 8;
    __shared__ __align__(16) float held[kJoinThreads][8];
    __shared__ float tops[kJoinThreads], sums[kJoinThreads];
    const CachedAttentionCall& c = a.c;
    for (int64_t b = blockIdx.x; b < c.n_seqs; b += gridDim.x) {
        if (cached_length(a, b)) continue;
        const int chunks = (int)c.d / 8;
        for (int64_t i = threadIdx.x; i < c.heads * chunks; i += kJoinThreads)
            *reinterpret_cast<v8*>(static_cast<T*>(c.out) + b * c.ldo[0] + i / chunks * c.ldo[1] + i % chunks * 8) = (v8){};
    }
    const int64_t units = c.kv_heads * a.head_groups;
    const int group = (int)(c.heads / c.kv_heads);
    const int64_t all = count_steps(a, per_step) * units;
    const int64_t workers = cached_workers(a.workers, all), here = blockIdx.x;
    if (here == 0 || here >= workers) return;
    const int64_t at = here * all / workers;
    int64_t b, before;
    if (!find_step(a, per_step, units, at, b, before)) return;
    const int64_t steps = max((int64_t)((cached_length(a, b) + (uint64_t)per_step - 1) / per_step), (int64_t)1);
    const int64_t unit = min((at - before * units) / steps, units - 1), from = before * units + unit * steps;
    auto worker = [&](int64_t step) { return ((step + 1) * workers - 1) / all; };
    // the first worker's part begins with the unit, the others' inside it
    const int64_t first = worker(from), last = min(worker(from + steps - 1), workers - 1);
    if (first + 1 != here) return;
    const int64_t hk = unit / a.head_groups;
    const int h0 = (int)(hk * group + unit % a.head_groups * 16);
    const int rows = min(a.rows, (int)((hk + 1) * group) - h0);
    const int tid = threadIdx.x, per = rows * kChunks, groups = kJoinThreads / per, g = tid / per;
    const int r = tid % per / kChunks, e = tid % per % kChunks * 8;
    float top = kLowest, sum = 0.0f, y[8] = {};
    if (g < groups) {
#pragma unroll 2
        for (int64_t w = first + g; w <= last; w += groups) {
            const float* p = a.parts + (2 * w + (w == first)) * part_floats(a.rows, kDp);
            const float4v lo = *reinterpret_cast<const float4v*>(p + r * kDp + e), hi = *reinterpret_cast<const float4v*>(p + r * kDp + e + 4);
            const float pt = p[a.rows * kDp + r], ps = p[a.rows * (kDp + 1) + r];
            const float now = fmaxf(top, pt), fa = exp2_fast((top - now) * a.c2), fb = exp2_fast((pt - now) * a.c2);
            top = now;
            sum = sum * fa + ps * fb;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k] = y[k] * fa + lo[k] * fb;
                y[4 + k] = y[4 + k] * fa + hi[k] * fb;
            }
        }
    }
    tops[tid] = top;
    sums[tid] = sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) held[tid][k] = y[k];
    __syncthreads();
    if (g > 0 || e >= c.d) return;
    float now = top;
    for (int i = 1; i < groups; ++i) now = fmaxf(now, tops[i * per + tid]);
    float f = exp2_fast((top - now) * a.c2);
    sum *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= f;
    for (int i = 1; i < groups; ++i) {
        f = exp2_fast((tops[i * per + tid] - now) * a.c2);
        sum = fmaf(sums[i * per + tid], f, sum);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = fmaf(held[i * per + tid][k], f, y[k]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    v8 out;
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = (T)(y[k] * inv);
    *reinterpret_cast<v8*>(static_cast<T*>(c.out) + b * c.ldo[0] + (h0 + r) * c.ldo[1] + e) = out;
}

constexpr int64_t kCachedWorkers = 512;   // at most
// Tokens up to which a unit is one workgroup's, without the join's launch: 333 tokens of 8
// key heads 8.7 us, divided 20.3; 900 tokens 14.3 and 16.7; 1500 tokens 18.7 and 16.6; 4000
// tokens 40.9 and 18.5.  (By the table, which the host knows, not by the lengths.  Many
// sequences would gain a little from more: 64 of 2000 tokens 94 us, divided 104.)
constexpr int64_t kCachedWhole = 1024;

inline int padded_head(int64_t d) { return d <= 64 ? 64 : 128; }
inline int64_t unit_rows(int64_t heads, int64_t kv_heads) { return std::min(heads / kv_heads, kHeadRows); }

template <typename T, int kDp, int kWaves>
hipError_t cached_waves(CachedArgs a, int64_t units, int64_t most, int cus, hipStream_t s) {
    if (most <= kCachedWhole) {
        const TimedLaunch t(K_CACHED_ATTENTION, s);
        GPTQ_LAUNCH(t, (cached_kernel<T, kDp, kWaves, false>), dim3((unsigned)units), dim3(kWaves * kWave), 0, s, a);
        return hipGetLastError();
    }
    constexpr int kStep = kWaves * 4 * kWave / (kDp / 8);
    a.workers = std::min({kCachedWorkers, (int64_t)(8 / kWaves) * cus, units * ((most + kStep - 1) / kStep)});
    const TimedLaunch t(K_CACHED_ATTENTION, s);
    GPTQ_LAUNCH(t, (cached_kernel<T, kDp, kWaves, true>), dim3((unsigned)a.workers), dim3(kWaves * kWave), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const TimedLaunch j(K_CACHED_JOIN, s);
    GPTQ_LAUNCH(j, (cached_join_kernel<T, kDp>), dim3((unsigned)a.workers), dim3(kJoinThreads), 0, s, a, (uint32_t)kStep);
    return hipGetLastError();
}

// Eight waves a workgroup, one a CU, while there is a CU for each unit (333 tokens of 8
// key heads 8.7 us, 9.5 with four waves; 900 tokens 14.2 and 17.4; 131072 tokens 108 us,
// 5.0 TB/s, and 112; 16 x 3000 tokens of 16 heads of 64 42 and 57).  Four waves, two
// workgroups a CU, for more units, since what a unit's begin and end take then lies beside
// another's copies (64 x 500 tokens 24.6 us, 28.9 with eight; in longer tables 999 x 50 and
// one of 7000 133 us and 216, 200 x 500 and one of 7000 103 and 111).
template <typename T, int kDp>
hipError_t cached_go(const CachedArgs& a, hipStream_t s) {
    const CachedAttentionCall& c = a.c;
    const int64_t units = c.n_seqs * c.kv_heads * a.head_groups, most = c.max_pages * c.cache.page_size;
    const int cus = device_cu_count();
    if (cus <= 0) return hipErrorInvalidDevice;
    return units <= cus ? cached_waves<T, kDp, 8>(a, units, most, cus, s) : cached_waves<T, kDp, 4>(a, units, most, cus, s);
}

}  // namespace

hipError_t launch_cache_store(const CacheStoreCall& c, hipStream_t s) {
    const TimedLaunch t(K_CACHE_STORE, s);
    const int chunks = (int)(c.d / 8);
    const int64_t threads = c.n * c.kv_heads * chunks;
    GPTQ_LAUNCH(t, cache_store_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, c, chunks);
    return hipGetLastError();
}

size_t cached_attention_workspace_bytes(int64_t n_seqs, int64_t heads, int64_t kv_heads, int64_t d, int64_t max_pages,
                                        int64_t page_size) {
    if (max_pages <= kCachedWhole && max_pages * std::min(page_size, kCachedWhole + 1) <= kCachedWhole) return 0;
    return (size_t)(2 * kCachedWorkers * part_floats(unit_rows(heads, kv_heads), padded_head(d))) * sizeof(float);
}

hipError_t launch_cached_attention(const CachedAttentionCall& c, int dtype, hipStream_t s) {
    CachedArgs a = {};
    a.c = c;
    a.rows = (int)unit_rows(c.heads, c.kv_heads);
    a.head_groups = (int)((c.heads / c.kv_heads + kHeadRows - 1) / kHeadRows);
    // pos / p = (t + (pos - t) / 2) >> (shift - 1), t = mulhi(mul, pos), shift = ceil(log2 p)
    while (((uint64_t)1 << a.page_shift) < (uint64_t)c.cache.page_size) ++a.page_shift;
    a.page_mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << a.page_shift) - (uint64_t)c.cache.page_size)) /
                                (uint64_t)c.cache.page_size + 1);
    a.c2 = c.scale * kLog2e;
    a.parts = static_cast<float*>(c.ws);
    if (c.d <= 64) return dtype == 0 ? cached_go<half_t, 64>(a, s) : cached_go<bf16_t, 64>(a, s);
    return dtype == 0 ? cached_go<half_t, 128>(a, s) : cached_go<bf16_t, 128>(a, s);
}

}  // namespace gptq
