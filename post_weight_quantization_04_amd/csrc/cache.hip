// Paged cache of keys and values: the store of new tokens, and the attention of
// one new token of each sequence over its pages.
#include "fp8_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

// One thread copies sixteen bytes of a key row and of the value row beside it.
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

__device__ __forceinline__ float wave_sum32(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// The plainest form: one wave a sequence and head, two values of the head a lane.
template <typename T>
__global__ __launch_bounds__(64) void cached_plain_kernel(CachedAttentionCall c) {
    const int lane = threadIdx.x;
    const int64_t b = blockIdx.x, h = blockIdx.y, hk = h / (c.heads / c.kv_heads);
    const CacheView& cache = c.cache;
    const int64_t count = min((int64_t)c.lengths[b], c.max_pages * cache.page_size);
    const T* q = static_cast<const T*>(c.q) + b * c.ldq[0] + h * c.ldq[1];
    float qv[2], acc[2] = {0.0f, 0.0f}, m = -__FLT_MAX__, l = 0.0f;
    for (int e = 0; e < 2; ++e) qv[e] = lane + 64 * e < c.d ? to_f32(q[lane + 64 * e]) : 0.0f;
    for (int64_t j = 0; j < count; ++j) {
        const int64_t page = c.table[b * c.ldt + j / cache.page_size], r = j % cache.page_size;
        if (page < 0 || page >= cache.pages) continue;
        const T* k = static_cast<const T*>(cache.keys) + page * cache.ldk[0] + hk * cache.ldk[1] + r * cache.ldk[2];
        const T* v = static_cast<const T*>(cache.values) + page * cache.ldv[0] + hk * cache.ldv[1] + r * cache.ldv[2];
        float s = 0.0f;
        for (int e = 0; e < 2; ++e)
            if (lane + 64 * e < c.d) s = fmaf(qv[e], to_f32(k[lane + 64 * e]), s);
        s = wave_sum32(s) * c.scale;
        const float top = fmaxf(m, s), keep = __expf(m - top), p = __expf(s - top);
        m = top;
        l = l * keep + p;
        for (int e = 0; e < 2; ++e)
            acc[e] = acc[e] * keep + (lane + 64 * e < c.d ? p * to_f32(v[lane + 64 * e]) : 0.0f);
    }
    T* o = static_cast<T*>(c.out) + b * c.ldo[0] + h * c.ldo[1];
    for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < c.d) o[lane + 64 * e] = (T)(l == 0.0f ? 0.0f : acc[e] / l);
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
    return 0;
}

hipError_t launch_cached_attention(const CachedAttentionCall& c, int dtype, hipStream_t s) {
    const TimedLaunch t(K_CACHED_ATTENTION, s);
    const dim3 grid((unsigned)c.n_seqs, (unsigned)c.heads);
    if (dtype == 0) GPTQ_LAUNCH(t, cached_plain_kernel<half_t>, grid, dim3(64), 0, s, c);
    else GPTQ_LAUNCH(t, cached_plain_kernel<bf16_t>, grid, dim3(64), 0, s, c);
    return hipGetLastError();
}

}  // namespace gptq
