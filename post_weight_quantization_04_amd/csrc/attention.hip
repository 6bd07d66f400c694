// Attention over whole prompts, several sequences packed one behind the other:
//   y[i, h] = sum_j p_ij v[j, h'],  p_ij = softmax over j of scale q[i, h] . k[j, h']
// The plainest form: one wave a token and head, two values of the head a lane.
#include "fp8_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

__device__ __forceinline__ float wave_sum32(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

template <typename T>
__global__ __launch_bounds__(64) void attention_plain_kernel(AttentionCall c) {
    const int lane = threadIdx.x;
    const int64_t i = blockIdx.x, h = blockIdx.y, hk = h / (c.heads / c.kv_heads);
    int64_t first = 0, last = c.n;
    bool found = !c.starts;
    for (int64_t s = 0; s < c.n_seqs && !found; ++s) {
        first = max(c.starts[s], 0);
        last = min((int64_t)c.starts[s + 1], c.n);
        found = i >= first && i < last;
    }
    if (!found) return;
    const T* q = static_cast<const T*>(c.q) + i * c.ldq[0] + h * c.ldq[1];
    float qv[2], acc[2] = {0.0f, 0.0f}, m = -__FLT_MAX__, l = 0.0f;
    for (int e = 0; e < 2; ++e) qv[e] = lane + 64 * e < c.d ? to_f32(q[lane + 64 * e]) : 0.0f;
    for (int64_t j = first; j < (c.causal ? i + 1 : last); ++j) {
        const T* k = static_cast<const T*>(c.k) + j * c.ldk[0] + hk * c.ldk[1];
        const T* v = static_cast<const T*>(c.v) + j * c.ldv[0] + hk * c.ldv[1];
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
    T* o = static_cast<T*>(c.out) + i * c.ldo[0] + h * c.ldo[1];
    for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < c.d) o[lane + 64 * e] = (T)(l == 0.0f ? 0.0f : acc[e] / l);
}

}  // namespace

hipError_t launch_attention(const AttentionCall& c, int dtype, hipStream_t s) {
    const TimedLaunch t(K_ATTENTION, s);
    const dim3 grid((unsigned)c.n, (unsigned)c.heads);
    if (dtype == 0) GPTQ_LAUNCH(t, attention_plain_kernel<half_t>, grid, dim3(64), 0, s, c);
    else GPTQ_LAUNCH(t, attention_plain_kernel<bf16_t>, grid, dim3(64), 0, s, c);
    return hipGetLastError();
}

}  // namespace gptq
