// Product with packed few-bit weights, bias, activation and residual:
//   y[t, o] = act( sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[t, k] + b[o] ) + r[t, o]
// The plainest form: one thread a result.
#include "fp8_common.hpp"
#include "kernels.hpp"

namespace gptq {

namespace {

struct PmArgs {
    PackedProduct c;
    int nw, ng;
};

__device__ __forceinline__ float activated(float v, int activation) {
    if (activation == 1) return v < 0.0f ? 0.0f : v;
    if (activation == 2) return v / (1.0f + __expf(-v));
    if (activation == 3) return 0.5f * v * (1.0f + erff(v * 0.70710678f));
    return v;
}

template <typename T, typename U>
__global__ __launch_bounds__(256) void packed_plain_kernel(PmArgs a) {
    const PackedProduct& c = a.c;
    const int64_t o = (int64_t)blockIdx.x * 16 + threadIdx.x / 16, t = (int64_t)blockIdx.y * 16 + threadIdx.x % 16;
    if (o >= c.M || t >= c.n) return;
    const uint32_t* row = c.packed + o * a.nw;
    const T* x = static_cast<const T*>(c.x) + t * c.ldx;
    const int64_t per = c.group ? c.group : c.K;
    float y = 0.0f;
    for (int64_t g = 0, k = 0; k < c.K; ++g) {
        const int z = c.zeros[o * a.ng + g];
        float part = 0.0f;
        for (int64_t e = min(k + per, c.K); k < e; ++k) {
            const int64_t at = k * c.bits;
            const int sh = (int)(at & 31);
            uint32_t q = row[at >> 5] >> sh;
            if (sh + c.bits > 32) q |= row[(at >> 5) + 1] << (32 - sh);
            part = fmaf((float)((int)(q & ((1u << c.bits) - 1u)) - z), to_f32(x[k]), part);
        }
        y = fmaf(part, c.scales[o * a.ng + g], y);
    }
    if (c.bias) y += to_f32(static_cast<const U*>(c.bias)[o]);
    y = activated(y, c.activation);
    if (c.residual) y += to_f32(static_cast<const U*>(c.residual)[t * c.ldr + o]);
    static_cast<U*>(c.y)[t * c.ldy + o] = (U)y;
}

template <typename T, typename U>
hipError_t packed_go(const PmArgs& a, hipStream_t s) {
    const TimedLaunch t(K_PACKED_MATMUL, s);
    const dim3 grid((unsigned)((a.c.M + 15) / 16), (unsigned)((a.c.n + 15) / 16));
    GPTQ_LAUNCH(t, (packed_plain_kernel<T, U>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_packed_matmul(const PackedProduct& c, int x_dtype, int y_dtype, hipStream_t s) {
    const PmArgs a = {c, (int)((c.K * c.bits + 31) / 32), (int)(c.group ? c.K / c.group : 1)};
    if (x_dtype == 0) return y_dtype == 1 ? packed_go<half_t, float>(a, s) : packed_go<half_t, half_t>(a, s);
    return y_dtype == 1 ? packed_go<bf16_t, float>(a, s) : packed_go<bf16_t, bf16_t>(a, s);
}

}  // namespace gptq
