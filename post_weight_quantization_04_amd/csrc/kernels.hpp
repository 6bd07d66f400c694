// Host-side launchers of the gfx950 kernels (one translation unit per stage)
// and the kernel-timing hook shared by them.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>
#include <stddef.h>
#include <stdint.h>

namespace gptq {

enum KernelId {
    K_HESS_F16 = 0,
    K_HESS_F32,
    K_HINV_LOAD,
    K_CHOL_STEP,
    K_HINV_STORE,
    K_Q_CONVERT,
    K_Q_GROUPGRID,
    K_Q_STEP,
    K_Q_TRAIL,
    K_PACK,
    K_DEQUANT,
    K_OUTERR,
    K_OBQ_HINV,
    K_OBQ_ROWS,
    K_PROPAGATE,
    K_HINV32_LOAD,
    K_CHOL32_STEP,
    K_HINV32_STORE,
    K_F8_WEIGHT,
    K_F8_ROWS,
    K_F8_COLUMNS,
    K_F8_NORM,
    K_F8_MATMUL,
    K_F8_GATED,
    K_PACKED_MATMUL,
    K_ATTENTION,
    K_CACHE_STORE,
    K_CACHED_ATTENTION,
    K_CACHED_JOIN,
    K_COUNT
};

// Kernel id of the launches in its scope, for the timing hook (see
// gptq_timing_enable).  Every launch goes through GPTQ_LAUNCH, which, while
// timing is enabled for that id, has the dispatch itself stamp a fresh HIP
// event pair with the kernel's start and end (no marker packets between the
// launches, so timed launches keep their spacing); a plain launch otherwise.
struct TimedLaunch {
    TimedLaunch(int kernel_id, hipStream_t) : id(kernel_id) {}
    int id;
};
struct LaunchEvents {
    explicit LaunchEvents(int id);
    hipEvent_t a = nullptr, b = nullptr;
};
#define GPTQ_LAUNCH(t, kernel, grid, block, shmem, stream, ...)                                        \
    do {                                                                                             \
        const ::gptq::LaunchEvents gptq_ev_((t).id);                                                 \
        hipExtLaunchKernelGGL(kernel, grid, block, shmem, stream, gptq_ev_.a, gptq_ev_.b, 0u, __VA_ARGS__); \
    } while (0)

// While alive, launches record no events on this thread (the timing hook
// creates HIP events, which entry points that must not allocate avoid).
struct TimingOff {
    TimingOff();
    ~TimingOff();
    bool prev;
};

// Compute units of the current device, queried once per device (0 on error).
int device_cu_count();

// ---- stage 1 ---------------------------------------------------------------
// nchunks token chunks Xs[0..nchunks) of ntok tokens each, one row stride;
// set: the first chunk writes H instead of adding into it.
hipError_t launch_hessian(float* H, int64_t n, const void* const* Xs, int64_t nchunks, int x_is_f16, int64_t ntok,
                          int64_t ldx, int set, hipStream_t s);

// ---- stages 2 + 3 ----------------------------------------------------------
constexpr int kCholNB = 64;  // panel width of the blocked factorization
size_t hinv_workspace_bytes(int64_t n);
hipError_t launch_prepare_hinv(const float* H, int64_t n, double damp_frac, float* U, uint8_t* dead,
                               int32_t* info, double* lambda_out, void* ws, hipStream_t s);
// Largest order the no-allocation entry point takes, its fixed scratch size,
// and the scratch's device address on the current device.
constexpr int64_t kNoAllocMaxDin = 4096;
size_t hinv_noalloc_scratch_bytes();
hipError_t hinv_noalloc_scratch(void** out);

// The same stages with float32 tiles and MFMA f32 products.
size_t hinv32_workspace_bytes(int64_t n);
hipError_t launch_prepare_hinv32(const float* H, int64_t n, double damp_frac, float* U, uint8_t* dead,
                                 int32_t* info, double* lambda_out, void* ws, hipStream_t s);

// ---- stage 4 ---------------------------------------------------------------
size_t quant_workspace_bytes(int64_t d_out, int64_t d_in, int64_t block, int split);
hipError_t launch_quantize(const void* W, int w_is_f16, int64_t d_out, int64_t d_in, const float* U,
                           const uint8_t* dead, int bits, int64_t group, int64_t block,
                           uint8_t* codes, float* scales, int32_t* zeros, float* err_row,
                           float* minmax, void* ws, int split, hipStream_t s);

// ---- few-bit storage, dequantization, output error ---------------------------
int64_t packed_words(int64_t d_in, int bits);
hipError_t launch_pack(const uint8_t* codes, int64_t d_out, int64_t d_in, int bits, uint32_t* packed,
                       hipStream_t s);
hipError_t launch_dequant(const uint32_t* packed, int bits, int64_t d_out, int64_t d_in, const float* scales,
                          const int32_t* zeros, int64_t group, void* out, int out_is_f16, hipStream_t s);
hipError_t launch_output_error(const void* W, int w_is_f16, const uint8_t* dead, const uint32_t* packed, int bits,
                               const float* scales, const int32_t* zeros, int64_t group, int64_t d_out,
                               int64_t d_in, const float* err_row, const double* lambda, float* out,
                               hipStream_t s);

// ---- greedy-order variant (small layers) -------------------------------------
size_t obq_workspace_bytes(int64_t d_in);
hipError_t launch_obq(const void* W, int w_is_f16, int64_t d_out, int64_t d_in, const float* U, const uint8_t* dead,
                      int bits, uint8_t* codes, float* scales, int32_t* zeros, int32_t* order, double* loss,
                      void* ws, hipStream_t s);

// ---- propagation to the next layer ------------------------------------------
hipError_t launch_propagate(const void* W, int64_t d_out, int64_t d_in, const void* X, int64_t ntok, int64_t ldx,
                            void* Y, int64_t ldy, int relu, hipStream_t s);

// ---- 8-bit operands (e4m3, a scale per block of 128) -------------------------
// dtype codes as gptq_dtype: 0 f16, 1 f32, 2 bf16
// Threads a workgroup: the entry points keep every launch below 2^32 threads.
constexpr int kF8WeightThreads = 1024;  // per 128 x 128 block
constexpr int kF8RowsThreads = 256;     // per 16 (token, block of 128) pairs
constexpr int kF8ColumnsThreads = 256;  // per 128 channels x 64 tokens
constexpr int kF8NormThreads = 512;     // per row, at most
hipError_t launch_f8_weight(const void* W, int dtype, int64_t d_out, int64_t d_in, int64_t ldw, uint8_t* q,
                            int64_t ldq, float* scales, int64_t lds, hipStream_t s);
hipError_t launch_f8_activations(const void* X, int dtype, int64_t n, int64_t d, int64_t ldx, int channel_major,
                                 uint8_t* q, int64_t ldq, float* scales, int64_t lds, hipStream_t s);
struct RmsNormCall {
    const void *x, *residual, *gain;  // residual, sum_out: or null
    void* sum_out;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldr, ldo, ldq, lds, n, d;
    double eps;
};
hipError_t launch_f8_rms_norm(const RmsNormCall& c, int dtype, hipStream_t s);
// X [n, K] against one (product) or two (gate, up) weights [M, K]
struct F8Product {
    const uint8_t* wq[2];
    const float* ws[2];
    const uint8_t* xq;
    const float* xs;
    void* y;
    int64_t ldw, ldws, ldx, ldxs, ldy, M, K, n;
    int channel_major, relu;
};
hipError_t launch_f8_matmul(const F8Product& c, int y_dtype, hipStream_t s);
// The kernel that sizes (n > 0, M > 0) are sent to on a device of `cus` compute units.
const char* f8_matmul_kernel_name(int64_t M, int64_t K, int64_t n, int y_dtype, int64_t cus);
const char* f8_gated_kernel_name(int64_t M, int64_t K, int64_t n, int64_t cus);
size_t f8_gated_workspace_bytes(int64_t n, int64_t d_ff);
hipError_t launch_f8_gated(const F8Product& c, uint8_t* q, int64_t ldq, float* scales, int64_t lds, void* ws,
                           hipStream_t s);

// ---- products with packed few-bit weights -------------------------------------
struct PackedProduct {
    const uint32_t* packed;
    const float* scales;
    const int32_t* zeros;
    const void *x, *bias, *residual;  // bias, residual: or null
    void* y;
    int64_t M, K, group, n, ldx, ldr, ldy;  // M: rows of the weights, group: 0 = one a row
    int bits, activation;
};
hipError_t launch_packed_matmul(const PackedProduct& c, int x_dtype, int y_dtype, hipStream_t s);
const char* packed_matmul_kernel_name(int64_t M, int64_t K, int64_t group, int64_t n, bool wide, int64_t cus);

// ---- attention ------------------------------------------------------------------
// Query heads that share a key head are rows of one tile, up to this many.
constexpr int64_t kHeadRows = 16;
// strides in elements: [.][0] per token, [.][1] per head
struct AttentionCall {
    const void *q, *k, *v;
    void* out;
    int64_t ldq[2], ldk[2], ldv[2], ldo[2];
    int64_t n, heads, kv_heads, d, n_seqs;
    const int32_t* starts;
    int causal;
    float scale;
};
// Pieces of 32 rows: no kernel has more workgroups.
inline int64_t attention_pieces(int64_t n, int64_t n_seqs, int64_t heads, int64_t kv_heads) {
    const int64_t group = heads / kv_heads, rows = group < kHeadRows ? group : kHeadRows;
    return (n / (32 / rows) + n_seqs) * kv_heads * ((group + kHeadRows - 1) / kHeadRows);
}
hipError_t launch_attention(const AttentionCall& c, int dtype, hipStream_t s);

// ---- paged cache ----------------------------------------------------------------
// strides in elements, per page, head and row
struct CacheView {
    void *keys, *values;
    int64_t ldk[3], ldv[3];
    int64_t pages, page_size;
};
struct CacheStoreCall {
    const void *k, *v;
    int64_t ldk[2], ldv[2];
    int64_t n, kv_heads, d;
    const int32_t* slots;
    CacheView cache;
};
hipError_t launch_cache_store(const CacheStoreCall& c, hipStream_t s);
struct CachedAttentionCall {
    const void* q;
    void* out;
    int64_t ldq[2], ldo[2];
    const int32_t *table, *lengths;
    int64_t ldt, max_pages, n_seqs, heads, kv_heads, d;
    CacheView cache;
    float scale;
    void* ws;
};
size_t cached_attention_workspace_bytes(int64_t n_seqs, int64_t heads, int64_t kv_heads, int64_t d, int64_t max_pages,
                                        int64_t page_size);
hipError_t launch_cached_attention(const CachedAttentionCall& c, int dtype, hipStream_t s);

}  // namespace gptq
