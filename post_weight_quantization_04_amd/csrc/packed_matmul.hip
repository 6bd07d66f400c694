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
// This file: which kernel a product is sent to.
#include <algorithm>

#include "packed_common.hpp"
#include "packed_tile.hpp"

namespace gptq {

namespace {

// Which kernel, by estimated time: rounds of workgroups over the CUs, each with a
// part of its own and one for a block of 128 columns, in us:
//                 few tokens (16 rows, a round)      32 x 64        64 x 128, one a CU   two   128 x 384
//   4-bit f16     1.7 + 0.1 (to 4), 0.12 (to 16), 0.2   2.0 + 0.4      2.0 + 0.9   2.0 + 1.4   3.5 + 2.65
// The same figures choose for the other forms, whose kernels change places at much the
// same sizes: over 4096 -> 4096 and 11008 -> 4096 with 8 to 2048 tokens, fourteen numbers of them,
// the chosen kernel takes 0.7% more than the fastest in geometric mean for 4-bit float16 in
// groups of 128, 2% for bfloat16, 1% for 2 and 3 bits, 4% for 8, 1% in groups of 64, 4% of
// 16, 0 to 1% for unaligned rows.  Furthest off are 33 to 64 tokens of 11008 columns, sent to
// 32 x 64 (of 8 bits 41 us, 32 with few tokens; in groups of 16 65 and 46), and 65 to 128
// unaligned ones in small groups, sent to 64 x 128 (62 us, 52 with few tokens).
// A kernel whose grid would be too large is left out, and so are those that a form lacks:
// 128 x 384 takes aligned rows of x and whole groups, 32 x 64 one of the two.
PmKernel choose(int64_t M, int64_t nb, int64_t n, bool vec, bool fine, int64_t cus) {
    if (n <= 4) return kPmFew;
    auto rounds = [&](int64_t tokens, int64_t rows, int64_t each) {
        return (double)((((n + tokens - 1) / tokens) * ((M + rows - 1) / rows) + cus * each - 1) / (cus * each));
    };
    auto fits = [&](int64_t tokens, int64_t rows, int64_t threads) {
        return ((n + tokens - 1) / tokens) * ((M + rows - 1) / rows) * threads < (int64_t)1 << 32;
    };
    const double none = 1e30;
    const double few = n <= 32 * 65535 ? rounds(32, 16, 1) * (1.7 + (n <= 16 ? 0.12 : 0.2) * nb) : none;
    const double small = (vec || !fine) && fits(32, 64, 1024) ? rounds(32, 64, 1) * (2.0 + 0.4 * nb) : none;
    const bool one = rounds(64, 128, 1) == 1.0;
    const double mid = one ? 2.0 + 0.9 * nb : rounds(64, 128, 2) * (2.0 + 1.4 * nb);
    const double big = vec && !fine ? rounds(128, 384, 1) * (3.5 + 2.65 * nb) : none;
    const double least = std::min(std::min(few, small), std::min(mid, big));
    return least == few ? kPmFew : least == small ? kPm32x64 : least == mid ? kPm64x128 : kPm128x384;
}

// Groups that do not consist of whole blocks.
bool fine_groups(int64_t K, int64_t group) { return group % kPmBlock != 0 && K > group; }

template <typename T, int kBits>
hipError_t bits_go(const PmArgs& a, hipStream_t s) {
    const bool fine = fine_groups(a.c.K, a.c.group);
    const int64_t cus = device_cu_count();
    if (cus <= 0) return hipErrorInvalidDevice;
    const PmKernel kernel = choose(a.c.M, a.nb, a.c.n, a.vec, fine, cus);
    if (kernel == kPmFew) return launch_packed_few<T, kBits>(a, fine, s);
    return launch_packed_tile<T, kBits>(a, kernel, fine, s);
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

const char* packed_matmul_kernel_name(int64_t M, int64_t K, int64_t group, int64_t n, bool wide, int64_t cus) {
    switch (choose(M, (K + kPmBlock - 1) / kPmBlock, n, wide && K % 8 == 0, fine_groups(K, group), cus)) {
        case kPmFew: return "few tokens";
        case kPm32x64: return "32 x 64";
        case kPm64x128: return "64 x 128";
        default: return "128 x 384";
    }
}

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
    a.vec = c.K % 8 == 0 && c.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(c.x) % 16 == 0;
    return x_dtype == 0 ? typed_go<half_t>(a, s) : typed_go<bf16_t>(a, s);
}

}  // namespace gptq
