"""Size limits of the 8-bit calls: every launch has fewer than 2^32 threads.
The first size past a limit is refused before any HIP call; the last one below
it passes the checks, and then fails for want of a device (these pointers are
not memory, so that half is skipped where there is one)."""
import ctypes
import os

import pytest

OK, EINVAL, EUNSUPPORTED, EHIP, EWORKSPACE = 0, 1, 2, 3, 4
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def clib():
    from post_weight_quantization_04_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def _no_device():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a device is there: the pointers of this test are not")


def weight(lib, m, k):
    ld = (k + 127) // 128 * 128
    return lib.gptq_fp8_weight(P, 0, m, k, k, P, ld, P, ld // 128, None)


# blocks of 128 x 128, one workgroup of 1024 threads each: below 2^22
@pytest.mark.parametrize("m,k", [(1 << 18, 1 << 18), (1 << 24, 32 * 128), (1 << 24, 31 * 128 + 1), ((1 << 18) - 127, 1 << 18)])
def test_weight_past_the_limit(clib, m, k):
    assert weight(clib, m, k) == EUNSUPPORTED


# (2049 x 2047 = 2^22 - 1)
@pytest.mark.parametrize("m,k", [(2049 * 128, 2047 * 128), (1 << 24, 31 * 128)])
def test_weight_below_the_limit(clib, m, k):
    _no_device()
    assert weight(clib, m, k) == EHIP


def acts(lib, n, d, cm=0):
    return lib.gptq_fp8_activations(P, 0, n, d, n if cm else d, cm, P, (d + 127) // 128 * 128, P, n, None)


# (token, block of 128) pairs, sixteen a workgroup of 256 threads: at most 2^28 - 16
@pytest.mark.parametrize("n,d", [((1 << 28) - 15, 128), ((1 << 28) - 1, 1), ((1 << 27) - 7, 129), (1 << 28, 128)])
def test_activations_past_the_limit(clib, n, d):
    assert acts(clib, n, d) == EUNSUPPORTED


@pytest.mark.parametrize("n,d", [((1 << 28) - 16, 128), ((1 << 27) - 8, 129)])
def test_activations_below_the_limit(clib, n, d):
    _no_device()
    assert acts(clib, n, d) == EHIP


# pieces of 128 channels by 64 tokens, 256 threads each: below 2^24
def test_channel_major_activations_at_the_limit(clib):
    assert acts(clib, (1 << 30) - 63, 128, 1) == EUNSUPPORTED
    assert acts(clib, (1 << 29) - 63, 129, 1) == EUNSUPPORTED
    _no_device()
    assert acts(clib, (1 << 30) - 64, 128, 1) == EHIP


# rows, up to 512 threads each: below 2^23
def test_norm_at_the_limit(clib):
    def norm(n):
        return clib.gptq_fp8_rms_norm(P, 128, None, 0, None, 0, P, 0, n, 128, 1e-6, P, 128, P, n, None)

    assert norm(1 << 23) == EUNSUPPORTED
    _no_device()
    assert norm((1 << 23) - 1) == EHIP


# products: up to 2^22 tiles of 256 x 256, in whatever tiles the choice takes
_GROUPS = {"few tokens": (16, 32, 512), "64 x 64, k in two groups": (64, 64, 512), "64 x 64": (64, 64, 256),
           "128 x 64, k in two groups": (128, 64, 512), "128 x 128": (128, 128, 512), "256 x 128": (256, 128, 512),
           "256 x 256": (256, 256, 512)}
_GATED_GROUPS = {"few tokens, then the quantizer": (16, 32, 512),
                 "32 channels x 64, k in two groups, then the quantizer": (32, 64, 512),
                 "64 channels x 64, k in two groups, then the quantizer": (64, 64, 512),
                 "128 channels x 64": (128, 64, 512), "128 channels x 128": (128, 128, 512), "128 channels x 256": (128, 256, 512)}


def _tiles(m, n, a, b):
    return -(-m // a) * -(-n // b)


def test_the_tiles_of_every_accepted_product_fit_a_launch(clib):
    """Over sizes up to the limits, on whole and partitioned devices: fewer
    than 2^32 threads in one dimension of the grid, fewer than 2^16 in the
    other."""
    sizes = sorted({min(1 << 24, max(1, (1 << e) + off)) for e in range(0, 25) for off in (-1, 0, 1)})
    seen = set()
    for m in sizes:
        for n in sizes:
            for d in (0, 1, 129, 1100, 9000, 1 << 22):
                for cus in (32, 256):
                    if _tiles(m, n, 256, 256) <= 1 << 22:
                        for dt in (0, 1):
                            name = clib.gptq_fp8_matmul_kernel(m, d, n, dt, cus).decode()
                            a, b, threads = _GROUPS[name]
                            if name == "few tokens":
                                assert -(-m // a) * threads < 1 << 32 and -(-n // (16 if n <= 16 else 32)) < 1 << 16
                            else:
                                assert _tiles(m, n, a, b) * threads < 1 << 32
                            seen.add((name, dt))
                    if _tiles(m, n, 128, 256) <= 1 << 22:
                        name = clib.gptq_fp8_gated_kernel(m, d, n, cus).decode()
                        a, b, threads = _GATED_GROUPS[name]
                        assert _tiles(m, n, a, b) * threads < 1 << 32
                        seen.add((name, 2))
    assert len(seen) == 7 + 6 + 6  # float32 products have no 128 x 128 tiles


def test_kernel_names_of_empty_and_refused_sizes(clib):
    for m, d, n in ((0, 128, 4), (4, 128, 0), (-1, 128, 4), (4, -1, 4), ((1 << 24) + 1, 128, 4), (4, (1 << 22) + 1, 4),
                    (4, 128, (1 << 24) + 1)):
        assert clib.gptq_fp8_matmul_kernel(m, d, n, 0, 256) is None and clib.gptq_fp8_gated_kernel(m, d, n, 256) is None
    assert clib.gptq_fp8_matmul_kernel(4, 128, 4, 3, 256) is None
    import torch
    from post_weight_quantization_04_amd import _lib
    assert _lib.fp8_matmul_kernel(4, 4, 128, torch.float64, 256) is None
    assert _lib.fp8_matmul_kernel(4, 4, 128, torch.bfloat16, 256) == "few tokens"
    _no_device()
    assert clib.gptq_fp8_matmul_kernel(400, 128, 400, 0, 0) is None and clib.gptq_fp8_gated_kernel(400, 128, 400, 0) is None


def test_the_gpu_tests_sizes_reach_the_kernels_they_name(clib):
    import fp8_cases
    import torch
    from post_weight_quantization_04_amd import _lib
    matmul, gated = fp8_cases.matmul(), fp8_cases.GATED
    less = [[(c[0] - 1,) + c[1:] for c in fp8_cases.batches(cases)] for cases in (matmul, gated)]
    for n, m, d, name, dtype in matmul + less[0]:
        assert _lib.fp8_matmul_kernel(n, m, d, getattr(torch, dtype), 256) == name, (n, m, d, dtype)
    for n, m, d, name in gated + less[1]:
        assert _lib.fp8_gated_kernel(n, m, d, 256) == name, (n, m, d)
    for dtype in ("float16", "bfloat16", "float32"):
        named = set(_GROUPS) - ({"128 x 128"} if dtype == "float32" else set())
        for cases in (matmul, less[0]):
            assert {c[3] for c in cases if c[4] == dtype} == named
    assert {c[3] for c in gated} == {c[3] for c in less[1]} == set(_GATED_GROUPS)
