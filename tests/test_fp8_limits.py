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
