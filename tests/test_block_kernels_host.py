"""Which kernel of the products with packed weights is named, for forms that
not every kernel has: rows of x at any alignment, groups of any size."""
import os

import pytest


@pytest.fixture(scope="module")
def kernel():
    from post_weight_quantization_04_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return lambda n, m, k, group, aligned: _lib.packed_matmul_kernel(n, m, k, group, aligned, 256)


# kernels there are, by (aligned rows, whole groups of 128 or one a row)
THERE = {(True, True): {"few tokens", "32 x 64", "64 x 128", "128 x 384"}, (True, False): {"few tokens", "32 x 64", "64 x 128"},
         (False, True): {"few tokens", "32 x 64", "64 x 128"}, (False, False): {"few tokens", "64 x 128"}}


def test_only_kernels_that_run_are_named(kernel):
    seen = {form: set() for form in THERE}
    for n in (1, 4, 5, 16, 17, 40, 64, 100, 250, 300, 530, 777, 1100, 2700, 4000, 8192):
        for m in (64, 301, 700, 1100, 1363, 2801, 4096, 11008):
            for k, group in ((384, 0), (512, 128), (640, 32), (640, 320), (192, 48), (4096, 64), (4096, 128), (1000, 0)):
                for aligned in (True, False):
                    form = aligned and k % 8 == 0, group % 128 == 0 or k <= group
                    seen[form].add(kernel(n, m, k, group, aligned))
    assert seen == THERE


def test_unaligned_rows_in_small_groups(kernel):
    assert kernel(250, 1100, 640, 32, True) == "32 x 64"
    assert kernel(250, 1100, 640, 32, False) == "64 x 128"
    assert kernel(64, 4096, 4096, 32, False) == "few tokens"
    assert kernel(2700, 2801, 192, 48, False) == "64 x 128"


def test_parts_of_the_cached_attention_are_aligned():
    """A part is read and written as sixteen bytes: 1024 of them, each a multiple of that, for any number of query heads
    that share a key head."""
    from post_weight_quantization_04_amd import _lib
    for rows in range(1, 20):
        for d in (64, 128):
            need = _lib.cached_attention_workspace(2, 2 * rows, 2, d, 400, 16)
            held = min(rows, 16)
            assert need % 1024 == 0 and need // 1024 % 16 == 0, (rows, d)
            assert 4 * held * (d + 2) <= need // 1024 < 4 * held * (d + 2) + 16, (rows, d)


def test_a_product_onto_its_own_input_is_refused():
    """Workgroups read all of X while others write Y (made before any HIP call: the pointer is never used)."""
    import ctypes
    from post_weight_quantization_04_amd import _lib
    p, other = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)
    rc = _lib.load().gptq_packed_matmul(other, 4, 256, 256, other, other, 128, p, 0, 4, 256, None, None, 0, p, 0, 256, 0, None)
    assert rc == 1
