"""Product with packed few-bit weights on the GPU: rows of x at any alignment
together with several groups a row, once for every kernel, width and type."""
import pytest
import torch

import block_ref as ref
from test_gpu_packed_matmul import make

pytestmark = pytest.mark.gpu
KINDS = ref.KINDS


def unaligned(x, shift=1):
    """x's values in rows of an odd stride that start `shift` elements into their memory, NaN around them."""
    n, d = x.shape
    ld = d + 1 + d % 2
    wide = torch.full((n * ld + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = wide[shift:shift + n * ld].view(n, ld)[:, :d]
    view.copy_(x)
    return view


# name, tokens, rows, columns, group: sizes that reach each kernel which takes unaligned rows
FORMS = [("few tokens", 3, 70, 384, 128), ("few tokens", 3, 70, 208, 16), ("few tokens", 30, 1000, 256, 32),
         ("few tokens", 30, 1000, 512, 128), ("32 x 64", 300, 700, 384, 128), ("32 x 64", 300, 700, 1280, 640),
         ("64 x 128", 250, 1100, 640, 32), ("64 x 128", 530, 301, 192, 48), ("64 x 128", 777, 1363, 384, 128),
         ("64 x 128", 777, 1363, 320, 64), ("64 x 128", 777, 1363, 640, 320)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("name,n,d_out,d,group", FORMS)
def test_unaligned_rows_in_groups(lib, name, n, d_out, d, group, bits, kind):
    from post_weight_quantization_04_amd import _lib, layer
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert _lib.packed_matmul_kernel(n, d_out, d, group, False) == name
    kind = KINDS[kind]
    # whole numbers, for which every sum is exact
    w, x, dense = make(n, d, d_out, bits, group, kind, seed=bits, whole=True)
    got = layer.packed_matmul(w, unaligned(x, bits % 2), dtype=torch.float32)
    assert torch.equal(got.double().cpu(), x.double() @ dense.t())
    # and any, with all of the epilogue
    w, x, dense = make(n, d, d_out, bits, group, kind, seed=bits)
    gen = torch.Generator().manual_seed(bits)
    b, r = torch.randn(d_out, generator=gen).to(kind), torch.randn(n, d_out, generator=gen).to(kind)
    got = layer.packed_matmul(w, unaligned(x), b.cuda(), "silu", r.cuda())
    want, off = ref.product(x.double(), dense, b.double(), "silu", r.double(), kind)
    ref.near(got, want, off, f"{name}: {n} x {d} -> {d_out}, {bits} bits, groups of {group}")
