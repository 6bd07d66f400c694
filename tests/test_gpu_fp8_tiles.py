"""Every kernel of the 8-bit product and gated block, by name: exact sums of
whole numbers, the accuracy of the e4m3 MFMA's sums, bad values, and results
that do not depend on the batch.  The sizes are those of ``fp8_cases``.

Tolerances.  Whole numbers: none.  The e4m3 MFMA adds groups of eight products
and cuts each product p below u = 2^-13 of a power of two that is at most the
largest magnitude of its group (``fp8_ref.product``), towards zero.  The
weights' signs are drawn independently of all magnitudes, so the seven cuts of
each group have independent signs and magnitudes below u, and u^2 is at most
2^-26 times the group's sum of p^2: over a row, the variance of the cuts' sum
stays below C = 7 2^-26 sum p^2.
  - One output: by Hoeffding's inequality the sum passes 8 sqrt(C) with
    probability below 2 exp(-32), 3e-14; over the 1e8 outputs tested, 3e-6.
  - All outputs together: a cut lies uniformly in [0, u) to first order, which
    is a third of its square: sqrt(7/3) 2^-13 = 1.9e-4 of the outputs' norm,
    since sum p^2 is an output's mean square under random signs; 2e-4 asserted
    beside half a step of the output type.  The float32 additions (128 in a
    block, a few for each block) round by at most two half steps of sums whose
    mean square is at most the output's: 2 2^-24 times the root of their number.
A product that is lost or counted twice moves an output by about sqrt(sum p^2 /
k), and the norm by as much of it: 7.7e-3 at k = 16500, where 8 sqrt(C) is
2.6e-3 of sqrt(sum p^2)."""
import numpy as np
import pytest

import fp8_cases
import fp8_ref as ref

pytestmark = pytest.mark.gpu


def say(*a):
    print("[fp8 tiles]", *a, flush=True)


def _t():
    import torch
    return torch


def held(v, scales):
    """An 8-bit matrix of values that e4m3 holds, zeros behind them."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rows, d = v.shape
    data = torch.zeros((rows, ref.blocks(d) * 128), dtype=torch.float8_e4m3fn, device="cuda")
    data[:, :d] = v.to(torch.float8_e4m3fn)
    return layer.Fp8(data, scales, d)


def by_rows(x8):
    """Activations in 64 bits."""
    return (x8.data.double() * x8.scales.t().double().repeat_interleave(128, 1))[:, :x8.cols].contiguous()


def by_tiles(w8):
    s = w8.scales.double().repeat_interleave(128, 0)[:w8.data.shape[0]].repeat_interleave(128, 1)
    return (w8.data.double() * s)[:, :w8.cols].contiguous()


def random_operands(gen, n, m, d):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    x = torch.randn((n, d), generator=gen, device="cuda") * torch.randn((1, d), generator=gen, device="cuda").exp()
    w = torch.randn((m, d), generator=gen, device="cuda") * 0.02
    return x, w, layer.fp8_activations(x), layer.fp8_weight(w)


def product_kernel(n, m, d, name, dtype):
    from post_weight_quantization_04_amd import _lib
    assert _lib.fp8_matmul_kernel(n, m, d, getattr(_t(), dtype)) == name


@pytest.mark.parametrize("channel_major", [False, True])
@pytest.mark.parametrize("n,m,d,name,dtype", fp8_cases.matmul())
def test_whole_numbers_are_exact(lib, n, m, d, name, dtype, channel_major):
    """Products are multiples of 1/4 of at most 64, so every sum is exact in
    float32 (below 2^24 quarters at k = 16500) and nothing is cut."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("whole numbers", n, m, d, name, dtype, channel_major)
    product_kernel(n, m, d, name, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    nb = ref.blocks(d)
    x = torch.randint(-4, 5, (n, d), generator=gen, device="cuda").float()
    w = torch.randint(-4, 5, (m, d), generator=gen, device="cuda").float()
    x8 = held(x, 2.0 ** torch.randint(-1, 2, (nb, n), generator=gen, device="cuda").float())
    w8 = held(w, 2.0 ** torch.randint(-1, 2, (ref.blocks(m), nb), generator=gen, device="cuda").float())
    want = by_rows(x8) @ by_tiles(w8).t().contiguous()
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype), channel_major=channel_major)
    assert torch.equal(y.t() if channel_major else y, want.to(y.dtype))
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype), channel_major=channel_major, relu=True)
    assert torch.equal(y.t() if channel_major else y, want.clamp(min=0).to(y.dtype))


@pytest.mark.parametrize("n,m,d,name,dtype", fp8_cases.matmul())
def test_accuracy_of_sums(lib, n, m, d, name, dtype):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("accuracy", n, m, d, name, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n * 3 + m + d)
    _, _, x8, w8 = random_operands(gen, n, m, d)
    xv, wt = by_rows(x8), by_tiles(w8).t().contiguous()
    want = xv @ wt
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype)).double()
    # float32: every addition and scaling rounds by at most two half steps of the sum of magnitudes
    dy = (128 + 2 * ref.blocks(d) + 4) * 2 * ref.U * (xv.abs() @ wt.abs())
    if dtype != "float32":
        dy += 8 * 7 ** 0.5 * 2.0 ** -13 * (xv.square() @ wt.square()).sqrt()
    off = (y - want).abs()
    assert bool((off <= dy + ref.HALF[dtype] * (want.abs() + dy) + ref.TINY[dtype]).all())
    steps = 128 + 2 * ref.blocks(d) + 4
    sums = 2 * ref.U * steps ** 0.5 + (0 if dtype == "float32" else 2e-4)
    assert float((y - want).norm() / want.norm()) <= sums + ref.HALF[dtype]


@pytest.mark.parametrize("n,m,d,name,dtype", fp8_cases.matmul())
def test_what_cancels(lib, n, m, d, name, dtype):
    """Products of 2^16 and -2^16, seven of 3.5 beside the first: float32
    results and the few-token kernel hold the rest, 24.5; the e4m3 MFMA may cut
    it, within 2^-10 of the sum of magnitudes."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("cancels", n, m, d, name, dtype)
    x, w = torch.zeros((n, d), device="cuda"), torch.zeros((m, d), device="cuda")
    x[:, 0] = x[:, d - 1] = w[:, 0] = 256
    w[:, d - 1] = -256
    x[:, 1:8], w[:, 1:8] = 3.5, 1
    x8 = held(x, torch.ones((ref.blocks(d), n), device="cuda"))
    w8 = held(w, torch.ones((ref.blocks(m), ref.blocks(d)), device="cuda"))
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype)).float()
    if dtype == "float32" or name == "few tokens":
        assert bool((y == 24.5).all())
    else:
        assert float((y - 24.5).abs().max()) <= 2.0 ** -10 * (2 * 65536 + 24.5)
    few = layer.fp8_matmul(w8, layer.Fp8(x8.data[:32], x8.scales[:, :32], d), dtype=getattr(torch, dtype))
    assert bool((few == 24.5).all())


@pytest.mark.parametrize("n,m,d,name,dtype", fp8_cases.matmul())
def test_bad_values_stay_where_they_belong(lib, n, m, d, name, dtype):
    """A NaN and infinities in tokens (the last one in the last block of k) and
    a NaN in a weight: those tokens and that block of 128 channels are NaN, and
    every other output keeps its bits."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("bad values", n, m, d, name, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    x, w, x8, w8 = random_operands(gen, n, m, d)
    last = (m - 1) // 128 * 128
    for relu in (False, True):
        clean = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype), relu=relu)
        assert not clean.isnan().any()
        xb, wb = x.clone(), w.clone()
        xb[1, d // 2], xb[2, 0], xb[n - 1, d - 1] = float("nan"), float("inf"), -float("inf")
        wb[m - 1, d - 1] = float("nan")
        bad = torch.zeros((n, m), dtype=torch.bool, device="cuda")
        bad[[1, 2, n - 1]] = True
        y = layer.fp8_matmul(w8, layer.fp8_activations(xb), dtype=clean.dtype, relu=relu)
        assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], clean[~bad])
        bad[:, last:] = True
        y = layer.fp8_matmul(layer.fp8_weight(wb), layer.fp8_activations(xb), dtype=clean.dtype, relu=relu)
        assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("n,m,d,name,dtype", fp8_cases.batches(fp8_cases.matmul()))
def test_results_do_not_depend_on_the_batch(lib, n, m, d, name, dtype):
    """The same tokens without the first, so that each moves to another lane
    or tile of the same kernel, and the same call twice: the same bits."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("batch", n, m, d, name, dtype)
    product_kernel(n, m, d, name, dtype)
    product_kernel(n - 1, m, d, name, dtype)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    _, _, x8, w8 = random_operands(gen, n, m, d)
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, dtype))
    assert torch.equal(y, layer.fp8_matmul(w8, x8, dtype=y.dtype))
    part = layer.Fp8(x8.data[1:], x8.scales[:, 1:], d)
    assert torch.equal(layer.fp8_matmul(w8, part, dtype=y.dtype), y[1:])


def gated_kernel(n, m, d, name):
    from post_weight_quantization_04_amd import _lib
    assert _lib.fp8_gated_kernel(n, m, d) == name


@pytest.mark.parametrize("n,m,d,name", fp8_cases.GATED)
def test_gated(lib, n, m, d, name):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("gated", n, m, d, name)
    gated_kernel(n, m, d, name)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    _, _, x8, g8 = random_operands(gen, n, m, d)
    u8 = layer.fp8_weight(torch.randn((m, d), generator=gen, device="cuda") * 0.02)
    xv = by_rows(x8)
    got = []
    for w8 in (g8, u8):
        wt = by_tiles(w8).t().contiguous()
        got += [(xv @ wt).cpu().numpy(), ((128 + 2 * ref.blocks(d) + 4) * 2 * ref.U * (xv.abs() @ wt.abs())).cpu().numpy()]
    h, dh = ref.silu_gate(got[0], got[2], got[1], got[3])
    out = layer.fp8_gated(g8, u8, x8)
    ref.check_quantized(out.data.view(torch.uint8).cpu().numpy(), out.scales.cpu().numpy(), h, dh)


@pytest.mark.parametrize("n,m,d,name", fp8_cases.GATED)
def test_gated_bad_values_stay_where_they_belong(lib, n, m, d, name):
    """A bad token is NaN in every block of the result, a bad gate or up weight
    in its own block of channels; every other code and scale keeps its bits."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("gated, bad values", n, m, d, name)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    x, g, x8, g8 = random_operands(gen, n, m, d)
    u = torch.randn((m, d), generator=gen, device="cuda") * 0.02
    u8 = layer.fp8_weight(u)
    clean = layer.fp8_gated(g8, u8, x8)
    assert not clean.scales.isnan().any()
    xb, gb, ub = x.clone(), g.clone(), u.clone()
    xb[1, d // 2], xb[n - 1, d - 1] = float("nan"), -float("inf")
    gb[m - 1, 0] = ub[0, d - 1] = float("nan")
    y = layer.fp8_gated(layer.fp8_weight(gb), layer.fp8_weight(ub), layer.fp8_activations(xb))
    bad = torch.zeros((n, ref.blocks(m)), dtype=torch.bool, device="cuda")
    bad[[1, n - 1]] = True
    bad[:, 0] = bad[:, -1] = True
    assert torch.equal(y.scales.isnan(), bad.t())
    assert torch.equal(y.scales[~bad.t()], clean.scales[~bad.t()])
    same = ~bad.repeat_interleave(128, 1)
    assert torch.equal(y.data.view(torch.uint8)[same], clean.data.view(torch.uint8)[same])


@pytest.mark.parametrize("n,m,d,name", fp8_cases.batches(fp8_cases.GATED))
def test_gated_does_not_depend_on_the_batch(lib, n, m, d, name):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("gated, batch", n, m, d, name)
    gated_kernel(n, m, d, name)
    gated_kernel(n - 1, m, d, name)
    gen = torch.Generator(device="cuda").manual_seed(n + m + d)
    _, _, x8, g8 = random_operands(gen, n, m, d)
    u8 = layer.fp8_weight(torch.randn((m, d), generator=gen, device="cuda") * 0.02)
    y, again = layer.fp8_gated(g8, u8, x8), layer.fp8_gated(g8, u8, x8)
    assert torch.equal(y.data.view(torch.uint8), again.data.view(torch.uint8)) and torch.equal(y.scales, again.scales)
    part = layer.fp8_gated(g8, u8, layer.Fp8(x8.data[1:], x8.scales[:, 1:], d))
    assert torch.equal(part.data.view(torch.uint8), y.data.view(torch.uint8)[1:])
    assert torch.equal(part.scales, y.scales[:, 1:])
