"""8-bit operators on the GPU against the definitions of ``fp8_ref``.

Tolerances.  Quantizers: the float32 steps are given, so scales and codes are
compared for equality.  Norm, product and gated block: the bound on float32
sums of ``fp8_ref`` (one step per addition, and what the e4m3 MFMA's adder
cuts where that runs) plus half a step of the output type, 2^-11 of the value for float16, 2^-8 bfloat16, 2^-24 float32, and half a
step of e4m3 (2^-4, or 2^-10 scales near zero) where the output is in 8 bits.
"""
import numpy as np
import pytest

import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = ("float16", "bfloat16", "float32")


def say(*a):
    print("[fp8]", *a, flush=True)


def _t():
    import torch
    return torch


def typed(a, name):
    """A device tensor of the type, and its values as float32."""
    torch = _t()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(getattr(torch, name))
    return t.cuda(), t.float().numpy()


def codes_of(f):
    return f.data.view(_t().uint8).cpu().numpy()


def strided(t, pad, offset):
    """The same values in a buffer with a longer row and an offset start."""
    torch = _t()
    ld = t.shape[1] + pad
    buf = torch.full((t.shape[0] * ld + offset + 8,), 7.0, dtype=t.dtype, device=t.device)
    v = torch.as_strided(buf, t.shape, (ld, 1), offset)
    v.copy_(t)
    return v


def values(rng, n, d):
    x = rng.standard_normal((n, d)) * np.exp(rng.standard_normal((1, d)))
    x[:, rng.integers(0, d, max(1, d // 100))] *= 30
    return x


# ---------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------
SIZES = [(1, 1), (1, 128), (3, 127), (64, 128), (65, 130), (17, 1000), (200, 257), (130, 1032)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
def test_quantizers_equal_the_definition(lib, n, d, name, pad, offset):
    from post_weight_quantization_04_amd import layer
    say("quantizers", n, d, name, pad, offset)
    rng = np.random.default_rng(n * 1000 + d)
    x, xf = typed(values(rng, n, d), name)
    want_q, want_s = ref.quantize_rows(xf)
    got = layer.fp8_activations(strided(x, pad, offset))
    np.testing.assert_array_equal(got.scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes_of(got), want_q)
    got = layer.fp8_activations(strided(x.t().contiguous(), pad, offset), channel_major=True)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes_of(got), want_q)
    want_q, want_s = ref.quantize_tiles(xf)
    got = layer.fp8_weight(strided(x, pad, offset))
    np.testing.assert_array_equal(got.scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes_of(got), want_q)


def test_every_rounding_of_e4m3(lib):
    """Every e4m3 value, every midpoint (a tie) and its float32 neighbours, in
    blocks whose peak 448 makes the scale 1."""
    from post_weight_quantization_04_amd import layer
    v = ref.TABLE[:127].astype(np.float32)
    mid = ((v[:-1].astype(np.float64) + v[1:]) / 2).astype(np.float32)
    x = np.concatenate([v, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1000))])
    x = np.concatenate([x, -x])
    x = np.concatenate([x, np.zeros(-len(x) % 127, np.float32)]).reshape(-1, 127)
    x = np.concatenate([np.full((len(x), 1), 448, np.float32), x], axis=1)
    t, xf = typed(x, "float32")
    got = layer.fp8_activations(t)
    assert np.all(got.scales.cpu().numpy() == 1.0)
    np.testing.assert_array_equal(codes_of(got), ref.encode(xf))


def test_special_blocks(lib):
    """Zeros, values far below the floor, the largest floats, infinities and
    NaN: a bad value spoils its own block only."""
    from post_weight_quantization_04_amd import layer
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 384)).astype(np.float32)
    x[0] = 0
    x[1, :128] = 1e-39
    x[2, 128:256] *= 5e37
    x[3, 130] = np.inf
    x[4, 5] = np.nan
    x[5, 300] = -np.inf
    t, xf = typed(x, "float32")
    want_q, want_s = ref.quantize_rows(xf)
    for got in (layer.fp8_activations(t), layer.fp8_activations(t.t().contiguous(), channel_major=True)):
        v = ref.rows_values(codes_of(got), got.scales.cpu().numpy(), 384)
        w = ref.rows_values(want_q, want_s, 384)
        np.testing.assert_array_equal(np.isnan(v), np.isnan(w))
        assert np.isnan(v[3, 128:256]).all() and np.isnan(v[4, :128]).all() and np.isnan(v[5, 256:]).all()
        assert np.isnan(v).sum() == 3 * 128
        np.testing.assert_array_equal(v[~np.isnan(w)], w[~np.isnan(w)])
    got = layer.fp8_weight(t)
    v = ref.tiles_values(codes_of(got), got.scales.cpu().numpy(), 384)
    assert np.isnan(v).all()   # all six rows share each 128 x 128 block, and each block holds a bad value


@pytest.mark.parametrize("channel_major", [False, True])
def test_what_lies_behind_is_left_alone(lib, channel_major):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    n, d = 70, 200
    x, xf = typed(np.random.default_rng(1).standard_normal((n, d)), "float16")
    data = torch.full((n + 3, 512), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, n + 5), 9.0, device="cuda")
    out = layer.Fp8(data[:n].view(torch.float8_e4m3fn), scales, d)
    layer.fp8_activations(x.t().contiguous() if channel_major else x, channel_major=channel_major, out=out)
    q, s = ref.quantize_rows(xf)
    h = data.cpu().numpy()
    np.testing.assert_array_equal(h[:n, :256], q)
    assert (h[n:] == 0x55).all() and (h[:, 256:] == 0x55).all()
    hs = scales.cpu().numpy()
    np.testing.assert_array_equal(hs[:2, :n], s)
    assert (hs[2:] == 9).all() and (hs[:, n:] == 9).all()
    # weights: d_out rows
    data.fill_(0x55)
    scales.fill_(9.0)
    layer.fp8_weight(x, out=layer.Fp8(data[:n].view(torch.float8_e4m3fn), scales, d))
    q, s = ref.quantize_tiles(xf)
    h, hs = data.cpu().numpy(), scales.cpu().numpy()
    np.testing.assert_array_equal(h[:n, :256], q)
    assert (h[n:] == 0x55).all() and (h[:, 256:] == 0x55).all()
    np.testing.assert_array_equal(hs[:1, :2], s)
    assert (hs[1:] == 9).all() and (hs[:, 2:] == 9).all()


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_ref(h, gain, eps):
    """y in 64 bits and its bound: a thread adds at most 32 squares (more only
    for the widest rows), ten additions join them; quotient, root, reciprocal
    and two products round once each."""
    rms = np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    y = h / rms * gain
    terms = max(32, h.shape[1] // 512 + 8) + 10 + 16
    return y, (terms + 10) * 2 * ref.U * np.abs(y)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("n,d,residual,pad", [
    (1, 1, True, 0), (5, 64, True, 0), (7, 127, False, 1), (9, 512, True, 8), (3, 520, True, 0), (2, 1000, False, 0),
    (4, 2048, True, 0), (1, 4096, True, 0), (33, 4096, True, 8), (3, 4100, True, 3), (2, 8192, False, 0),
    (2, 11008, True, 0), (2, 16384, True, 0), (2, 16392, True, 0), (3, 20001, True, 0),
])
def test_rms_norm(lib, n, d, residual, pad, name):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("norm", n, d, residual, pad, name)
    rng = np.random.default_rng(n + d)
    x, xf = typed(values(rng, n, d), name)
    r, rf = typed(values(rng, n, d) * 3, name)
    g, gf = typed(1 + 0.3 * rng.standard_normal(d), name)
    eps = 1e-5
    out, total = layer.fp8_rms_norm(strided(x, pad, pad), g, eps, residual=strided(r, pad, 0) if residual else None)
    h32 = xf + rf if residual else xf
    # the kernel norms the float32 sum: known to half a step of it
    y, dy = norm_ref(h32.astype(np.float64), gf.astype(np.float64), eps)
    ref.check_quantized(codes_of(out), out.scales.cpu().numpy(), y, dy)
    if residual:
        assert torch.equal(total.cpu(), torch.from_numpy(h32).to(x.dtype))
    else:
        assert total is None


@pytest.mark.parametrize("d", [500, 4096, 20000])
@pytest.mark.parametrize("into", ["residual", "x"])
def test_rms_norm_in_place(lib, d, into):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(d)
    x, _ = typed(values(rng, 6, d), "bfloat16")
    r, _ = typed(values(rng, 6, d), "bfloat16")
    g, _ = typed(rng.standard_normal(d), "bfloat16")
    want, total = layer.fp8_rms_norm(x, g, residual=r)
    x2, r2 = x.clone(), r.clone()
    got, same = layer.fp8_rms_norm(x2, g, residual=r2, sum_out=r2 if into == "residual" else x2)
    assert same is (r2 if into == "residual" else x2)
    assert torch.equal(same, total)
    assert torch.equal(x2 if into == "residual" else r2, x if into == "residual" else r)
    np.testing.assert_array_equal(codes_of(got), codes_of(want))
    assert torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("d", [300, 4096, 20000])
def test_rms_norm_extremes(lib, d):
    """Rows of zeros, of values whose squares leave float32, with an infinity,
    with a NaN: the others stay right."""
    from post_weight_quantization_04_amd import layer
    rng = np.random.default_rng(d)
    h = rng.standard_normal((6, d)).astype(np.float32)
    h[1] = 0
    h[2] *= 1e30
    h[3, 7] = np.inf
    h[4, 200] = np.nan
    h[5] *= 1e-18
    x, xf = typed(h, "float32")
    g, gf = typed(1 + 0.1 * rng.standard_normal(d), "float32")
    out, _ = layer.fp8_rms_norm(x, g, 1e-20)
    q, s = codes_of(out), out.scales.cpu().numpy()
    fine = [0, 1, 2, 5]
    y, dy = norm_ref(xf[fine].astype(np.float64), gf.astype(np.float64), 1e-20)
    ref.check_quantized(q[fine], s[:, fine], y, dy)
    v = ref.rows_values(q, s, d)
    assert np.isnan(v[3, :128]).all() and (v[3, 128:] == 0).all()   # x / infinity elsewhere
    assert np.isnan(v[4]).all()


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def operands(rng, n, m, d):
    """8-bit activations and weights as the quantizers write them."""
    from post_weight_quantization_04_amd import layer
    x, _ = typed(values(rng, n, d), "float16")
    w, _ = typed(rng.standard_normal((m, d)) * 0.02, "float16")
    x8, w8 = layer.fp8_activations(x), layer.fp8_weight(w)
    xv = ref.rows_values(codes_of(x8), x8.scales.cpu().numpy(), d)
    wv = ref.tiles_values(codes_of(w8), w8.scales.cpu().numpy(), d)
    return x8, w8, xv, wv


MM = [(1, 1, 1), (1, 16, 128), (1, 4096, 256), (2, 17, 129), (15, 100, 1000), (16, 64, 1100), (17, 200, 384), (33, 130, 640),
      (64, 256, 512), (65, 257, 300), (100, 1363, 1000), (129, 128, 1152), (200, 520, 136), (256, 512, 256), (300, 700, 2000),
      (513, 1025, 513), (1030, 260, 128)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("n,m,d", MM)
@pytest.mark.parametrize("channel_major", [False, True])
def test_matmul(lib, n, m, d, name, channel_major):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("matmul", n, m, d, name, channel_major)
    rng = np.random.default_rng(n * 7 + m + d)
    x8, w8, xv, wv = operands(rng, n, m, d)
    relu = (n + m) % 2 == 1
    shape = (m, n) if channel_major else (n, m)
    # a view with a longer row: what lies behind has to stay
    buf = torch.full((shape[0] + 1, shape[1] + 5), 3.0, dtype=getattr(torch, name), device="cuda")
    y = layer.fp8_matmul(w8, x8, relu=relu, channel_major=channel_major, out=buf[:shape[0], :shape[1]])
    got = y.float().cpu().numpy().astype(np.float64)
    want, dy = ref.product(xv, wv, ref.cuts(n, name))
    if relu:
        want = np.maximum(want, 0)
    if channel_major:
        want, dy = want.T, dy.T
    most = dy + ref.HALF[name] * (np.abs(want) + dy) + ref.TINY[name]
    off = np.abs(got - want)
    assert np.all(off <= most), float(np.max(off / most))
    rest = buf.float().cpu().numpy()
    assert (rest[shape[0]:] == 3).all() and (rest[:, shape[1]:] == 3).all()


# tiles from 64 x 64 to 256 x 256 and once the few-token kernel, most in ragged
# sizes, mostly of a few blocks of k (``fp8_cases`` holds sizes of every kernel by name)
LARGE = [(4090, 4100, 300), (2040, 4096, 200), (1020, 4096, 260), (500, 4096, 128), (700, 4000, 8400), (90, 300, 16520),
         (1030, 1025, 72), (500, 4096, 1300), (4090, 4096, 600), (4000, 4090, 250)]


@pytest.mark.parametrize("name", ("float16", "float32"))
@pytest.mark.parametrize("n,m,d", LARGE)
@pytest.mark.parametrize("channel_major", [False, True])
def test_matmul_tiles(lib, n, m, d, name, channel_major):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("matmul tiles", n, m, d, name, channel_major)
    rng = np.random.default_rng(n + m + d)
    x8, w8, xv, wv = operands(rng, n, m, d)
    y = layer.fp8_matmul(w8, x8, dtype=getattr(torch, name), channel_major=channel_major)
    got = (y.t() if channel_major else y).float().cpu().numpy()
    want, dy = ref.product(xv, wv, ref.cuts(n, name))
    most = dy + ref.HALF[name] * (np.abs(want) + dy) + ref.TINY[name]
    off = np.abs(got - want)
    assert np.all(off <= most), float(np.max(off / most))


@pytest.mark.parametrize("n,m,d", [(1, 200, 512), (40, 300, 700), (300, 512, 1024)])
def test_matmul_of_whole_numbers_is_exact(lib, n, m, d):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(n)
    xi = rng.integers(-3, 4, (n, d)).astype(np.float32)
    wi = rng.integers(-3, 4, (m, d)).astype(np.float32)

    def held(v, scales):
        data = np.zeros((v.shape[0], ref.blocks(d) * 128), np.uint8)
        data[:, :d] = ref.encode(v)
        return layer.Fp8(torch.from_numpy(data).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda(), d)

    sx = (2.0 ** rng.integers(0, 3, (ref.blocks(d), n))).astype(np.float32)
    sw = (2.0 ** rng.integers(0, 3, (ref.blocks(m), ref.blocks(d)))).astype(np.float32)
    x8, w8 = held(xi, sx), held(wi, sw)
    want = ref.rows_values(codes_of(x8), sx, d) @ ref.tiles_values(codes_of(w8), sw, d).T
    assert np.abs(want).max() < 2 ** 24
    y = layer.fp8_matmul(w8, x8, dtype=torch.float32)
    np.testing.assert_array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("name", ("float16", "float32"))
@pytest.mark.parametrize("channel_major", [False, True])
def test_matmul_of_long_rows_is_exact(lib, name, channel_major):
    """The largest tiles over 65 blocks of k: a round of 64 scales, and one
    more.  Every sum is exact, and float16 rounds it once."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, m, d = 3840, 4096, 65 * 128
    say("long rows", n, m, d, name, channel_major)
    x, w = (torch.randint(-1, 2, (rows, d), generator=gen, device="cuda").float() for rows in (n, m))
    xs = 2.0 ** torch.randint(-1, 2, (65, n), generator=gen, device="cuda").float()
    ws = 2.0 ** torch.randint(-1, 2, (m // 128, 65), generator=gen, device="cuda").float()
    y = layer.fp8_matmul(layer.Fp8(w.to(torch.float8_e4m3fn), ws, d), layer.Fp8(x.to(torch.float8_e4m3fn), xs, d),
                         dtype=getattr(torch, name), channel_major=channel_major)
    # every product is a multiple of 1/4 of at most 4, and float32 holds all sums
    want = (x * xs.t().repeat_interleave(128, 1)) @ (w * ws.repeat_interleave(128, 0).repeat_interleave(128, 1)).t()
    assert torch.equal(y.t() if channel_major else y, want.to(y.dtype))


@pytest.mark.parametrize("n,m", [(3, 200), (300, 300)])
def test_matmul_carries_bad_values(lib, n, m):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(3)
    d = 300
    x = rng.standard_normal((n, d)).astype(np.float32)
    x[1, 150] = np.nan
    x[2, 0] = np.inf
    x8 = layer.fp8_activations(typed(x, "float32")[0])
    w8 = layer.fp8_weight(typed(rng.standard_normal((m, d)), "float32")[0])
    for relu in (False, True):
        y = layer.fp8_matmul(w8, x8, dtype=torch.float32, relu=relu)
        bad = torch.isnan(y)
        assert bad[1].all() and bad[2].all() and int(bad.sum()) == 2 * m


def test_matmul_empty(lib):
    from post_weight_quantization_04_amd import layer
    torch = _t()
    e = torch.float8_e4m3fn
    w = layer.Fp8(torch.empty((5, 0), dtype=e, device="cuda"), torch.empty((1, 0), device="cuda"), 0)
    x = layer.Fp8(torch.empty((7, 0), dtype=e, device="cuda"), torch.empty((0, 7), device="cuda"), 0)
    y = torch.full((7, 5), 4.0, device="cuda")
    assert torch.equal(layer.fp8_matmul(w, x, out=y), torch.zeros((7, 5), device="cuda"))
    for n in (7, 70):   # both kernels of the gated block
        x0 = layer.Fp8(torch.empty((n, 0), dtype=e, device="cuda"), torch.empty((0, n), device="cuda"), 0)
        h = layer.fp8_gated(w, w, x0)
        assert h.values.shape == (n, 5) and not h.data.view(torch.uint8).any()
        assert bool((h.scales == 2.0 ** -96 / 448).all())
        y = layer.fp8_matmul(w, x0)
        assert not y.any()
    none = layer.fp8_activations(torch.empty((0, 256), device="cuda"))
    w8 = layer.fp8_weight(torch.ones((5, 256), device="cuda"))
    assert layer.fp8_matmul(w8, none).shape == (0, 5)
    assert layer.fp8_gated(w8, w8, none).values.shape == (0, 5)
    assert layer.fp8_weight(torch.empty((0, 256), device="cuda")).values.shape == (0, 256)


# ---------------------------------------------------------------------------
# gated block
# ---------------------------------------------------------------------------
GATED = [(1, 1, 1), (1, 128, 256), (1, 1000, 520), (2, 130, 129), (16, 256, 512), (17, 200, 384), (40, 640, 300), (64, 129, 256),
         (65, 384, 640), (130, 257, 200), (256, 256, 384), (300, 700, 513),
         (200, 5000, 136), (1024, 11008, 128), (4090, 2040, 200), (33, 140, 16600),
         (990, 500, 1000), (100, 5590, 1300), (70, 5500, 8300), (200, 5000, 8300), (4090, 2040, 300)]


@pytest.mark.parametrize("n,m,d", GATED)
def test_gated(lib, n, m, d):
    from post_weight_quantization_04_amd import layer
    say("gated", n, m, d)
    rng = np.random.default_rng(n + m + d)
    x8, g8, xv, gv = operands(rng, n, m, d)
    _, u8, _, uv = operands(rng, 1, m, d)
    out = layer.fp8_gated(g8, u8, x8)
    g, dg = ref.product(xv, gv)
    u, du = ref.product(xv, uv)
    h, dh = ref.silu_gate(g, u, dg, du)
    ref.check_quantized(codes_of(out), out.scales.cpu().numpy(), h, dh)


@pytest.mark.parametrize("n", [4, 200])
def test_gated_far_gates(lib, n):
    """Gates of plus and minus several hundred: exp overflows, silu does not."""
    from post_weight_quantization_04_amd import layer
    rng = np.random.default_rng(8)
    m, d = 256, 256
    x8, g8, xv, gv = operands(rng, n, m, d)
    x8.scales.mul_(100.0)
    xv = ref.rows_values(codes_of(x8), x8.scales.cpu().numpy(), d)
    _, u8, _, uv = operands(rng, 1, m, d)
    g, dg = ref.product(xv, gv)
    u, du = ref.product(xv, uv)
    assert g.min() < -100 and g.max() > 100
    h, dh = ref.silu_gate(g, u, dg, du)
    out = layer.fp8_gated(g8, u8, x8)
    ref.check_quantized(codes_of(out), out.scales.cpu().numpy(), h, dh)


# ---------------------------------------------------------------------------
# together, as they are used
# ---------------------------------------------------------------------------
def test_a_feed_forward_block(lib):
    """norm -> gate, up, product -> down -> the next norm's residual sum, each
    step against the definition fed with the step before."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(12)
    for n in (1, 5, 90):
        d, ff = 512, 1400
        x, xf = typed(rng.standard_normal((n, d)), "bfloat16")
        r, rf = typed(values(rng, n, d), "bfloat16")
        gain, gainf = typed(1 + 0.1 * rng.standard_normal(d), "bfloat16")
        weights = [layer.fp8_weight(typed(rng.standard_normal(s) * 0.05, "bfloat16")[0]) for s in ((ff, d), (ff, d), (d, ff))]
        gate, up, down = weights
        a, stream = layer.fp8_rms_norm(x, gain, residual=r)
        h = layer.fp8_gated(gate, up, a)
        y = layer.fp8_matmul(down, h, dtype=torch.bfloat16)
        b, stream2 = layer.fp8_rms_norm(y, gain, residual=stream)
        y1, dy1 = norm_ref((xf + rf).astype(np.float64), gainf.astype(np.float64), 1e-6)
        ref.check_quantized(codes_of(a), a.scales.cpu().numpy(), y1, dy1)
        av = ref.rows_values(codes_of(a), a.scales.cpu().numpy(), d)
        gv, uv = (ref.tiles_values(codes_of(w), w.scales.cpu().numpy(), d) for w in (gate, up))
        g, dg = ref.product(av, gv)
        u, du = ref.product(av, uv)
        hv, dh = ref.silu_gate(g, u, dg, du)
        ref.check_quantized(codes_of(h), h.scales.cpu().numpy(), hv, dh)
        got_h = ref.rows_values(codes_of(h), h.scales.cpu().numpy(), ff)
        yv, dy = ref.product(got_h, ref.tiles_values(codes_of(down), down.scales.cpu().numpy(), ff), ref.cuts(n, "bfloat16"))
        off = np.abs(y.float().cpu().numpy() - yv)
        assert np.all(off <= dy + 2.0 ** -8 * (np.abs(yv) + dy) + 2.0 ** -134)
        s2 = stream.float().cpu().numpy() + y.float().cpu().numpy()
        assert torch.equal(stream2.cpu(), torch.from_numpy(s2).bfloat16())


def test_propagate_fp8_feeds_the_next_hessian(lib):
    """A chain layer kept in 8 bits: its output is the next layer's input."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(4)
    X, Xf = typed(rng.standard_normal((200, 264)), "float16")
    w8 = layer.fp8_weight(typed(rng.standard_normal((144, 200)) * 0.1, "float16")[0])
    Y = layer.propagate_fp8(w8, X, relu=True)
    assert Y.shape == (144, 264) and Y.dtype == torch.float16
    xq, xs = ref.quantize_rows(np.ascontiguousarray(Xf.T))
    want, dy = ref.product(ref.rows_values(xq, xs, 200), ref.tiles_values(codes_of(w8), w8.scales.cpu().numpy(), 200),
                           ref.cuts(264, "float16"))
    want = np.maximum(want, 0)
    got = Y.float().cpu().numpy().T
    assert np.all(np.abs(got - want) <= dy + 2.0 ** -11 * (np.abs(want) + dy) + 2.0 ** -25)
    H = layer.hessian(Y).cpu().numpy()
    full = 2 * got.astype(np.float64).T @ got
    assert np.linalg.norm(np.tril(H) - np.tril(full)) <= 1e-5 * np.linalg.norm(np.tril(full))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("d,n,m,relu", [(200, 5, 144, False), (130, 264, 300, True), (640, 1000, 257, False)])
def test_propagate_fp8_of_every_type_feeds_the_next_hessian(lib, d, n, m, relu, name):
    """float16 and float32 come back as they were, bfloat16 as float32; the
    Hessian takes each, and a second layer of the chain the first one's."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    say("propagate", d, n, m, relu, name)
    rng = np.random.default_rng(d + n)
    X, Xf = typed(rng.standard_normal((d, n)), name)
    w8 = layer.fp8_weight(typed(rng.standard_normal((m, d)) * 0.1, name)[0])
    Y = layer.propagate_fp8(w8, X, relu=relu)
    back = "float32" if name == "bfloat16" else name
    assert Y.shape == (m, n) and Y.dtype == getattr(torch, back)
    xq, xs = ref.quantize_rows(np.ascontiguousarray(Xf.T))
    want, dy = ref.product(ref.rows_values(xq, xs, d), ref.tiles_values(codes_of(w8), w8.scales.cpu().numpy(), d),
                           ref.cuts(n, back))
    want = np.maximum(want, 0) if relu else want
    got = Y.float().cpu().numpy().T
    assert np.all(np.abs(got - want) <= dy + ref.HALF[back] * (np.abs(want) + dy) + ref.TINY[back])
    H = layer.hessian(Y).cpu().numpy()
    full = 2 * got.astype(np.float64).T @ got
    assert np.linalg.norm(np.tril(H) - np.tril(full)) <= 1e-5 * np.linalg.norm(np.tril(full))
    v8 = layer.fp8_weight(typed(rng.standard_normal((64, m)) * 0.1, name)[0])
    assert layer.propagate_fp8(v8, Y).dtype == Y.dtype
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    assert layer.propagate_fp8(w8, X, relu=relu, out=out) is out
    _, dy = ref.product(ref.rows_values(xq, xs, d), ref.tiles_values(codes_of(w8), w8.scales.cpu().numpy(), d),
                        ref.cuts(n, "bfloat16"))
    off = np.abs(out.float().cpu().numpy().T - want)
    assert np.all(off <= dy + 2.0 ** -8 * (np.abs(want) + dy) + 2.0 ** -134)


@pytest.mark.parametrize("n", [2, 150])
def test_graphs_and_streams(lib, n):
    """The chain captured twice on a side stream, replayed in turn with eager
    work between, equals the eager result on new inputs every time."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(n)
    d, ff = 384, 640
    x = torch.empty((n, d), dtype=torch.float16, device="cuda")
    r = torch.empty_like(x)
    gain = typed(1 + 0.1 * rng.standard_normal(d), "float16")[0]
    gate, up, down = (layer.fp8_weight(typed(rng.standard_normal(s) * 0.05, "float16")[0]) for s in ((ff, d), (ff, d), (d, ff)))
    ws = layer.Workspace()

    def chain(ws=None):
        a, total = layer.fp8_rms_norm(x, gain, residual=r)
        h = layer.fp8_gated(gate, up, a, ws=ws)
        return h.data, h.scales, layer.fp8_matmul(down, h), total

    def fill(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn((n, d), generator=gen, device="cuda"))
        r.copy_(torch.randn((n, d), generator=gen, device="cuda"))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for share in (None, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(share)
        graphs.append((g, out))
    for seed in range(1, 5):
        fill(seed)
        want = [t.clone() for t in chain()]
        torch.cuda.synchronize()
        for g, out in graphs:
            g.replay()
            for a, b in zip(out, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        chain(ws)
    # a stream given by hand
    fill(9)
    torch.cuda.synchronize()
    want = layer.fp8_rms_norm(x, gain, residual=r)[0]
    torch.cuda.synchronize()
    got = layer.fp8_rms_norm(x, gain, residual=r, stream=side)[0]
    side.synchronize()
    assert torch.equal(got.data.view(torch.uint8), want.data.view(torch.uint8))


def test_a_workspace_that_grows_keeps_a_graphs_buffer(lib):
    """A graph captured with a small workspace, which then grows: the replay
    writes to the buffer it was captured with, which nobody else was given."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(6)
    x8, g8, _, _ = operands(rng, 2, 300, 256)
    _, u8, _, _ = operands(rng, 1, 300, 256)
    want = layer.fp8_gated(g8, u8, x8)
    ws = layer.Workspace()
    layer.fp8_gated(g8, u8, x8, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.fp8_gated(g8, u8, x8, ws=ws)
    small = ws.buf.numel()
    ws.get(small * 4)
    assert ws.buf.numel() >= small * 4
    others = [torch.full((small,), 77, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.data.view(torch.uint8), want.data.view(torch.uint8)) and torch.equal(out.scales, want.scales)
        assert all(bool((t == 77).all()) for t in others)


def test_offsets_past_32_bits(lib):
    """Activations, codes and outputs of more than 4 GiB: the last rows are
    those of a small call."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(1)
    # (4096 tokens: like the long call, in a tile that does not share k among groups of waves, and not few)
    n, d, m, tail = 1_100_000, 4096, 2048, 4096
    w8 = layer.fp8_weight(torch.randn((m, d), generator=gen, device="cuda").half())
    x = torch.zeros((n, d), dtype=torch.float16, device="cuda")
    x[-tail:] = torch.randn((tail, d), generator=gen, device="cuda").half()
    gain = torch.ones(d, dtype=torch.float16, device="cuda")
    say("past 32 bits: norm and quantizer")
    a, b = layer.fp8_activations(x), layer.fp8_activations(x[-tail:])
    assert a.data.numel() > 2 ** 32
    assert torch.equal(a.data[-tail:].view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales[:, -tail:], b.scales)
    r, total = layer.fp8_rms_norm(x, gain, residual=x, sum_out=None)
    s, part = layer.fp8_rms_norm(x[-tail:], gain, residual=x[-tail:])
    assert torch.equal(total[-tail:], part)
    assert torch.equal(r.data[-tail:].view(torch.uint8), s.data.view(torch.uint8)) and torch.equal(r.scales[:, -tail:], s.scales)
    del r, total, x
    say("past 32 bits: product")
    y, z = layer.fp8_matmul(w8, a), layer.fp8_matmul(w8, b)
    assert y.numel() * 2 > 2 ** 32 and torch.equal(y[-tail:], z) and bool((y[:1000] == 0).all())
    yt = layer.fp8_matmul(w8, a, channel_major=True)
    assert torch.equal(yt[:, -tail:].t(), z)
    del y, yt
    say("past 32 bits: gated")
    g, h = layer.fp8_gated(w8, w8, a), layer.fp8_gated(w8, w8, b)
    assert torch.equal(g.data[-tail:].view(torch.uint8), h.data.view(torch.uint8)) and torch.equal(g.scales[:, -tail:], h.scales)


def test_millions_of_tokens(lib):
    """Sixteen output channels, more tokens than a grid's second dimension
    counts in 32s."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, d, m = 2_200_000, 1920, 16
    say("millions of tokens", n, d, m)
    w8 = layer.fp8_weight(torch.randn((m, d), generator=gen, device="cuda").half())
    x8 = layer.Fp8(torch.randint(0, 120, (n, d), generator=gen, device="cuda", dtype=torch.uint8),
                   torch.rand((d // 128, n), generator=gen, device="cuda") + 0.5, d)
    y = layer.fp8_matmul(w8, x8)
    wv = ref.tiles_values(codes_of(w8), w8.scales.cpu().numpy(), d)
    for at in (0, n // 2, 2 ** 21 - 32, n - 64):
        part = slice(at, at + 64)
        xv = ref.rows_values(x8.data[part].cpu().numpy(), x8.scales[:, part].cpu().numpy(), d)
        want, dy = ref.product(xv, wv, ref.cuts(n, "float16"))
        got = y[part].double().cpu().numpy()
        big = np.abs(want) + dy > 65504.0     # leaves float16: infinite, or the largest value
        most = dy + ref.HALF["float16"] * (np.abs(want) + dy) + ref.TINY["float16"]
        assert np.all((np.abs(got - want) <= most) | big)
        assert np.all(np.abs(got[big]) > 6e4) and big.mean() < 0.9


def test_results_do_not_depend_on_the_batch(lib):
    """The same rows alone and inside a batch of the same variant, and the
    same call twice: the same bits."""
    from post_weight_quantization_04_amd import layer
    torch = _t()
    rng = np.random.default_rng(2)
    x8, w8, _, _ = operands(rng, 300, 300, 640)
    a, b = layer.fp8_matmul(w8, x8), layer.fp8_matmul(w8, x8)
    assert torch.equal(a, b)
    half = layer.Fp8(x8.data[:150], x8.scales[:, :150], 640)
    assert torch.equal(layer.fp8_matmul(w8, half), a[:150])


def test_binding_refusals(lib):
    from post_weight_quantization_04_amd import GptqError, layer
    torch = _t()
    x = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    a, w = layer.fp8_activations(x), layer.fp8_weight(torch.zeros((8, 256), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        layer.fp8_activations(x.double())
    with pytest.raises(ValueError):
        layer.fp8_activations(x.t())                                   # column stride
    with pytest.raises(ValueError):
        layer.fp8_activations(x, out=layer.Fp8(a.data, a.scales, 200))
    with pytest.raises(ValueError):
        layer.fp8_activations(x, out=layer.Fp8(a.data[:, :128], a.scales, 256))
    with pytest.raises(ValueError):
        layer.fp8_matmul(w, a, out=torch.empty((8, 4), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        layer.fp8_matmul(w, a, dtype=torch.float32, out=torch.empty((4, 8), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        layer.fp8_matmul(w, layer.Fp8(a.data, a.scales[:1], 256))
    with pytest.raises(ValueError):
        layer.fp8_rms_norm(x, torch.ones(256, device="cuda"))          # gain's type
    with pytest.raises(GptqError):
        layer.fp8_rms_norm(x, torch.ones(256, dtype=torch.float16, device="cuda"), eps=0.0)
    with pytest.raises(GptqError):
        layer.fp8_rms_norm(x, torch.ones(256, dtype=torch.float16, device="cuda"), sum_out=x)
    with pytest.raises(ValueError):
        layer.fp8_gated(w, layer.fp8_weight(torch.zeros((9, 256), dtype=torch.float16, device="cuda")), a)
