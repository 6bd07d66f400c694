"""Host side of the product with packed weights, the attention and the paged
cache: argument checks of the C ABI (made before any HIP call, so no GPU is
needed), the limits, and the binding's refusals."""
import ctypes
import os

import numpy as np
import pytest

import block_ref as ref

OK, EINVAL, EUNSUPPORTED, EHIP, EWORKSPACE = 0, 1, 2, 3, 4
F16, F32, BF16 = 0, 1, 2
P = ctypes.c_void_p(4096)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4100)


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


def test_the_reference_packs_as_documented():
    rng = np.random.default_rng(0)
    for bits in range(2, 9):
        codes = rng.integers(0, 1 << bits, (3, 37)).astype(np.uint8)
        words = ref.pack(codes, bits).view(np.uint32)
        assert words.shape == (3, (37 * bits + 31) // 32)
        for r in range(3):
            stream = sum(int(w) << (32 * i) for i, w in enumerate(words[r]))
            assert [(stream >> (j * bits)) & ((1 << bits) - 1) for j in range(37)] == codes[r].tolist()


def product(lib, packed=P, bits=4, m=8, k=256, s=P, z=P, g=128, x=P, xt=F16, n=4, ldx=256, b=None, r=None, ldr=0, y=P,
            yt=F16, ldy=8, act=0):
    return lib.gptq_packed_matmul(packed, bits, m, k, s, z, g, x, xt, n, ldx, b, r, ldr, y, yt, ldy, act, None)


def test_product_refusals(clib):
    for bad in (dict(m=-1), dict(k=-1), dict(n=-1), dict(bits=1), dict(bits=9), dict(g=-16), dict(g=96), dict(xt=3), dict(yt=-1),
                dict(act=4), dict(act=-1), dict(ldx=255), dict(ldy=7), dict(r=P, ldr=7), dict(packed=None), dict(s=None),
                dict(z=None), dict(x=None), dict(y=None)):
        assert product(clib, **bad) == EINVAL, bad
    for bad in (dict(xt=F32, yt=F32), dict(yt=BF16), dict(xt=BF16, yt=F16), dict(k=240, ldx=240, g=24), dict(k=(1 << 21) + 16, ldx=1 << 22, g=0),
                dict(ldx=(1 << 21) + 1), dict(m=(1 << 24) + 1, ldy=1 << 25), dict(n=(1 << 24) + 1),
                dict(m=1 << 24, ldy=1 << 24, n=1 << 15)):
        assert product(clib, **bad) == EUNSUPPORTED, bad
    assert product(clib, n=0, y=None, x=None) == OK
    assert product(clib, m=0, y=None) == OK


def attend(lib, q=P, qt=512, qh=64, k=P, kt=128, kh=64, v=P, vt=128, vh=64, o=P, ot=512, oh=64, dt=F16, n=10, h=8, kv=2, d=64,
           starts=P, seqs=2, causal=1, scale=0.125):
    return lib.gptq_attention(q, qt, qh, k, kt, kh, v, vt, vh, o, ot, oh, dt, n, h, kv, d, starts, seqs, causal, scale, None)


def test_attention_refusals(clib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(n=-1), dict(h=-8), dict(kv=-2), dict(kv=3), dict(kv=0), dict(d=-8), dict(seqs=-1), dict(causal=2), dict(dt=5),
                dict(qt=63), dict(qh=63), dict(kt=63), dict(kh=63), dict(vt=63), dict(vh=63), dict(ot=63), dict(oh=63),
                dict(starts=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(scale=1e-60),
                dict(scale=1e60), dict(scale=1e-38), dict(scale=2e38), dict(q=None), dict(k=None), dict(v=None), dict(o=None)):
        assert attend(clib, **bad) == EINVAL, bad
    wide = dict(qt=2048, qh=256, kt=512, kh=256, vt=512, vh=256, ot=2048, oh=256)
    for bad in (dict(dt=F32), dict(d=136, **wide), dict(d=60), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(qt=516),
                dict(qh=68), dict(kt=132), dict(kh=68), dict(vt=132), dict(vh=68), dict(ot=516), dict(oh=68), dict(kt=(1 << 22) + 8),
                dict(qt=1 << 23), dict(vt=1 << 23), dict(ot=1 << 23), dict(n=(1 << 24) + 1), dict(seqs=(1 << 24) + 1), dict(n=1 << 24, h=64),
                dict(h=1 << 17)):
        assert attend(clib, **bad) == EUNSUPPORTED, bad
    assert attend(clib, n=0, q=None, k=None, v=None, o=None) == OK
    assert attend(clib, h=0, kv=0) == OK
    assert attend(clib, seqs=0) == OK
    assert attend(clib, starts=None, seqs=1, n=0) == OK


def store(lib, k=P, kt=128, kh=64, v=P, vt=128, vh=64, dt=F16, n=10, kv=2, d=64, slots=P, ck=P, c0=2048, c1=1024, c2=64, cv=P,
          w0=2048, w1=1024, w2=64, pages=5, page=16):
    return lib.gptq_cache_store(k, kt, kh, v, vt, vh, dt, n, kv, d, slots, ck, c0, c1, c2, cv, w0, w1, w2, pages, page, None)


def test_store_refusals(clib):
    for bad in (dict(n=-1), dict(kv=-1), dict(d=-1), dict(pages=-1), dict(page=0), dict(dt=4), dict(kt=63), dict(kh=63), dict(vt=63),
                dict(vh=63), dict(c0=63), dict(c1=63), dict(c2=63), dict(w0=63), dict(w1=63), dict(w2=63), dict(k=None),
                dict(v=None), dict(slots=None), dict(ck=None), dict(cv=None)):
        assert store(clib, **bad) == EINVAL, bad
    for bad in (dict(dt=F32), dict(d=60), dict(k=ODD), dict(v=ODD), dict(ck=ODD), dict(cv=ODD), dict(kt=132), dict(kh=68), dict(vt=132),
                dict(vh=68), dict(c0=2052), dict(c1=1028), dict(c2=68), dict(w0=2052), dict(w1=1028), dict(w2=68),
                dict(c2=1 << 23), dict(c0=1 << 31), dict(w0=1 << 31), dict(pages=1 << 27), dict(pages=1 << 40), dict(page=1 << 40), dict(n=1 << 27), dict(n=1 << 40),
                dict(d=136, kt=272, kh=136, vt=272, vh=136, c2=136, w2=136)):
        assert store(clib, **bad) == EUNSUPPORTED, bad
    assert store(clib, n=0, k=None, v=None, slots=None) == OK
    assert store(clib, pages=0, ck=None, cv=None) == OK


def cached(lib, q=P, qs=512, qh=64, ck=P, c0=2048, c1=1024, c2=64, cv=P, w0=2048, w1=1024, w2=64, pages=5, page=16, table=P,
           ldt=4, most=4, lengths=P, n=3, h=8, kv=2, d=64, o=P, os_=512, oh=64, dt=F16, scale=0.125, ws=P, room=1 << 40):
    return lib.gptq_cached_attention(q, qs, qh, ck, c0, c1, c2, cv, w0, w1, w2, pages, page, table, ldt, most, lengths, n, h, kv, d,
                                     o, os_, oh, dt, scale, ws, room, None)


def test_cached_refusals(clib):
    nan = float("nan")
    for bad in (dict(n=-1), dict(h=-1), dict(kv=-1), dict(kv=3), dict(d=-1), dict(pages=-1), dict(page=0), dict(most=-1), dict(most=5),
                dict(dt=9), dict(scale=0.0), dict(scale=nan), dict(scale=1e-38), dict(scale=2e38), dict(qs=63), dict(qh=63), dict(os_=63), dict(oh=63), dict(c0=63),
                dict(c1=63), dict(c2=63), dict(w0=63), dict(w1=63), dict(w2=63), dict(q=None), dict(o=None), dict(lengths=None),
                dict(table=None), dict(ck=None), dict(cv=None)):
        assert cached(clib, **bad) == EINVAL, bad
    for bad in (dict(dt=F32), dict(d=60), dict(q=ODD), dict(o=ODD), dict(ck=ODD), dict(cv=ODD), dict(qs=516), dict(qh=68), dict(c0=2052),
                dict(c1=1028), dict(c2=68), dict(w2=68), dict(os_=516), dict(oh=68), dict(n=(1 << 20) + 1), dict(pages=1 << 27),
                dict(ldt=1 << 40, most=1 << 40), dict(ldt=1 << 28, most=1 << 28), dict(c2=1 << 23), dict(w2=1 << 23), dict(n=1 << 20, h=16)):
        assert cached(clib, **bad) == EUNSUPPORTED, bad
    assert cached(clib, n=0, q=None, o=None) == OK
    assert cached(clib, h=0, kv=0) == OK
    need = clib.gptq_cached_attention_workspace(3, 8, 2, 64, 400, 16)
    for bad in (dict(ws=None), dict(ws=ODD), dict(room=need - 1)):
        assert need > 0 and cached(clib, ldt=400, most=400, **bad) == EWORKSPACE, bad
    for none in ((0, 8, 2, 64, 400, 16), (3, 8, 3, 64, 400, 16), (3, 8, 0, 64, 400, 16), (3, 8, 2, 60, 400, 16), (3, 8, 2, 64, -1, 16),
                 (3, 8, 2, 64, 400, 0)):
        assert clib.gptq_cached_attention_workspace(*none) == 0, none


def test_binding_refusals(clib):
    """Tensors that are on no device, or whose shapes do not fit."""
    import torch
    from post_weight_quantization_04_amd import layer
    h = torch.zeros(4, 8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        layer.attention(h, h, h)
    w = layer.Packed(torch.zeros(8, 8, dtype=torch.int32), torch.ones(8, 1), torch.zeros(8, 1, dtype=torch.int32), 4, 64, 0)
    with pytest.raises(ValueError):
        layer.packed_matmul(w, torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        layer.packed_matmul(w, torch.zeros(2, 64, dtype=torch.float16), activation="tanh")
    cache = layer.kv_cache(3, 8, 16, 64, device="cpu")
    one = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        layer.cache_store(cache, h, h, one)
    with pytest.raises(ValueError):
        layer.cached_attention(h, cache, one[:, None], one)


def test_product_kernels_by_name(clib):
    import torch
    from post_weight_quantization_04_amd import _lib
    for name, n, m, k, group in ref.PACKED_KERNELS:
        assert _lib.packed_matmul_kernel(n, m, k, group, True, 256) == name, (n, m, k, group)
    assert {c[0] for c in ref.PACKED_KERNELS} == set(_PACKED_GROUPS)
    # tiles of 128 x 384 take whole groups of aligned rows
    assert _lib.packed_matmul_kernel(2700, 2801, 384, 128, False, 256) == "64 x 128"
    for bad in ((0, 256, 0, 4), (8, -1, 0, 4), (8, 256, 0, 0), (8, 256, -16, 4), (8, 256, 24, 4), (8, 256, 96, 4), (8, (1 << 21) + 16, 0, 4),
                ((1 << 24) + 1, 256, 0, 4), (8, 256, 0, (1 << 24) + 1), (1 << 24, 256, 0, (1 << 12) + 1)):
        assert clib.gptq_packed_matmul_kernel(*bad, 1, 256) is None, bad
    assert clib.gptq_packed_matmul_kernel(1 << 24, 256, 0, 1 << 12, 1, 256) is not None
    if torch.cuda.device_count() == 0:
        assert clib.gptq_packed_matmul_kernel(8, 256, 0, 4, 1, 0) is None


_PACKED_GROUPS = {"few tokens": None, "32 x 64": (32, 64, 1024), "64 x 128": (64, 128, 256), "128 x 384": (128, 384, 512)}


def test_product_grids(clib):
    """Over sizes up to the limits: fewer than 2^32 threads in one dimension of
    the grid, fewer than 2^16 in the other."""
    sizes = sorted({min(1 << 24, max(1, (1 << e) + off)) for e in range(0, 25) for off in (-1, 0, 1)})
    seen = set()
    for m in sizes:
        for n in sizes:
            if -(-m // 256) * -(-n // 256) > 1 << 20:
                continue
            for d in (0, 16, 1024, 9000, 1 << 21):
                for cus in (32, 256):
                    for aligned in (0, 1):
                        name = clib.gptq_packed_matmul_kernel(m, d, 0, n, aligned, cus).decode()
                        seen.add(name)
                        if name == "few tokens":
                            assert -(-m // 16) * 512 < 1 << 32 and -(-n // (4 if n <= 4 else 16 if n <= 16 else 32)) < 1 << 16
                        else:
                            a, b, threads = _PACKED_GROUPS[name]
                            assert -(-n // a) * -(-m // b) * threads < 1 << 32
    assert seen == set(_PACKED_GROUPS)


def test_attention_of_no_channels(clib):
    """The default scale of rows without channels (they are refused, or empty, like others)."""
    import torch
    from post_weight_quantization_04_amd import layer
    h = torch.zeros(4, 8, 0, dtype=torch.float16)
    with pytest.raises(ValueError):
        layer.attention(h, h, h)
    cache = layer.kv_cache(3, 8, 16, 0, device="cpu")
    one = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        layer.cached_attention(h, cache, one[:, None], one)
