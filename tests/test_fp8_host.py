"""Host side of the 8-bit operators: the reference's own format against
torch's e4m3, argument checks of the C ABI (made before any HIP call, so no
GPU is needed), and the binding's refusals."""
import ctypes
import os

import numpy as np
import pytest

import fp8_ref as ref

OK, EINVAL, EUNSUPPORTED, EHIP, EWORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def clib():
    from post_weight_quantization_04_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


P = ctypes.c_void_p(4096)   # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4100)


def test_reference_codes_are_torchs_e4m3():
    import torch
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.randn(20000), torch.randn(20000) * 2.0 ** -8,
                   torch.from_numpy((ref.TABLE[:126] + ref.TABLE[1:127]).astype(np.float32) / 2)])
    got = ref.encode(v.numpy())
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, want)
    codes = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(ref.decode(codes), torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())


def weight(lib, W=P, dt=0, m=8, k=200, ldw=200, q=P, ldq=256, s=P, lds=2):
    return lib.gptq_fp8_weight(W, dt, m, k, ldw, q, ldq, s, lds, None)


def test_weight_refusals(clib):
    for bad in (dict(m=-1), dict(k=-1), dict(ldw=199), dict(ldq=255), dict(ldq=200), dict(lds=1), dict(dt=3), dict(dt=-1),
                dict(W=None), dict(q=None), dict(s=None)):
        assert weight(clib, **bad) == EINVAL, bad
    for bad in (dict(q=ODD), dict(ldq=264), dict(m=(1 << 24) + 1), dict(k=(1 << 24) + 1, ldw=1 << 25, ldq=1 << 25, lds=1 << 20),
                dict(m=1 << 19, k=1 << 19, ldw=1 << 19, ldq=1 << 19, lds=1 << 12)):
        assert weight(clib, **bad) == EUNSUPPORTED, bad
    assert weight(clib, m=0, W=None, q=None, s=None) == OK
    assert weight(clib, k=0, W=None, q=None, s=None, ldw=0, ldq=0, lds=0) == OK


def acts(lib, X=P, dt=0, n=8, d=200, ldx=200, cm=0, q=P, ldq=256, s=P, lds=8):
    return lib.gptq_fp8_activations(X, dt, n, d, ldx, cm, q, ldq, s, lds, None)


def test_activations_refusals(clib):
    for bad in (dict(n=-1), dict(d=-1), dict(ldx=199), dict(cm=1, ldx=7), dict(cm=2), dict(ldq=255), dict(lds=7), dict(dt=3),
                dict(X=None), dict(q=None), dict(s=None)):
        assert acts(clib, **bad) == EINVAL, bad
    for bad in (dict(q=ODD), dict(ldq=264), dict(n=1 << 31, lds=1 << 31), dict(n=1 << 27, lds=1 << 27),
                dict(n=1 << 29, lds=1 << 29, ldx=1 << 29, cm=1)):
        assert acts(clib, **bad) == EUNSUPPORTED, bad
    assert acts(clib, n=0, X=None, q=None, s=None) == OK


def norm(lib, x=P, ldx=200, r=P, ldr=200, o=P, ldo=200, g=P, dt=0, n=8, d=200, eps=1e-6, q=P, ldq=256, s=P, lds=8):
    return lib.gptq_fp8_rms_norm(x, ldx, r, ldr, o, ldo, g, dt, n, d, eps, q, ldq, s, lds, None)


def test_rms_norm_refusals(clib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(n=-1), dict(d=-1), dict(ldx=199), dict(ldr=199), dict(ldo=199), dict(r=None), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=1e-21), dict(eps=nan), dict(eps=inf), dict(ldq=255), dict(lds=7), dict(dt=3), dict(x=None),
                dict(g=None), dict(q=None), dict(s=None)):
        assert norm(clib, **bad) == EINVAL, bad
    for bad in (dict(q=ODD), dict(ldq=264), dict(n=1 << 23, lds=1 << 23)):
        assert norm(clib, **bad) == EUNSUPPORTED, bad
    assert norm(clib, n=0, x=None, g=None, q=None, s=None) == OK


def mm(lib, wq=P, ldw=256, ws=P, ldws=2, m=8, k=200, xq=P, ldx=256, xs=P, ldxs=5, n=5, Y=P, dt=0, ldy=8, cm=0, act=0):
    return lib.gptq_fp8_matmul(wq, ldw, ws, ldws, m, k, xq, ldx, xs, ldxs, n, Y, dt, ldy, cm, act, None)


def test_matmul_refusals(clib):
    for bad in (dict(m=-1), dict(k=-1), dict(n=-1), dict(ldw=255), dict(ldws=1), dict(ldx=255), dict(ldxs=4), dict(ldy=7),
                dict(cm=1, ldy=4), dict(cm=2), dict(act=2), dict(dt=3), dict(Y=None), dict(wq=None), dict(ws=None),
                dict(xq=None), dict(xs=None)):
        assert mm(clib, **bad) == EINVAL, bad
    big = (1 << 22) + 16
    for bad in (dict(wq=ODD), dict(xq=ODD), dict(ldw=264), dict(ldx=264), dict(ldw=big), dict(ldx=big),
                dict(m=(1 << 24) + 1, ldy=1 << 25), dict(n=(1 << 24) + 1, ldxs=1 << 25)):
        assert mm(clib, **bad) == EUNSUPPORTED, bad
    assert mm(clib, m=1 << 24, n=1 << 24, ldy=1 << 24, ldxs=1 << 24) == EUNSUPPORTED
    assert mm(clib, n=0, wq=None, ws=None, xq=None, xs=None, Y=None) == OK
    assert mm(clib, m=0, wq=None, ws=None, xq=None, xs=None, Y=None) == OK


def gated(lib, gq=P, gs=P, uq=P, us=P, ldw=256, ldws=2, m=130, k=200, xq=P, ldx=256, xs=P, ldxs=5, n=5, q=P, ldq=256, s=P,
          lds=5, ws=P, size=1 << 30):
    return lib.gptq_fp8_gated(gq, gs, uq, us, ldw, ldws, m, k, xq, ldx, xs, ldxs, n, q, ldq, s, lds, ws, size, None)


def test_gated_refusals(clib):
    for bad in (dict(m=-1), dict(k=-1), dict(n=-1), dict(ldw=255), dict(ldws=1), dict(ldx=255), dict(ldxs=4), dict(ldq=255),
                dict(ldq=130), dict(lds=4), dict(q=None), dict(s=None), dict(gq=None), dict(gs=None), dict(uq=None),
                dict(us=None), dict(xq=None), dict(xs=None)):
        assert gated(clib, **bad) == EINVAL, bad
    for bad in (dict(gq=ODD), dict(uq=ODD), dict(xq=ODD), dict(q=ODD), dict(ldw=264), dict(ldx=264), dict(ldq=264),
                dict(m=1 << 24, n=1 << 24, ldq=1 << 24, ldxs=1 << 24, lds=1 << 24)):
        assert gated(clib, **bad) == EUNSUPPORTED, bad
    need = clib.gptq_fp8_gated_workspace(5, 130)
    assert need > 0
    for bad in (dict(ws=None), dict(size=need - 1), dict(ws=ODD)):
        assert gated(clib, **bad) == EWORKSPACE, bad
    assert clib.gptq_fp8_gated_workspace(0, 130) == 0 and clib.gptq_fp8_gated_workspace(-1, 130) == 0
    assert gated(clib, n=0, gq=None, uq=None, xq=None, q=None, ws=None, size=0) == OK


@pytest.mark.parametrize("n", [5, 64, 1000])
def test_calls_without_a_device_return_an_error(clib, n):
    """Every variant of the products asks for the device's size or launches:
    without a device both come back as a status."""
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a device is there: the pointers of this test are not")
    for dt in (0, 1, 2):
        assert mm(clib, n=n, ldxs=n, dt=dt) == EHIP
    assert gated(clib, n=n, ldxs=n, lds=n) == EHIP
    assert gated(clib, n=n, ldxs=n, lds=n, m=20000, ldq=20096) == EHIP
    assert weight(clib) == EHIP and acts(clib, n=n, lds=n) == EHIP and norm(clib, n=n, lds=n) == EHIP


def test_binding_refuses_host_tensors():
    import torch
    from post_weight_quantization_04_amd import layer
    x = torch.zeros(4, 128)
    for call in (lambda: layer.fp8_weight(x), lambda: layer.fp8_activations(x),
                 lambda: layer.fp8_rms_norm(x, torch.ones(128))):
        with pytest.raises(ValueError):
            call()
    a = layer.Fp8(torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(1, 4), 128)
    with pytest.raises(ValueError):
        layer.fp8_matmul(a, a)
    with pytest.raises(ValueError):
        layer.fp8_gated(a, a, a)
    with pytest.raises(ValueError):
        layer.fp8_matmul(a, layer.Fp8(a.data, a.scales, 100))


def test_propagate_fp8_gives_a_type_that_hessian_takes(monkeypatch):
    """The chain's next call accepts what comes back, for every type of X."""
    import torch
    from post_weight_quantization_04_amd import _lib, layer
    monkeypatch.setattr(layer, "fp8_activations", lambda X, **_: X)
    monkeypatch.setattr(layer, "fp8_matmul", lambda w, x, dtype=None, out=None, **_: torch.empty(1, dtype=dtype) if out is None else out)
    for given, back in ((torch.float16, torch.float16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)):
        X = torch.zeros(4, 4, dtype=given)
        Y = layer.propagate_fp8(None, X)
        assert Y.dtype == back
        _lib._dtype_code(Y)
        out = torch.empty(4, 4, dtype=torch.bfloat16)
        assert layer.propagate_fp8(None, X, out=out) is out


def test_a_workspace_asks_only_whether_its_stream_is_captured(monkeypatch):
    """Every call of the framework takes its scratch memory here: a host
    buffer asks nothing, a device buffer the one question."""
    import torch
    from post_weight_quantization_04_amd import layer
    asked = []
    monkeypatch.setattr(torch.cuda, "is_available", lambda: asked.append("available"))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: asked.append("capturing") or True)
    ws = layer.Workspace("cpu")
    assert ws.get(1000).numel() == 1000 and ws.get(10) is ws.buf and asked == []

    class Device:
        is_cuda = True

        def numel(self):
            return 5000

    ws.buf = held = Device()
    assert ws.get(5000) is held and asked == ["capturing"]
    ws.get(6000)                   # handed out during a capture: kept for its graph
    assert ws.buf is not held and ws._kept == [held]
