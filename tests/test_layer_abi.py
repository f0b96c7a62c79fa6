"""Refusals of the operators around the core (CPU only): every call here fails
validation, or is a no-op, before any launch; the buffers are host canaries
that stay untouched."""
import ctypes

import pytest
import torch

from tests.test_abi import Canary, kda, make_cfg  # noqa: F401  (fixture)

NAN = float("nan")


@pytest.fixture
def buf():
    c = Canary(1 << 12)
    yield c
    assert c.untouched()


def at(c, off=0):
    base = c.a.ctypes.data
    return ctypes.c_void_p(base + (-base) % 256 + off)


def test_add_rmsnorm(kda, buf):
    lib, p = kda.library(), at(buf)
    cfg, _ = make_cfg(kda)
    plain = lambda c=cfg, n=4, hid=64, x=p, r=p, w=p, eps=1e-6, h=p, y=p: lib.kda_add_rmsnorm(
        None if c is None else ctypes.byref(c), n, hid, x, r, w, eps, h, y, None)
    fp8 = lambda c=cfg, n=4, hid=64, x=p, r=p, w=p, eps=1e-6, h=p, y=p, s=p: lib.kda_add_rmsnorm_fp8(
        None if c is None else ctypes.byref(c), n, hid, x, r, w, eps, h, y, s, None)
    for f in (plain, fp8):
        for bad in (dict(c=None), dict(n=-1), dict(hid=0), dict(hid=-8), dict(eps=NAN), dict(eps=-1e-3), dict(x=None),
                    dict(w=None), dict(y=None), dict(x=at(buf, 2)), dict(r=at(buf, 8)), dict(w=at(buf, 4)),
                    dict(h=at(buf, 2)), dict(y=at(buf, 4))):
            assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(hid=20), dict(hid=32776), dict(c=make_cfg(kda, io_dtype=2)[0]),
                    dict(c=make_cfg(kda, out_dtype=5)[0]), dict(n=1 << 60)):
            assert f(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
        assert f(n=0, x=None, w=None, y=None) == kda.KDA_OK
    assert fp8(s=None) == kda.KDA_ERR_INVALID_ARGUMENT
    assert fp8(s=at(buf, 2)) == kda.KDA_ERR_INVALID_ARGUMENT
    assert plain(y=at(buf, 8)) == kda.KDA_ERR_INVALID_ARGUMENT


def test_add_rmsnorm_backward(kda, buf):
    lib, p = kda.library(), at(buf)
    cfg, _ = make_cfg(kda)
    q = lambda c, n, hid: lib.kda_add_rmsnorm_backward_workspace_bytes(ctypes.byref(c), n, hid)
    f = lambda c=cfg, n=4, hid=64, h=p, w=p, eps=1e-6, dy=p, dh=p, dx=p, dw=p, ws=p, size=1 << 30: \
        lib.kda_add_rmsnorm_backward(None if c is None else ctypes.byref(c), n, hid, h, w, eps, dy, dh, dx, dw, ws,
                                     size, None)
    for bad in (dict(c=None), dict(n=-1), dict(hid=0), dict(eps=NAN), dict(eps=-1.0), dict(h=None), dict(w=None),
                dict(dy=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(dx=at(buf, 4)), dict(ws=at(buf, 8))):
        assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(hid=12), dict(hid=1 << 20), dict(c=make_cfg(kda, io_dtype=9)[0])):
        assert f(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    need = q(cfg, 4, 64)
    assert need >= 4 * 64 * 4 and need % 256 == 0 and q(cfg, 1 << 30, 64) < 1 << 20
    assert f(size=need - 1) == kda.KDA_ERR_WORKSPACE_TOO_SMALL
    assert q(cfg, 0, 64) > 0 and q(cfg, -1, 64) == 0 and q(cfg, 4, 12) == 0


def test_output_gate_fp8_and_backward(kda, buf):
    lib, p = kda.library(), at(buf)
    cfg, _ = make_cfg(kda)
    f = lambda c=cfg, n=4, o=p, g=p, w=p, eps=1e-6, y=p, s=p: lib.kda_output_gate_fp8(
        None if c is None else ctypes.byref(c), n, o, g, w, eps, y, s, None)
    b = lambda c=cfg, n=4, o=p, g=p, w=p, eps=1e-6, dy=p, do=p, dg=p, dw=p, ws=p, size=1 << 30: \
        lib.kda_output_gate_backward(None if c is None else ctypes.byref(c), n, o, g, w, eps, dy, do, dg, dw, ws, size,
                                     None)
    for call in (f, b):
        for bad in (dict(c=None), dict(n=-1), dict(eps=NAN), dict(eps=-1.0), dict(o=None), dict(g=None), dict(w=None),
                    dict(o=at(buf, 8)), dict(g=at(buf, 2)), dict(w=at(buf, 4)), dict(c=make_cfg(kda, H=0)[0])):
            assert call(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(c=make_cfg(kda, dk=48, dv=48)[0]), dict(c=make_cfg(kda, H=70000)[0]),
                    dict(c=make_cfg(kda, out_dtype=4)[0]), dict(n=1 << 61)):
            assert call(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    for bad in (dict(y=None), dict(s=None), dict(y=at(buf, 4)), dict(s=at(buf, 2))):
        assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(dy=None), dict(do=None), dict(dg=None), dict(dw=None), dict(ws=None), dict(dg=at(buf, 8))):
        assert b(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    assert f(n=0, o=None, g=None, w=None, y=None, s=None) == kda.KDA_OK
    need = lib.kda_output_gate_backward_workspace_bytes(ctypes.byref(cfg), 4)
    assert need > 0 and need % 256 == 0 and b(size=need - 1) == kda.KDA_ERR_WORKSPACE_TOO_SMALL
    assert lib.kda_output_gate_backward_workspace_bytes(ctypes.byref(make_cfg(kda, dk=48, dv=48)[0]), 4) == 0


def test_fp8_matmul(kda, buf):
    lib, p = kda.library(), at(buf)
    cfg, _ = make_cfg(kda)
    f = lambda c=cfg, M=4, N=8, K=32, a=p, sa=p, w=p, sw=p, y=p: lib.kda_fp8_matmul(
        None if c is None else ctypes.byref(c), M, N, K, a, sa, w, sw, y, None)
    for bad in (dict(c=None), dict(M=-1), dict(N=0), dict(K=0), dict(K=-16), dict(a=None), dict(sa=None), dict(w=None),
                dict(sw=None), dict(y=None), dict(a=at(buf, 8)), dict(w=at(buf, 4)), dict(y=at(buf, 8)),
                dict(sa=at(buf, 2)), dict(sw=at(buf, 1))):
        assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(K=24), dict(K=1 << 21), dict(N=1 << 21), dict(M=1 << 31), dict(c=make_cfg(kda, out_dtype=2)[0])):
        assert f(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    assert f(M=0, a=None, sa=None, w=None, sw=None, y=None) == kda.KDA_OK


def test_binding_refuses_before_the_library(kda):
    """Shapes, types and devices are checked in the binding: host tensors never reach a kernel."""
    cfg = kda.Config(None, None, None, None, None, num_heads=2, head_k_dim=64, head_v_dim=64)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm(cfg, bf(4, 64), bf(4, 64), torch.ones(64))               # not on the GPU
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm(cfg, torch.zeros(4, 64), None, torch.ones(64))           # not the io dtype
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm_fp8(cfg, bf(4, 64), bf(5, 64), torch.ones(64))           # residual of another shape
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm_backward(cfg, bf(4, 64), torch.ones(32), bf(4, 64))      # weight of another length
    with pytest.raises(ValueError):
        kda.kda_output_gate_fp8(cfg, bf(4, 3, 64), bf(4, 3, 64), torch.ones(64))     # not num_heads
    with pytest.raises(ValueError):
        kda.kda_output_gate_backward(cfg, bf(4, 2, 64), bf(4, 2, 64), torch.ones(64), torch.zeros(4, 2, 64))
    with pytest.raises(ValueError):
        kda.kda_fp8_matmul(cfg, f8(4, 256), torch.ones(4, 1), f8(8, 256), torch.ones(1, 2))   # scales do not fit K
    with pytest.raises(ValueError):
        kda.kda_fp8_matmul(cfg, bf(4, 256), torch.ones(4, 2), f8(8, 256), torch.ones(1, 2))   # a in bf16
