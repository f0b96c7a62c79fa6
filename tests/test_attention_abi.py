"""Refusals of the full-attention layers' operators (CPU only): every call here fails validation, or is a no-op, before
any launch; the buffers are host canaries that stay untouched."""
import ctypes

import pytest
import torch

from tests.test_abi import kda, make_cfg  # noqa: F401  (fixture)
from tests.test_layer_abi import at, buf  # noqa: F401  (fixture)

NAN, INF = float("nan"), float("inf")


def ref(c):
    return None if c is None else ctypes.byref(c)


def cfg_of(kda, **kw):  # noqa: F811
    a = dict(H=4, dk=64, dv=64)
    a.update(kw)
    return make_cfg(kda, **a)[0]


def rope_of(kda, p, **kw):  # noqa: F811
    c = kda.KdaRopeC(32, 0, 1, p, None)
    for name, val in kw.items():
        setattr(c, name, val)
    return c


def cache_of(kda, p, **kw):  # noqa: F811
    c = kda.KdaKvCacheC(p, p, p, p, 4, 64, 2, 2, p, p, p)
    for name, val in kw.items():
        setattr(c, name, val)
    return c


def test_structs_match_the_header(kda):  # noqa: F811
    assert ctypes.sizeof(kda.KdaRopeC) == 32 and kda.KdaRopeC.inv_freq.offset == 16
    assert ctypes.sizeof(kda.KdaKvCacheC) == 4 * 8 + 4 * 4 + 3 * 8 and kda.KdaKvCacheC.page_table.offset == 48
    assert kda.NUM_STAGES == 12


def test_qk_norm_rope(kda, buf):  # noqa: F811
    lib, p = kda.library(), at(buf)
    f = lambda c=cfg_of(kda), r=rope_of(kda, p), n=4, kv=2, q=p, qs=256, k=p, ks=128, wq=p, wk=p, eps=1e-6, pos=p, qo=p, ko=p: \
        lib.kda_qk_norm_rope(ref(c), ref(r), n, kv, q, qs, k, ks, wq, wk, eps, pos, qo, ko, None)
    b = lambda c=cfg_of(kda), r=rope_of(kda, p), n=4, kv=2, q=p, qs=256, k=p, ks=128, wq=p, wk=p, eps=1e-6, pos=p, gq=p, gk=p, \
        dq=p, dk=p, dw=p, ws=p, size=1 << 30: \
        lib.kda_qk_norm_rope_backward(ref(c), ref(r), n, kv, q, qs, k, ks, wq, wk, eps, pos, gq, gk, dq, dk, dw, ws, size, None)
    for call in (f, b):
        for bad in (dict(c=None), dict(n=-1), dict(kv=-1), dict(eps=NAN), dict(eps=-1.0), dict(q=None), dict(k=None),
                    dict(pos=None), dict(qs=255), dict(qs=248), dict(qs=-256), dict(ks=120), dict(ks=0), dict(q=at(buf, 8)), dict(k=at(buf, 2)),
                    dict(wq=at(buf, 4)), dict(wk=at(buf, 8)), dict(pos=at(buf, 2)), dict(r=rope_of(kda, p, rotary_dim=-16)),
                    dict(r=rope_of(kda, p, num_axes=0)), dict(r=rope_of(kda, p, interleaved=2)),
                    dict(r=rope_of(kda, None)), dict(c=cfg_of(kda, H=0))):
            assert call(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(c=cfg_of(kda, dk=32, dv=32)), dict(c=cfg_of(kda, dk=64, dv=128)), dict(c=cfg_of(kda, dk=96, dv=96)),
                    dict(c=cfg_of(kda, H=70000)), dict(kv=70000, ks=1 << 40), dict(c=cfg_of(kda, io_dtype=2)), dict(c=cfg_of(kda, out_dtype=4)),
                    dict(n=1 << 60), dict(n=1 << 40, qs=1 << 40), dict(r=rope_of(kda, p, rotary_dim=24)),
                    dict(r=rope_of(kda, p, rotary_dim=80)), dict(r=rope_of(kda, p, num_axes=5))):
            assert call(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    for bad in (dict(qo=None), dict(ko=None), dict(qo=at(buf, 8))):
        assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(gq=None), dict(gk=None), dict(dq=None), dict(dk=None), dict(dw=None), dict(ws=None), dict(dw=at(buf, 4)),
                dict(gk=at(buf, 8)), dict(ws=at(buf, 8))):
        assert b(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    assert f(n=0, q=None, k=None, qo=None, ko=None, pos=None) == kda.KDA_OK
    w = lambda c, n, kv: lib.kda_qk_norm_rope_backward_workspace_bytes(ref(c), n, kv)
    need = w(cfg_of(kda), 4, 2)
    assert need > 0 and need % 256 == 0 and b(size=need - 1) == kda.KDA_ERR_WORKSPACE_TOO_SMALL
    assert w(cfg_of(kda), 0, 0) > 0 and w(cfg_of(kda), 1 << 40, 2) < 1 << 21
    assert w(cfg_of(kda), -1, 2) == 0 and w(cfg_of(kda), 4, -1) == 0 and w(cfg_of(kda, dk=32, dv=32), 4, 2) == 0


CACHE_BAD = [dict(k=None), dict(k_scale=None), dict(v=None), dict(v_scale=None), dict(lengths=None), dict(page_table=None),
             dict(num_pages=-1), dict(max_pages=-1), dict(page_size=0), dict(num_kv_heads=0)]


def test_append_and_read(kda, buf):  # noqa: F811
    lib, p = kda.library(), at(buf)
    a = lambda c=cfg_of(kda), r=rope_of(kda, p), m=cache_of(kda, p), N=2, n=4, k=p, ks=128, v=p, vs=128, w=p, eps=1e-6, pos=p: \
        lib.kda_append_kv(ref(c), ref(r), ref(m), N, n, k, ks, v, vs, w, eps, pos, None)
    g = lambda c=cfg_of(kda), m=cache_of(kda, p), N=2, n=4, k=p, v=p: lib.kda_read_kv(ref(c), ref(m), N, n, k, v, None)
    for call in (a, g):
        for bad in (dict(c=None), dict(m=None), dict(N=-1), dict(n=-1), dict(k=at(buf, 8)), dict(v=at(buf, 2)),
                    *[dict(m=cache_of(kda, p, **x)) for x in CACHE_BAD], dict(m=cache_of(kda, p, k=at(buf, 8).value)),
                    dict(m=cache_of(kda, p, v_scale=at(buf, 4).value)), dict(m=cache_of(kda, p, lengths=at(buf, 2).value)),
                    dict(m=cache_of(kda, p, cu_seqlens=at(buf, 1).value))):
            assert call(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(m=cache_of(kda, p, page_size=16)), dict(m=cache_of(kda, p, page_size=96)), dict(N=(1 << 24) + 1),
                    dict(m=cache_of(kda, p, num_kv_heads=70000)), dict(c=cfg_of(kda, dk=32, dv=32)), dict(n=1 << 60)):
            if call is a and "m" in bad and bad["m"].num_kv_heads == 70000:
                bad.update(ks=1 << 30, vs=1 << 30)
            assert call(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
        assert call(N=0) == kda.KDA_OK and call(n=0) == kda.KDA_OK
    for bad in (dict(k=None), dict(v=None), dict(ks=120), dict(vs=132), dict(eps=NAN), dict(eps=-1.0), dict(w=at(buf, 4)),
                dict(pos=at(buf, 2)), dict(r=rope_of(kda, None))):
        assert a(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    assert a(r=rope_of(kda, p, rotary_dim=128)) == kda.KDA_ERR_UNSUPPORTED
    assert g(k=None, v=None) == kda.KDA_OK


def test_paged_attention(kda, buf):  # noqa: F811
    lib, p = kda.library(), at(buf)
    f = lambda c=cfg_of(kda), m=cache_of(kda, p), N=2, n=4, mq=2, q=p, s=0.125, o=p, lse=p, ws=p, size=1 << 30: \
        lib.kda_paged_attention(ref(c), ref(m), N, n, mq, q, s, o, lse, ws, size, None)
    for bad in (dict(c=None), dict(m=None), dict(N=-1), dict(n=-1), dict(mq=-1), dict(q=None), dict(o=None), dict(ws=None), dict(s=NAN),
                dict(s=INF), dict(q=at(buf, 8)), dict(o=at(buf, 8)), dict(lse=at(buf, 2)), dict(ws=at(buf, 8)),
                dict(m=cache_of(kda, p, num_kv_heads=3)), *[dict(m=cache_of(kda, p, **x)) for x in CACHE_BAD]):
        assert f(**bad) == kda.KDA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(N=4097), dict(n=(1 << 28) + 1), dict(m=cache_of(kda, p, page_size=48)), dict(c=cfg_of(kda, dk=16, dv=16)),
                dict(c=cfg_of(kda, io_dtype=2))):
        assert f(**bad) == kda.KDA_ERR_UNSUPPORTED, bad
    assert f(N=0) == kda.KDA_OK and f(n=0) == kda.KDA_OK
    w = lambda c=cfg_of(kda), kv=2, N=2, n=4, mq=2: lib.kda_paged_attention_workspace_bytes(ref(c), kv, N, n, mq)
    need = w()
    assert need > 0 and need % 256 == 0 and f(size=need - 1) == kda.KDA_ERR_WORKSPACE_TOO_SMALL
    assert w(kv=3) == 0 and w(kv=0) == 0 and w(N=4097) == 0 and w(n=-1) == 0 and w(mq=-1) == 0
    assert kda.kda_paged_attention_workspace_bytes(kda.Config(None, None, None, None, None, 4, 64, 64), 2, 2**40, 4) == 0


def test_binding_refuses_before_the_library(kda):  # noqa: F811
    """Shapes, types and devices are checked in the binding: host tensors never reach a kernel."""
    cfg = kda.Config(None, None, None, None, None, num_heads=4, head_k_dim=64, head_v_dim=64)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = kda.KvCache.empty(3, 2, 64, 32, device="cpu")
    with pytest.raises(ValueError):
        kda.KvCache(cache.k, cache.k_scale, cache.v, cache.v_scale[:, :1])
    with pytest.raises(ValueError):
        kda.KvCache(cache.k.float(), cache.k_scale, cache.v, cache.v_scale)
    with pytest.raises(ValueError):
        kda.Rope(z(16, t=torch.float64))
    with pytest.raises(ValueError):
        kda.Rope(z(16, t=torch.float32), axis=i(15))
    with pytest.raises(ValueError):
        kda.Rope.build(64, sections=(8, 8, 8), device="cpu")
    rope = kda.Rope.build(32, 1e6, sections=(4, 8, 4), device="cpu")
    assert rope.axis.tolist() == [0] * 4 + [1] * 8 + [2] * 4 and rope.num_axes == 3
    assert abs(rope.inv_freq[8].item() - 1e-3) < 1e-9
    for call in (lambda: kda.kda_qk_norm_rope(cfg, rope, z(2, 4, 64), None, None, None, i(3, 2)),            # not on the GPU
                 lambda: kda.kda_qk_norm_rope(cfg, rope, z(2, 3, 64), None, None, None, i(3, 2)),            # not num_heads
                 lambda: kda.kda_qk_norm_rope(cfg, rope, z(2, 4, 64), None, None, None, i(2, 2)),            # not the axes
                 lambda: kda.kda_qk_norm_rope(cfg, rope, z(2, 64, 4).transpose(1, 2), None, None, None, i(3, 2)),
                 lambda: kda.kda_qk_norm_rope(cfg, rope, z(2, 4, 64), z(2, 2, 64), None, z(64), i(3, 2)),    # weight not fp32
                 lambda: kda.kda_qk_norm_rope_backward(cfg, rope, z(2, 4, 64), None, None, None, i(3, 2), z(2, 4, 64), z(2, 2, 64)),
                 lambda: kda.kda_append_kv(cfg, cache, i(3), i(2, 2), i(2), z(4, 2, 64), z(4, 2, 64)),       # not on the GPU
                 lambda: kda.kda_append_kv(cfg, cache, i(2), i(2, 2), i(2), z(4, 2, 64), z(4, 2, 64)),       # cu_seqlens
                 lambda: kda.kda_append_kv(cfg, cache, i(3), i(3, 2), i(2), z(4, 2, 64), z(4, 2, 64)),       # page_table
                 lambda: kda.kda_read_kv(cfg, cache, i(3), i(2, 2), i(2).long(), 4),
                 lambda: kda.kda_paged_attention(cfg, cache, z(4, 4, 128), i(3), i(2, 2), i(2)),
                 lambda: kda.kda_paged_attention(cfg, kda.KvCache.empty(3, 2, 128, 32, device="cpu"), z(4, 4, 64), i(3), i(2, 2), i(2)),
                 lambda: kda.kda_paged_attention(cfg, cache, z(4, 4, 64), i(3), i(2, 2), i(2))):
        with pytest.raises(ValueError):
            call()
