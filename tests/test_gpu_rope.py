"""Norm and rotation of query and key heads, and their gradients, against the definitions in 64 bits
(tests/attention_reference.py)."""
import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import U, check
from tests.test_gpu_layer import BF, F32, Rand, guarded

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_03_amd as m
    return m


def make_cfg(kda, hq, d, io=BF, out=BF):
    return kda.Config(None, None, None, None, None, num_heads=hq, head_k_dim=d, head_v_dim=d, io_dtype=io, out_dtype=out)


def make_rope(kda, rot, axes=1, inter=False, theta=1e6):
    half = rot // 2
    inv = (theta ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()
    axis = None if axes == 1 else (torch.arange(half) * axes // half).int().cuda()
    return kda.Rope(inv, axis, axes, inter)


def expected(x, w, rope, pos, eps=EPS):
    y = ref.normed(x, w, eps)
    rot = 2 * len(rope.inv_freq)
    if not rot:
        return y, y.abs()
    return (ref.rotate(y, ref.angles(rope.inv_freq, rope.axis, pos), rot, rope.interleaved),
            ref.pair_magnitude(y, rot, rope.interleaved))


CASES = [(1, 16, 2, 256, 64, 1, False), (3, 1, 1, 64, 16, 1, False), (5, 7, 1, 64, 48, 1, True), (17, 6, 3, 128, 128, 3, False),
         (2, 3, 2, 128, 96, 2, False), (33, 5, 5, 256, 256, 4, True), (9, 4, 0, 128, 64, 1, False), (4, 9, 2, 256, 0, 1, False),
         (1031, 2, 1, 64, 64, 2, True), (700, 40, 8, 128, 32, 1, False), (2, 3, 1, 256, 208, 3, True),
         (9000, 16, 2, 256, 64, 1, False)]


@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,inter", CASES)
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_norm_rope(kda, n, hq, hkv, d, rot, axes, inter, io, out):
    r = Rand(n + hq)
    q, k = r(n, hq, d, dtype=io, scale=3), r(n, hkv, d, dtype=io) if hkv else None
    wq, wk = r.weight(d), r.weight(d)
    rope = make_rope(kda, rot, axes, inter)
    pos = torch.randint(-300000, 300000, (axes, n), generator=r.g, device="cuda", dtype=torch.int32)
    cfg = make_cfg(kda, hq, d, io, out)
    y, ok_y = guarded((n, hq, d), out)
    z, ok_z = guarded((n, max(hkv, 1), d), out)
    kda.kda_qk_norm_rope(cfg, rope, q, k, wq, wk, pos, EPS, q_out=y, k_out=z if hkv else None)
    assert ok_y() and ok_z()
    check(y.cpu(), *expected(q, wq, rope, pos), ref.ROPE_REL)
    if hkv:
        check(z.cpu(), *expected(k, wk, rope, pos), ref.ROPE_REL)


def test_positions_far_and_near(kda):
    """Every bit of an int32 position counts: the lowest, the largest, and their neighbours."""
    at = [-2**31, -2**31 + 1, -1, 0, 1, 2**20, 2**24 + 1, 2**30 - 1, 2**31 - 2, 2**31 - 1]
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    r = Rand(2)
    q = r(len(at), 3, 128)
    rope = make_rope(kda, 128)
    y, _ = kda.kda_qk_norm_rope(make_cfg(kda, 3, 128, F32, F32), rope, q, None, None, None, pos)
    # the rate in 64 bits is off by 2^-53, the angle of position 2^31 by 2^-22 turns of the fastest pair: 2 pi 2^31 2^-53
    # radians, 1.5e-6
    e, m = expected(q, None, rope, pos)
    check(y.cpu(), e, m, ref.ROPE_REL + 3e-6)
    check(y.cpu()[3:6], e[3:6], m[3:6], ref.ROPE_REL)


def test_views_in_place_and_leading_row(kda):
    """q and k as views into one projection, outputs over their inputs, one-axis positions as a vector."""
    r = Rand(3)
    n, hq, hkv, d = 37, 5, 2, 128
    wide = r(n, (hq + 2 * hkv) * d + 24, dtype=BF)
    q, k = wide[:, :hq * d].view(n, hq, d), wide[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    cfg, rope, w = make_cfg(kda, hq, d), make_rope(kda, 64), r.weight(d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    y, z = kda.kda_qk_norm_rope(cfg, rope, q, k, w, w, pos)
    y1, z1 = kda.kda_qk_norm_rope(cfg, rope, q.contiguous(), k.contiguous(), w, w, pos[None])
    assert torch.equal(y, y1) and torch.equal(z, z1)
    q2, k2 = q.contiguous(), k.contiguous()
    y2, z2 = kda.kda_qk_norm_rope(cfg, rope, q2, k2, w, w, pos, q_out=q2, k_out=k2)
    assert y2 is q2 and torch.equal(q2, y) and torch.equal(k2, z)
    one = wide[:1, :hq * d].view(1, hq, d)
    assert torch.equal(kda.kda_qk_norm_rope(cfg, rope, one, None, w, None, pos[:1])[0], y[:1])
    none, nk = kda.kda_qk_norm_rope(cfg, rope, q[:0], k[:0], w, w, pos[:0])
    assert none.shape == (0, hq, d) and nk.shape == (0, hkv, d)


@pytest.mark.parametrize("io", [BF, F32])
def test_special_rows(kda, io):
    """NaN, infinities, zeros and values beyond fp32's squares stay in their own row, and unrotated channels in theirs
    where there is no norm."""
    r = Rand(5)
    n, d = 8, 128
    q = r(n, 2, d, dtype=io)
    q[1, 0, 3] = float("nan")
    q[2, 1, 70] = float("inf")
    q[3] = 0
    q[4, 0] = 3e38
    w, rope = r.weight(d), make_rope(kda, 64)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    cfg = make_cfg(kda, 2, d, io, F32)
    y, _ = kda.kda_qk_norm_rope(cfg, rope, q, None, w, None, pos)
    e, m = expected(q, w, rope, pos)
    y = y.cpu()
    assert y[1, 0].isnan().all() and not y[1, 1].isnan().any() and (y[3] == 0).all() and (y[4, 0] == 0).all()
    rows = [0, 5, 6, 7]
    check(y[rows], e[rows], m[rows], ref.ROPE_REL)
    x, _ = kda.kda_qk_norm_rope(cfg, rope, q, None, None, None, pos)
    x = x.cpu()
    bad = x[2, 1].isfinite().logical_not()
    assert bad.nonzero().tolist() == [[70]] and x[1, 0].isnan().nonzero().flatten().tolist() == [3, 35]
    zero = torch.zeros((1, 2, d), dtype=io, device="cuda")
    assert kda.kda_qk_norm_rope(cfg, rope, zero, None, w, None, pos[:, :1], 0.0)[0].isnan().all()


@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,inter", CASES)
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (F32, BF)])
def test_backward(kda, n, hq, hkv, d, rot, axes, inter, io, out):
    r = Rand(n + 7)
    q, k = r(n, hq, d, dtype=io, scale=3), r(n, hkv, d, dtype=io) if hkv else None
    wq, wk = r.weight(d), r.weight(d)
    rope = make_rope(kda, rot, axes, inter)
    pos = torch.randint(-300000, 300000, (axes, n), generator=r.g, device="cuda", dtype=torch.int32)
    gq, gk = r(n, hq, d, dtype=out), r(n, hkv, d, dtype=out) if hkv else None
    cfg = make_cfg(kda, hq, d, io, out)
    got = kda.kda_qk_norm_rope_backward(cfg, rope, q, k, wq, wk, pos, gq, gk, EPS)
    again = kda.kda_qk_norm_rope_backward(cfg, rope, q, k, wq, wk, pos, gq, gk, EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
    angle = ref.angles(rope.inv_freq, rope.axis, pos)
    for x, w, g, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        if x is None:
            assert dx is None and (dw == 0).all()
            continue
        edx, edw, mx, mw = ref.qk_backward(x, w, g, angle, rot, inter, EPS)
        # two norms' sums in each term instead of one
        check(dx.cpu(), edx, mx, 3 * ref.ROPE_REL)
        # a lane's rows (at most n * heads over the groups of 768 workgroups), the lanes of a channel, the partial rows
        chain = n * x.shape[1] / (min(768, n * (hq + hkv) * d / 16 / 256 + 1) * 256 * 16 / d) + 64 + 128
        check(dw.cpu(), edw, mw, 2 * ref.ROPE_REL + chain * U)


def test_backward_without_norm_views_and_no_tokens(kda):
    r = Rand(11)
    n, hq, hkv, d = 21, 3, 2, 64
    wide = r(n, (hq + hkv) * d + 8, dtype=BF)
    q, k = wide[:, :hq * d].view(n, hq, d), wide[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    cfg, rope, w = make_cfg(kda, hq, d, BF, F32), make_rope(kda, 32), r.weight(d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    gq, gk = r(n, hq, d), r(n, hkv, d)
    dq, dk, dwq, dwk = kda.kda_qk_norm_rope_backward(cfg, rope, q, k, None, w, pos, gq, gk)
    angle = ref.angles(rope.inv_freq, None, pos[None])
    check(dq.cpu(), ref.rotate(gq.double().cpu(), -angle, 32, False), ref.pair_magnitude(gq.double().cpu(), 32, False), ref.ROPE_REL)
    assert (dwq == 0).all()
    e = ref.qk_backward(k, w, gk, angle, 32, False, EPS)
    check(dk.cpu(), e[0], e[2], 3 * ref.ROPE_REL)
    check(dwk.cpu(), e[1], e[3], 2 * ref.ROPE_REL + 300 * U)
    out = kda.kda_qk_norm_rope_backward(cfg, rope, q[:0], k[:0], w, w, pos[:0], gq[:0], gk[:0])
    assert (out[2] == 0).all() and (out[3] == 0).all() and out[0].shape == (0, hq, d)


def test_backward_against_differences(kda):
    """Central differences of the forward in fp32 along random directions."""
    r = Rand(13)
    n, hq, hkv, d = 6, 3, 2, 64
    q, k, wq, wk = r(n, hq, d), r(n, hkv, d), r.weight(d), r.weight(d)
    cfg, rope = make_cfg(kda, hq, d, F32, F32), make_rope(kda, 48, 2, True, 100.0)
    pos = torch.randint(0, 50, (2, n), generator=r.g, device="cuda", dtype=torch.int32)
    gq, gk = r(n, hq, d), r(n, hkv, d)
    grads = kda.kda_qk_norm_rope_backward(cfg, rope, q, k, wq, wk, pos, gq, gk)

    def loss(*a):
        y, z = kda.kda_qk_norm_rope(cfg, rope, *a, pos)
        return (y.double() * gq).sum() + (z.double() * gk).sum()

    args = [q, k, wq, wk]
    for i, g in enumerate(grads):
        u = r(*g.shape)
        h = 2.0 ** -9
        step = [a + (h * u if j == i else 0) for j, a in enumerate(args)], [a - (h * u if j == i else 0) for j, a in enumerate(args)]
        fd = (loss(*step[0]) - loss(*step[1])) / (2 * h)
        an = (g.double() * u).sum()
        # the third derivative's h^2 / 6 (terms of the size of the gradient's own, |u| ~ 1 against rows of norm 8), and the
        # loss's own rounding over 2 h: sqrt(terms) * 24 U / (2 h)
        terms = gq.numel() + gk.numel()
        lim = 3 * h * h * g.double().norm() * u.double().norm() + terms ** 0.5 * 24 * U * 4 / (2 * h)
        assert abs(fd - an) <= lim, (i, float(fd), float(an), float(lim))


def test_streams_and_graph(kda):
    """On another stream than the current one, and captured: replays give the eager bits, eager work in between."""
    r = Rand(17)
    n, hq, hkv, d = 300, 4, 2, 128
    q, k, w = r(n, hq, d, dtype=BF), r(n, hkv, d, dtype=BF), r.weight(d)
    gq, gk = r(n, hq, d, dtype=BF), r(n, hkv, d, dtype=BF)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    cfg, rope = make_cfg(kda, hq, d), make_rope(kda, 64)
    f = lambda **a: (*kda.kda_qk_norm_rope(cfg, rope, q, k, w, w, pos, **a),
                     *kda.kda_qk_norm_rope_backward(cfg, rope, q, k, w, w, pos, gq, gk, **a))
    eager = [t.clone() for t in f()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = f(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for i in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out)), i
        f()
