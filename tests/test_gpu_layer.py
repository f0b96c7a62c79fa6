"""The operators around the core on the GPU against their definitions in 64
bits (tests/layer_reference.py): the residual RMS norm, the output epilogue's
e4m3 form, both backward passes and the block-scaled product; alone at the
sizes where they can go wrong, and together as a layer uses them."""
import numpy as np
import pytest
import torch

import oracle
from kda_inputs import BF16
from tests import layer_reference as ref
from tests.layer_reference import U, check, check_rows_fp8

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_03_amd as m
    return m


def make_cfg(kda, io=BF, out=BF, H=1, d=128):
    return kda.Config(A_log=None, dt_bias=None, conv_w_q=None, conv_w_k=None, conv_w_v=None, num_heads=H,
                      head_k_dim=d, head_v_dim=d, io_dtype=io, out_dtype=out)


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def __call__(self, *shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype)

    def weight(self, n):
        return 0.5 + torch.rand((n,), generator=self.g, device="cuda")


def guarded(shape, dtype):
    """A tensor inside a larger buffer, and a check that its surroundings stay as they were."""
    n, m = int(np.prod(shape)), 256
    buf = torch.full((n * dtype.itemsize + 2 * m,), 0x5a, dtype=torch.uint8, device="cuda")
    t = buf[m:m + n * dtype.itemsize].view(dtype).view(shape)
    return t, lambda: bool((buf[:m] == 0x5a).all()) and bool((buf[m + n * dtype.itemsize:] == 0x5a).all())


# ---- the norm -------------------------------------------------------------

ROWS = [(1, 8), (5, 72), (3, 512), (9, 520), (1, 2048), (7, 2056), (2, 4096), (5, 4104), (3, 8192), (2, 8200),
        (3, 16384), (2, 16392), (1, 32768), (1031, 128), (4099, 264), (4001, 640), (7, 784), (13, 1288), (3, 6144)]


@pytest.mark.parametrize("n,hidden", ROWS)
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (BF, F32), (BF, F8), (F32, F8)])
def test_add_rmsnorm(kda, n, hidden, io, out):
    r = Rand(hidden + n)
    x, res, w = r(n, hidden, dtype=io), r(n, hidden, dtype=io, scale=3), r.weight(hidden)
    cfg = make_cfg(kda, io, F32 if out == F8 else out)
    y, ok_y = guarded((n, hidden), out)
    h, ok_h = guarded((n, hidden), io)
    rel = ref.norm_chain(hidden) * U
    expect = ref.rmsnorm(ref.sum_h(x, res), w, EPS)
    if out == F8:
        s, ok_s = guarded((n, (hidden + 127) // 128), F32)
        kda.kda_add_rmsnorm_fp8(cfg, x, res, w, EPS, h=h, y=y, y_scale=s)
        check_rows_fp8(y, s, expect, rel)
        assert ok_s()
    else:
        kda.kda_add_rmsnorm(cfg, x, res, w, EPS, h=h, y=y)
        check(y, expect, expect.abs(), rel)
    assert torch.equal(h, ref.sum_h(x, res)) and ok_y() and ok_h()


def test_add_rmsnorm_without_residual_and_in_place(kda):
    r = Rand(3)
    x, res, w = r(33, 1000, dtype=BF), r(33, 1000, dtype=BF), r.weight(1000)
    cfg = make_cfg(kda)
    y0, h0 = kda.kda_add_rmsnorm(cfg, x, None, w)
    assert h0 is x
    check(y0, ref.rmsnorm(x, w, EPS), ref.rmsnorm(x, w, EPS).abs(), ref.norm_chain(1000) * U)
    y, h = kda.kda_add_rmsnorm(cfg, x, res, w)
    for target in ("x", "residual"):
        x2, r2 = x.clone(), res.clone()
        y2, h2 = kda.kda_add_rmsnorm(cfg, x2, r2, w, h=x2 if target == "x" else r2)
        assert torch.equal(y2, y) and torch.equal(h2, h) and h2 is (x2 if target == "x" else r2)
    x2 = x.clone()
    assert torch.equal(kda.kda_add_rmsnorm(cfg, x2, None, w, y=x2)[0], y0)   # the documented alias
    # leading axes, and eps
    y3, h3 = kda.kda_add_rmsnorm(cfg, x.view(3, 11, 1000), res.view(3, 11, 1000), w, 0.5)
    e = ref.rmsnorm(h, w, 0.5).view(3, 11, 1000)
    assert h3.shape == (3, 11, 1000)
    check(y3, e, e.abs(), ref.norm_chain(1000) * U)


@pytest.mark.parametrize("io", [BF, F32])
def test_add_rmsnorm_special_rows(kda, io):
    """Rows and blocks of zeros, far values, infinities and NaN, each in a row of its own: the others are untouched."""
    r = Rand(5)
    hidden = 392
    x, w = r(9, hidden, dtype=io), r.weight(hidden)
    x[1] = 0
    x[2, 128:256] = 0
    x[3, 5] = float("nan")
    x[4, 300] = float("inf")
    x[5] *= 1e-8
    x[6] *= 1e8
    x[7, :256] = 0
    cfg = make_cfg(kda, io, F32)
    q, s, _ = kda.kda_add_rmsnorm_fp8(cfg, x, None, w)
    y, _ = kda.kda_add_rmsnorm(cfg, x, None, w)
    fine = [0, 1, 2, 5, 6, 7, 8]
    e = ref.rmsnorm(x, w, EPS)
    rel = ref.norm_chain(hidden) * U
    check_rows_fp8(q[fine], s[fine], e[fine], rel)
    check(y[fine], e[fine], e[fine].abs(), rel)
    assert (q[1].float() == 0).all() and (q[2, 128:256].float() == 0).all()
    assert torch.isnan(s[3]).all() and torch.isnan(y[3]).all()
    # an infinity's row: 1 / rms is 0, so its own block is NaN and the others are 0
    assert torch.isnan(s[4, 2]) and torch.isnan(y[4, 300]) and (q[4, :256].float() == 0).all()


def test_fp8_rows_of_far_values_with_a_small_eps(kda):
    """Rows so small that 448 / amax has no fp32 value, while 1 / rms (1 / sqrt(eps): their squares are 0) lifts them."""
    r = Rand(6)
    x, w = r(4, 256) * torch.tensor([[1.0], [1e-30], [2e-37], [3e-36]], device="cuda"), r.weight(256)
    q, s, _ = kda.kda_add_rmsnorm_fp8(make_cfg(kda, F32), x, None, w, 1e-30)
    check_rows_fp8(q, s, ref.rmsnorm(x, w, 1e-30), ref.norm_chain(256) * U)
    gate = r(4, 2, 128)
    cfg = make_cfg(kda, F32, F32, 2)
    q, s = kda.kda_output_gate_fp8(cfg, x.view(4, 2, 128), gate, w[:128].contiguous(), 1e-30)
    e = ref.output_gate(x.view(4, 2, 128), gate, w[:128], 1e-30).view(4, -1)
    check_rows_fp8(q, s, e, (ref.norm_chain(128) + 22) * U)


def test_fp8_rows_of_far_values_with_a_large_weight(kda):
    """Rows whose weighted values are so large that 448 / amax is near fp32's smallest normal number."""
    r = Rand(7)
    x, w = r(4, 256) * torch.tensor([[1.0], [1e12], [1e17], [3e17]], device="cuda"), r.weight(256) * 1e18
    q, s, _ = kda.kda_add_rmsnorm_fp8(make_cfg(kda, F32), x, None, w)
    check_rows_fp8(q, s, ref.rmsnorm(x, w, EPS), ref.norm_chain(256) * U)
    gate = r(4, 2, 128)
    q, s = kda.kda_output_gate_fp8(make_cfg(kda, F32, F32, 2), x.view(4, 2, 128), gate, w[:128].contiguous())
    e = ref.output_gate(x.view(4, 2, 128), gate, w[:128], EPS).view(4, -1)
    check_rows_fp8(q, s, e, (ref.norm_chain(128) + 22) * U)


@pytest.mark.parametrize("n,hidden", ROWS)
@pytest.mark.parametrize("io,out,with_dh", [(BF, BF, True), (F32, F32, True), (BF, F32, False), (F32, BF, True)])
def test_add_rmsnorm_backward(kda, n, hidden, io, out, with_dh):
    r = Rand(hidden + n + 1)
    h, w, dy = r(n, hidden, dtype=io, scale=2), r.weight(hidden), r(n, hidden, dtype=out)
    d_h = r(n, hidden) if with_dh else None
    cfg = make_cfg(kda, io, out)
    dx, ok = guarded((n, hidden), F32)
    _, dw = kda.kda_add_rmsnorm_backward(cfg, h, w, dy, d_h, EPS, dx=dx)
    e, edw, m, mdw = ref.rmsnorm_backward(h, w, dy, d_h, EPS)
    rel = 2 * ref.norm_chain(hidden) * U + 8 * U
    check(dx, e, m, rel, "dx")
    # rows of a workgroup, then the partial sums: at most 768 rows of them in 16 chains, joined
    check(dw, edw, mdw, rel + (n / 768 + 64 + 16 + 4) * U, "dw")
    assert ok()
    if with_dh:   # in place
        dx2, dw2 = kda.kda_add_rmsnorm_backward(cfg, h, w, dy, d_h, EPS, dx=d_h)
        assert dx2 is d_h and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_add_rmsnorm_backward_against_differences(kda):
    r = Rand(11)
    h, w, dy, d_h = r(6, 40, scale=2), r.weight(40), r(6, 40), r(6, 40)
    dx, dw = kda.kda_add_rmsnorm_backward(make_cfg(kda, F32, F32), h, w, dy, d_h, EPS)
    loss = lambda h_, w_: (ref.rmsnorm(h_, w_, EPS) * dy.double()).sum() + (h_ * d_h.double()).sum()
    vh, vw = r(6, 40).double(), r(40).double()
    t = 1e-5   # central differences in 64 bits: off by ~t^2 of the third derivative, and 1e-16 / t
    fd = (loss(h.double() + t * vh, w.double() + t * vw) - loss(h.double() - t * vh, w.double() - t * vw)) / (2 * t)
    got = (dx.double() * vh).sum() + (dw.double() * vw).sum()
    scale = (dx.double() * vh).abs().sum() + (dw.double() * vw).abs().sum()
    assert abs(got - fd) <= 1e-5 * scale


# ---- the output epilogue ----------------------------------------------------

GATES = [(1, 1, 16), (5, 3, 16), (37, 5, 32), (3, 2, 64), (19, 7, 64), (1, 32, 128), (41, 3, 128), (2500, 9, 16),
         (300, 33, 128)]


@pytest.mark.parametrize("n,H,d", GATES)
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_output_gate_fp8_and_backward(kda, n, H, d, io, out):
    r = Rand(1000 * d + n + H)
    o, gate, w = r(n, H, d, dtype=out) * 10.0 ** r(n, H, 1).to(out).clamp(-2, 2), r(n, H, d, dtype=io, scale=2), r.weight(d)
    dy = r(n, H, d, dtype=out)
    cfg = make_cfg(kda, io, out, H, d)
    q, ok_q = guarded((n, H * d), F8)
    s, ok_s = guarded((n, (H * d + 127) // 128), F32)
    kda.kda_output_gate_fp8(cfg, o, gate, w, EPS, y=q, y_scale=s)
    # |gate| stays under 12: sigmoid is off by at most 1.3 * 12 + 6 half steps
    rel = (ref.norm_chain(d) + 22) * U
    check_rows_fp8(q, s, ref.output_gate(o, gate, w, EPS).view(n, H * d), rel)
    assert ok_q() and ok_s()
    d_o, d_gate, dw = kda.kda_output_gate_backward(cfg, o, gate, w, dy, EPS)
    e, eg, ew, m, mg, mw = ref.output_gate_backward(o, gate, w, dy, EPS)
    rel = 2 * rel + 8 * U
    check(d_o, e, m, rel, "d_o")
    check(d_gate, eg, mg, rel, "d_gate")
    rows = n * H * d / 8 / 256 / 768   # passes of a workgroup over the tensor
    check(dw, ew, mw, rel + (rows + 1 + 128 + 128 + 16) * U, "dw")


def test_output_gate_backward_against_differences(kda):
    r = Rand(21)
    o, gate, w, dy = r(5, 3, 32), r(5, 3, 32), r.weight(32), r(5, 3, 32)
    d_o, d_gate, dw = kda.kda_output_gate_backward(make_cfg(kda, F32, F32, 3, 32), o, gate, w, dy, EPS)
    vo, vg, vw = r(5, 3, 32).double(), r(5, 3, 32).double(), r(32).double()
    loss = lambda t: (ref.output_gate(o.double() + t * vo, gate.double() + t * vg, w.double() + t * vw, EPS)
                      * dy.double()).sum()
    fd = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [d_o.double() * vo, d_gate.double() * vg, dw.double() * vw]
    assert abs(sum(t.sum() for t in terms) - fd) <= 1e-5 * sum(t.abs().sum() for t in terms)


def test_output_gate_special_values(kda):
    """Gates far out, heads of zeros, a NaN in one head: the values of the other blocks stay."""
    r = Rand(23)
    n, H, d = 4, 5, 32   # blocks of four heads; the last one holds a single head
    o, gate, w, dy = r(n, H, d), r(n, H, d), r.weight(d), r(n, H, d)
    gate[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), 200.0, -200.0])
    o[1, 2] = 0
    o[2, 4, 3] = float("nan")
    o[3] = 0
    cfg = make_cfg(kda, F32, F32, H, d)
    q, s = kda.kda_output_gate_fp8(cfg, o, gate, w)
    d_o, d_gate, dw = kda.kda_output_gate_backward(cfg, o, gate, w, dy)
    rel = (ref.norm_chain(d) + 22) * U
    e = ref.output_gate(o, gate, w, EPS).view(n, -1)
    check_rows_fp8(q[[0, 1, 3]], s[[0, 1, 3]], e[[0, 1, 3]], rel)
    check_rows_fp8(q[2:3, :128], s[2:3, :1], e[2:3, :128], rel)
    assert torch.isnan(s[2, 1]) and (q[3].float() == 0).all()
    ref_o, ref_g, _, m, mg, _ = ref.output_gate_backward(o, gate, w, dy, EPS)
    for t in (0, 1, 3):
        check(d_o[t], ref_o[t], m[t], 2 * rel + 8 * U)
        check(d_gate[t], ref_g[t], mg[t], 2 * rel + 8 * U)
    assert torch.isnan(d_o[2, 4]).all() and torch.isfinite(d_o[2, :4]).all() and torch.isnan(dw).any()


# ---- the product -------------------------------------------------------------

def fp8_operands(r, M, N, K):
    """Rows as the producers leave them (each block reaches 448), scales over a wide range."""
    a, w = r(M, K), r(N, K)
    sa = ref.block_scale(a)
    q = (a / sa.repeat_interleave(128, -1)[:, :K]).to(F8)
    wq, sw = ref.quantise_weight(w)
    return q, sa * torch.exp(2 * r(*sa.shape)), wq, sw * torch.exp(2 * r(*sw.shape))


PRODUCTS = [(1, 1, 16), (1, 17, 48), (1, 4096, 4096), (2, 130, 128), (16, 64, 112), (17, 33, 144), (33, 129, 2032),
            (64, 256, 256), (65, 320, 1024), (100, 1000, 400), (128, 128, 128), (129, 257, 384), (250, 515, 4096),
            (256, 256, 4096), (257, 300, 272), (300, 16416, 128), (511, 512, 528), (1000, 1002, 1008),
            (2049, 260, 640), (4100, 1028, 1040), (5000, 4200, 272), (4500, 4400, 1168), (70000, 264, 128),
            (80, 520, 2048), (200, 1000, 1024), (300, 4100, 2048), (700, 3000, 2560), (900, 4200, 1024), (1300, 3500, 1536),
            (275, 228, 800), (322, 767, 1968), (518, 486, 16), (609, 781, 48), (762, 663, 272), (419, 591, 1024),
            (393, 628, 4096), (1059, 589, 7680), (1226, 1615, 1376), (1266, 1611, 1280), (1854, 2262, 1024),
            (3505, 3049, 144), (2323, 3339, 128), (3589, 3397, 416), (5337, 5563, 432), (12, 6000, 1040), (3, 8200, 4112), (2, 40, 2576)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("out", [BF, F32])
def test_fp8_matmul(kda, M, N, K, out):
    r = Rand(M + 3 * N + 5 * K)
    a, sa, w, sw = fp8_operands(r, M, N, K)
    y, ok = guarded((M, N), out)
    kda.kda_fp8_matmul(make_cfg(kda, out=out), a, sa, w, sw, y=y)
    ref.check_matmul(y, a, sa, w, sw)
    assert ok()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_fp8_matmul_special_values(kda, M):
    """A NaN or infinite scale stays in its token's row (its 128 columns for the weight's)."""
    r = Rand(M)
    N, K = 300, 272
    a, sa, w, sw = fp8_operands(r, M, N, K)
    sw[1, 2] = float("nan")
    sa[M - 1, 1] = float("inf")
    y = kda.kda_fp8_matmul(make_cfg(kda, out=F32), a, sa, w, sw)
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[128:256] = False
    assert torch.isnan(y[:, ~cols]).all()
    assert not torch.isfinite(y[M - 1]).any()
    if M > 1:
        ref.check_matmul(y, a, sa, w, torch.nan_to_num(sw), slice(0, M - 1), cols)
    a.view(torch.uint8)[0, 0] = 0x7f   # NaN in e4m3
    sa[M - 1, 1] = 1.0
    y = kda.kda_fp8_matmul(make_cfg(kda, out=F32), a, sa, w, sw)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1:, cols]).all()


# ---- offsets beyond 32 bits ----------------------------------------------------

def big(*shape, dtype=BF):
    """Zeros of more than 2^31 values."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free memory")
    t = torch.zeros(shape, dtype=dtype, device="cuda")
    assert t.numel() > 2**31
    return t


def test_add_rmsnorm_large(kda):
    r, n, hidden = Rand(41), 65600, 32768
    x, w = big(n, hidden), r.weight(hidden)
    x[-3:], x[0] = r(3, hidden, dtype=BF), r(hidden, dtype=BF)
    rows = [0, n - 3, n - 2, n - 1]
    cfg = make_cfg(kda)
    e, rel = ref.rmsnorm(x[rows], w, EPS), ref.norm_chain(hidden) * U
    q, s, h = kda.kda_add_rmsnorm_fp8(cfg, x, None, w)
    assert h is x
    check_rows_fp8(q[rows], s[rows], e, rel)
    assert (q[n // 2].float() == 0).all()
    del q, s
    dy = big(n, hidden)
    dy[-2:] = r(2, hidden, dtype=BF)
    dx, dw = kda.kda_add_rmsnorm_backward(cfg, x, w, dy)
    ex, ew, m, mw = ref.rmsnorm_backward(x[rows], w, dy[rows], None, EPS)
    rel = 2 * rel + 8 * U
    check(dx[rows], ex, m, rel)
    check(dw, ew, mw, rel + (-(-n // 768) + 768) * U)
    assert (dx[n // 2] == 0).all()


def test_output_gate_large(kda):
    r, n, H, d = Rand(42), 131200, 128, 128
    o, gate, w = big(n, H, d), big(n, H, d), r.weight(d)
    rows = [0, n - 2, n - 1]
    o[rows], gate[rows] = r(3, H, d, dtype=BF), r(3, H, d, dtype=BF)
    cfg = make_cfg(kda, BF, BF, H, d)
    q, s = kda.kda_output_gate_fp8(cfg, o, gate, w)
    rel = (ref.norm_chain(d) + 22) * U
    check_rows_fp8(q[rows], s[rows], ref.output_gate(o[rows], gate[rows], w, EPS).view(3, -1), rel)
    del q, s
    dy = torch.zeros_like(o)
    dy[rows] = r(3, H, d, dtype=BF)
    d_o, d_gate, dw = kda.kda_output_gate_backward(cfg, o, gate, w, dy)
    e, eg, ew, m, mg, mw = ref.output_gate_backward(o[rows], gate[rows], w, dy[rows], EPS)
    check(d_o[rows], e, m, 2 * rel + 8 * U)
    check(d_gate[rows], eg, mg, 2 * rel + 8 * U)
    check(dw, ew, mw, 2 * rel + (8 + 5500 + 128 + 128 + 16) * U)


@pytest.mark.parametrize("M,N,K", [(131200, 16416, 16384), (1, 262200, 8208), (40, 262200, 8208), (300, 262200, 8208)])
def test_fp8_matmul_large(kda, M, N, K):
    """The operand or the output of more than 2^31 values, by its first and last rows and columns."""
    r, f = Rand(43), 64
    a, w = torch.zeros(M, K, dtype=F8, device="cuda"), torch.zeros(N, K, dtype=F8, device="cuda")
    assert max(a.numel(), w.numel()) > 2**31
    kb, m, n = -(-K // 128), min(M, f), min(N, f)
    sa, sw = r(M, kb).exp(), r(-(-N // 128), kb).exp()
    rows, cols = sorted({*range(m), *range(M - m, M)}), [*range(n), *range(N - n, N)]
    q = lambda k: r(k, K).to(F8).view(torch.uint8)   # noqa: E731  (indexed as bytes)
    a.view(torch.uint8)[rows], w.view(torch.uint8)[cols] = q(len(rows)), q(len(cols))
    y = kda.kda_fp8_matmul(make_cfg(kda), a, sa, w, sw)
    a, sa = a.view(torch.uint8)[rows].view(F8), sa[rows]
    scale = sw.repeat_interleave(128, 0)[cols]   # a row's own scale
    x = ref.dequantised(a, sa)
    z = w.view(torch.uint8)[cols].view(F8).double() * scale.double().repeat_interleave(128, -1)[:, :K]
    e = x @ z.T.contiguous()
    lim = (128 + kb + 19) * U * (x.abs() @ z.abs().T.contiguous())
    lim = lim + 128 * 2.0 ** -13 * (ref.blocks_of(x).abs().amax(-1) @ ref.blocks_of(z).abs().amax(-1).T.contiguous())
    check(y[rows][:, cols], e, lim, 1.0)
    assert (y[M // 2, n:N - n] == 0).all()


def test_sizes_beyond_32_bits_are_refused(kda):
    """Sizes that an int32 argument would cut to small ones."""
    empty = lambda *s, dtype=F8: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    k = 2**32 + 16
    with pytest.raises(kda.KdaError) as e:
        kda.kda_fp8_matmul(make_cfg(kda), empty(0, k), empty(0, k // 128 + 1, dtype=F32), empty(1, k),
                           empty(1, k // 128 + 1, dtype=F32))
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm(make_cfg(kda), empty(0, 2**32 + 8, dtype=BF), None, empty(8, dtype=F32))


# ---- streams, graphs, repeats ------------------------------------------------

def everything(kda, r, stream=None):
    """One call of each operator at small sizes; the outputs."""
    n, H, d = 70, 3, 64
    cfg = make_cfg(kda, BF, BF, H, d)
    x, res, w = r(n, H * d, dtype=BF), r(n, H * d, dtype=BF), r.weight(H * d)
    o, gate, ow, dy = r(n, H, d, dtype=BF), r(n, H, d, dtype=BF), r.weight(d), r(n, H, d, dtype=BF)
    wq, sw = ref.quantise_weight(r(200, H * d))
    tiles = [fp8_operands(r, 300, 520, 1024), fp8_operands(r, 1100, 1000, 512), fp8_operands(r, 4500, 4400, 272)]
    torch.cuda.synchronize()

    def call():
        y, ys, h = kda.kda_add_rmsnorm_fp8(cfg, x, res, w, stream=stream)
        p = kda.kda_fp8_matmul(cfg, y, ys, wq, sw, stream=stream)
        z, zs = kda.kda_output_gate_fp8(cfg, o, gate, ow, stream=stream)
        p2 = kda.kda_fp8_matmul(cfg, z, zs, wq, sw, stream=stream)
        yb, _ = kda.kda_add_rmsnorm(cfg, x, res, w, stream=stream)
        grads = kda.kda_output_gate_backward(cfg, o, gate, ow, dy, stream=stream)
        products = [kda.kda_fp8_matmul(cfg, *t, stream=stream) for t in tiles]
        return (y, ys, h, p, z, zs, p2, yb, *grads, *products,
                *kda.kda_add_rmsnorm_backward(cfg, h, w, dy.view(n, H * d), stream=stream))
    return call


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_repeats_and_streams(kda):
    """The same bits on every call, on another stream, and on two streams at once."""
    first = everything(kda, Rand(31))()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = [everything(kda, Rand(31), s) for s in streams]
    outs = [c() for _ in range(3) for c in calls]
    torch.cuda.synchronize()
    assert all(same(first, o) for o in outs)


def test_graph_replays(kda):
    r = Rand(31)
    call = everything(kda, r)
    expect = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert same(expect, outs)
        assert same(expect, call())   # eager work between the replays


# ---- together ------------------------------------------------------------------

def test_layer_forward(kda):
    """A KDA layer's steps in a row, prefill then decode: the norm, six projections, the core, the epilogue, the
    projection back.  Each step is checked against its definition on what the step before it stored."""
    from kda_inputs import make_problem, make_tokens
    from kda_inputs.torch_io import from_torch_bf16, make_config
    H, d, lens = 2, 128, [70, 0, 1, 200]
    hidden = 320
    p = make_problem(4100, lens, H, d, d, BF16, conv_state=False)
    dev = torch.device("cuda:0")
    cfg = make_config(p, dev, out_dtype=BF)
    r = Rand(41)
    weights = {k: ref.quantise_weight(r(n, hidden, scale=hidden ** -0.5)) for k, n in
               (("q", H * d), ("k", H * d), ("v", H * d), ("alpha", H * d), ("b", H), ("gate", H * d))}
    back = ref.quantise_weight(r(hidden, H * d, scale=(H * d) ** -0.5))
    norm_w, onorm_w = r.weight(hidden), r.weight(d)

    def project(y, ys, wq):
        out = kda.kda_fp8_matmul(cfg, y, ys, *wq)
        ref.check_matmul(out, y, ys, *wq)
        return out

    def front(n):
        x, res = r(n, hidden, dtype=BF), r(n, hidden, dtype=BF, scale=3)
        y, ys, h = kda.kda_add_rmsnorm_fp8(cfg, x, res, norm_w)
        check_rows_fp8(y, ys, ref.rmsnorm(ref.sum_h(x, res), norm_w, EPS), ref.norm_chain(hidden) * U)
        t = {k: project(y, ys, wq) for k, wq in weights.items()}
        t["alpha"], t["gate"] = t["alpha"].view(n, H, d), t["gate"].view(n, H, d)
        return t

    def behind(o, gate):
        z, zs = kda.kda_output_gate_fp8(cfg, o, gate, onorm_w)
        check_rows_fp8(z, zs, ref.output_gate(o, gate, onorm_w, EPS).flatten(1), (ref.norm_chain(d) + 22) * U)
        return project(z, zs, back)

    T, N = sum(lens), len(lens)
    t = front(T)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    S = torch.empty((N, H, d, d), device=dev)
    conv = torch.empty((N, 3, cfg.ctot), dtype=BF, device=dev)
    o, _, _ = kda.kda_varlen_prefill(cfg, cu, t["q"], t["k"], t["v"], t["alpha"], t["b"], final_state=S,
                                     conv_state_out=conv)
    for name in ("q", "k", "v", "alpha", "b"):   # the oracle on the projections as stored
        setattr(p, name, from_torch_bf16(t[name]))
    p.initial_state = None
    p.conv_state = None
    o_ref, S_ref, _, _ = oracle.forward(p)
    rms = float(np.sqrt(np.mean(o_ref ** 2)))
    off = np.abs(o.double().cpu().numpy() - o_ref)
    assert np.all(off <= 2e-3 * rms + 2.0 ** -8 * np.abs(o_ref)), off.max() / rms
    behind(o, t["gate"])

    t = front(N)   # one token for each sequence
    Sd = S.clone()
    od = kda.kda_decode_step(cfg, t["q"], t["k"], t["v"], t["alpha"], t["b"], Sd, conv)
    assert torch.isfinite(od).all()
    behind(od, t["gate"])


def test_layer_gradients(kda):
    """The gradient of a loss through epilogue, core and norm: dL/dz -> d_o -> the core's backward -> the norm's, each
    on what the step before it stored, against the gradient oracle and the formulas."""
    from kda_inputs import make_problem
    from kda_inputs.torch_io import problem_to_device
    H, d = 2, 64
    p = make_problem(4200, [90, 33], H, d, d, BF16, state_seqs=[0, 1], conv_state=True)
    dev = torch.device("cuda:0")
    cfg, t = problem_to_device(p, dev, out_dtype=F32)
    n = p.total_T
    r = Rand(43)
    gate, ow, dz = r(n, H, d, dtype=BF), r.weight(d), r(n, H, d)
    args = (t["cu_seqlens"], t["q"], t["k"], t["v"], t["alpha"], t["b"], t["initial_state"], t["conv_state"])
    o, _, _ = kda.kda_varlen_prefill(cfg, *args)
    d_o, d_gate, _ = kda.kda_output_gate_backward(cfg, o, gate, ow, dz)
    e, eg, _, m, mg, _ = ref.output_gate_backward(o, gate, ow, dz, EPS)
    rel = 2 * (ref.norm_chain(d) + 22) * U + 8 * U
    check(d_o, e, m, rel)
    check(d_gate, eg, mg, rel)
    g = kda.kda_varlen_backward(cfg, *args, d_o=d_o)
    g_ref = oracle.backward(p, d_o.double().cpu().numpy(), None)
    for name in ("dq", "dk", "dv", "dalpha", "db"):
        a, b = g[name].double().cpu().numpy(), g_ref[name].reshape(g[name].shape)
        assert np.max(np.abs(a - b) / (np.sqrt(np.mean(b ** 2)) + np.abs(b))) <= 5e-5, name
    # q's projection taken as the identity: dq is the gradient of the normalised rows
    hidden = H * d
    h, w = r(n, hidden, dtype=BF), r.weight(hidden)
    dx, dw = kda.kda_add_rmsnorm_backward(cfg, h, w, g["dq"], g["dk"])
    ex, ew, mx, mw = ref.rmsnorm_backward(h, w, g["dq"], g["dk"], EPS)
    rel = 2 * ref.norm_chain(hidden) * U + 8 * U
    check(dx, ex, mx, rel)
    check(dw, ew, mw, rel + 100 * U)
