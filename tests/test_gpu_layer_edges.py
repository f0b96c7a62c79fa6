"""The operators around the core where a value, an alias or an order is at its
edge: weighted values beyond fp32 that the row's norm brings back, gates far
out, an output over its input, products that cancel."""
import pytest
import torch

from tests import layer_reference as ref
from tests.layer_reference import U, check, check_rows_fp8
from tests.product_shapes import BF16
from tests.test_gpu_layer import BF, EPS, F8, F32, Rand, kda, make_cfg  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def test_norm_over_its_input_returns_no_h(kda):
    """y=x without a residual overwrites h, which is x: the call has no h to return."""
    r = Rand(61)
    x, w = r(9, 320, dtype=BF), r.weight(320)
    cfg = make_cfg(kda)
    y0, h0 = kda.kda_add_rmsnorm(cfg, x, None, w)
    assert h0 is x
    for view in (lambda t: t, lambda t: t.view(9, 320)):
        x2 = x.clone()
        y, h = kda.kda_add_rmsnorm(cfg, x2, None, w, y=view(x2))
        assert h is None and torch.equal(y, y0)
    x2, stream = x.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    y, h = kda.kda_add_rmsnorm(cfg, x2, None, w, y=x2, stream=stream)
    torch.cuda.synchronize()
    assert h is None and torch.equal(y, y0)
    # an output of its own leaves x, and returns it
    y, h = kda.kda_add_rmsnorm(cfg, x, None, w, y=torch.empty_like(x))
    assert h is x and torch.equal(y, y0)


@pytest.mark.parametrize("h_scale,w_scale,eps", [(1e17, 1e22, EPS), (1e-18, 1e-24, 1e-38), (1e12, 1e27, EPS)])
def test_fp8_rows_whose_weighted_values_leave_fp32(kda, h_scale, w_scale, eps):
    """h * weight passes fp32's range (or its normal numbers), h / rms * weight does not."""
    r = Rand(62)
    x, w = r(5, 392) * h_scale, r.weight(392) * w_scale
    e = ref.rmsnorm(x, w, eps)
    assert e.abs().max() < 1e38 and ref.block_scale(e).min() > 1e-30
    q, s, _ = kda.kda_add_rmsnorm_fp8(make_cfg(kda, F32, F32), x, None, w, eps)
    check_rows_fp8(q, s, e, ref.norm_chain(392) * U)
    for d in (16, 32, 64):   # (the products o * weight of wider heads have a range of their own, see kda.h)
        o, gate, ow = r(7, 3, d) * h_scale, r(7, 3, d), r.weight(d) * w_scale
        q, s = kda.kda_output_gate_fp8(make_cfg(kda, F32, F32, 3, d), o, gate, ow, eps)
        check_rows_fp8(q, s, ref.output_gate(o, gate, ow, eps).view(7, -1), (ref.norm_chain(d) + 22) * U)


@pytest.mark.parametrize("io", [BF, F32])
def test_fp8_rows_whose_squares_leave_fp32(kda, io):
    """The row's 1 / rms is 0 then, and so is its y, also where h * weight passes fp32's range; its neighbours stay."""
    r = Rand(66)
    x, w = r(4, 392, dtype=io), 1.25 + r.weight(392)
    x[1] = torch.finfo(BF).min
    x[2, ::3] = 1e20
    cfg = make_cfg(kda, io, F32)
    q, s, _ = kda.kda_add_rmsnorm_fp8(cfg, x, None, w)
    y, _ = kda.kda_add_rmsnorm(cfg, x, None, w)
    e = ref.rmsnorm(x, w, EPS)
    check_rows_fp8(q[[0, 3]], s[[0, 3]], e[[0, 3]], ref.norm_chain(392) * U)
    assert (y[1:3] == 0).all() and (q[1:3].float() == 0).all() and torch.isfinite(s).all()
    o, gate, ow = r(4, 3, 32, dtype=io), r(4, 3, 32, dtype=io), 1.25 + r.weight(32)
    o[1, 1] = torch.finfo(BF).min
    q, s = kda.kda_output_gate_fp8(make_cfg(kda, io, io, 3, 32), o, gate, ow)
    assert (q[1, 32:64].float() == 0).all() and torch.isfinite(s).all()


@pytest.mark.parametrize("d", [16, 128])
def test_output_gate_far_gates(kda, d):
    """Gates of 64 to 85 and of -64 to -85, where a product x * log2(e) rounded to fp32 is off by 44 U in e^x.

    Roundings on the way to d_gate, in U (half a step of fp32): the row's squares 8 + 4, the mean's eps 1, halved by the
    root, the root 2 and the division 1: 1 / rms 10.  e^-gate 4 (2 ulp), 1 + x 1, the reciprocal 2: the sigmoid 7; one
    minus it 4 + 7 + 1.  d_gate = dy sig w n (1 - sig): 7 + 11 + 12 and four products: 34.  Two more for the second
    order."""
    r = Rand(63)
    n, H = 64, 4
    o, w, dy = r(n, H, d), r.weight(d), r(n, H, d) * 1e6
    far = 64 + 21 * torch.rand((n, H, d), generator=r.g, device="cuda")
    gate = torch.where(r(n, H, d) < 0, far, -far)
    d_o, d_gate, dw = kda.kda_output_gate_backward(make_cfg(kda, F32, F32, H, d), o, gate, w, dy, EPS)
    e, _, ew, m, _, mw = ref.output_gate_backward(o, gate, w, dy, EPS)
    eg = dy * ref.output_gate(o, gate, w, EPS) * torch.sigmoid(-gate.double())   # 1 - sigmoid(64) is 0 in 64 bits too
    off = ((d_gate.double() - eg) / eg).abs()
    assert off.max() <= 36 * U, f"d_gate {off.max() / U:.1f} U"
    check(d_o, e, m, (2 * 36 + 8) * U, "d_o")
    check(dw, ew, mw, (36 + 64 + 256) * U, "dw")


def test_output_gate_backward_gates_at_the_ends(kda):
    """The type's largest and lowest values, infinities and NaN as gates: the sigmoid is 0 or 1, both gradients of it 0."""
    r = Rand(65)
    n, H, d = 6, 2, 128
    o, w, dy = r(n, H, d), r.weight(d), r(n, H, d)
    for dtype in (F32, BF):
        top = torch.finfo(dtype).max
        gate = r(n, H, d)
        gate[:, :, ::16] = torch.tensor([top, -top, float("inf"), -float("inf"), 1e30, -1e30, 104.0, -104.0], device="cuda")
        gate[5, 1, 3] = float("nan")
        gate = gate.to(dtype)
        d_o, d_gate, dw = kda.kda_output_gate_backward(make_cfg(kda, dtype, F32, H, d), o, gate, w, dy, EPS)
        assert (d_gate[:, :, ::16].abs() <= 1e-37).all() and torch.isnan(d_gate[5, 1, 3]) and torch.isnan(dw[3])
        e, eg, _, m, mg, _ = ref.output_gate_backward(o, gate, w, dy, EPS)
        rel = 2 * (ref.norm_chain(d) + 22) * U + 8 * U
        check(d_o[:5], e[:5], m[:5], rel)
        check(d_gate[:5], eg[:5], mg[:5], rel)
        assert torch.isfinite(d_o[5, 0]).all() and torch.isnan(d_o[5, 1]).all()


@pytest.mark.parametrize("io", [BF, F32])
def test_backward_rows_whose_squares_leave_fp32(kda, io):
    """y is 0 on such a row whatever its values are: its gradients are 0, and d_h passes through; the others stay."""
    r = Rand(67)
    h, w, dy, d_h = r(5, 392, dtype=io), 1.25 + r.weight(392), r(5, 392, dtype=F32), r(5, 392)
    h[1] = torch.finfo(BF).min
    h[2, ::3] = 1e38
    fine = [0, 3, 4]
    dx, dw = kda.kda_add_rmsnorm_backward(make_cfg(kda, io, F32), h, w, dy, d_h, EPS)
    e, edw, m, mdw = ref.rmsnorm_backward(h[fine], w, dy[fine], d_h[fine], EPS)
    rel = 2 * ref.norm_chain(392) * U + 8 * U
    check(dx[fine], e, m, rel, "dx")
    check(dw, edw, mdw, rel + 100 * U, "dw")
    assert torch.equal(dx[1:3], d_h[1:3])
    for d in (32, 128):
        o, gate, ow, dz = r(5, 2, d, dtype=io), r(5, 2, d), 1.25 + r.weight(d), r(5, 2, d, dtype=io)
        o[1] = torch.finfo(BF).min
        d_o, d_gate, dw = kda.kda_output_gate_backward(make_cfg(kda, F32, io, 2, d), o, gate, ow, dz, EPS)
        keep = [0, 2, 3, 4]
        e, eg, ew, m, mg, mw = ref.output_gate_backward(o[keep], gate[keep], ow, dz[keep], EPS)
        rel = 2 * (ref.norm_chain(d) + 22) * U + 8 * U
        check(d_o[keep], e, m, rel, "d_o")
        check(d_gate[keep], eg, mg, rel, "d_gate")
        check(dw, ew, mw, rel + 300 * U, "d_weight")
        assert (d_o[1] == 0).all() and (d_gate[1] == 0).all()


# ---- the product's sums --------------------------------------------------------

def exponent(v):
    """The power of two of an e4m3 value; -6, that of its smallest normal numbers, for those below and for 0."""
    return (torch.frexp(v.float())[1] - 1).clamp(min=-6)


def cut_bound(a, a_scale, w, w_scale):
    """What an e4m3 step may lose of each output.  The step sums the products of 8 neighbouring channels in units of 2^-13
    of the power of two of the largest of them (of their exponents' sum); what lies below a unit is cut.  The largest
    loses nothing, so a group loses less than 7 units."""
    k = a.shape[1]
    ea, ew = exponent(a), exponent(w)
    bound = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64, device=a.device)
    for g in range(0, k, 8):
        top = (ea[:, None, g:g + 8] + ew[None, :, g:g + 8]).amax(-1).double()
        bound += 7 * torch.exp2(top - 13) * (a_scale[:, g // 128].double()[:, None] * w_scale[:, g // 128].double()[None])
    return bound


def outliers(r, M, N, K):
    """Operands with three channels 50 times larger in each block, two of which cancel in every output exactly."""
    a, w = r(M, K), r(N, K)
    for b in range(0, K, 128):
        a[:, b + 3] *= 50
        a[:, b + 9] *= 50
        w[:, b + 3] *= 4
    sa = ref.block_scale(a)
    qa = (a / sa.repeat_interleave(128, -1)[:, :K]).to(F8)
    wq, sw = ref.quantise_weight(w)
    one, other = list(range(3, K, 128)), [min(b + 12, K - 1) for b in range(0, K, 128)]
    a8, w8 = qa.view(torch.uint8), wq.view(torch.uint8)
    a8[:, other] = a8[:, one]
    w8[:, other] = w8[:, one] ^ 0x80
    return qa, sa, wq, sw


@pytest.mark.parametrize("M,N,K", [s for ss in BF16.values() for s in ss[:1] if s[2] > 16] + [(1, 500, 4112), (7, 4000, 272)])
def test_product_of_outliers_that_cancel(kda, M, N, K):
    """Fp32 outputs keep fp32's sums; bf16 outputs stay within what an e4m3 step cuts."""
    a, sa, w, sw = outliers(Rand(M + N), M, N, K)
    rows = sorted({*range(min(M, 40)), *range(max(0, M - 24), M)})
    cols = sorted({*range(min(N, 140)), *range(max(0, N - 60), N)})
    ra, rs = a.float()[rows], sa[rows]
    rw, rws = w.float()[cols], sw.repeat_interleave(128, 0)[cols]
    x = ra.double() * rs.double().repeat_interleave(128, -1)[:, :K]
    z = rw.double() * rws.double().repeat_interleave(128, -1)[:, :K]
    e, m = x @ z.T.contiguous(), x.abs() @ z.abs().T.contiguous()
    lim = (min(K, 128) + (K + 127) // 128 + 19) * U * m
    y = kda.kda_fp8_matmul(make_cfg(kda, out=F32), a, sa, w, sw)
    check(y[rows][:, cols], e, lim, 1.0, "fp32")
    y = kda.kda_fp8_matmul(make_cfg(kda), a, sa, w, sw)
    check(y[rows][:, cols], e, lim + cut_bound(ra, rs, rw, rws), 1.0, "bf16")


@pytest.mark.parametrize("M,N", [(1, 40), (300, 520), (5337, 5563)])
@pytest.mark.parametrize("at", [(0, 1), (5, 100)])
def test_product_of_two_large_values_that_cancel(kda, M, N, at):
    """448 * 448 - 448 * 448 + 126 ones: 126 in fp32.  In an e4m3 step the ones beside a large product, in its group of 8
    channels, lie below its unit (2^(8 + 8 - 13) = 8) and are cut; the others stay."""
    a, w = torch.ones(M, 128, device="cuda"), torch.ones(N, 128, device="cuda")
    a[:, at[0]] = a[:, at[1]] = w[:, at[0]] = 448
    w[:, at[1]] = -448
    one = lambda n: torch.ones(n, 1, device="cuda")   # noqa: E731
    args = (a.to(F8), one(M), w.to(F8), one(-(-N // 128)))
    assert (kda.kda_fp8_matmul(make_cfg(kda, out=F32), *args) == 126).all()
    assert (kda.kda_fp8_matmul(make_cfg(kda), *args) == (120 if at[0] // 8 == at[1] // 8 else 112)).all()


def test_product_bf16_loss_by_data(kda):
    """The loss of bf16 outputs on Gaussian operands, and with two channels in 128 up to a hundred times larger.  A value
    off by c before its rounding ends at most 2 c further from its exact value than the nearest bf16 value is."""
    r = Rand(64)
    M, N, K = 600, 520, 1024
    for k in (1, 5, 20, 100):
        a = r(M, K)
        a.view(M, -1, 128)[:, :, :2] *= k
        sa = ref.block_scale(a)
        q = (a / sa.repeat_interleave(128, -1)).to(F8)
        wq, sw = ref.quantise_weight(r(N, K))
        y = kda.kda_fp8_matmul(make_cfg(kda), q, sa, wq, sw).double()
        x, z = ref.dequantised(q, sa), ref.dequantised(wq, sw, 128)
        e, m = x @ z.T.contiguous(), x.abs() @ z.abs().T.contiguous()
        nearest = e.to(BF).double()
        cut = cut_bound(q.float(), sa, wq.float(), sw.repeat_interleave(128, 0)[:N]) + (128 + 8 + 19) * U * m
        off, best, most = ((y - e).norm() / e.norm()).item(), ((nearest - e).norm() / e.norm()).item(), (cut.norm() / e.norm()).item()
        print(f"outliers x {k}: off by {off:.6e}, rounding alone {best:.6e}, not the nearest "
              f"{(y != nearest).double().mean().item():.4f}, the cut's bound {most:.2e}", flush=True)
        assert off <= best + 2 * most
        assert ((y - e).abs() <= (nearest - e).abs() + 2 * cut).all()
