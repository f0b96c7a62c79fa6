"""The operators around the core where a workgroup goes through its loop more
than once, on dense data and in full: several rows of the norm and of its
backward in one workgroup, several passes of the output gate's backward."""
import pytest
import torch

from tests import layer_reference as ref
from tests.layer_reference import U, check, check_rows_fp8
from tests.test_gpu_layer import BF, EPS, F8, F32, Rand, guarded, kda, make_cfg, same  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# Rows that share a workgroup of the backward: 1, 2 or 3 rows where a row has all of one (256 or 1024 lanes, one to four
# steps of 8 channels), several at a time below.
SHARED = [(2100, 4096, BF), (2100, 4096, F32), (1600, 2056, BF), (1600, 2056, F32), (700, 1544, BF), (700, 776, F32),
          (3100, 4104, BF), (800, 6144, BF), (900, 8192, BF), (900, 8192, F32), (800, 16384, BF), (780, 16392, F32),
          (600, 24584, BF), (13000, 128, BF), (9000, 256, F32), (3500, 1024, BF), (3300, 1536, BF)]


@pytest.mark.parametrize("n,hidden,io", SHARED)
def test_norm_backward_rows_of_one_workgroup(kda, n, hidden, io):
    r = Rand(n + hidden)
    h, w, dy, d_h = r(n, hidden, dtype=io, scale=2), r.weight(hidden), r(n, hidden, dtype=io), r(n, hidden)
    cfg = make_cfg(kda, io, io)
    dx, dw = kda.kda_add_rmsnorm_backward(cfg, h, w, dy, d_h, EPS)
    e, edw, m, mdw = ref.rmsnorm_backward(h, w, dy, d_h, EPS)
    rel = 2 * ref.norm_chain(hidden) * U + 8 * U
    check(dx, e, m, rel, "dx")
    # a workgroup's rows (at most 6 below 3000 of them, else 768 workgroups share them), its lanes joined (16), then the
    # partial sums: 48 rows a wave in 8 chains, joined, 16 waves joined
    check(dw, edw, mdw, rel + (max(6, n / 768 + 1) + 16 + 48 + 8 + 16) * U, "dw")
    assert same((dx, dw), kda.kda_add_rmsnorm_backward(cfg, h, w, dy, d_h, EPS))


@pytest.mark.parametrize("n,hidden,io,out", [(66000, 2048, BF, BF), (66000, 1544, BF, F8), (65600, 1024, F32, F32),
                                             (263000, 264, BF, F8), (65537, 4104, BF, F8)])
def test_norm_more_rows_than_workgroups(kda, n, hidden, io, out):
    """The grid holds 65536 workgroups (of four rows up to 1536 channels)."""
    r = Rand(n)
    x, res, w = r(n, hidden, dtype=io), r(n, hidden, dtype=io, scale=3), r.weight(hidden)
    cfg = make_cfg(kda, io, F32 if out == F8 else out)
    if out == F8:
        y, s, h = kda.kda_add_rmsnorm_fp8(cfg, x, res, w)
    else:
        y, h = kda.kda_add_rmsnorm(cfg, x, res, w)
    assert torch.equal(h, ref.sum_h(x, res))
    rel = ref.norm_chain(hidden) * U
    for i in range(0, n, 16384):   # in parts: the 64-bit values of all rows are large
        t = slice(i, i + 16384)
        e = ref.rmsnorm(h[t], w, EPS)
        if out == F8:
            check_rows_fp8(y[t], s[t], e, rel)
        else:
            check(y[t], e, e.abs(), rel)


@pytest.mark.parametrize("n,hidden", [(5, 72), (9, 520), (7, 2056), (3, 8192), (2, 16392)])
def test_norm_fp32_in_bf16_out(kda, n, hidden):
    r = Rand(hidden)
    x, res, w = r(n, hidden), r(n, hidden, scale=3), r.weight(hidden)
    y, ok = guarded((n, hidden), BF)
    _, h = kda.kda_add_rmsnorm(make_cfg(kda, F32, BF), x, res, w, y=y)
    e = ref.rmsnorm(h, w, EPS)
    check(y, e, e.abs(), ref.norm_chain(hidden) * U)
    assert torch.equal(h, x + res) and ok()


# more than 768 workgroups' worth of rows
GATE_PASSES = [(1500, 33, 128, BF, BF), (1500, 33, 128, F32, F32), (9000, 11, 16, BF, F32), (3000, 17, 32, F32, BF),
               (2500, 21, 64, BF, BF)]


@pytest.mark.parametrize("n,H,d,io,out", GATE_PASSES)
def test_output_gate_several_passes(kda, n, H, d, io, out):
    r = Rand(n + H + d)
    o, gate, w = r(n, H, d, dtype=out), r(n, H, d, dtype=io, scale=2), r.weight(d)
    dy = r(n, H, d, dtype=out)
    cfg = make_cfg(kda, io, out, H, d)
    q, s = kda.kda_output_gate_fp8(cfg, o, gate, w, EPS)
    rel = (ref.norm_chain(d) + 22) * U   # |gate| stays under 12
    check_rows_fp8(q, s, ref.output_gate(o, gate, w, EPS).view(n, H * d), rel)
    d_o, d_gate, dw = kda.kda_output_gate_backward(cfg, o, gate, w, dy, EPS)
    e, eg, ew, m, mg, mw = ref.output_gate_backward(o, gate, w, dy, EPS)
    rel = 2 * rel + 8 * U
    check(d_o, e, m, rel, "d_o")
    check(d_gate, eg, mg, rel, "d_gate")
    # a lane's passes, the lanes of a channel (at most 256 / 2), the partial sums as in the norm's backward
    check(dw, ew, mw, rel + (n * H * d / 8 / 256 / 768 + 2 + 128 + 48 + 8 + 16) * U, "dw")
    assert same((d_o, d_gate, dw), kda.kda_output_gate_backward(cfg, o, gate, w, dy, EPS))
