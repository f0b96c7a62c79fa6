"""The operators around the core where a value, an alias or an order is at its
edge."""
import pytest
import torch

from tests import layer_reference as ref
from tests.layer_reference import U, check, check_rows_fp8
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
