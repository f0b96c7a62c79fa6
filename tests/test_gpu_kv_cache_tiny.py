"""Keys next to a boundary between two codes where fp32 has fewer bits: blocks of the least scale."""
import pytest
import torch

from tests import attention_reference as ref
from tests.test_gpu_kv_cache import Batch
from tests.test_gpu_layer import F32
from tests.test_gpu_rope import expected, kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [2.0 ** -23, 2.0 ** -24, 2.0 ** -26])
@pytest.mark.parametrize("d", [64, 256])
def test_boundaries_of_the_least_scale(kda, d, eps):  # noqa: F811
    """Rows of ones are normed to 1 / sqrt(1 + eps), just below 1; weights at the boundaries of the scale 2^-126 (and one step
    of fp32 on either side) give keys that fp32 cannot tell from them."""
    b = Batch(kda, [(4, 4)], 1, d, 32)
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    w = (middle * 2.0 ** -126).repeat(d // 8)
    w[8:16] += 2.0 ** -149
    w[16:24] -= 2.0 ** -149
    w, x = w.cuda(), torch.ones(4, 1, d, device="cuda")
    x[1] = -1
    cfg, rope = make_cfg(kda, 1, d, F32, F32), make_rope(kda, 0)
    kda.kda_append_kv(cfg, b.cache, *b.where, x, x, w, eps, rope=rope)
    want, _ = expected(x, w, rope, None, eps)
    code, e = ref.quantised(want)
    got, _ = kda.kda_read_kv(cfg, b.cache, *b.where, 4)
    assert torch.equal(got.double().cpu(), ref.values(code, e))
