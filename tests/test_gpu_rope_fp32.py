"""The sines of the all-fp32 norm and rotation: as near as fp32 holds them, also next to 0."""
import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import U
from tests.test_gpu_layer import F32, Rand
from tests.test_gpu_rope import kda, make_cfg, make_rope  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot,axes,inter", [(64, 64, 1, False), (128, 96, 2, True), (256, 256, 3, False), (256, 64, 1, True)])
@pytest.mark.parametrize("n", [3, 333, 5000])
def test_rotation_alone(kda, d, rot, axes, inter, n):  # noqa: F811
    """Without a norm a value has the rounding of its sine, of a product and of the sum: 3 U of |a cos| + |b sin|.  The angle
    is formed in 64 bits: at 3e5 / (2 pi) turns three roundings of 2^-53 are 1e-10 radians."""
    r = Rand(n + d)
    x, g = r(n, 2, d), r(n, 2, d)
    rope = make_rope(kda, rot, axes, inter)
    pos = torch.randint(-300000, 300000, (axes, n), generator=r.g, device="cuda", dtype=torch.int32)
    pos[:, : n // 3] = torch.randint(0, 3, (axes, n // 3), generator=r.g, device="cuda", dtype=torch.int32)
    cfg = make_cfg(kda, 2, d, F32, F32)
    angle = ref.angles(rope.inv_freq, rope.axis, pos)
    y = kda.kda_qk_norm_rope(cfg, rope, x, None, None, None, pos)[0]
    dx = kda.kda_qk_norm_rope_backward(cfg, rope, x, None, None, None, pos, g, None)[0]
    for got, of, t in ((y, x, angle), (dx, g, -angle)):
        of = of.double().cpu()
        e = ref.rotate(of, t, rot, inter)
        a, b = ref.pair_channels(rot, inter)
        c, s = t.cos().abs()[:, None], t.sin().abs()[:, None]
        m, near = of.abs().clone(), of.abs().clone()
        m[..., a], m[..., b] = of[..., a].abs() * c + of[..., b].abs() * s, of[..., a].abs() * s + of[..., b].abs() * c
        near[..., a] = near[..., b] = of[..., a].abs() + of[..., b].abs()
        ratio = ((got.double().cpu() - e).abs() / (3 * U * m + 1e-10 * near + 1e-37)).max().item()
        assert ratio <= 1, ratio
