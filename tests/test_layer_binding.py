"""Sizes and arguments that the binding of the operators around the core passes
to the library (CPU only)."""
import pytest

from tests.test_abi import kda  # noqa: F401  (fixture)


def cfg(kda, H=2, d=64):
    return kda.Config(None, None, None, None, None, num_heads=H, head_k_dim=d, head_v_dim=d)


@pytest.mark.parametrize("n,hidden", [(4, 2**32 + 64), (4, -2**32 + 64), (4, 2**31 + 64), (2**64 + 4, 64),
                                      (2**63, 64), (-2**64 + 4, 64), (-1, 64), (4, 0), (4, 12)])
def test_norm_workspace_of_sizes_that_do_not_fit(kda, n, hidden):
    """No size is cut to a small one: what the library refuses has no workspace."""
    assert kda.kda_add_rmsnorm_backward_workspace_bytes(cfg(kda), n, hidden) == 0


@pytest.mark.parametrize("n,H,d", [(2**64 + 4, 2, 64), (-2**64 + 4, 2, 64), (2**63, 2, 64), (4, 2**32 + 2, 64),
                                   (4, 2, 2**32 + 64), (4, -2**32 + 2, 64), (4, 70000, 64)])
def test_gate_workspace_of_sizes_that_do_not_fit(kda, n, H, d):
    assert kda.kda_output_gate_backward_workspace_bytes(cfg(kda, H, d), n) == 0


def test_workspaces_of_sizes_that_fit(kda):
    assert kda.kda_add_rmsnorm_backward_workspace_bytes(cfg(kda), 4, 64) >= 4 * 64 * 4
    assert kda.kda_add_rmsnorm_backward_workspace_bytes(cfg(kda), 0, 64) > 0
    assert kda.kda_output_gate_backward_workspace_bytes(cfg(kda), 4) > 0
