"""Infinite and extreme values in the operators around a layer's scan, against what their formulas give."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("d", [16, 17])
def test_selscan_without_a_skip_takes_infinite_inputs(d):
    """y = sum_n h C has no term in u itself then: an infinite u gives infinite outputs from its token on, not NaN."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    u = torch.ones(1, 20, d, device="cuda")
    u[0, 5, 3] = float("inf")
    dt, A, bc = torch.ones(1, 20, d, device="cuda"), -torch.ones(d, 16, device="cuda"), torch.ones(1, 20, 1, 16, device="cuda")
    y, h = ssm.selscan_fwd(u, dt, A, bc, bc)
    assert torch.isposinf(y[0, 5:, 3]).all() and torch.isposinf(h[0, 3]).all()
    others = torch.arange(d, device="cuda") != 3
    assert torch.isfinite(y[0, :5]).all() and torch.isfinite(y[..., others]).all() and torch.isfinite(h[0, others]).all()
    y, h = ssm.selscan_step(u[:, 5], dt[:, 0], A, bc[:, 0], bc[:, 0])
    assert torch.isposinf(y[0, 3]) and torch.isposinf(h[0, 3]).all() and torch.isfinite(y[0, others]).all()
