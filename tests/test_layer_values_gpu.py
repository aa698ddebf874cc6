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


@pytest.mark.parametrize("where", ["u", "h0"])
def test_selscan_infinite_states_cross_the_parts_of_a_split_time_axis(where):
    """exp(A delta) over a whole part is 0 in f32, over each of its tokens it is not: an infinite state stays one."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    assert ssm.selscan_fwd_workspace_bytes(1, 400, 16, 16) > 0  # split
    u = torch.ones(1, 400, 16, device="cuda")
    dt, A, bc = torch.ones(1, 400, 16, device="cuda"), -torch.ones(16, 16, device="cuda"), torch.ones(1, 400, 1, 16, device="cuda")
    h0 = torch.zeros(1, 16, 16, device="cuda")
    if where == "u":
        u[0, 100, 3] = float("inf")
    else:
        h0[0, 3] = float("inf")
    y, h = ssm.selscan_fwd(u, dt, A, bc, bc, h0=h0)
    first = 100 if where == "u" else 0
    assert torch.isposinf(y[0, first:, 3]).all() and torch.isposinf(h[0, 3]).all()
    others = torch.arange(16, device="cuda") != 3
    assert torch.isfinite(y[0, :first]).all() and torch.isfinite(y[..., others]).all() and torch.isfinite(h[0, others]).all()


def test_selscan_growing_states_of_zero_cross_the_parts():
    """A decay that grows (A > 0) over a part is infinite in f32: a state of 0 stays 0."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    u = torch.zeros(1, 400, 16, device="cuda")
    u[0, 390:] = 1
    dt, A, bc = torch.ones(1, 400, 16, device="cuda"), torch.ones(16, 16, device="cuda"), torch.ones(1, 400, 1, 16, device="cuda")
    y, h = ssm.selscan_fwd(u, dt, A, bc, bc)
    assert not y[0, :390].any() and torch.isfinite(y).all() and torch.isfinite(h).all() and (y[0, 390:] > 0).all()
