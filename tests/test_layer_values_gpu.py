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


@pytest.mark.parametrize("rate", ["lowest", "infinite"])
@pytest.mark.parametrize("d", [16, 17])
def test_selscan_decay_rates_at_the_end_of_the_range(d, rate):
    """A of the lowest value, or minus infinity: a token forgets all before it, a step of 0 and padding change nothing."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, N = 2, 37, 16
    g = torch.Generator("cuda").manual_seed(2)
    u, B, C = (torch.randn(*n, device="cuda", generator=g) for n in ((b, L, d), (b, L, 1, N), (b, L, 1, N)))
    low = torch.finfo(torch.float32).min if rate == "lowest" else float("-inf")
    A, h0 = torch.full((d, N), low, device="cuda"), torch.randn(b, d, N, device="cuda", generator=g)
    dt = torch.full((b, L, d), 0.5, device="cuda")
    lens = torch.tensor([L, 20], dtype=torch.int32, device="cuda")
    y, h = ssm.selscan_fwd(u, dt, A, B, C, h0=h0, lens=lens, softplus=False)
    own = 0.5 * u[..., None] * B  # [b, L, d, N]
    want = (own * C).sum(-1)
    want[1, 20:] = 0
    assert torch.allclose(y, want, rtol=1e-5, atol=1e-5)
    assert torch.equal(h, torch.stack([own[0, -1], own[1, 19]]))
    y1, h1 = ssm.selscan_step(u[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], state=h0, softplus=False)
    assert torch.equal(h1, own[:, 0]) and torch.allclose(y1, want[:, 0], rtol=1e-5, atol=1e-5)
    y, h = ssm.selscan_fwd(u, 0 * dt, A, B, C, h0=h0, lens=lens, softplus=False)
    assert torch.equal(h, h0) and torch.isfinite(y).all()
    y1, h1 = ssm.selscan_step(u[:, 0], 0 * dt[:, 0], A, B[:, 0], C[:, 0], state=h0, softplus=False)
    assert torch.equal(h1, h0) and torch.isfinite(y1).all()


def test_selscan_a_rate_that_is_no_number_stays_none():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    A = -torch.ones(8, 16, device="cuda")
    A[3, 5] = float("nan")
    x, bc = torch.ones(1, 5, 8, device="cuda"), torch.ones(1, 5, 1, 16, device="cuda")
    y, h = ssm.selscan_fwd(x, x, A, bc, bc)
    y1, h1 = ssm.selscan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])
    for a, s in ((y[0], h[0]), (y1, h1[0])):
        assert torch.isnan(a[:, 3]).all() and torch.isnan(s[3, 5])
        assert torch.isfinite(a[:, :3]).all() and torch.isfinite(a[:, 4:]).all() and int(torch.isnan(s).sum()) == 1
