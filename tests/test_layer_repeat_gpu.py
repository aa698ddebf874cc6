"""The operators around a layer's scan, called again and again: the same bits every time.

The selective scan's raw tiles are refilled by tensor copies while other warps go on; a refill that overtook a read
would show as a few wrong values in one call of many."""
import pytest

from test_layer_workspace_gpu import scan_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(1, 4000, 1536), (3, 777, 2048), (7, 1300, 1472), (13, 1100, 1544), (2, 600, 1025)], ids=str)
def test_selscan_repeats(cuda_lib, case, dtype):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    args = scan_case(case, 11, dtype)
    y0, h0 = ssm.selscan_fwd(*args)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        y, h = ssm.selscan_fwd(*args)
        differ += (y != y0).sum() + (h != h0).sum()
    assert int(differ) == 0 and torch.isfinite(y0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_norm_and_steps_repeat(cuda_lib, dtype):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator("cuda").manual_seed(3)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
    x, w, weight = rand(2, 900, 2048).to(t), rand(2048, 4), rand(2048)
    u, dt, A, B, C, D, z = scan_case((64, 1, 2048), 12, dtype)
    state = rand(64, 2048, 16)
    calls = [lambda: ssm.conv_fwd(x, w), lambda: ssm.conv_step(x[0, :64], w), lambda: ssm.rmsnorm_fwd(x, weight, x),
             lambda: ssm.rmsnorm_fp8_fwd(x, weight, x, group=128)[1:],
             lambda: ssm.selscan_step(u[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], D, z[:, 0], None, state)]
    for call in calls:
        first = call()
        for _ in range(40):
            assert all(torch.equal(a, b) for a, b in zip(first, call()))
