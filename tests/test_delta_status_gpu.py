"""GPU tests of the status of delta_fwd: of calls without a workspace, and of those that need one and do not use it."""
import pytest

from test_delta_gpu import inputs, on_device, rng_of

pytestmark = pytest.mark.gpu
STALL_CHAIN = 1 << 40  # CTA 0 of the chains makes no copies


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def with_fault(t, **kw):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    try:
        ssm.debug_set_lookback_fault(STALL_CHAIN, 5_000_000)
        out = ssm.delta_fwd(**t, **kw)
        torch.cuda.synchronize()
    finally:
        ssm.debug_set_lookback_fault()
    return out


def test_status_of_a_call_without_a_workspace():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    t = on_device(inputs(rng_of("status"), 2, 300, 4, 2, 64, 128, "bf16"), "bf16")
    want = ssm.delta_fwd(**t)
    assert ssm.check_device_status(kind="delta") == 0
    lost = with_fault(t)
    assert bool(lost[0].isnan().any())
    ssm.delta_fwd(**{k: v[:, :5] if v.dim() > 1 else v for k, v in t.items()})  # needs none
    assert ssm.check_device_status(kind="delta") == _lib.SSM_ERR_TIMEOUT
    assert ssm.check_device_status(kind="delta") == 0
    with_fault(t)
    got = ssm.delta_fwd(**t)
    assert ssm.check_device_status(kind="delta", device="cuda:0") == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with_fault(t, workspace=ssm.Workspace("cuda"))  # not the kept one
    assert ssm.check_device_status(kind="delta") == 0
    with_fault(t)
    assert ssm.check_device_status(kind="selscan") == 0
    with pytest.raises(ssm.SsmError):  # a call that is refused leaves no memory with a status
        ssm.delta_fwd(**t, y=t["v"])
    assert ssm.check_device_status(kind="delta") == 0


def test_status_of_a_call_that_goes_token_by_token():
    """Sizes that need a workspace, rows that tensor copies cannot read: no waits, and none of an earlier call's."""
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("status of tokens"), 2, 300, 4, 2, 64, 128, "bf16")
    ws = ssm.Workspace("cuda")
    with_fault(on_device(s, "bf16"), workspace=ws)
    assert ws.buf[:8].any()
    for _ in range(2):
        with ssm.KernelTimer() as timer:
            ssm.delta_fwd(**on_device(s, "bf16", 1), workspace=ws)
        assert timer.launches["delta"] == 1 and timer.launches["delta_chain"] == 0
        assert ssm.check_device_status(ws) == 0
        ws.buf[:256] = 0xff  # it may hold anything


def test_status_of_tokens_without_a_workspace():
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("status of tokens"), 2, 300, 4, 2, 64, 128, "bf16")
    with_fault(on_device(s, "bf16"))
    ssm.delta_fwd(**on_device(s, "bf16", 1))
    assert ssm.check_device_status(kind="delta") == 0
