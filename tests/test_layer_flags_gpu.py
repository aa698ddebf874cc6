"""Truth values of the layer operators' Python calls that have none: their own error, before anything runs."""
import pytest

pytestmark = pytest.mark.gpu


def test_flags_without_a_truth_value(cuda_lib):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x, w = torch.ones(2, 3, 16, device="cuda"), torch.ones(16, 4, device="cuda")
    A, bc = -torch.ones(16, 16, device="cuda"), torch.ones(2, 3, 1, 16, device="cuda")
    neither = torch.ones(2)

    class Odd:
        def __bool__(self):
            raise KeyError("odd")

    calls = [lambda f: ssm.conv_fwd(x, w, silu=f), lambda f: ssm.conv_fwd(x, w, return_final_state=f),
             lambda f: ssm.conv_step(x[:, 0], w, silu=f),
             lambda f: ssm.conv_step(x[:, 0], w, state=torch.ones(2, 3, 16, device="cuda"), inplace=f),
             lambda f: ssm.selscan_fwd(x, x, A, bc, bc, softplus=f), lambda f: ssm.selscan_fwd(x, x, A, bc, bc, return_final_state=f),
             lambda f: ssm.selscan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], softplus=f)]
    for call in calls:
        with pytest.raises(RuntimeError, match="ambiguous"):
            call(neither)
        with pytest.raises(KeyError, match="odd"):
            call(Odd())
        call(True), call(1)
