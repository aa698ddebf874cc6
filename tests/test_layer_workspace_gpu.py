"""The selective scan's workspace: shared with the other operations, and what a wait that runs out leaves."""
import numpy as np
import pytest

import parity as P
from oracle import linscan as olin
from oracle import native
from selective_state_space_mamba_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


# b, L, d: one whose time axis is split, one of few items (a queue with a CTA an SM), one of many
SPLIT, QUEUE_ONE, QUEUE_TWO = (1, 400, 48), (7, 1300, 1472), (13, 1100, 1544)


def scan_case(case, seed, dtype="bf16"):
    """Random inputs of selscan_fwd, in the order of its arguments."""
    import torch
    b, L, d = case
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    u, dt, z = (torch.randn(b, L, d, device="cuda", generator=g).to(t) for _ in range(3))
    B, C = (torch.randn(b, L, 1, 16, device="cuda", generator=g).to(t) for _ in range(2))
    A = -torch.rand(d, 16, device="cuda", generator=g) - 0.1
    return u, dt, A, B, C, torch.ones(d, device="cuda"), z


def header(ws):
    """(status, counter, done, epoch) of a workspace."""
    b = ws.buf[:24].cpu().numpy()
    return int(b[:8].view(np.uint64)[0]), *(int(v) for v in b[8:20].view(np.uint32))


@pytest.mark.parametrize("case", [SPLIT, QUEUE_ONE, QUEUE_TWO], ids=str)
def test_header_is_left_as_the_other_operations_need_it(case):
    """They keep their flag epoch in the header, and find their claim counters at 0."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    ws = ssm.Workspace("cuda", 32 << 20)
    a = torch.rand(2, 70000, device="cuda")
    ssm.linscan_fwd(a, a, workspace=ws)
    ssm.linscan_fwd(a, a, workspace=ws)
    before = header(ws)
    assert before == (0, 0, 0, before[3]) and before[3] > 0
    ssm.selscan_fwd(*scan_case(case, 1), workspace=ws)
    assert header(ws) == before


def test_operations_in_turn_on_one_workspace():
    """linscan_fwd, ssd_fwd and selscan_fwd in every order, on changing inputs."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    ws = ssm.Workspace("cuda", 256 << 20)
    shape = synth.SSDShape("ws", 2, 2000, 4, 64, 128, 1, 256, "bf16", h0=True)

    def linscan(seed):
        inp = synth.scan_inputs(2, 300000, seed=seed)
        h = ssm.linscan_fwd(P.to_dev(inp["a"]), P.to_dev(inp["b"]), workspace=ws)
        P.assert_rows_close(P.to_np(h), native.linscan(inp["a"], inp["b"]), f"linscan {seed}")

    def short_linscan(seed):
        inp = synth.scan_inputs(3, 5000, seed=seed)
        h = ssm.linscan_fwd(P.to_dev(inp["a"]), P.to_dev(inp["b"]), workspace=ws)
        P.assert_rows_close(P.to_np(h), olin.linscan(inp["a"], inp["b"]), f"linscan {seed}")

    def ssd(seed):
        inp = synth.ssd_inputs(shape, seed=seed)
        args = [P.to_dev(inp[k], "bf16") for k in ("x", "dt")] + [P.to_dev(inp["A"])] + \
            [P.to_dev(inp[k], "bf16") for k in ("B", "C")] + [P.to_dev(inp["D"]), P.to_dev(inp["h0"])]
        y, h = ssm.ssd_fwd(*args, workspace=ws)
        y2, h2 = ssm.ssd_fwd(*args, workspace=ssm.Workspace("cuda"))
        P.assert_ssd_close("bf16", P.to_np(y), P.to_np(y2), P.to_np(h), P.to_np(h2), f"ssd {seed}")

    def selscan(case):
        def run(seed):
            args = scan_case(case, seed)
            y, h = ssm.selscan_fwd(*args, workspace=ws)
            y2, h2 = ssm.selscan_fwd(*args, workspace=ssm.Workspace("cuda"))
            assert torch.equal(y, y2) and torch.equal(h, h2), f"selscan {case} {seed}"
        return run

    ops = [linscan, short_linscan, ssd] + [selscan(c) for c in (SPLIT, QUEUE_ONE, QUEUE_TWO)]
    seed = 0
    for first in ops:  # each right after each
        for second in ops:
            for op in (first, second):
                seed += 1
                op(seed)
                assert ssm.check_device_status(ws) == 0


def test_leftover_error_ends_no_wait_of_another_operation():
    """A scan's error that nobody has read yet does not count for the look-back calls that follow."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    ws = ssm.Workspace("cuda", 64 << 20)
    a = torch.rand(2, 70000, device="cuda")
    ssm.linscan_fwd(a, a, workspace=ws)
    assert header(ws)[3] == 1  # the epoch of the next launch
    try:
        ssm.debug_set_lookback_fault(3, 2_000_000)
        ssm.selscan_fwd(*scan_case(QUEUE_TWO, 2), workspace=ws)
        torch.cuda.synchronize()
    finally:
        ssm.debug_set_lookback_fault()
    assert header(ws)[0] & 0xffffffff == _lib.SSM_ERR_TIMEOUT and header(ws)[0] >> 32 != 1
    inp = synth.scan_inputs(2, 300000, seed=3)
    h = ssm.linscan_fwd(P.to_dev(inp["a"]), P.to_dev(inp["b"]), workspace=ws)
    P.assert_rows_close(P.to_np(h), native.linscan(inp["a"], inp["b"]), "linscan after the error")
    assert ssm.check_device_status(ws) == _lib.SSM_ERR_TIMEOUT and ssm.check_device_status(ws) == 0


@pytest.mark.parametrize("case", [(1, 8, 16), SPLIT], ids=str)
def test_workspace_of_another_device_or_type_is_refused(case):
    """On the host: the kernels would follow its pointer."""
    import torch
    import selective_state_space_mamba_gb300 as ssm

    class Floats(ssm.Workspace):
        def ensure(self, nbytes):
            return super().ensure(nbytes).view(torch.float32)

    class EverySecond(ssm.Workspace):
        def ensure(self, nbytes):
            return super().ensure(2 * nbytes)[::2]

    args = scan_case(case, 1)
    for ws in (ssm.Workspace("cpu"), Floats("cuda"), EverySecond("cuda")):
        with pytest.raises(ValueError, match="workspace"):
            ssm.selscan_fwd(*args, workspace=ws)
    ssm.selscan_fwd(*args, workspace=ssm.Workspace("cuda"))
    torch.cuda.synchronize()
