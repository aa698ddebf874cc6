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


STALL_COPIES = 1 << 40  # this and an item's index: the item's copies give up


def run_with_fault(args, stall, lens=None, workspace=None):
    """(y, h_final, what is right, their values without the fault).  Outputs start as a value that is nobody's."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    y0, h0 = ssm.selscan_fwd(*args, lens=lens)
    y, h = torch.full_like(y0, 777.0), torch.full_like(h0, 777.0)
    try:
        ssm.debug_set_lookback_fault(stall, 2_000_000)
        ssm.selscan_fwd(*args, lens=lens, y=y, h_final=h, workspace=workspace)
        torch.cuda.synchronize()
    finally:
        ssm.debug_set_lookback_fault()
    return y, h, y0, h0


def all_right_or_nan(got, want, what):
    import torch
    bad = ~(torch.isnan(got) | (got == want))
    assert not bad.any(), f"{what}: {int(bad.sum())} elements are neither right nor NaN, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case,lens", [(QUEUE_ONE, None), (QUEUE_TWO, None), (QUEUE_TWO, [1100, 0, 300, 256, 257, 1, 700] + 6 * [900])],
                         ids=str)
def test_an_item_that_hands_no_state_on(case, lens, dtype):
    """The rest of its chain is NaN, everything else right or NaN, and the call reports it."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    b, L, d = case
    ws = ssm.Workspace("cuda")
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = scan_case(case, 4, dtype)
    y, h, y0, h0 = run_with_fault(args, 3, n, ws)
    assert ssm.check_device_status(ws) == _lib.SSM_ERR_TIMEOUT
    all_right_or_nan(y, y0, "y")
    all_right_or_nan(h, h0, "h_final")
    # item 3 of the queue: the first 512 tokens of channels 192 to 255 of sequence 0
    assert torch.equal(y[:, :512], y0[:, :512])
    assert torch.isnan(y[0, 512:, 192:256]).all() and torch.isnan(h[0, 192:256]).all()
    again, h2 = ssm.selscan_fwd(*args, lens=n, workspace=ws)
    assert ssm.check_device_status(ws) == 0 and torch.equal(again, y0) and torch.equal(h2, h0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case,item,where", [
    ((2, 70, 72), 1, (0, slice(0, None), slice(64, None))),           # an item a CTA, no workspace
    ((2, 70, 73), 2, (1, slice(0, None), slice(0, 64))),              # rows that are not aligned
    (SPLIT, 1, (0, slice(200, None), slice(0, None))),                # a part of the time axis, both kernels
    (QUEUE_ONE, 5, (0, slice(0, 256), slice(320, 384))),              # the first item of a CTA
    (QUEUE_ONE, 200, None), (QUEUE_TWO, 330, None), (QUEUE_TWO, 900, None),  # others are in its hands
    ((13, 1100, 1537), 700, None)], ids=str)
def test_an_item_whose_copies_give_up(case, item, where, dtype):
    """The waits between a CTA's warps run out: what it had claimed is NaN, nothing is left unwritten."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    b, L, d = case
    ws = ssm.Workspace("cuda", 1 << 20)
    args = scan_case(case, 5, dtype)
    y, h, y0, h0 = run_with_fault(args, STALL_COPIES + item, None, ws)
    need = ssm.selscan_fwd_workspace_bytes(b, L, d, 16)
    assert ssm.check_device_status(ws) == (_lib.SSM_ERR_TIMEOUT if need else 0)
    all_right_or_nan(y, y0, "y")
    all_right_or_nan(h, h0, "h_final")
    assert torch.isnan(y).any() and torch.isnan(h).any()
    if where is not None:
        assert torch.isnan(y[where]).all()
    again, h2 = ssm.selscan_fwd(*args, workspace=ws)
    assert ssm.check_device_status(ws) == 0 and torch.equal(again, y0) and torch.equal(h2, h0)


def test_padding_and_empty_sequences_after_a_fault():
    """Items without a token pass the lost state on, and padding stays 0 where it is written."""
    import torch
    case = (13, 1100, 1544)
    n = torch.tensor([0, 1100] + 11 * [30], dtype=torch.int32, device="cuda")
    y, h, y0, h0 = run_with_fault(scan_case(case, 6), STALL_COPIES + 40, n)
    all_right_or_nan(y, y0, "y")
    all_right_or_nan(h, h0, "h_final")
    assert not y[0].any() and not y[2:, 30:].any()


def test_every_wait_with_no_time_at_all():
    """A limit of a nanosecond: whichever waits run out, the outputs are right or NaN."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    for case in ((2, 70, 72), (2, 70, 73), SPLIT, QUEUE_ONE, QUEUE_TWO):
        args = scan_case(case, 7)
        y0, h0 = ssm.selscan_fwd(*args)
        y, h = torch.full_like(y0, 777.0), torch.full_like(h0, 777.0)
        try:
            ssm.debug_set_lookback_fault(-1, 1)
            ssm.selscan_fwd(*args, y=y, h_final=h)
            torch.cuda.synchronize()
        finally:
            ssm.debug_set_lookback_fault()
        all_right_or_nan(y, y0, f"y {case}")
        all_right_or_nan(h, h0, f"h_final {case}")


@pytest.mark.parametrize("case", [SPLIT, QUEUE_ONE], ids=str)
def test_status_of_a_call_without_a_workspace(case):
    """The workspace that such a call allocates is kept until the next one, for its status."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    args = scan_case(case, 8)
    run_with_fault(args, STALL_COPIES + 1)
    small = scan_case((1, 4, 16), 8)
    ssm.selscan_fwd(*small)  # needs none
    assert ssm.check_device_status(kind="selscan") == _lib.SSM_ERR_TIMEOUT
    assert ssm.check_device_status(kind="selscan") == 0
    run_with_fault(args, STALL_COPIES + 1)
    ssm.selscan_fwd(*args)
    assert ssm.check_device_status(kind="selscan", device="cuda:0") == 0
    run_with_fault(args, STALL_COPIES + 1, None, ssm.Workspace("cuda"))  # not the kept one
    assert ssm.check_device_status(kind="selscan") == 0
    torch.cuda.synchronize()
