"""GPU tests of the gated delta rule's ways through a prompt: orders of strides, segments of the workspace, offsets beyond 32
bits, workspaces of the caller, streams, and waits that run out."""
import numpy as np
import pytest

from oracle import delta as od
from test_delta_gpu import OUT, SPLIT, close, dev, host, inputs, ints, on_device, rng_of, rows_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def launched(timer):
    return {k for k, n in timer.launches.items() if n}


def agree(a, b):
    """Two ways through the same bf16 prompt: each within the bounds of its own arithmetic, about 2^-7 of the output's size
    (operands and outputs of 2^-9 each) and 2^-14 of the state's."""
    (y, h), (y2, h2) = a, b
    assert float((y.float() - y2.float()).norm()) <= 2.0 ** -7 * float(y2.float().norm())
    assert float((h - h2).norm()) <= 2.0 ** -14 * float(h2.norm())
    assert not bool(y.isnan().any()) and not bool(h.isnan().any())


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("how", ["tokens first", "batch of one row", "same tensor", "wide", "odd"])
def test_strides(how, N):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H = 3, 150, 4, 2, 64
    s = inputs(rng_of("strides", how, N), b, L, nh, G, H, N, "bf16")
    if how == "batch of one row":
        for k in ("q", "k", "v", "dt", "beta"):
            s[k][:] = s[k][:1]
    if how == "same tensor":
        s["q"] = s["k"]
    t = on_device(s, "bf16")
    chunks = True
    if how == "tokens first":  # [L, b, ...] in memory
        t = {k: v.transpose(0, 1).contiguous().transpose(0, 1) if v.dim() > 1 else v for k, v in t.items()}
    elif how == "batch of one row":
        t = {k: v[:1].expand(b, *v.shape[1:]) if v.dim() > 1 else v for k, v in t.items()}
        chunks = False  # rows on one another
    elif how == "same tensor":
        t["q"] = t["k"]
    else:
        pad, c = (8, True) if how == "wide" else (1, False)
        t, chunks = on_device(s, "bf16", pad), c
    y_ref, ey, h_ref, eh = od.delta(**s, split=SPLIT, out=OUT)
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**t, h0=dev(s["h0"]))
    assert launched(timer) == ({"delta_prepare", "delta_chain"} if chunks else {"delta"})
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("heads", [(4, 4), (8, 1), (6, 1), (10, 2)])
def test_heads_of_a_group(heads):
    """As many heads as groups, and more of a group than a CTA takes at once."""
    import selective_state_space_mamba_gb300 as ssm
    nh, G = heads
    s = inputs(rng_of("heads", heads), 2, 100, nh, G, 24, 64, "bf16")
    y_ref, ey, h_ref, eh = od.delta(**s, split=SPLIT, out=OUT)
    y, h = ssm.delta_fwd(**on_device(s, "bf16"), h0=dev(s["h0"]))
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("shift", [1, 2])
def test_states_and_outputs_off_16_bytes(shift):
    """h0 and h_final may start at any float; a y off 16 bytes goes token by token."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("off", shift), 2, 140, 2, 1, 64, 128, "bf16")
    t = on_device(s, "bf16")
    want = ssm.delta_fwd(**t, h0=dev(s["h0"]))
    h0, h = (torch.full((s["h0"].size + shift,), float("nan"), device="cuda")[shift:].view(s["h0"].shape) for _ in range(2))
    h0.copy_(dev(s["h0"]))
    got = ssm.delta_fwd(**t, h0=h0, h_final=h)
    assert torch.equal(got[0], want[0]) and got[1] is h and torch.equal(h, want[1])
    y = torch.empty(want[0].numel() + shift, device="cuda", dtype=torch.bfloat16)[shift:].view(want[0].shape)
    agree(ssm.delta_fwd(**t, h0=dev(s["h0"]), y=y), want)


def test_segments():
    """More chunks than the workspace holds records of: the states go from segment to segment.  Two sequences' heads against
    the definition, all of them against the prompt token by token (odd rows)."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N = 40, 2200, 32, 16, 64, 64
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.nn.functional.silu(torch.randn(s, device="cuda", generator=g)).bfloat16()  # noqa: E731
    q, k, v, dt, beta = r(b, L, G, N), r(b, L, G, N), r(b, L, nh, H), r(b, L, nh), r(b, L, nh)
    A, h0 = -torch.rand(nh, device="cuda", generator=g), 0.3 * torch.randn(b, nh, H, N, device="cuda", generator=g)
    lens = torch.randint(0, L + 1, (b,), device="cuda", generator=g).int()
    lens[0], lens[39] = L, 2048  # the end of the first segment
    with ssm.KernelTimer() as timer:
        got = ssm.delta_fwd(q, k, v, dt, beta, A, None, h0, lens)
    assert timer.launches["delta_chain"] == 2
    odd = torch.empty(b, L, G * N + 1, device="cuda", dtype=torch.bfloat16)[..., 1:].unflatten(-1, (G, N))
    odd.copy_(q)
    with ssm.KernelTimer() as timer:
        tokens = ssm.delta_fwd(odd, k, v, dt, beta, A, None, h0, lens)
    assert launched(timer) == {"delta"}
    agree(got, tokens)
    for i in (0, 39):
        part = [host(x[i : i + 1, :, :1]) for x in (q, k)] + [host(x[i : i + 1, :, :2]) for x in (v, dt, beta)]
        y_ref, ey, h_ref, eh = od.delta(*part, host(A[:2]), None, host(h0[i : i + 1, :2]), [int(lens[i])], split=SPLIT, out=OUT)
        close(host(got[0][i : i + 1, :, :2]), y_ref, ey, "y", "bf16")
        rows_close(host(got[1][i : i + 1, :2]), h_ref, eh, "h")


def test_offsets_beyond_32_bits():
    """v and y of 2^31 elements and more, in segments; the end of the prompt against a call of its own."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    L, nh, H, N, tail = (1 << 19) + 37, 64, 64, 64, 5000
    g = torch.Generator("cuda").manual_seed(4)
    r = lambda *s: torch.randn(s, device="cuda", generator=g, dtype=torch.bfloat16)  # noqa: E731
    a = [r(1, L, 1, N), r(1, L, 1, N), r(1, L, nh, H), r(1, L, nh), r(1, L, nh)]
    A = -0.1 * torch.rand(nh, device="cuda", generator=g)
    whole = ssm.delta_fwd(*a, A)
    head = [x[:, : L - tail] for x in a]
    _, h = ssm.delta_fwd(*head, A)
    agree(ssm.delta_fwd(*[x[:, L - tail :] for x in a], A, h0=h), (whole[0][:, L - tail :], whole[1]))
    # token by token, from the same state
    odd = torch.empty(1, tail, 1, N + 1, device="cuda", dtype=torch.bfloat16)[..., 1:]
    odd.copy_(a[0][:, L - tail :])
    agree(ssm.delta_fwd(odd, *[x[:, L - tail :] for x in a[1:]], A, h0=h), (whole[0][:, L - tail :], whole[1]))
    del whole, head
    # states of 2^31 elements and more, a step
    n = (1 << 31) // (nh * 128 * 128) + 3
    state = torch.zeros(n, nh, 128, 128, device="cuda")
    slots = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    x = [r(2, 1, 128), r(2, 1, 128), r(2, nh, 128), r(2, nh), r(2, nh)]
    y, _ = ssm.delta_step(*x, A, state=state, slots=slots, inplace=True)
    y2, h2 = ssm.delta_step(*x, A)
    assert torch.equal(y, y2) and torch.equal(state[n - 1], h2[0]) and torch.equal(state[0], h2[1])
    assert not bool(state[1 : n - 1].any())


def test_workspace_of_the_caller():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("workspace"), 1, 300, 2, 1, 64, 128, "bf16")
    t = on_device(s, "bf16")
    want = ssm.delta_fwd(**t)
    ws = ssm.Workspace("cuda")
    need = ssm.delta_fwd_workspace_bytes(1, 300, 2, 64, 128, 1)
    assert need > 0
    ws.ensure(need)
    ws.buf.fill_(0xff)  # it may hold anything
    got = ssm.delta_fwd(**t, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ssm.check_device_status(ws) == 0
    with pytest.raises(ValueError, match="workspace"):
        from selective_state_space_mamba_gb300 import _layer
        _layer._load().delta_fwd(*t.values(), None, None, None, True, True, True, None, None, True, ws.buf.cpu())


def test_two_streams_at_once():
    """Calls without a workspace on two streams, and a captured one beside an eager one."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    ts = [on_device(inputs(rng_of("two", i), 2, 1000, 4, 2, 64, 128, "bf16"), "bf16") for i in range(2)]
    want = [ssm.delta_fwd(**t) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for st, t in zip(streams, ts):
            with torch.cuda.stream(st):
                got.append(ssm.delta_fwd(**t))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = ssm.delta_fwd(**ts[0])
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            eager = ssm.delta_fwd(**ts[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0][0]) and torch.equal(eager[0], want[1][0]) and torch.equal(eager[1], want[1][1])


@pytest.mark.parametrize("pieces", [False, True])
@pytest.mark.parametrize("where", ["prepare", "chain"])
def test_waits_that_run_out(where, pieces):
    """A CTA that gives up: its outputs are NaN, the others right, and the status says so; the next call is right again."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    lib = _lib.load()
    L = 3000 if pieces else 300
    s = inputs(rng_of("waits", where, pieces), 1, L, 2, 2, 64, 128, "bf16")
    t = on_device(s, "bf16")
    ws = ssm.Workspace("cuda")
    want = ssm.delta_fwd(**t, workspace=ws)
    assert ssm.check_device_status(ws) == 0
    # CTA 0 of the kernel that prepares the chunks has the first head's first; CTA 0 of the chains is of the first head
    lib.ssm_debug_set_lookback_fault(0 if where == "prepare" else 1 << 40, 5_000_000)
    try:
        y, h = ssm.delta_fwd(**t, workspace=ws)
        torch.cuda.synchronize()
    finally:
        lib.ssm_debug_set_lookback_fault(-1, 0)
    assert ssm.check_device_status(ws) == _lib.SSM_ERR_TIMEOUT
    assert torch.equal(y[:, :, 1], want[0][:, :, 1]) and torch.equal(h[:, 1], want[1][:, 1])
    assert bool(y[:, :, 0].isnan().any()) and bool(h[:, 0].isnan().all())
    ok = ~y[:, :, 0].isnan()
    assert torch.equal(y[:, :, 0][ok], want[0][:, :, 0][ok])
    again = ssm.delta_fwd(**t, workspace=ws)
    assert ssm.check_device_status(ws) == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
