"""Ways through the layer operators that the other tests do not take: queues of every state size and of several groups,
split time axes with a queue, bounds without room for a split where nothing is split, and sentinels around every output
and workspace."""
import numpy as np
import pytest

from oracle import layer as ol
from test_guards_gpu import Guarded
from test_layer_gpu import SCAN, close, dev, host, ints, norm_inputs, rng_of, rounded, run_scan, scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def some_of(r, d, G, each):
    """Channels of every group, `each` of it."""
    per = d // G
    return np.concatenate([g * per + np.sort(r.choice(per, each, replace=False)) for g in range(G)])


def against_the_definition(case, dtype, lens, pieces, step):
    """A scan of many chains: some of its channels against the definition and, without a split, bit for bit what the
    same tokens give in calls of `step` tokens."""
    b, L, d, N, G, pad = case
    r = rng_of("cover", case, dtype, lens)
    inp = scan_inputs(r, (b, L), d, N, G, dtype)
    h0 = (0.3 * r.standard_normal((b, d, N))).astype(np.float32)
    bs, cs = np.unique([0, b // 2, b - 1]), some_of(r, d, G, 12)
    sub = {k: (v[cs] if k in ("A", "D", "dt_bias") else v[bs] if k in ("B", "C") else v[bs][..., cs]) for k, v in inp.items()}
    some = None if lens is None else [lens[i] for i in bs]
    y_ref, ey, h_ref, eh = ol.selscan(**sub, h0=h0[bs][:, cs], lens=some, pieces=pieces)
    if lens is not None:
        for i, n in enumerate(lens):
            for k in ("u", "dt", "B", "C", "z"):
                inp[k][i, n:] = np.nan
    y, h = run_scan(inp, dtype, pad, h0, lens)
    close(host(h)[bs][:, cs], h_ref, eh, "h")
    close(host(y)[bs][..., cs], y_ref, ey, "y", dtype)
    if step == 0:
        return
    state, parts = h0, []
    for t0 in range(0, L, step):
        p = {k: (v[:, t0 : t0 + step] if k in ("u", "dt", "B", "C", "z") else v) for k, v in inp.items()}
        n = None if lens is None else [min(max(m - t0, 0), step) for m in lens]
        part, state = run_scan(p, dtype, pad, state, n)
        parts.append(host(part))
        state = host(state)
    assert np.array_equal(np.concatenate(parts, 1), host(y)) and np.array_equal(state, host(h))


QUEUES = [  # b, L, d, N, G, pad: chains a little over the SMs, and over two a SM
    (7, 1100, 1472, 8, 1, 0), (13, 1100, 1600, 8, 2, 0), (7, 1100, 736, 32, 1, 8), (13, 1060, 800, 32, 1, 0),
    (7, 1100, 368, 64, 1, 0), (13, 1060, 400, 64, 2, 8), (13, 1060, 1536, 16, 3, 0),
    (7, 1100, 1471, 8, 1, 0), (13, 1060, 390, 64, 2, 1), (13, 1060, 1580, 16, 2, 3),  # rows that are not aligned
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_lens", [False, True])
@pytest.mark.parametrize("case", QUEUES, ids=str)
def test_queue_of_every_state_size(case, with_lens, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, N, G, _ = case
    assert ssm.selscan_fwd_workspace_bytes(b, L, d, N, G) > 0
    lens = [max(0, L - 97 * i) for i in range(b)] if with_lens else None
    against_the_definition(case, dtype, lens, 1, 256)


SPLIT_QUEUES = [(1, 9600, 1280, 16, 1, 0), (1, 9600, 1280, 8, 1, 8), (2, 9700, 320, 32, 2, 0), (1, 9600, 320, 64, 1, 0),
                (1, 9600, 1279, 16, 1, 0), (2, 9611, 318, 64, 3, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_lens", [False, True])
@pytest.mark.parametrize("case", SPLIT_QUEUES, ids=str)
def test_split_time_axis_with_a_queue(case, with_lens, dtype):
    """Parts of about 600 tokens, each of several items; a last sequence that ends in an earlier part."""
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, N, G, _ = case
    # a state of every chain's scan threads lies in the workspace where there is a queue
    assert ssm.selscan_fwd_workspace_bytes(b, L, d, N, G) > 300 * 128 * 8 * 4
    lens = [L - 5 - 3333 * (b - 1 - i) for i in range(b)] if with_lens else None
    against_the_definition(case, dtype, lens, 700, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_prompt_within_the_bound_of_its_way(case, dtype):
    """As test_selscan_prompt, with no room for a sum of delta where the time axis is not split."""
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, N, G, pad, has_h0, lens, has_z, has_bias = case
    if ssm.selscan_fwd_workspace_bytes(b, L, d, N, G) > 0:
        pieces = L // 2  # two parts at least
    else:
        pieces = 1
    r = rng_of("bound", case, dtype)
    inp = scan_inputs(r, (b, L), d, N, G, dtype)
    if not has_z:
        inp["z"] = None
    if not has_bias:
        inp["dt_bias"] = inp["D"] = None
    h0 = (0.3 * r.standard_normal((b, d, N))).astype(np.float32) if has_h0 else None
    y_ref, ey, h_ref, eh = ol.selscan(**inp, h0=h0, lens=lens, pieces=pieces)
    y, h = run_scan(inp, dtype, pad, h0, lens)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref, ey, "y", dtype)


# ------------------------------------------------------------------------------ sentinels

def guarded(shape, dtype):
    """(Guarded, its middle as a tensor)."""
    import torch
    t = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[dtype]
    g = Guarded(int(np.prod(shape)) * t.itemsize)
    return g, g.view(t, shape)


def checked(**guards):
    for name, g in guards.items():
        g.check(name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 5, 2), (2, 33, 130, 3), (3, 70, 257, 4), (1, 301, 1792, 4), (2, 129, 1001, 4)], ids=str)
def test_conv_outputs_guarded(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, W = case
    r = rng_of("guard conv", case, dtype)
    x, w = rounded(r.standard_normal((b, L, d)), dtype), r.standard_normal((d, W)).astype(np.float32)
    state = rounded(r.standard_normal((b, W - 1, d)), dtype)
    lens = [L] + [max(0, L - 17 * i) for i in range(1, b)]
    y_ref, err, s_ref = ol.conv(x, w, None, state, lens)
    gy, y = guarded((b, L, d), dtype)
    gs, s = guarded((b, W - 1, d), dtype)
    ssm.conv_fwd(dev(x, dtype), dev(w), None, dev(state, dtype), ints(lens), y=y, state_out=s)
    checked(y=gy, state=gs)
    close(host(y), y_ref, err, "y", dtype)
    assert np.array_equal(host(s), s_ref)
    y_ref, err, s_ref = ol.conv(x[:, :1], w, None, state)
    gy, y = guarded((b, d), dtype)
    gs, s = guarded((b, W - 1, d), dtype)
    ssm.conv_step(dev(x[:, 0], dtype), dev(w), None, dev(state, dtype), y=y, state_out=s)
    checked(y=gy, state=gs)
    close(host(y), y_ref[:, 0], err[:, 0], "y", dtype)
    assert np.array_equal(host(s), s_ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [
    (1, 1, 1, 8, 1), (2, 33, 40, 16, 1), (2, 70, 73, 16, 1), (3, 50, 72, 32, 3), (2, 47, 36, 64, 2), (1, 400, 24, 8, 1),
    (1, 700, 65, 16, 1), (7, 1060, 1472, 16, 1), (13, 1060, 390, 64, 2)], ids=str)
def test_selscan_outputs_and_workspace_guarded(case, dtype):
    """Twice with one workspace of exactly the bytes that are asked for."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, N, G = case
    inp = scan_inputs(rng_of("guard scan", case, dtype), (b, L), d, N, G, dtype)
    need = ssm.selscan_fwd_workspace_bytes(b, L, d, N, G)
    gw = Guarded(need)

    class Exact:
        def ensure(self, nbytes):
            assert nbytes == need
            return gw.view(torch.uint8, (need,))

    lens = [L] + [max(0, L - 17 * i) for i in range(1, b)]
    want = run_scan(inp, dtype, 0, None, lens)
    for _ in range(2):
        gy, y = guarded((b, L, d), dtype)
        gh, h = guarded((b, d, N), "f32")
        run_scan(inp, dtype, 0, None, lens, y=y, h_final=h, workspace=Exact())
        checked(y=gy, h_final=gh, workspace=gw)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 8, 1), (3, 33, 16, 1), (5, 72, 32, 2), (2, 30, 64, 3), (81, 2050, 16, 1), (40, 4104, 8, 2)], ids=str)
def test_selscan_step_outputs_guarded(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, d, N, G = case
    r = rng_of("guard step", case, dtype)
    inp = scan_inputs(r, (b,), d, N, G, dtype)
    state = (0.3 * r.standard_normal((b, d, N))).astype(np.float32)
    one = {k: (v if k in ("A", "D", "dt_bias") else v[:, None]) for k, v in inp.items()}
    y_ref, ey, h_ref, eh = ol.selscan(**one, h0=state)
    gy, y = guarded((b, d), dtype)
    gh, h = guarded((b, d, N), "f32")
    ssm.selscan_step(dev(inp["u"], dtype), dev(inp["dt"], dtype), dev(inp["A"]), dev(inp["B"], dtype), dev(inp["C"], dtype),
                     dev(inp["D"]), dev(inp["z"], dtype), dev(inp["dt_bias"]), dev(state), y=y, state_out=h)
    checked(y=gy, state=gh)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref[:, 0], ey[:, 0], "y", dtype)


@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", [(1, 1), (3, 257), (2, 2560), (613, 100), (613, 257), (613, 1031), (610, 2561), (609, 10248), (2, 16391)],
                         ids=str)
def test_rmsnorm_outputs_guarded(shape, dtype, res):
    import selective_state_space_mamba_gb300 as ssm
    rows, d = shape
    x, w, residual = norm_inputs("guard", rows, d, dtype, res)
    v, err, r = ol.rmsnorm(x, w, residual)
    xr, gr, ro = dev(x, dtype), None, None
    gy, y = guarded((rows, d), dtype)
    if residual is not None:
        gr, ro = guarded((rows, d), res)
    ssm.rmsnorm_fwd(xr, dev(w), dev(residual, res), y=y, residual_out=ro)
    gy.check("y")
    close(host(y), v, err, "y", dtype)
    if gr:
        gr.check("residual_out")
        close(host(ro), r, ol.U * np.abs(r), "residual", res)
    for group in (0, 128):
        gq, q = guarded((rows, d), "e4m3")
        gs, s = guarded((rows, -(-d // 128)) if group else (rows,), "f32")
        if residual is not None:
            gr, ro = guarded((rows, d), res)
        ssm.rmsnorm_fp8_fwd(xr, dev(w), dev(residual, res), group=group, q=q, scale=s, residual_out=ro)
        checked(q=gq, scale=gs)
        if gr:
            gr.check("residual_out")
        each = np.repeat(host(s).reshape(rows, -1), group or d, axis=1)[:, :d]
        close(host(q) * each, v, err + 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * each + 4 * ol.U * np.abs(v), f"q {group}")
