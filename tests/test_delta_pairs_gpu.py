"""GPU tests of the gated delta rule where a CTA runs two chains of up to 64 rows: more heads than SMs, and long chains whose
pieces are more."""
import numpy as np
import pytest

from oracle import delta as od
from test_delta_gpu import OUT, SPLIT, close, dev, host, inputs, ints, on_device, rng_of, rows_close
from test_delta_paths_gpu import agree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


CASES = [  # b, L, nh, G, H, N, h0, lens
    (5, 130, 33, 3, 64, 128, True, [130, 0, 64, 129, 200]),  # an odd number of chains
    (5, 193, 33, 33, 40, 64, True, None),
    (3, 72, 60, 4, 8, 128, False, None),
    (2, 321, 80, 8, 64, 64, True, [1, 320]),
    (4, 66, 64, 8, 56, 128, True, [66, 65, 0, 2]),           # neighbours of unequal lengths
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(case):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N, h0, lens = case
    s = inputs(rng_of("pairs", case), b, L, nh, G, H, N, "bf16", h0)
    y_ref, ey, h_ref, eh = od.delta(**s, lens=lens, split=SPLIT, out=OUT)
    if lens is not None:
        for i, n in enumerate(od._lens(lens, b, L)):
            for k in ("q", "k", "v", "dt", "beta"):
                s[k][i, n:] = np.nan
    t = on_device(s, "bf16")
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**t, h0=dev(s["h0"]), lens=ints(lens))
    assert timer.launches["delta_chain"] == 1
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")
    y2, none = ssm.delta_fwd(**t, h0=dev(s["h0"]), lens=ints(lens), return_final_state=False)
    assert none is None and torch.equal(y2, y)


@pytest.mark.parametrize("sizes", [(8, 2048, 24, 8, 64, 128), (1, 8192, 24, 24, 64, 128), (2, 8192, 32, 8, 64, 64), (1, 4096, 160, 5, 32, 128)],
                         ids=str)
def test_heads_by_themselves(sizes):
    """The same heads one group at a time, a chain in a CTA (whole or in other pieces); and repeats are equal."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N = sizes
    t = on_device(inputs(rng_of("alone", sizes), b, L, nh, G, H, N, "bf16", h0=False, slow=True), "bf16")
    y, h = ssm.delta_fwd(**t)
    for _ in range(5):
        y2, h2 = ssm.delta_fwd(**t)
        assert torch.equal(y, y2) and torch.equal(h, h2)
    for i, g in ((0, 0), (b - 1, G - 1)):
        of = slice(g * (nh // G), (g + 1) * (nh // G))
        part = dict(q=t["q"][i:i + 1, :, g:g + 1], k=t["k"][i:i + 1, :, g:g + 1], v=t["v"][i:i + 1, :, of],
                    dt=t["dt"][i:i + 1, :, of], beta=t["beta"][i:i + 1, :, of], A=t["A"][of], dt_bias=t["dt_bias"][of])
        agree((y[i:i + 1, :, of], h[i:i + 1, of]), ssm.delta_fwd(**part))


@pytest.mark.parametrize("pieces", [False, True])
def test_waits_that_run_out(pieces):
    """A CTA that gives up: the outputs of its two chains are NaN, those of the other heads right."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    lib = _lib.load()
    L, nh = (8192, 24) if pieces else (300, 160)
    t = on_device(inputs(rng_of("waits of pairs", pieces), 1, L, nh, 8, 64, 128, "bf16"), "bf16")
    ws = ssm.Workspace("cuda")
    want = ssm.delta_fwd(**t, workspace=ws)
    assert ssm.check_device_status(ws) == 0
    lib.ssm_debug_set_lookback_fault(1 << 40, 5_000_000)
    try:
        y, h = ssm.delta_fwd(**t, workspace=ws)
        torch.cuda.synchronize()
    finally:
        lib.ssm_debug_set_lookback_fault(-1, 0)
    assert ssm.check_device_status(ws) == _lib.SSM_ERR_TIMEOUT
    lost = y.isnan().any(dim=3).any(dim=1)[0]
    assert bool(lost[0]) and int(lost.sum()) == (1 if pieces else 2)
    assert torch.equal(y[:, :, ~lost], want[0][:, :, ~lost]) and torch.equal(h[:, ~lost], want[1][:, ~lost])
    ok = ~y.isnan()
    assert torch.equal(y[ok], want[0][ok])
    again = ssm.delta_fwd(**t, workspace=ws)
    assert ssm.check_device_status(ws) == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
