"""GPU tests of the gated delta rule: how far a NaN or an infinity reaches, gates that are infinite, decays above 1, and long
prompts token by token."""
import numpy as np
import pytest

from oracle import delta as od
from test_delta_gpu import OUT, SPLIT, close, dev, host, inputs, on_device, rng_of, rows_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


# way: b, L, nh, G, H, N, type, the token with the value; the kernels
WAYS = {
    "tokens f32": ((2, 200, 4, 2, 40, 64), "f32", 101, {"delta"}),
    "tokens, many heads": ((11, 130, 8, 4, 64, 128), "f32", 77, {"delta"}),
    "tokens bf16": ((2, 60, 4, 2, 40, 128), "bf16", 33, {"delta"}),
    "tokens of 32 columns": ((2, 200, 4, 2, 40, 32), "bf16", 101, {"delta"}),
    "chunks": ((2, 300, 4, 2, 72, 128), "bf16", 140, {"delta_prepare", "delta_chain"}),
    "chunks of 64 columns": ((2, 300, 4, 2, 128, 64), "bf16", 140, {"delta_prepare", "delta_chain"}),
    "pairs": ((3, 200, 60, 10, 64, 128), "bf16", 90, {"delta_prepare", "delta_chain"}),
    "pairs of 64 columns": ((3, 200, 60, 10, 56, 64), "bf16", 90, {"delta_prepare", "delta_chain"}),
    "pieces": ((1, 2700, 2, 2, 64, 128), "bf16", 1000, {"delta_prepare", "delta_states", "delta_join", "delta_chain"}),
}


def launched(timer):
    return {k for k, n in timer.launches.items() if n}


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("of,value", [("q", NAN), ("k", NAN), ("v", NAN), ("dt", NAN), ("beta", NAN), ("q", INF), ("k", INF), ("v", INF)])
@pytest.mark.parametrize("way", WAYS)
def test_reach_of_a_value(way, of, value):
    """One NaN or infinity: everything that it does not enter by the definition is as without it, to the last bit, except, in chunks,
    the tokens before it in its chunk, of its heads (of v: its row).  A NaN in q spoils its token alone; in the others
    everything from its token on."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    (b, L, nh, G, H, N), dtype, at, kernels = WAYS[way]
    s = inputs(rng_of("reach", way), b, L, nh, G, H, N, dtype, slow=True)
    t, h0 = on_device(s, dtype), dev(s["h0"])
    want = ssm.delta_fwd(**t, h0=h0)
    t[of] = t[of].clone()
    i, g, row = b - 1, G - 1, 5
    heads = torch.zeros(nh, dtype=torch.bool, device="cuda")
    if of in "qk":
        t[of][i, at, g, 3] = value
        heads[g * (nh // G):] = True
    else:
        t[of][(i, at, nh - 1, row) if of == "v" else (i, at, nh - 1)] = value
        heads[-1] = True
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**t, h0=h0)
    assert launched(timer) == kernels
    touched = torch.zeros_like(y, dtype=torch.bool)
    start = at if kernels == {"delta"} else at // 64 * 64
    stop = at + 1 if of == "q" else L
    rows = slice(row, row + 1) if of == "v" else slice(0, H)
    touched[i, start:stop, heads, rows] = True
    assert torch.equal(y[~touched], want[0][~touched])
    assert not torch.isfinite(y[i, at:stop, heads, rows]).any()
    touched_h = torch.zeros_like(h, dtype=torch.bool)
    if of != "q":
        touched_h[i, heads, rows] = True
        assert not torch.isfinite(h[touched_h]).any()
    assert torch.equal(h[~touched_h], want[1][~touched_h])


@pytest.mark.parametrize("way", WAYS)
def test_infinite_gates_are_their_limits(way):
    """dt of +-infinity: no state left, no decay; beta of +-infinity: 1 and 0.  As with values that are large enough."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    (b, L, nh, G, H, N), dtype, at, _ = WAYS[way]
    s = inputs(rng_of("infinite gates", way), b, L, nh, G, H, N, dtype)
    got = []
    for big in (1e30, INF):
        t = on_device(s, dtype)
        for i, (k, sign) in enumerate((k, sign) for k in ("dt", "beta") for sign in (1, -1)):
            t[k][:, at + 3 * i :: 50] = sign * big
        got.append(ssm.delta_fwd(**t, h0=dev(s["h0"])))
    assert torch.isfinite(got[1][0]).all() and torch.isfinite(got[1][1]).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# Decays above 1 do not change the bound: an error that a row has is carried on with a factor of at most a token's decay, and what
# an evaluation in chunks adds goes by the largest |v| + a |S| so far.
GROWTH = [  # b, L, nh, G, H, N, lowest and highest dt (A is 1)
    (2, 200, 4, 2, 64, 128, -0.1, 0.3), (2, 80, 4, 2, 64, 64, 0.6, 1.1), (3, 150, 60, 10, 48, 64, -0.2, 0.5),
    (1, 2700, 2, 1, 64, 128, -0.01, 0.012), (11, 70, 4, 4, 128, 128, 0.7, 1.2),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("case", GROWTH, ids=str)
def test_decays_above_one(case, negative, dtype):
    """A > 0, or a negative dt without the softplus."""
    import selective_state_space_mamba_gb300 as ssm
    from test_delta_gpu import rounded
    b, L, nh, G, H, N, low, high = case
    r = rng_of("growth", case, dtype)
    s = inputs(r, b, L, nh, G, H, N, dtype, bias=False)
    s["dt"] = rounded((-1 if negative else 1) * r.uniform(low, high, s["dt"].shape), dtype)
    s["A"] = np.full(nh, -1.0 if negative else 1.0, np.float32)
    y_ref, ey, h_ref, eh = od.delta(**s, softplus=False, **(dict(split=SPLIT, out=OUT) if dtype == "bf16" else {}))
    y, h = ssm.delta_fwd(**on_device(s, dtype), h0=dev(s["h0"]), softplus=False)
    close(host(y), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")


LONG = [  # b, L, nh, G, H, N, type
    (1, 3001, 2, 1, 40, 128, "f32"), (5, 1100, 16, 4, 64, 64, "f32"), (5, 777, 16, 4, 64, 128, "f32"), (2, 1500, 4, 2, 24, 32, "f32"),
    (2, 1500, 4, 2, 24, 32, "bf16"), (1, 2003, 2, 1, 41, 64, "bf16"),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_prompts_token_by_token(case):
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N, dtype = case
    s = inputs(rng_of("long", case), b, L, nh, G, H, N, dtype, slow=True)
    y_ref, ey, h_ref, eh = od.delta(**s)
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**on_device(s, dtype), h0=dev(s["h0"]))
    assert launched(timer) == {"delta"}
    close(host(y), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")


# What test_delta_gpu.py has of options, heads of a group, and chunks of fewer than 64 tokens, at lengths that go in chunks.
@pytest.mark.parametrize("options", [dict(softplus=False), dict(sigmoid=False), dict(l2norm=False), dict(scale=0.7),
                                     dict(softplus=False, sigmoid=False, l2norm=False, scale=-2.0)], ids=str)
def test_options_in_chunks(options):
    import selective_state_space_mamba_gb300 as ssm
    from test_delta_gpu import rounded
    r = rng_of("options in chunks", options)
    s = inputs(r, 2, 150, 2, 1, 64, 128, "bf16", bias=False)
    if not options.get("softplus", True):
        s["dt"] = np.abs(s["dt"]) * 0.125
    if not options.get("sigmoid", True):
        s["beta"] = rounded(r.uniform(0, 1, s["beta"].shape), "bf16")
    if not options.get("l2norm", True):  # lengths below 1
        s["q"], s["k"] = (rounded(v / (1.01 * np.linalg.norm(v, axis=-1, keepdims=True)), "bf16") for v in (s["q"], s["k"]))
    y_ref, ey, h_ref, eh = od.delta(**s, **options, split=SPLIT, out=OUT)
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**on_device(s, "bf16"), h0=dev(s["h0"]), **options)
    assert launched(timer) == {"delta_prepare", "delta_chain"}
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


CHUNKS = [  # b, L, nh, G, H, N, lens
    (2, 120, 4, 4, 24, 64, None), (2, 120, 8, 1, 24, 64, None), (2, 113, 6, 1, 24, 64, [112, 65]), (2, 127, 10, 2, 24, 64, None),
    (64, 24, 64, 16, 8, 64, None), (32, 33, 128, 8, 8, 64, [33, 1, 32, 31, 0, 16, 17, 33] * 4), (8, 56, 40, 4, 8, 128, [56, 1, 0, 55, 33, 32, 16, 2]),
    (16, 40, 16, 2, 64, 128, [40, 1, 0, 39, 33, 32, 16, 2] * 2),
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: str(c[:6]))
def test_short_prompts_in_chunks(case):
    import selective_state_space_mamba_gb300 as ssm
    from test_delta_gpu import ints
    b, L, nh, G, H, N, lens = case
    s = inputs(rng_of("short", case), b, L, nh, G, H, N, "bf16")
    y_ref, ey, h_ref, eh = od.delta(**s, lens=lens, split=SPLIT, out=OUT)
    if lens is not None:  # padding may hold anything
        for i, n in enumerate(od._lens(lens, b, L)):
            for k in ("q", "k", "v", "dt", "beta"):
                s[k][i, n:] = np.nan
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**on_device(s, "bf16"), h0=dev(s["h0"]), lens=ints(lens))
    assert launched(timer) == {"delta_prepare", "delta_chain"}
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


def test_a_token_before_chunks():
    """The last length that goes token by token."""
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("before chunks"), 2, 111, 4, 2, 24, 64, "bf16")
    y_ref, ey, h_ref, eh = od.delta(**s)
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**on_device(s, "bf16"), h0=dev(s["h0"]))
    assert launched(timer) == {"delta"}
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")
