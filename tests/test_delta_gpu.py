"""GPU parity of the gated delta rule (prompts and single tokens) against the float64 definition in
oracle/delta.py.

Every element is held to the bound that oracle/delta.py derives from the arithmetic; a bf16 output may be off by
2^-8 of its value besides.  NaN stands in every place that a call must not read: padding, unused slots, columns
beside a strided tensor.

bf16 prompts of states of 64 and 128 may go through the tensor cores in chunks of 64 tokens: operands in f32 are split
into two bf16 halves, each half a rounding of at most 2^-9, together 2^-18 (SPLIT), and the operands of the
output's sums are rounded once to bf16, 2^-9 each for the weights and the corrections (OUT, their root sum of squares).
"""
import zlib

import numpy as np
import pytest

from oracle import delta as od

pytestmark = pytest.mark.gpu

SPLIT, OUT = 2.0 ** -18, 2.0 ** -8.5


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def rng_of(*key):
    return np.random.Generator(np.random.PCG64(zlib.crc32(repr(key).encode())))


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.array(a, dtype=np.float32, order="C")).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def ints(a):
    import torch
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def rounded(a, dtype):
    from selective_state_space_mamba_gb300 import synth
    a = np.ascontiguousarray(a, np.float32)
    return synth.round_to_bf16(a) if dtype == "bf16" else a


def strided(a, dtype, pad, tail=2):
    """A device tensor of a's values; its last `tail` dimensions lie in rows with `pad` columns of NaN on each side."""
    import torch
    if pad == 0:
        return dev(a, dtype)
    flat = a.reshape(*a.shape[:-tail], -1)
    wide = torch.full((*flat.shape[:-1], flat.shape[-1] + 2 * pad), float("nan"), device="cuda",
                      dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    wide[..., pad:-pad] = dev(flat, dtype)
    return wide[..., pad:-pad].unflatten(-1, a.shape[-tail:])


def close(got, ref, err, what, dtype="f32"):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    tol = err + 1e-30 + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[i] <= 0, f"{what}: {got[i]!r} for {ref[i]!r} at {i}, off by more than {np.broadcast_to(tol, ref.shape)[i]:.3e}"


def rows_close(got, ref, err, what):
    """Rows of a state: the 2-norm of the difference."""
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    over = np.linalg.norm(got - ref, axis=-1) - err - 1e-30
    i = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[i] <= 0, f"{what}: row {i} off by {np.linalg.norm((got - ref)[i]):.3e}, more than {err[i]:.3e}"


def inputs(r, b, L, nh, G, H, N, dtype, h0=True, bias=True, slow=False):
    silu = lambda x: x / (1 + np.exp(-x))  # noqa: E731
    s = {"q": rounded(silu(r.standard_normal((b, L, G, N))), dtype), "k": rounded(silu(r.standard_normal((b, L, G, N))), dtype),
         "v": rounded(silu(r.standard_normal((b, L, nh, H))), dtype), "dt": rounded(r.standard_normal((b, L, nh)), dtype),
         "beta": rounded(r.standard_normal((b, L, nh)), dtype),
         "A": (-np.exp(r.uniform(0, np.log(16.0), nh)) * (0.01 if slow else 1)).astype(np.float32),
         "dt_bias": r.uniform(-7, -2, nh).astype(np.float32) if bias else None,
         "h0": (0.3 * r.standard_normal((b, nh, H, N))).astype(np.float32) if h0 else None}
    return s


def on_device(s, dtype, pad=0):
    return dict(q=strided(s["q"], dtype, pad), k=strided(s["k"], dtype, pad), v=strided(s["v"], dtype, pad),
                dt=strided(s["dt"], dtype, pad, 1), beta=strided(s["beta"], dtype, pad, 1), A=dev(s["A"]),
                dt_bias=dev(s["dt_bias"]))


CASES = [  # b, L, nh, G, H, N, pad, h0, lens
    (1, 1, 1, 1, 8, 64, 0, False, None),
    (1, 1, 2, 2, 64, 128, 0, True, None),
    (2, 7, 3, 1, 5, 32, 0, True, None),
    (1, 64, 2, 1, 64, 128, 0, False, None),
    (1, 63, 2, 2, 128, 128, 0, True, None),
    (2, 65, 4, 2, 128, 64, 8, True, None),
    (3, 130, 2, 1, 96, 128, 0, True, [130, 0, 64]),
    (2, 200, 2, 2, 72, 64, 16, False, [1, 199]),
    (2, 97, 2, 1, 33, 128, 3, True, [200, -5]),          # odd rows; lengths outside 0 .. L are clamped
    (1, 300, 1, 1, 200, 128, 0, True, None),             # rows of more than one tile
    (1, 129, 3, 3, 16, 32, 1, False, None),
    (5, 128, 8, 4, 64, 64, 64, True, [128, 127, 65, 3, 0]),
    (2, 257, 6, 2, 128, 128, 0, False, [257, 192]),
    # heads enough that short prompts go in chunks too: one chunk and its ends
    (10, 33, 4, 2, 128, 128, 0, True, [33, 1, 32, 31, 0, 16, 17, 33, 33, 2]),
    (10, 63, 4, 4, 128, 64, 8, False, None),
    (10, 64, 4, 1, 128, 128, 0, True, [64, 63, 1, 64, 0, 65, 33, 32, 2, 64]),
    (11, 65, 4, 2, 120, 128, 0, True, [65, 64, 63, 1, 0, 65, 33, 32, 2, 64, 66]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N, pad, h0, lens = case
    s = inputs(rng_of("delta", case, dtype), b, L, nh, G, H, N, dtype, h0)
    y_ref, ey, h_ref, eh = od.delta(**s, lens=lens, **(dict(split=SPLIT, out=OUT) if dtype == "bf16" else {}))
    if lens is not None:  # padding may hold anything
        for i, n in enumerate(od._lens(lens, b, L)):
            for k in ("q", "k", "v", "dt", "beta"):
                s[k][i, n:] = np.nan
    t = on_device(s, dtype, pad)
    y, h = ssm.delta_fwd(**t, h0=dev(s["h0"]), lens=ints(lens))
    close(host(y), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")
    y2, none = ssm.delta_fwd(**t, h0=dev(s["h0"]), lens=ints(lens), return_final_state=False)
    assert none is None and np.array_equal(host(y2), host(y))


PIECES = [  # b, L, nh, G, H, N, h0, lens: few chains of many chunks, which are cut into pieces that run at once
    (1, 2661, 1, 1, 64, 128, True, None),
    (2, 2700, 2, 1, 128, 64, True, [2700, 700]),      # a length inside a piece, empty pieces behind it
    (3, 2624, 1, 1, 136, 128, False, [1, 2624, 0]),   # rows of two tiles
    (1, 4100, 3, 3, 72, 64, True, None),
]


@pytest.mark.parametrize("case", PIECES, ids=str)
def test_pieces(case):
    import selective_state_space_mamba_gb300 as ssm
    b, L, nh, G, H, N, h0, lens = case
    s = inputs(rng_of("pieces", case), b, L, nh, G, H, N, "bf16", h0, slow=True)
    y_ref, ey, h_ref, eh = od.delta(**s, lens=lens, split=SPLIT, out=OUT)
    if lens is not None:
        for i, n in enumerate(od._lens(lens, b, L)):
            for k in ("q", "k", "v", "dt", "beta"):
                s[k][i, n:] = np.nan
    t = on_device(s, "bf16")
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(**t, h0=dev(s["h0"]), lens=ints(lens))
    assert timer.launches["delta_states"] == 1
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("options", [dict(softplus=False), dict(sigmoid=False), dict(l2norm=False), dict(scale=0.7),
                                     dict(softplus=False, sigmoid=False, l2norm=False, scale=-2.0)], ids=str)
@pytest.mark.parametrize("step", [False, True])
def test_options(options, dtype, step):
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("options", options, dtype)
    s = inputs(r, 2, 100, 2, 1, 64, 128, dtype, bias=False)
    if not options.get("softplus", True):
        s["dt"] = np.abs(s["dt"]) * 0.125
    if not options.get("sigmoid", True):
        s["beta"] = rounded(r.uniform(0, 1, s["beta"].shape), dtype)
    if not options.get("l2norm", True):  # lengths below 1
        s["q"], s["k"] = (rounded(v / (1.01 * np.linalg.norm(v, axis=-1, keepdims=True)), dtype) for v in (s["q"], s["k"]))
    n = 1 if step else 100
    for k in ("q", "k", "v", "dt", "beta"):
        s[k] = s[k][:, :n]
    y_ref, ey, h_ref, eh = od.delta(**s, **options, **(dict(split=SPLIT, out=OUT) if dtype == "bf16" else {}))
    t = on_device(s, dtype)
    if step:
        t = {k: v[:, 0] if v is not None and v.dim() > 2 else v for k, v in t.items()}
        y, h = ssm.delta_step(**t, state=dev(s["h0"]), **options)
        y = y[:, None]
    else:
        y, h = ssm.delta_fwd(**t, h0=dev(s["h0"]), **options)
    close(host(y), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slow_and_fast_decays(dtype):
    """States that hardly decay (errors add up over the whole prompt), and heads that forget all of it in a token."""
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("decays", dtype), 1, 700, 4, 1, 64, 128, dtype, slow=True)
    s["A"][1], s["A"][2], s["A"][3] = -1e-6, -3e4, -3e38
    s["dt"][0, ::5, 2] = -60.0  # now and then no decay at all
    s["dt"][0, ::7, 3] = 60.0
    y_ref, ey, h_ref, eh = od.delta(**s, **(dict(split=SPLIT, out=OUT) if dtype == "bf16" else {}))
    y, h = ssm.delta_fwd(**on_device(s, dtype), h0=dev(s["h0"]))
    close(host(y), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("N", [64, 128])
def test_keys_that_repeat(N):
    """One key over and over, beta 1: each correction replaces what the key answered; the inverse has a row of -1s."""
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("repeat", N), 1, 192, 2, 1, 64, N, "bf16", slow=True)
    s["k"][:] = s["k"][:, :1]
    s["beta"][:] = 30.0
    y_ref, ey, h_ref, eh = od.delta(**s, split=SPLIT, out=OUT)
    y, h = ssm.delta_fwd(**on_device(s, "bf16"), h0=dev(s["h0"]))
    close(host(y), y_ref, ey, "y", "bf16")
    rows_close(host(h), h_ref, eh, "h")


STEPS = [  # b, nh, G, H, N, pad, slots, n
    (1, 1, 1, 1, 32, 0, None, 1), (3, 4, 2, 64, 128, 0, None, 3), (2, 2, 1, 33, 64, 1, None, 2),
    (5, 3, 3, 16, 128, 8, [6, -1, 0, 7, 3], 8), (4, 24, 24, 64, 128, 0, [2, 9, 1, 1 << 30], 4),
    (2, 2, 2, 130, 32, 3, [1, 0], 2), (3, 2, 1, 100, 64, 0, [-1, -1, 5], 5),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("case", STEPS, ids=str)
def test_step(case, dtype, shift):
    """shift: states that are not aligned to 16 bytes."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, nh, G, H, N, pad, slots, n = case
    r = rng_of("delta step", case, dtype)
    s = inputs(r, b, 1, nh, G, H, N, dtype, False)
    state = (0.3 * r.standard_normal((n, nh, H, N))).astype(np.float32)
    at = np.arange(b) if slots is None else np.asarray(slots)
    used = (at >= 0) & (at < n)
    part = {k: v[used] if k in ("q", "k", "v", "dt", "beta") else v for k, v in s.items()}
    y_ref, ey, h_new, eh = od.delta(**{**part, "h0": state[at[used]]})
    want, e, want_h, eh_all = np.zeros((b, nh, H)), np.zeros((b, nh, H)), state.astype(np.float64), np.zeros((n, nh, H))
    want[used], e[used], want_h[at[used]], eh_all[at[used]] = y_ref[:, 0], ey[:, 0], h_new, eh
    for k in ("q", "k", "v", "dt", "beta"):  # unused places may hold anything
        s[k][~used] = np.nan
    t = {k: v[:, 0] if v is not None and v.dim() > 1 else v for k, v in on_device(s, dtype, pad).items()}
    st = torch.empty(state.size + shift, device="cuda")[shift:].view(state.shape)
    st.copy_(dev(state))
    y, h = ssm.delta_step(**t, state=st, slots=ints(slots))
    close(host(y), want, e, "y", dtype)
    rows_close(host(h), want_h, eh_all, "state")
    assert np.array_equal(host(st), state)
    y2, h2 = ssm.delta_step(**t, state=st, slots=ints(slots), inplace=True)
    assert h2.data_ptr() == st.data_ptr() and np.array_equal(host(h2), host(h)) and np.array_equal(host(y2), host(y))


def test_step_from_zeros():
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("zeros"), 3, 1, 2, 1, 40, 64, "f32", False)
    y_ref, ey, h_ref, eh = od.delta(**s)
    t = {k: v[:, 0] if v is not None and v.dim() > 1 else v for k, v in on_device(s, "f32").items()}
    y, h = ssm.delta_step(**t)
    close(host(y)[:, None], y_ref, ey, "y")
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("dtype,L", [("f32", 90), ("bf16", 90), ("bf16", 200)])
def test_prompt_then_steps(dtype, L):
    """A prompt in two parts, then tokens one by one, against the whole."""
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("then", dtype, L), 2, L, 4, 2, 64, 128, dtype)
    y_ref, ey, h_ref, eh = od.delta(**s, **(dict(split=SPLIT, out=OUT) if dtype == "bf16" else {}))
    t = on_device(s, dtype)
    cut = lambda a, c: {k: v[:, a:c] if v is not None and v.dim() > 1 else v for k, v in t.items()}  # noqa: E731
    y1, h = ssm.delta_fwd(**cut(0, 70), h0=dev(s["h0"]))
    y2, h = ssm.delta_fwd(**cut(70, L - 3), h0=h)
    ys = [y1, y2]
    for i in range(L - 3, L):
        one = {k: v[:, i] if v is not None and v.dim() > 1 else v for k, v in t.items()}
        y, h = ssm.delta_step(**one, state=h, inplace=True)
        ys.append(y[:, None])
    import torch
    close(host(torch.cat(ys, 1)), y_ref, ey, "y", dtype)
    rows_close(host(h), h_ref, eh, "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_of_the_caller(dtype):
    """y, h_final and state_out given by the caller; no tokens at all; no sequences."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    s = inputs(rng_of("given", dtype), 2, 70, 2, 1, 64, 64, dtype)
    t = on_device(s, dtype)
    want_y, want_h = ssm.delta_fwd(**t, h0=dev(s["h0"]))
    y, h = torch.full_like(want_y, float("nan")), torch.full_like(want_h, float("nan"))
    got = ssm.delta_fwd(**t, h0=dev(s["h0"]), y=y, h_final=h)
    assert got[0] is y and got[1] is h and torch.equal(y, want_y) and torch.equal(h, want_h)
    none = {k: v[:, :0] if v is not None and v.dim() > 1 else v for k, v in t.items()}
    y, h = ssm.delta_fwd(**none, h0=dev(s["h0"]))
    assert y.shape == (2, 0, 2, 64) and np.array_equal(host(h), s["h0"])
    y, h = ssm.delta_fwd(**none)
    assert not host(h).any()
    y, h = ssm.delta_fwd(**{k: v[:0] if v is not None and v.dim() > 1 else v for k, v in t.items()})
    assert y.shape == (0, 70, 2, 64) and h.shape == (0, 2, 64, 64)


def test_h0_of_zeros_is_no_h0():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    for dtype in ("f32", "bf16"):
        t = on_device(inputs(rng_of("no h0"), 1, 100, 2, 1, 64, 128, dtype), dtype)
        a, b = ssm.delta_fwd(**t), ssm.delta_fwd(**t, h0=torch.zeros(1, 2, 64, 128, device="cuda"))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_and_streams(dtype):
    """A captured prompt and an in-place step, replayed with new inputs, on a stream of their own."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    first, second = (on_device(inputs(rng_of("graph", i), 2, 150, 4, 2, 64, 128, dtype), dtype) for i in (0, 1))
    state = torch.zeros(2, 4, 64, 128, device="cuda")

    def run(t, state):
        y, h = ssm.delta_fwd(**t)
        one = {k: v[:, 0] if v.dim() > 1 else v for k, v in t.items()}
        y1, _ = ssm.delta_step(**one, state=state, inplace=True)
        return y, h, y1

    want = []
    for t in (first, second):
        st = torch.zeros_like(state)
        want.append((*(x.clone() for x in run(t, st)), st))
    stream = torch.cuda.Stream()
    live = {k: v.clone() for k, v in first.items()}
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        run(live, state)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = run(live, state)
    for t, (y, h, y1, st) in zip((first, second, first), (want[0], want[1], want[0])):
        for k in live:
            live[k].copy_(t[k])
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((*out, state), (y, h, y1, st)):
            assert torch.equal(got, ref)


def test_repeats_are_equal():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    t = on_device(inputs(rng_of("repeat calls"), 3, 500, 8, 4, 128, 128, "bf16"), "bf16")
    y, h = ssm.delta_fwd(**t)
    for _ in range(20):
        y2, h2 = ssm.delta_fwd(**t)
        assert torch.equal(y, y2) and torch.equal(h, h2)
