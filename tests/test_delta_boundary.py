"""CPU tests of the gated delta rule and of the norms with a gate and a residual: the entry points refuse bad
arguments on the host before anything is enqueued, and the float64 definitions agree with closed forms."""
import numpy as np
import pytest

from oracle import delta as od
from selective_state_space_mamba_gb300 import _lib
from selective_state_space_mamba_gb300._lib import SsmDeltaArgs, SsmTokens

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or enqueues nothing
FAR = 1 << 40   # the outputs' place, away from the inputs'
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (_lib.SSM_ERR_INVALID_ARG, _lib.SSM_ERR_UNSUPPORTED, _lib.SSM_ERR_ALIGNMENT,
                                              _lib.SSM_ERR_WORKSPACE)
OK = _lib.SSM_OK


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def delta(lib, step=False, slots=None, nslots=None, ws=(3 * FAR, 1 << 40), **kw):
    a = SsmDeltaArgs()
    v = dict(q=FAKE, k=FAKE, v=FAKE, dt=FAKE, beta=FAKE, A=FAKE, dt_bias=None, h0=None, lens=None, y=FAR, h_final=2 * FAR,
             batch=2, seqlen=64, nheads=4, headdim=64, dstate=64, ngroups=2, softplus=1, sigmoid=1, l2norm=1, scale=1.0,
             dtype=1, bs=1 << 20, ts=512)
    v.update(kw)
    for k in ("q", "k", "v", "dt", "beta"):
        setattr(a, k, SsmTokens(v[k], v["bs"], v["ts"]))
    for k in ("A", "dt_bias", "h0", "lens", "y", "h_final", "batch", "seqlen", "nheads", "headdim", "dstate", "ngroups",
              "softplus", "sigmoid", "l2norm", "scale", "dtype"):
        setattr(a, k, v[k])
    if step:
        return lib.ssm_delta_step(a, slots, v["batch"] if nslots is None else nslots, None)
    return lib.ssm_delta_fwd(a, ws[0], ws[1], None)


def test_delta_refusals(lib):
    for step in (False, True):
        f = lambda **kw: delta(lib, step, **kw)  # noqa: B023,E731
        assert f(batch=-1) == INVALID and f(nheads=0) == INVALID and f(ngroups=0) == INVALID and f(headdim=0) == INVALID
        assert f(ngroups=3) == INVALID and f(dtype=3) == INVALID
        assert f(dstate=16) == UNSUPPORTED and f(dstate=0) == UNSUPPORTED and f(dstate=256) == UNSUPPORTED
        assert f(batch=65536) == UNSUPPORTED and f(headdim=1 << 29) == UNSUPPORTED
        assert f(nheads=1 << 28, ngroups=1 << 28, headdim=1) == UNSUPPORTED
        for k in ("q", "k", "v", "dt", "beta", "A", "y"):
            assert f(**{k: None}) == INVALID, k
        for k in ("q", "k", "v", "dt", "beta"):
            assert f(**{k: FAKE + 1}) == ALIGNMENT, k
        for k in ("A", "dt_bias", "h0"):
            assert f(**{k: FAKE + 2}) == ALIGNMENT, k
        assert f(bs=-1) == INVALID and f(bs=1 << 62) == INVALID
        assert f(y=FAKE + 96) == INVALID and f(y=2 * FAR + 4) == INVALID
        assert f(h0=2 * FAR + 4) == INVALID
    assert delta(lib, seqlen=-1) == INVALID
    assert delta(lib, h0=2 * FAR) == INVALID           # a prompt does not update in place
    assert delta(lib, ts=-1) == INVALID
    assert delta(lib, True, nslots=3) == INVALID       # without slots, a state row for each sequence
    assert delta(lib, True, nslots=-1, slots=FAKE) == INVALID
    assert delta(lib, True, h_final=None) == INVALID
    assert delta(lib, batch=0) == OK and delta(lib, True, batch=0) == OK
    assert delta(lib, seqlen=0, h_final=None) == OK
    assert lib.ssm_delta_fwd(None, None, 0, None) == INVALID
    assert lib.ssm_delta_step(None, None, 0, None) == INVALID


def test_delta_workspace(lib):
    f = lib.ssm_delta_fwd_workspace_bytes
    for bad in ((-1, 64, 4, 64, 64, 2, 1), (1, -1, 4, 64, 64, 2, 1), (1, 64, 0, 64, 64, 1, 1), (1, 64, 4, 64, 65, 2, 1),
                (1, 64, 4, 64, 64, 3, 1), (65536, 64, 4, 64, 64, 2, 1), (0, 64, 4, 64, 64, 2, 1)):
        assert f(*bad) == 0
    assert f(1, 64, 4, 64, 64, 2, 0) == 0 and f(1, 64, 4, 64, 32, 2, 1) == 0 and f(1, 64, 4, 60, 64, 2, 1) == 0
    assert f(1, 1, 4, 64, 64, 2, 1) == 0                       # one token
    assert f(1, 64, 4, 64, 64, 2, 1) == 0                      # few tokens
    one, two = f(1, 128, 4, 64, 64, 2, 1), f(1, 129, 4, 64, 64, 2, 1)
    assert two - one == 4 * 25600 and one == 256 + 2 * 4 * 25600
    long = f(4, 1 << 20, 32, 128, 128, 16, 1)                  # in segments, with the states between them
    assert 4 * 32 * 128 * 128 * 4 < long < 4 * 32 * (1 << 14) * 25600
    assert delta(lib, seqlen=128, ws=(None, 0)) == WORKSPACE and delta(lib, seqlen=128, ws=(3 * FAR, one)) == WORKSPACE
    assert delta(lib, seqlen=128, ws=(3 * FAR + 16, 1 << 40)) == ALIGNMENT


def gated(lib, **kw):
    a = dict(x=FAKE, xs=64, z=FAKE, zs=64, w=FAKE, ww=64, y=FAR, rows=4, d=64, group=0, first=0, dtype=1)
    a.update(kw)
    return lib.ssm_gatednorm_fwd(a["x"], a["xs"], a["z"], a["zs"], a["w"], a["ww"], a["y"], a["rows"], a["d"], a["group"],
                                 a["first"], 1e-5, a["dtype"], None)


def block(lib, **kw):
    a = dict(x=FAKE, xs=64, w=FAKE, z=None, zs=64, res=FAKE, rout=2 * FAR, w2=FAKE, y=FAR, rows=4, d=64, dtype=1, rdtype=1)
    a.update(kw)
    return lib.ssm_blocknorm_fwd(a["x"], a["xs"], a["w"], a["z"], a["zs"], a["res"], a["rout"], a["w2"], a["y"], a["rows"],
                                 a["d"], 1.0, 1e-5, a["dtype"], a["rdtype"], None)


def test_norm_refusals(lib):
    for f in (gated, block):
        assert f(lib, rows=-1) == INVALID and f(lib, d=0) == INVALID and f(lib, dtype=2) == INVALID
        for k in ("x", "w", "y") + (("z",) if f is gated else ("res", "w2")):
            assert f(lib, **{k: None}) == INVALID, k
        for k in ("x", "w", "z"):
            assert f(lib, **{k: FAKE + 1}) == ALIGNMENT, k
        assert f(lib, xs=-64) == INVALID and f(lib, xs=1 << 62) == INVALID
        assert f(lib, y=FAKE + 2 * 64) == INVALID
        assert f(lib, rows=0) == OK
        assert f(lib, rows=1 << 31, y=1 << 58, rout=1 << 60) == UNSUPPORTED if f is block else True
    assert gated(lib, group=-1) == INVALID and gated(lib, group=48) == INVALID and gated(lib, group=128) == INVALID
    assert gated(lib, group=32, ww=16) == INVALID and gated(lib, ww=32) == INVALID
    assert gated(lib, rows=1 << 31) == UNSUPPORTED and gated(lib, rows=1 << 30, group=16) == UNSUPPORTED
    assert gated(lib, d=(1 << 30) + 8, ww=(1 << 30) + 8) == UNSUPPORTED
    assert block(lib, rdtype=7) == INVALID and block(lib, dtype=0, rdtype=1) == INVALID
    assert block(lib, rout=FAKE + 4) == INVALID and block(lib, res=FAKE + 1) == ALIGNMENT
    assert block(lib, d=(1 << 30) + 8) == UNSUPPORTED


WRAPS = (1 << 32) + 256  # 256 in 32 bits


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_python_sizes_that_wrap_are_refused(dtype):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    t = lambda *n: torch.empty(n, device="meta", dtype=getattr(torch, dtype))  # noqa: E731
    f = lambda *n: torch.empty(n, device="meta")  # noqa: E731
    n = WRAPS
    calls = [
        lambda: ssm.delta_fwd(t(1, 1, n, 64), t(1, 1, n, 64), t(1, 1, 8, 64), t(1, 1, 8), t(1, 1, 8), f(8)),
        lambda: ssm.delta_fwd(t(1, 1, 1, n), t(1, 1, 1, n), t(1, 1, 8, 64), t(1, 1, 8), t(1, 1, 8), f(8)),
        lambda: ssm.delta_fwd(t(1, 1, 1, 64), t(1, 1, 1, 64), t(1, 1, n, 64), t(1, 1, n), t(1, 1, n), f(n)),
        lambda: ssm.delta_fwd(t(1, 1, 1, 64), t(1, 1, 1, 64), t(1, 1, 8, n), t(1, 1, 8), t(1, 1, 8), f(8)),
        lambda: ssm.delta_step(t(1, n, 64), t(1, n, 64), t(1, 8, 64), t(1, 8), t(1, 8), f(8)),
        lambda: ssm.delta_step(t(1, 1, 64), t(1, 1, 64), t(1, 8, n), t(1, 8), t(1, 8), f(8)),
        lambda: ssm.gatednorm_fwd(t(1, n), t(1, n), f(n)), lambda: ssm.gatednorm_fwd(t(1, 8), t(1, 8), f(8), group=1 << 32),
        lambda: ssm.blocknorm_fwd(t(1, n), f(n), t(1, n), f(n)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ssm.SsmError, match="SSM_ERR_UNSUPPORTED"):
            call()
            pytest.fail(f"call {i} was taken")


def test_python_refusals():
    """Shapes, types and devices: refused before anything is enqueued (tensors of the CPU: the device last)."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    t = lambda *n: torch.zeros(n)  # noqa: E731
    good = dict(q=t(2, 5, 2, 64), k=t(2, 5, 2, 64), v=t(2, 5, 4, 16), dt=t(2, 5, 4), beta=t(2, 5, 4), A=t(4))
    bad = [dict(q=t(2, 5, 64)), dict(k=t(2, 5, 1, 64)), dict(k=t(2, 4, 2, 64)), dict(v=t(2, 5, 64)), dict(v=t(1, 5, 4, 16)),
           dict(dt=t(2, 5, 2)), dict(beta=t(2, 5)), dict(A=t(2)), dict(A=t(4).double()), dict(dt_bias=t(3)),
           dict(k=t(2, 5, 2, 64).bfloat16()), dict(q=t(2, 5, 2, 128)[..., ::2]), dict(q=t(2, 5, 4, 64)[:, :, ::2]),
           dict(v=t(2, 5, 8, 16)[:, :, ::2]), dict(k=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            ssm.delta_fwd(**{**good, **kw})
    with pytest.raises(TypeError, match="unsupported dtype"):
        ssm.delta_fwd(**{**good, "q": t(2, 5, 2, 64).half()})
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.delta_fwd(**good)
    with pytest.raises(TypeError):
        ssm.delta_fwd(**good, scale="x")
    one = dict(q=t(2, 2, 64), k=t(2, 2, 64), v=t(2, 4, 16), dt=t(2, 4), beta=t(2, 4), A=t(4))
    for kw in (dict(q=t(2, 1, 2, 64)), dict(v=t(2, 64)), dict(dt=t(2, 5))):
        with pytest.raises(ValueError):
            ssm.delta_step(**{**one, **kw})
    for kw in (dict(x=t(2, 8), z=t(2, 7), weight=t(8)), dict(x=t(2, 8), z=t(2, 8), weight=t(4)), dict(x=t(2, 8), z=None, weight=t(8)),
               dict(x=t(2, 8), z=t(2, 8), weight=t(2, 4))):
        with pytest.raises(ValueError):
            ssm.gatednorm_fwd(**kw)
    with pytest.raises(TypeError):
        ssm.gatednorm_fwd(t(2, 8), t(2, 8), t(8), group="x")
    for kw in (dict(x=t(2, 8), weight=t(8), residual=None, next_weight=t(8)),
               dict(x=t(2, 8), weight=t(7), residual=t(2, 8), next_weight=t(8))):
        with pytest.raises(ValueError):
            ssm.blocknorm_fwd(**kw)


# ------------------------------------------------------------------------------ the definitions

def test_delta_by_products():
    """S_t = a_t S_{t-1} (I - beta k k^T) + beta v k^T, written with matrices; one token gives beta v k^T."""
    r = np.random.default_rng(1)
    b, L, nh, G, H, N = 2, 9, 4, 2, 3, 5
    q, k = r.standard_normal((2, b, L, G, N))
    v, dt, beta = r.standard_normal((b, L, nh, H)), r.standard_normal((b, L, nh)), r.standard_normal((b, L, nh))
    A, bias, h0 = -r.uniform(0, 2, nh), r.standard_normal(nh), r.standard_normal((b, nh, H, N))
    y, ey, h, eh = od.delta(q, k, v, dt, beta, A, bias, h0, lens=[L, 4], scale=0.3)
    for i in range(b):
        for j in range(nh):
            S, g = h0[i, j], j // 2
            for t in range([L, 4][i]):
                kt, qt = (x[i, t, g] / np.sqrt(x[i, t, g] @ x[i, t, g] + 1e-6) for x in (k, q))
                a, be = np.exp(A[j] * np.log1p(np.exp(dt[i, t, j] + bias[j]))), 1 / (1 + np.exp(-beta[i, t, j]))
                S = a * S @ (np.eye(N) - be * np.outer(kt, kt)) + be * np.outer(v[i, t, j], kt)
                assert np.allclose(y[i, t, j], 0.3 * S @ qt)
            assert np.allclose(h[i, j], S)
    assert not y[1, 4:].any() and (ey >= 0).all() and (eh >= 0).all()


def test_delta_answers_its_keys():
    """beta 1 and no decay: after a token the state answers its key with its value, and keeps the answers to
    orthogonal keys."""
    r = np.random.default_rng(2)
    N = 8
    k = np.linalg.qr(r.standard_normal((N, N)))[0][None, :, None]
    v = r.standard_normal((1, N, 1, 3))
    y, _, h, _ = od.delta(k, k, v, np.zeros((1, N, 1)), np.ones((1, N, 1)), np.zeros(1), scale=1.0, softplus=False,
                          sigmoid=False, l2norm=False)
    assert np.allclose(y, v) and np.allclose(h[0, 0] @ k[0, :, 0].T, v[0, :, 0].T)


def test_norms_by_hand():
    x, z = np.array([[3.0, 4.0, 0.0, 2.0]]), np.array([[0.0, 1.0, 2.0, -1.0]])
    silu = z / (1 + np.exp(-z))
    y, e = od.gatednorm(x, z, np.array([1.0, 2.0]), group=2, eps=0.0)
    want = np.array([[3 / np.sqrt(12.5), 8 / np.sqrt(12.5), 0.0, 4 / np.sqrt(2.0)]]) * silu
    assert np.allclose(y, want) and (e >= 0).all()
    y, e = od.gatednorm(x, z, np.ones(4), gate_first=True, eps=0.5)
    u = x * silu
    assert np.allclose(y, u / np.sqrt((u ** 2).mean() + 0.5)) and (e >= 0).all()
    y, e, r, er = od.blocknorm(x, np.ones(4), z, np.full(4, 2.0), alpha=0.5, eps=0.0)
    assert np.allclose(r, 0.5 * z + x / np.sqrt(29 / 4)) and np.allclose((y / 2) ** 2 @ np.ones(4), 4)
    assert (e >= 0).all() and (er >= 0).all()
