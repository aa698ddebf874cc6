"""GPU parity of the norms with a gate and a residual (gatednorm, blocknorm) against the float64 definitions in
oracle/delta.py, each element held to the bound derived there; a bf16 output may be off by 2^-8 of its value besides."""
import numpy as np
import pytest

from oracle import delta as od
from test_delta_gpu import close, dev, host, rng_of, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def rows_of(a, dtype, pad):
    """A device tensor of a's rows, with `pad` columns of NaN on each side."""
    import torch
    if pad == 0:
        return dev(a, dtype)
    wide = torch.full((a.shape[0], a.shape[1] + 2 * pad), float("nan"), device="cuda",
                      dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    wide[:, pad:-pad] = dev(a, dtype)
    return wide[:, pad:-pad]


GATED = [  # rows, d, group, shared weight, pad
    (1, 1, 0, False, 0), (1, 64, 0, False, 0), (3, 1536, 64, True, 0), (2, 4096, 128, True, 8), (7, 5120, 0, False, 0),
    (5, 120, 40, True, 3), (4, 77, 7, False, 1), (2, 300, 0, True, 0), (700, 256, 128, False, 64), (1300, 96, 32, True, 0),
    (640, 1000, 200, False, 0), (620, 1023, 341, True, 0), (2, 20001, 0, False, 0), (611, 2048, 256, True, 8),
    (700, 20480, 0, False, 0), (9, 512, 512, True, 16), (650, 64, 8, True, 0), (3, 24, 8, False, 0), (615, 1024, 1024, True, 4),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gatednorm(case, first, dtype):
    import selective_state_space_mamba_gb300 as ssm
    rows, d, group, shared, pad = case
    r = rng_of("gatednorm", case, first, dtype)
    x, z = (rounded(r.standard_normal((rows, d)), dtype) for _ in range(2))
    x[0] *= 2.0 ** -20  # a row that eps decides
    w = (1 + 0.2 * r.standard_normal((group or d) if shared else d)).astype(np.float32)
    ref, err = od.gatednorm(x, z, w, group, first)
    y = ssm.gatednorm_fwd(rows_of(x, dtype, pad), rows_of(z, dtype, pad), dev(w), group=group, gate_first=first)
    close(host(y), ref, err, "y", dtype)


BLOCK = [  # rows, d, pad
    (1, 1, 0), (1, 2560, 0), (3, 77, 3), (5, 1001, 1), (2, 4096, 8), (700, 2560, 0), (640, 333, 0), (3, 20001, 0),
    (620, 13000, 0), (615, 256, 16), (1, 12288, 0),
]


@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("case", BLOCK, ids=str)
def test_blocknorm(case, gate, dtype, res):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    rows, d, pad = case
    r = rng_of("blocknorm", case, gate, dtype, res)
    x, z = (rounded(r.standard_normal((rows, d)), dtype) for _ in range(2))
    residual = rounded(4 * r.standard_normal((rows, d)), res)
    w, w2 = ((1 + 0.2 * r.standard_normal(d)).astype(np.float32) for _ in range(2))
    ref, err, r_ref, r_err = od.blocknorm(x, w, residual, w2, z if gate else None, 0.75)
    args = [rows_of(x, dtype, pad), dev(w), dev(residual, res), dev(w2), rows_of(z, dtype, pad) if gate else None]
    y, out = ssm.blocknorm_fwd(*args, alpha=0.75)
    close(host(y), ref, err, "y", dtype)
    close(host(out), r_ref, r_err, "residual", res)
    assert np.array_equal(host(args[2]), residual)
    y2, out2 = ssm.blocknorm_fwd(*args, alpha=0.75, residual_out=args[2])  # in place
    assert out2 is args[2] and torch.equal(out2, out) and torch.equal(y2, y)


def test_nan_and_infinity_stay_in_their_group():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x = torch.ones(4, 256, device="cuda")
    z = torch.ones_like(x)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    for first in (False, True):
        y = ssm.gatednorm_fwd(x, z, torch.ones(128, device="cuda"), group=128, gate_first=first)
        bad = ~torch.isfinite(y)
        assert bad[1, :128].all() and not bad[1, 128:].any() and not bad[2, :128].any() and bad[2, 200]
        assert not bad[0].any() and not bad[3].any()
    y, r = ssm.blocknorm_fwd(x, z[0], z, z[0])
    assert torch.isnan(y[1]).all() and not torch.isnan(y[0]).any() and not torch.isnan(y[3]).any()


def test_shapes_and_graph():
    """Leading dimensions, no rows, outputs of the caller, and a captured call on new inputs."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    g = torch.Generator("cuda").manual_seed(5)
    x, z, res = (torch.randn(2, 3, 512, device="cuda", generator=g) for _ in range(3))
    w = torch.ones(512, device="cuda")
    y, b = ssm.gatednorm_fwd(x, z, w[:64], group=64), ssm.blocknorm_fwd(x, w, res, w, z)
    assert y.shape == x.shape and torch.equal(y.view(6, 512), ssm.gatednorm_fwd(x.view(6, 512), z.view(6, 512), w, group=64))
    given = [torch.empty_like(x) for _ in range(3)]
    assert ssm.gatednorm_fwd(x, z, w[:64], group=64, y=given[0]) is given[0] and torch.equal(given[0], y)
    got = ssm.blocknorm_fwd(x, w, res, w, z, y=given[1], residual_out=given[2])
    assert got[0] is given[1] and got[1] is given[2] and all(torch.equal(p, q) for p, q in zip(got, b))
    assert ssm.gatednorm_fwd(x[:0], z[:0], w).shape == (0, 3, 512)
    assert ssm.blocknorm_fwd(x[:0], w, res[:0], w)[0].shape == (0, 3, 512)
    live, graph = [t.clone() for t in (x, z, res)], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssm.gatednorm_fwd(live[0], live[1], w, group=128), *ssm.blocknorm_fwd(live[0], w, live[2], w, live[1])
    for scale in (1.0, -3.0):
        for t, s in zip(live, (x, z, res)):
            t.copy_(s * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = ssm.gatednorm_fwd(live[0], live[1], w, group=128), *ssm.blocknorm_fwd(live[0], w, live[2], w, live[1])
        assert all(torch.equal(p, q) for p, q in zip(out, want))
