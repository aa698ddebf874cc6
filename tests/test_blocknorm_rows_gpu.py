"""GPU parity of the norms with a gate and a residual over many rows: every number of vectors that a thread may hold, aligned and
not (the rules in csrc/blocknorm.cu go by rows, by columns in eights, and by alignment)."""
import numpy as np
import pytest

from oracle import delta as od
from test_blocknorm_gpu import rows_of
from test_delta_gpu import close, dev, host, rng_of, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


GATED = [  # rows, d, group, pad
    (700, 5120, 0, 0), (640, 2561, 0, 0), (620, 5001, 0, 0), (610, 9001, 0, 0), (620, 1024, 512, 0), (320, 1056, 528, 8),
    (612, 5120, 0, 4), (310, 4098, 2049, 0), (9800, 136, 8, 0), (9800, 120, 120, 8),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gatednorm(case, first, dtype):
    import selective_state_space_mamba_gb300 as ssm
    rows, d, group, pad = case
    r = rng_of("gatednorm rows", case, first, dtype)
    x, z = (rounded(r.standard_normal((rows, d)), dtype) for _ in range(2))
    x[0] *= 2.0 ** -20  # a row that eps decides
    w = (1 + 0.2 * r.standard_normal(d)).astype(np.float32)
    ref, err = od.gatednorm(x, z, w, group, first)
    y = ssm.gatednorm_fwd(rows_of(x, dtype, pad), rows_of(z, dtype, pad), dev(w), group=group, gate_first=first)
    close(host(y), ref, err, "y", dtype)


BLOCK = [  # rows, d, pad
    (640, 2561, 0), (620, 5001, 0), (610, 9001, 0), (610, 13001, 0), (620, 640, 0), (611, 200, 3), (609, 700, 1), (610, 20480, 0),
    (609, 12288, 8),
]


@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("case", BLOCK, ids=str)
def test_blocknorm(case, gate, dtype, res):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    rows, d, pad = case
    r = rng_of("blocknorm rows", case, gate, dtype, res)
    x, z = (rounded(r.standard_normal((rows, d)), dtype) for _ in range(2))
    residual = rounded(4 * r.standard_normal((rows, d)), res)
    w, w2 = ((1 + 0.2 * r.standard_normal(d)).astype(np.float32) for _ in range(2))
    ref, err, r_ref, r_err = od.blocknorm(x, w, residual, w2, z if gate else None, 0.75)
    args = [rows_of(x, dtype, pad), dev(w), dev(residual, res), dev(w2), rows_of(z, dtype, pad) if gate else None]
    y, out = ssm.blocknorm_fwd(*args, alpha=0.75)
    close(host(y), ref, err, "y", dtype)
    close(host(out), r_ref, r_err, "residual", res)
    y2, out2 = ssm.blocknorm_fwd(*args, alpha=0.75, residual_out=args[2])  # in place
    assert out2 is args[2] and torch.equal(out2, out) and torch.equal(y2, y)
