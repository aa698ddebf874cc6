"""Offsets beyond 32 bits in the operators around a layer's scan: long sequences, many rows, large caches of states."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room(cuda_lib):
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 45 << 30:
        pytest.skip("needs 40 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed=1):
    import torch
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("d", [1, 2])
def test_conv_of_more_tokens_than_31_bits(d):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    L, n = (1 << 31) + 1000, 3000
    x = torch.zeros(1, L, d, device="cuda", dtype=torch.bfloat16)
    x[:, -n:] = randn(1, n, d)
    w, bias = randn(d, 4, seed=2), randn(d, seed=3)
    y, s = ssm.conv_fwd(x, w, bias)
    y2, s2 = ssm.conv_fwd(x[:, -n:], w, bias)  # the tokens before them are zeros
    assert torch.equal(y[:, -n:], y2) and torch.equal(s, s2)
    assert torch.equal(y[:, (1 << 31) - 2500 : -n], y[:, :1].expand(1, L - n - (1 << 31) + 2500, d))


def test_selscan_ragged_rows_of_more_tokens_than_31_bits():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    L, n = (1 << 31) + 1000, 4096
    x = torch.zeros(1, L, 1, device="cuda", dtype=torch.bfloat16)
    x[:, -n:] = randn(1, n, 1)
    B = torch.zeros(1, 1, 1, 8, device="cuda", dtype=torch.bfloat16) + 1
    A = -torch.ones(1, 8, device="cuda")
    y, h = ssm.selscan_fwd(x, x, A, B.expand(1, L, 1, 8), B.expand(1, L, 1, 8))
    y2, h2 = ssm.selscan_fwd(x[:, -n:], x[:, -n:], A, B.expand(1, n, 1, 8), B.expand(1, n, 1, 8))
    # parts of the time axis begin elsewhere: sums of a few terms in f32, a rounding of bf16 apart at most
    assert torch.allclose(y[:, -n:].float(), y2.float(), rtol=2.0 ** -7, atol=1e-4) and torch.allclose(h, h2, rtol=1e-4, atol=1e-5)
    assert y2.any() and not y[:, (1 << 31) - 5000 : -n].any()


@pytest.mark.parametrize("d", [4096, 4097])
def test_rmsnorm_of_more_elements_than_32_bits(d):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    rows, n = (1 << 20) + 600, 700
    x = torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16)
    x[-n:], x[:n] = randn(n, d), randn(n, d, seed=5)
    w = randn(d, seed=2)
    y, r = ssm.rmsnorm_fwd(x, w, x)
    for part in (slice(0, n), slice(rows - n, rows)):
        y2, r2 = ssm.rmsnorm_fwd(x[part], w, x[part])
        assert torch.equal(y[part], y2) and torch.equal(r[part], r2)
    assert not y[n : 2 * n].any() and not y[-2 * n : -n].any()
    del y, r
    q, s, _ = ssm.rmsnorm_fp8_fwd(x, w, group=128)
    q2, s2, _ = ssm.rmsnorm_fp8_fwd(x[-n:], w, group=128)
    assert torch.equal(q[-n:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-n:], s2)


@pytest.mark.parametrize("b", [3, 90])
def test_steps_in_caches_of_more_elements_than_32_bits(b):
    """The cache's last slots, in place, against the same states in a cache of their own."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    d, N, slots = 4104, 16, 70000
    state = torch.zeros(slots, d, N, device="cuda")
    state[-b:] = randn(b, d, N)
    at = torch.arange(slots - b, slots, device="cuda", dtype=torch.int32)
    u, dt, B, C = randn(b, d, seed=2), randn(b, d, seed=3), randn(b, 1, N, seed=4), randn(b, 1, N, seed=5)
    A = -torch.rand(d, N, device="cuda")
    own = state[-b:].clone()
    y, _ = ssm.selscan_step(u, dt, A, B, C, state=state, slots=at, inplace=True)
    y2, h2 = ssm.selscan_step(u, dt, A, B, C, state=own)
    assert torch.equal(y, y2) and torch.equal(state[-b:], h2) and not state[:b].any() and not state[-2 * b : -b].any()
    del state
    conv = torch.zeros(200000, 3, d, device="cuda", dtype=torch.bfloat16)
    conv[-b:] = randn(b, 3, d, seed=6)
    at = torch.arange(200000 - b, 200000, device="cuda", dtype=torch.int32)
    x, w, own = u.bfloat16(), randn(d, 4, seed=7), conv[-b:].clone()
    y, _ = ssm.conv_step(x, w, state=conv, slots=at, inplace=True)
    y2, s2 = ssm.conv_step(x, w, state=own)
    assert torch.equal(y, y2) and torch.equal(conv[-b:], s2) and not conv[:b].any() and not conv[-2 * b : -b].any()
