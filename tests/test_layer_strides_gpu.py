"""Orders of strides, and sequences of more than 2^31 tokens, in the operators around a layer's scan."""
import pytest

from test_layer_workspace_gpu import scan_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def inside(t):
    """The same values with sequences inside tokens: [L, b, ...] in memory."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def wide(t, columns=48, rows=5):
    """The same values in wider rows, and a sequence's rows followed by others."""
    import torch
    b, L, d = t.shape[0], t.shape[1], t[0, 0].numel()
    buf = torch.full((b, L + rows, d + columns), float("nan"), device=t.device, dtype=t.dtype)
    buf[:, :L, 16 : 16 + d] = t.reshape(b, L, d)
    return buf[:, :L, 16 : 16 + d].unflatten(-1, t.shape[2:])


def skewed(t):
    """The same values with sequences apart by no whole number of rows, each on 16 bytes."""
    import torch
    b, L, d = t.shape[0], t.shape[1], t[0, 0].numel()
    row, seq = d + 24, L * (d + 24) + 16
    buf = torch.full((b * seq,), float("nan"), device=t.device, dtype=t.dtype)
    v = buf.as_strided((b, L, d), (seq, row, 1))
    v.copy_(t.reshape(b, L, d))
    return v.unflatten(-1, t.shape[2:])


def skewed_inside(t):
    """Sequences inside tokens, and tokens apart by no whole number of sequences."""
    import torch
    b, L, d = t.shape[0], t.shape[1], t[0, 0].numel()
    row, tok = d + 8, b * (d + 8) + 24
    buf = torch.full((L * tok,), float("nan"), device=t.device, dtype=t.dtype)
    v = buf.as_strided((b, L, d), (row, tok, 1))
    v.copy_(t.reshape(b, L, d))
    return v.unflatten(-1, t.shape[2:])


LAYOUTS = {"plain": lambda t: t, "inside": inside, "wide": wide, "skewed": skewed, "skewed_inside": skewed_inside,
           "wide_inside": lambda t: wide(t.transpose(0, 1).contiguous()).transpose(0, 1)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", [(3, 50, 72), (3, 50, 73), (2, 1, 64), (2, 400, 40), (7, 1300, 1472)], ids=str)
def test_selscan_order_of_strides(case, layout, dtype):
    """Each tensor in turn, and all of them, against the same values in plain tensors.  (Both ways of copying give
    the same values to the same arithmetic.)"""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    names = ("u", "dt", "A", "B", "C", "D", "z")
    plain = dict(zip(names, scan_case(case, 21, dtype)))
    want = ssm.selscan_fwd(**plain)
    change = LAYOUTS[layout]
    for which in [("u",), ("dt",), ("B",), ("C",), ("z",), ("u", "dt", "B", "C", "z")]:
        got = ssm.selscan_fwd(**{k: change(v) if k in which else v for k, v in plain.items()})
        assert all(torch.equal(a, b) for a, b in zip(got, want)), which


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", [(3, 50, 72), (3, 50, 73), (2, 300, 514)], ids=str)
def test_conv_order_of_strides(case, layout, dtype):
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x = scan_case(case, 22, dtype)[0]
    w = torch.randn(case[2], 4, device="cuda")
    want = ssm.conv_fwd(x, w)
    assert all(torch.equal(a, b) for a, b in zip(ssm.conv_fwd(LAYOUTS[layout](x), w), want))


def test_selscan_of_more_tokens_than_31_bits():
    """2^31 + 1000 tokens of eight channels (whole vectors: 32 GiB, and as much of y).  All inputs are one tensor, zeros
    but for the last 4096 tokens: y there is that of those tokens by themselves."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    L, last = (1 << 31) + 1000, 4096
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 70 GiB of device memory")
    x = torch.zeros(1, L, 8, device="cuda", dtype=torch.bfloat16)
    x[:, -last:] = torch.randn(1, last, 8, device="cuda")
    A, g = -torch.ones(8, 8, device="cuda"), x.view(1, L, 1, 8)
    y, h = ssm.selscan_fwd(x, x, A, g, g)
    y2, h2 = ssm.selscan_fwd(x[:, -last:], x[:, -last:], A, g[:, -last:], g[:, -last:])
    tail = y[:, -last:].clone()
    near = y[:, : -last].count_nonzero() if last == 0 else y[:, (1 << 31) - 5000 : -last].count_nonzero()
    del x, g, y
    torch.cuda.empty_cache()
    assert int(near) == 0 and tail.any()
    # both start from zeros; parts of the time axis begin elsewhere, a rounding of bf16 apart
    assert torch.allclose(tail.float(), y2.float(), rtol=2.0 ** -7, atol=1e-4) and torch.allclose(h, h2, rtol=1e-4, atol=1e-5)
