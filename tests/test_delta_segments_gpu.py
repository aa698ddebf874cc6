"""GPU tests of the gated delta rule over prompts of several workspace segments whose chains are cut into pieces: what a
segment leaves for the next one."""
import pytest

from test_delta_paths_gpu import agree

pytestmark = pytest.mark.gpu

SEGMENT = 655 * 64  # tokens of a segment of 64 heads: 2^30 bytes of records of 25,600 bytes a head and chunk
PIECE = 82 * 64     # ... of one of its eight pieces


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("ends", [[0, 1, 2, 3, 4, 5, 6, 12], [7, 0, 3, 15, -1, 7, -8, 11]], ids=str)
def test_lengths_that_end_in_pieces_of_the_middle_segment(ends):
    """ends: the piece, counted from the middle segment's first, in which a sequence ends.  The states hardly decay and are hardly
    overwritten, so that one that is wrong at a segment's start shows to its end.  Whole segments are cut the same way
    in a call of their own, which keeps no states between segments: equal to the last bit.  The last one has fewer pieces here."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b, nh, G, H, N, L = 8, 8, 2, 64, 64, 2 * SEGMENT + 20000
    g = torch.Generator("cuda").manual_seed(11)
    r = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()  # noqa: E731
    t = [r(b, L, G, N), r(b, L, G, N), r(b, L, nh, H), r(b, L, nh), r(b, L, nh) - 7]  # beta about 0.001
    A, bias = -torch.rand(nh, device="cuda", generator=g), torch.full((nh,), -11.0, device="cuda")
    h0 = torch.randn(b, nh, H, N, device="cuda", generator=g)
    n = [min(L, max(0, SEGMENT + PIECE * e + 1 + 333 * i)) for i, e in enumerate(ends)]
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    with ssm.KernelTimer() as timer:
        y, h = ssm.delta_fwd(*t, A, bias, h0, lens)
    assert timer.launches["delta_states"] == timer.launches["delta_chain"] == 3
    state = h0
    for start in range(0, L, SEGMENT):
        part = [x[:, start : start + SEGMENT] for x in t]
        left = (lens - start).clamp(0, SEGMENT).int()
        y1, state = ssm.delta_fwd(*part, A, bias, state, left)
        if start + SEGMENT < L:
            assert torch.equal(y[:, start : start + SEGMENT], y1), start
        else:
            agree((y[:, start:], h), (y1, state))
            ended = left == 0
            assert torch.equal(h[ended], state[ended])
    # the states were worth the test: what a sequence that goes on ends with is not forgotten within a segment
    on = lens > 2 * SEGMENT
    again = ssm.delta_fwd(*(x[on][:, :SEGMENT] for x in t), A, bias, torch.zeros_like(h0[on]))[1]
    first = ssm.delta_fwd(*(x[on][:, :SEGMENT] for x in t), A, bias, h0[on])[1]
    assert float((first - again).norm()) > 0.1 * float(h0[on].norm())
