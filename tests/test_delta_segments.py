"""CPU tests of the workspace that the gated delta rule asks for prompts of several segments."""
import pytest

from selective_state_space_mamba_gb300 import _lib


@pytest.mark.parametrize("sizes", [(8, 8, 64, 64), (1, 32, 128, 128), (40, 32, 64, 64), (1, 3, 8, 64)], ids=str)
def test_a_segment_reads_and_writes_states_in_different_places(sizes):
    """CTAs that read what a segment enters with and those that write what it leaves run at the same time: from the third
    segment on there is a place for each.  (The second of two segments leaves h_final, the first enters with h0.)"""
    b, nh, H, N = sizes
    f = lambda chunks: _lib.load().ssm_delta_fwd_workspace_bytes(b, 64 * chunks, nh, H, N, 1, _lib.SSM_BF16)  # noqa: E731
    most = (1 << 30) // 25600 // (b * nh)  # chunks of a segment
    state = (b * nh * H * N * 4 + 255) // 256 * 256
    one, two, three = f(most), f(most + 1), f(2 * most + 1)
    assert two - one == state and f(2 * most) == two
    assert three - two == state and f(3 * most + 1) == three and f(9 * most) == three
