"""CPU tests of the rules by which a prompt of the gated delta rule is run, seen through the workspace that it asks for."""
from selective_state_space_mamba_gb300 import _lib


def need(b, L, nh, H, N):
    return _lib.load().ssm_delta_fwd_workspace_bytes(b, L, nh, H, N, 1, _lib.SSM_BF16)


def pieces(b, L, nh, H, N):
    """Of the chains: all but the last leave a state, all but the first and the last a map of states besides."""
    left = need(b, L, nh, H, N) - 256 - b * nh * -(-L // 64) * 25600
    state, passing = b * nh * H * N * 4, b * nh * N * N * 4
    n = next((n for n in range(1, 33) if (n - 1) * state + max(n - 2, 0) * passing == left), None)
    assert n, left
    return n


def test_chains_are_cut_as_measured():
    """The faster of two ways by at least 5 % in calls of 128 to 512 chunks (by themselves; in pairs it would be the other number)."""
    assert pieces(1, 64 * 128, 16, 64, 128) == 6   # 155 us, in pairs 8: 167
    assert pieces(1, 64 * 128, 20, 64, 128) == 5   # 177, 11: 194
    assert pieces(1, 64 * 96, 40, 64, 128) == 3    # 206, 6: 229
    assert pieces(1, 64 * 512, 9, 64, 128) == 16   # 327, 24: 350
    assert pieces(1, 64 * 32, 32, 64, 64) == 3     # 77, 4: 81
    assert pieces(4, 4096, 32, 64, 128) == 1 and pieces(2, 8192, 32, 64, 128) == 3


def test_prompts_go_in_chunks_where_that_is_shorter():
    """From the first length on that is named; the measured times that it comes from stand beside the rule in csrc/delta_tc.cu."""
    for b, nh, H, N, first in ((1, 24, 64, 128, 112), (1, 8, 64, 64, 112), (1, 32, 128, 64, 112), (1, 19, 128, 128, 112), (1, 20, 128, 128, 72),
                               (1, 38, 128, 128, 72), (1, 39, 128, 128, 56), (8, 24, 64, 64, 56), (255, 1, 64, 64, 56), (256, 1, 64, 64, 40),
                               (4, 32, 128, 128, 40), (1023, 1, 64, 128, 40), (1024, 1, 64, 128, 24), (32, 32, 128, 128, 24)):
        assert need(b, first - 1, nh, H, N) == 0 and need(b, first, nh, H, N) > 0, (b, nh, H, N)
