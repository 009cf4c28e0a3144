"""Host side of the recurrent-layer operators on the CPU: what their argument checks compare, beside the
refusals themselves.  No call here reaches a kernel."""
import retentive_network_scale_amd as rn
from tests.test_recurrent_abi_cpu import INVALID, P, _bwd


def test_scan_bwd_workspace_is_what_the_call_needs():
    """An arena passed with its full size meets neighbours only within the bytes that the call uses: the next check
    (the workspace's alignment) is reached."""
    need = rn.lib().selective_scan_bwd_workspace_bytes(2, 60, 64, 16, 2)
    assert 0 < need < 1 << 24
    assert _bwd(ws=P(21, 8), wb=1 << 28, dh0=P(22), du=P(23)) == INVALID
    assert b"aligned" in rn.lib().retention_last_error()
    assert _bwd(ws=P(21, 8), wb=1 << 28, dh0=P(21, 64)) == INVALID
    assert b"overlaps" in rn.lib().retention_last_error()
