"""Host side of the recurrent-layer operators on the CPU: what their argument checks compare, beside the
refusals themselves.  No call here reaches a kernel."""
import importlib.util

import pytest
import torch

import retentive_network_scale_amd as rn
from tests.test_recurrent_abi_cpu import INVALID, P, _bwd, _conv_bwd, _scan


def test_scan_bwd_workspace_is_what_the_call_needs():
    """An arena passed with its full size meets neighbours only within the bytes that the call uses: the next check
    (the workspace's alignment) is reached."""
    need = rn.lib().selective_scan_bwd_workspace_bytes(2, 60, 64, 16, 2)
    assert 0 < need < 1 << 24
    assert _bwd(ws=P(21, 8), wb=1 << 28, dh0=P(22), du=P(23)) == INVALID
    assert b"aligned" in rn.lib().retention_last_error()
    assert _bwd(ws=P(21, 8), wb=1 << 28, dh0=P(21, 64)) == INVALID
    assert b"overlaps" in rn.lib().retention_last_error()


LENGTHS = [*range(1, 1200), *range(1200, 6000, 13), *range(6000, 70000, 997), *(1 << i for i in range(17, 24))]


@pytest.mark.parametrize("B,D,N,G", [(1, 512, 64, 1), (1, 2048, 64, 1), (1, 2048, 16, 1), (2, 64, 16, 2), (3, 500, 32, 1),
                                     (8, 1000, 8, 2), (1, 1, 1, 1), (16, 4096, 4, 4), (2, 4096, 16, 1), (1, 16, 24, 1)])
def test_scan_workspace_holds_for_shorter_sequences(B, D, N, G):
    """The queries grow with L, and cover what a call of that L asks for: one workspace, of the longest, serves all."""
    lib = rn.lib()
    before = (0, 0)
    for L in (n for n in LENGTHS if B * n <= 1 << 24):
        need = (lib.selective_scan_workspace_bytes(B, L, D, N, G), lib.selective_scan_bwd_workspace_bytes(B, L, D, N, G))
        assert need[0] >= before[0] and need[1] >= before[1], (L, before, need)
        before = need
        big = dict(bt=B, L=L, d=D, n=N, g=G, uld=D, dld=D, zld=D, bld=G * N, cld=G * N)
        # stand-ins far apart; a workspace that is large enough is refused for its alignment only
        at = {k: P(i << 24) for i, k in enumerate(("u", "delta", "A", "B", "C", "D", "z", "bias"), 1)}
        if need[0]:
            assert _scan(**big, **at, out=P(20 << 24), h0=None, hT=None, ws=P(30 << 24, 8), wb=need[0]) == INVALID
            assert b"16-byte aligned" in lib.retention_last_error()
        grads = {k: P(i << 24) for i, k in enumerate(("d_o", "du", "dd", "dA", "dB", "dC", "dD", "dz", "db"), 20)}
        assert _bwd(**big, **at, **grads, h0=None, dhT=None, dh0=None, ws=P(40 << 24, 8), wb=need[1]) == INVALID
        assert b"16-byte aligned" in lib.retention_last_error()


@pytest.mark.parametrize("B,D", [(1, 4096), (1, 1), (3, 1000), (4, 4096), (16, 67), (2, 64)])
def test_conv_workspace_holds_for_shorter_sequences(B, D):
    lib = rn.lib()
    before = 0
    for L in (n for n in LENGTHS if B * n <= 1 << 24):
        need = lib.causal_conv1d_bwd_workspace_bytes(B, L, D, 4)
        assert need >= before, (L, before, need)
        before = need
        at = {k: P(i << 24) for i, k in enumerate(("x", "w", "bias", "d_o", "dx", "dw", "db"), 1)}
        assert _conv_bwd(**at, s0=None, dsT=None, ds0=None, bt=B, L=L, d=D, xld=D, ws=P(20 << 24, 8), wb=need) == INVALID
        assert b"16-byte aligned" in lib.retention_last_error()


def test_binding_imports_without_a_gpu_runtime(monkeypatch):
    """torch built for the CPU alone lacks the stream and device queries: that shows at a call, not at import."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location(rn.__name__ + ".recurrent_again", rn.recurrent.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    with pytest.raises(TypeError):
        module.linear_w4(torch.zeros(1, 32), torch.zeros(1, 16), torch.zeros(1, 1))
