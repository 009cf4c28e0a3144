"""GPU tests of the operators around the layers (include/language.h) at the edges of what their calls take:
row strides beyond 32 bits within a tile."""
import pytest
import torch

import retentive_network_scale_amd as rn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(seed, *shape, dt=F32):
    return torch.randn(*shape, generator=_gen(seed)).to(dt)


# ------------------------------------------------------------------------------------ linear
@pytest.mark.parametrize("ld", [(1 << 26) + (1 << 22) + 8, (1 << 26) + (1 << 22) + 7])
@pytest.mark.parametrize("M,N,K", [(70, 320, 136), (128, 32000, 72), (128, 2100, 65), (9, 40, 72), (3, 40, 72)])
def test_linear_rows_far_apart(M, N, K, ld):
    """The last token of each of many long prompts: rows of x so far apart that a tile's offsets pass 2^32
    elements.  The result is that of the same rows one behind the other, and so is dw: each is the same
    sum in the same order."""
    rows = _r(1, M, K, dt=BF).to(DEV)
    far = torch.empty(M * ld, dtype=BF, device=DEV).as_strided((M, K), (ld, 1))  # what lies between has no values
    far.copy_(rows)
    w, b, d_o = (_r(2, N, K) * K ** -0.5).to(BF).to(DEV), _r(3, N, dt=BF).to(DEV), _r(4, M, N, dt=BF).to(DEV)
    assert torch.equal(rn.linear(far, w, b), rn.linear(rows, w, b))
    far_g, g = (rn.linear_bwd(x, w, d_o, dbias=True) for x in (far, rows))
    assert all(torch.equal(s, t) for s, t in zip(far_g, g))
