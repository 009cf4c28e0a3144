"""C-ABI checks of the operators around the layers (include/language.h) that need no GPU: exports, and the
refusal of bad arguments on the host before any launch (no call here reaches a kernel)."""
import ctypes
import os
import re

import pytest
import torch

import retentive_network_scale_amd as rn
from tests.test_recurrent_abi_cpu import P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16 = 0, 1


def test_every_declared_symbol_is_exported_and_bound():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "language.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:embedding|group|linear|beam)\w*)\s*\(", src))
    assert names == set(rn.LANGUAGE_SYMBOLS)
    for n in names:
        assert hasattr(rn.lib(), n) and n in rn.__all__, n


def _embed(**kw):
    v = dict(ids=P(1), table=P(2), out=P(3), n=100, V=1000, D=64, scale=2.0, ind=BF16, outd=BF16)
    v.update(kw)
    return rn.lib().embedding(*v.values(), None)


def _embed_bwd(**kw):
    v = dict(ids=P(1), d_o=P(2), dt=P(3), n=100, V=1000, D=64, ld=64, scale=2.0, ind=BF16, outd=BF16, ws=P(4), wb=1 << 20)
    v.update(kw)
    return rn.lib().embedding_bwd(*v.values(), None)


SIZES = [(dict(n=-1), INVALID), (dict(V=0), INVALID), (dict(D=0), INVALID), (dict(ind=5), INVALID), (dict(outd=-1), INVALID),
         (dict(ids=None), INVALID), (dict(n=(1 << 28) + 1), UNSUPPORTED), (dict(V=(1 << 24) + 1), UNSUPPORTED),
         (dict(D=(1 << 20) + 1, ld=1 << 21), UNSUPPORTED), (dict(n=1 << 28, D=1 << 10, ld=1 << 10), UNSUPPORTED),
         (dict(V=1 << 24, D=1 << 14, ld=1 << 14), UNSUPPORTED), (dict(ids=P(1, 2)), INVALID)]


@pytest.mark.parametrize("kw,code", [(({k: v for k, v in kw.items() if k != "ld"}), c) for kw, c in SIZES] + [
    (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(table=P(2, 1)), INVALID), (dict(out=P(3, 1)), INVALID),
    (dict(out=P(2, 1000)), INVALID), (dict(out=P(1)), INVALID)])
def test_embedding_refuses(kw, code):
    assert _embed(**kw) == code
    assert rn.lib().retention_last_error() != b""


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(d_o=None), INVALID), (dict(dt=None), INVALID), (dict(ld=63), INVALID), (dict(ld=1 << 32), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wb=100), WORKSPACE), (dict(ws=P(4, 8)), INVALID), (dict(ws=P(2)), INVALID),
    (dict(dt=P(2)), INVALID), (dict(dt=P(4)), INVALID), (dict(dt=P(1)), INVALID), (dict(d_o=P(2, 1)), INVALID)])
def test_embedding_bwd_refuses(kw, code):
    assert _embed_bwd(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_embedding_workspace_query():
    q = rn.lib().embedding_bwd_workspace_bytes
    assert q(0, 1000, 64) == 0 == q(-1, 1000, 64) == q(100, 0, 64) == q(100, 1000, 1 << 21)
    assert q(100, 1000, 64) >= 100 * 4 + 1001 * 4
    assert _embed(n=0, ids=None, table=None, out=None) == 0


def _norm(**kw):
    v = dict(x=P(1), gate=P(2), w=P(3), b=P(4), out=P(5), lengths=None, B=2, H=3, L=10, W=64, sb=1920, sh=640, sl=64,
             gld=192, silu=1, eps=1e-5, ind=BF16, outd=BF16)
    v.update(kw)
    return rn.lib().group_norm_gate(*v.values(), None)


def _norm_bwd(**kw):
    v = dict(x=P(1), gate=P(2), w=P(3), b=P(4), d_o=P(5), lengths=None, dx=P(6), dgate=P(7), dw=P(8), db=P(9), B=2, H=3, L=10,
             W=64, sb=1920, sh=640, sl=64, gld=192, silu=1, eps=1e-5, ind=BF16, outd=BF16, ws=P(10), wb=1 << 20)
    v.update(kw)
    return rn.lib().group_norm_gate_bwd(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(L=-1), INVALID), (dict(W=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(ind=2), INVALID),
    (dict(outd=9), INVALID), (dict(x=None), INVALID), (dict(sb=10), INVALID), (dict(sh=63), INVALID), (dict(sl=63), INVALID),
    (dict(sl=-64), INVALID), (dict(gld=191), INVALID), (dict(x=P(1, 1)), INVALID), (dict(gate=P(2, 1)), INVALID),
    (dict(w=P(3, 2)), INVALID), (dict(b=P(4, 1)), INVALID), (dict(lengths=P(11, 2)), INVALID),
    (dict(W=1025, sl=1025, sh=10250, sb=30750, gld=3 * 1025), UNSUPPORTED), (dict(sl=1 << 32), UNSUPPORTED),
    (dict(sb=1 << 40), UNSUPPORTED), (dict(gld=1 << 32), UNSUPPORTED), (dict(B=1 << 20, L=1 << 10), UNSUPPORTED),
    (dict(H=1 << 16, W=8, gld=1 << 19, sh=80, sb=80 << 16, sl=8), UNSUPPORTED),
    (dict(B=1 << 18, L=1 << 8, H=64, W=64, gld=64 * 64), UNSUPPORTED),
])
def test_norm_refuses(kw, code):
    assert _norm(**kw) == code
    assert _norm_bwd(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_norm_refuses_overlaps_and_workspaces():
    for kw in (dict(out=P(1)), dict(out=P(2, 64)), dict(out=P(3)), dict(out=P(4)), dict(out=None), dict(out=P(5, 1)),
               dict(lengths=P(5))):
        assert _norm(**kw) == INVALID, kw
    for kw in (dict(dx=P(1)), dict(dgate=P(2)), dict(dgate=P(6)), dict(dw=P(3)), dict(db=P(8)), dict(dx=P(5)), dict(dx=None),
               dict(dgate=None), dict(gate=None), dict(d_o=None), dict(ws=P(1)), dict(ws=P(10, 4)), dict(ws=P(6)),
               dict(dw=P(8, 2))):
        assert _norm_bwd(**kw) == INVALID, kw
    assert _norm_bwd(ws=None) == WORKSPACE == _norm_bwd(wb=64)
    assert _norm(L=0, x=None, out=None) == 0
    q = rn.lib().group_norm_gate_bwd_workspace_bytes
    assert q(2, 3, 10, 64) > 0 and q(2, 3, 0, 64) == 0 == q(2, 3, 10, 4096) == q(0, 3, 10, 64)


def _linear(**kw):
    v = dict(x=P(1), w=P(2), bias=P(3), res=P(4), out=P(5), pre=P(6), M=100, N=48, K=64, ld=64, act=1, rd=BF16, od=BF16,
             ws=P(7), wb=1 << 23)
    v.update(kw)
    return rn.lib().linear(*v.values(), None)


def _linear_bwd(**kw):
    v = dict(x=P(1), w=P(2), d_o=P(3), pre=P(4), dx=P(5), dw=P(6), db=P(7), M=100, N=48, K=64, ld=64, act=1, od=BF16, ws=P(8),
             wb=1 << 23)
    v.update(kw)
    return rn.lib().linear_bwd(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(od=2), INVALID), (dict(act=3), INVALID),
    (dict(act=-1), INVALID), (dict(ld=63), INVALID), (dict(ld=1 << 32), UNSUPPORTED), (dict(N=(1 << 22) + 1), UNSUPPORTED),
    (dict(K=(1 << 22) + 1, ld=1 << 23), UNSUPPORTED), (dict(M=(1 << 28) + 1), UNSUPPORTED),
    (dict(M=1 << 28, N=1 << 10), UNSUPPORTED), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=P(1, 1)), INVALID),
    (dict(w=P(2, 1)), INVALID),
])
def test_linear_refuses(kw, code):
    assert _linear(**kw) == code
    assert _linear_bwd(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_linear_refuses_overlaps_and_workspaces():
    for kw in (dict(out=P(1)), dict(out=P(2)), dict(out=P(3)), dict(out=P(4, 2)), dict(out=P(4), od=F32), dict(pre=P(5)),
               dict(pre=P(1)), dict(out=None), dict(rd=7), dict(bias=P(3, 1)), dict(res=P(4, 1)), dict(out=P(5, 1)),
               dict(pre=P(6, 1))):
        assert _linear(**kw) == INVALID, kw
    big = dict(M=100, N=48, K=4096, ld=4096)
    need = rn.lib().linear_workspace_bytes(100, 48, 4096)
    assert need > 0
    assert _linear(**big, ws=None) == WORKSPACE == _linear(**big, wb=need - 1)
    assert _linear(**big, ws=P(7, 8)) == INVALID == _linear(**big, ws=P(4))
    for kw in (dict(dx=P(1)), dict(dw=P(2)), dict(dw=P(5)), dict(db=P(3)), dict(dx=P(4)), dict(d_o=None), dict(pre=None),
               dict(ws=P(3)), dict(ws=P(8, 4)), dict(db=P(7, 2)), dict(pre=P(4, 1))):
        assert _linear_bwd(**kw) == INVALID, kw
    assert _linear_bwd(ws=None) == WORKSPACE == _linear_bwd(wb=64)
    assert _linear(M=0, x=None, w=None, out=None) == 0
    # calls without tokens are checked as well, and need no workspace
    assert _linear_bwd(M=0, dw=P(7), ws=None) == INVALID == _norm_bwd(L=0, db=P(8), ws=None)
    q = rn.lib()
    assert q.linear_workspace_bytes(0, 48, 64) == 0 == q.linear_workspace_bytes(1, 48, 4096)
    assert q.linear_bwd_workspace_bytes(0, 48, 64) == 0 and q.linear_bwd_workspace_bytes(100, 48, 64) >= 100 * 48 * 2


def _select(**kw):
    v = dict(z=P(1), s=P(2), e=P(3), tok=P(4), par=P(5), out=P(6), B=2, W=4, V=100, K=8, ld=100, eos=2, dt=BF16, ws=P(7),
             wb=1 << 20)
    v.update(kw)
    return rn.lib().beam_select(*v.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(W=0), INVALID), (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(W=1, V=7), INVALID),
    (dict(ld=99), INVALID), (dict(ld=1 << 32), UNSUPPORTED), (dict(eos=-1), INVALID), (dict(eos=100), INVALID),
    (dict(dt=3), INVALID), (dict(z=None), INVALID), (dict(s=None), INVALID), (dict(tok=None), INVALID),
    (dict(par=None), INVALID), (dict(out=None), INVALID), (dict(z=P(1, 1)), INVALID), (dict(s=P(2, 2)), INVALID),
    (dict(tok=P(4, 1)), INVALID), (dict(K=65), UNSUPPORTED), (dict(W=65), UNSUPPORTED),
    (dict(W=64, V=1 << 24, ld=1 << 24), UNSUPPORTED), (dict(W=64, V=65537, ld=65537), UNSUPPORTED),
    (dict(V=(1 << 24) + 1, ld=1 << 25), UNSUPPORTED),
    (dict(B=1 << 23), UNSUPPORTED), (dict(V=20000, ld=20000, ws=None), WORKSPACE), (dict(V=20000, ld=20000, wb=16), WORKSPACE),
    (dict(V=20000, ld=20000, ws=P(7, 8)), INVALID), (dict(K=33, ws=None), WORKSPACE),
    (dict(tok=P(1)), INVALID), (dict(out=P(2)), INVALID), (dict(par=P(4)), INVALID), (dict(V=20000, ld=20000, ws=P(6)), INVALID),
    (dict(V=20000, ld=20000, ws=P(1)), INVALID), (dict(tok=P(3)), INVALID),
])
def test_select_refuses(kw, code):
    assert _select(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_select_without_requests():
    assert _select(B=0, z=None, ws=None, wb=0) == 0
    q = rn.lib().beam_select_workspace_bytes
    assert q(0, 4, 100, 8) == 0 == q(2, 65, 100, 8) and q(2, 4, 20000, 8) > 0


def _reorder(states=((21, 4096), (22, 4096)), parents=P(30), B=2, W=4, count=None, null=False):
    n = len(states)
    at = (ctypes.c_void_p * max(n, 1))(*(a if a is None else a << 24 for a, _ in states))
    size = (ctypes.c_longlong * max(n, 1))(*(s for _, s in states))
    return rn.lib().beam_reorder(None if null else at, size, n if count is None else count, parents, B, W, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(W=0), INVALID), (dict(W=65), UNSUPPORTED), (dict(count=-1), INVALID), (dict(null=True), INVALID),
    (dict(count=65), UNSUPPORTED), (dict(B=1 << 16), UNSUPPORTED), (dict(parents=None), INVALID), (dict(parents=P(30, 2)), INVALID),
    (dict(states=((21, -1),)), INVALID), (dict(states=((None, 64),)), INVALID), (dict(states=((21, 64), (21, 64))), INVALID),
    (dict(states=((21, 1 << 22), (22, 64))), INVALID), (dict(states=((30, 64),)), INVALID),
    (dict(states=((21, 1 << 41),)), UNSUPPORTED), (dict(states=tuple((1 + i << 17, 1 << 24) for i in range(60)), W=1, B=65535), UNSUPPORTED),
])
def test_reorder_refuses(kw, code):
    assert _reorder(**kw) == code
    assert rn.lib().retention_last_error() != b""


def test_reorder_of_nothing():
    assert _reorder(states=()) == 0 == _reorder(B=0) == _reorder(states=((21, 0),))


def test_binding_refuses_what_is_not_on_a_gpu():
    t, i = torch.zeros(2, 4, 8), torch.zeros(2, 4, dtype=torch.int32)
    for fn in (lambda: rn.embedding(i, t[0]), lambda: rn.embedding_bwd(i, t, 10), lambda: rn.group_norm_gate(t[None]),
               lambda: rn.group_norm_gate_bwd(t[None], t), lambda: rn.linear(t, t[0]), lambda: rn.linear_bwd(t, t[0], t),
               lambda: rn.beam_select(t, t[..., 0], 2), lambda: rn.beam_reorder([t], i)):
        with pytest.raises(TypeError):
            fn()
