"""Refusals of the cross-attention calls, before any launch (no GPU needed), and the definition the GPU tests use."""
import math

import pytest
import torch

from cross_plain import attend

P = 1 << 20   # a 256-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_75_b200 as fa
    return fa


def fwd(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, sl=P, B=2, Hq=8, Hkv=2, Nq=5, Nk=9, d=128, scale=0.1, od=0)
    a.update(kw)
    return fa.library().fa_fwd_cross(*a.values(), None)


def fwd_packed(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, cq=P, ck=P, S=2, Tq=10, Tk=18, mq=6, mk=10, Hq=8, Hkv=2, d=64, scale=0.1, od=1)
    a.update(kw)
    return fa.library().fa_fwd_varlen_cross(*a.values(), None)


def bwd(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, do=P, lse=P, dq=P, dk=P, dv=P, sl=P, B=2, Hq=8, Hkv=2, Nq=5, Nk=9, d=128, scale=0.1, ws=P,
             wsb=1 << 30)
    a.update(kw)
    return fa.library().fa_bwd_cross(*a.values(), None)


def bwd_packed(fa, **kw):
    a = dict(q=P, k=P, v=P, o=P, do=P, lse=P, dq=P, dk=P, dv=P, cq=P, ck=P, S=2, Tq=10, Tk=18, mq=6, mk=10, Hq=8, Hkv=2, d=64,
             scale=0.1, ws=P, wsb=1 << 30)
    a.update(kw)
    return fa.library().fa_bwd_varlen_cross(*a.values(), None)


SIZES = [(dict(Hq=0), -1), (dict(Hkv=3), -1), (dict(scale=0.0), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
         (dict(d=96), -2), (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(o=0), -1), (dict(q=P + 8), -3),
         (dict(v=P + 2), -3), (dict(o=P + 4), -3), (dict(lse=P + 2), -3)]
DENSE = [(dict(B=-1), -1), (dict(Nq=-1), -1), (dict(Nk=-2), -1), (dict(sl=P + 1), -3), (dict(B=1 << 20, Nk=1 << 11), -2)]
PACKED = [(dict(S=-1), -1), (dict(Tq=-1), -1), (dict(Tk=-1), -1), (dict(mq=-1), -1), (dict(mk=-1), -1), (dict(cq=0), -1),
          (dict(ck=0), -1), (dict(cq=P + 2), -3), (dict(ck=P + 1), -3)]
GRADS = [(dict(do=0), -1), (dict(lse=0), -1), (dict(dq=0), -1), (dict(dk=0), -1), (dict(dv=0), -1), (dict(do=P + 8), -3),
         (dict(dk=P + 2), -3), (dict(ws=0), -4), (dict(wsb=64), -4), (dict(ws=P + 16), -3)]


@pytest.mark.parametrize("kw,status", SIZES + DENSE + [(dict(od=2), -1)])
def test_fwd_rejects(fa, kw, status):
    assert fwd(fa, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + PACKED + [(dict(od=-1), -1)])
def test_fwd_packed_rejects(fa, kw, status):
    assert fwd_packed(fa, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + DENSE + GRADS)
def test_bwd_rejects(fa, kw, status):
    assert bwd(fa, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + PACKED + GRADS)
def test_bwd_packed_rejects(fa, kw, status):
    assert bwd_packed(fa, **kw) == status


def test_nothing_to_do(fa):
    assert fwd(fa, B=0) == 0 and fwd(fa, Nq=0) == 0 and fwd_packed(fa, S=0) == 0 and fwd_packed(fa, Tq=0) == 0
    assert bwd(fa, B=0) == 0 and bwd(fa, Nq=0, Nk=0) == 0 and bwd_packed(fa, S=0) == 0


def test_binding_refuses(fa):
    t = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(fa.FAError):
        fa.fwd_cross(t, t, t)                                  # not CUDA tensors


def test_definition_against_differences():
    """The definition's gradients against central differences of sum(do * o)."""
    g = torch.Generator().manual_seed(7)
    q, k, v, do = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 4, 8), (5, 2, 8), (5, 2, 8), (3, 4, 8)))
    got = attend(q, k, v, 0.3, do)
    h = 1e-5
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        num = torch.zeros_like(x)
        for i in range(x.numel()):
            old = x.view(-1)[i].item()
            f = []
            for step in (h, -h):
                x.view(-1)[i] = old + step
                f.append((attend(q, k, v, 0.3)["o"][0] * do).sum().item())
            x.view(-1)[i] = old
            num.view(-1)[i] = (f[0] - f[1]) / (2 * h)
        # central differences: O(h^2) ~ 1e-10 of third derivatives of order 1, and 1e-16 / h ~ 1e-11 of cancellation
        assert (num - got[name][0]).abs().max() < 1e-8


def test_definition_without_keys():
    q = torch.ones((2, 2, 8))
    none = torch.zeros((0, 1, 8))
    r = attend(q, none, none, 0.5, q)
    assert (r["o"][0] == 0).all() and torch.isneginf(r["lse"][0]).all() and (r["dq"][0] == 0).all()
