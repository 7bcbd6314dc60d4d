"""Refusals of fa_decode_shared and fa_decode_cross, before any launch (no GPU needed)."""
import math

import pytest
import torch

P = 1 << 20   # a 256-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_75_b200 as fa
    return fa


def shared(fa, **kw):
    a = dict(q=P, k=P, v=P, bt=P, sl=P, cg=P, pl=P, o=P, lse=P, sinks=P, S=4, ng=2, np=100, Hq=8, Hkv=2, d=128, ps=16, maxp=10,
             scale=0.1, ws=P, wsb=1 << 40)
    a.update(kw)
    return fa.library().fa_decode_shared(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), -1), (dict(ng=-1), -1), (dict(ng=5), -1), (dict(np=-1), -1), (dict(np=0), -1), (dict(maxp=0), -1),
    (dict(Hq=7), -1), (dict(Hkv=0), -1), (dict(scale=-1.0), -1), (dict(scale=math.nan), -1), (dict(d=80), -2), (dict(ps=32), -2),
    (dict(S=1025), -2), (dict(Hq=258, Hkv=2), -2), (dict(np=1 << 27), -2), (dict(maxp=1 << 22), -2), (dict(S=1024, maxp=1 << 21), -2),
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(bt=0), -1), (dict(sl=0), -1), (dict(cg=0), -1), (dict(pl=0), -1),
    (dict(o=0), -1), (dict(q=P + 8), -3), (dict(k=P + 2), -3), (dict(bt=P + 2), -3), (dict(cg=P + 1), -3), (dict(pl=P + 2), -3),
    (dict(lse=P + 2), -3), (dict(sinks=P + 3), -3), (dict(ws=0), -4), (dict(wsb=1000), -4), (dict(ws=P + 16), -3)])
def test_shared_rejects(fa, kw, status):
    assert shared(fa, **kw) == status


def cross(fa, **kw):
    a = dict(q=P, k=P, v=P, sl=P, o=P, lse=P, B=3, Hq=8, Hkv=2, Nq=1, Nk=50, d=64, scale=0.1, ws=P, wsb=1 << 40)
    a.update(kw)
    return fa.library().fa_decode_cross(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(Nq=-1), -1), (dict(Nk=-1), -1), (dict(Hq=7), -1), (dict(scale=0.0), -1), (dict(d=32), -2),
    (dict(Hq=258, Hkv=2), -2), (dict(Nq=140000), -2), (dict(B=1 << 20, Nk=1 << 12), -2), (dict(B=1, Nk=1 << 27), -2),
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(o=0), -1), (dict(q=P + 8), -3), (dict(sl=P + 2), -3),
    (dict(lse=P + 1), -3), (dict(ws=0), -4), (dict(wsb=64), -4), (dict(ws=P + 128), -3)])
def test_cross_rejects(fa, kw, status):
    assert cross(fa, **kw) == status


def test_nothing_to_do(fa):
    assert shared(fa, S=0, ng=0) == 0 and cross(fa, B=0) == 0 and cross(fa, Nq=0) == 0


def test_workspace_bytes(fa):
    f, g = fa.decode_shared_workspace_bytes, fa.decode_cross_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(1025, 8, 2, 128) == 0 and f(4, 9, 2, 128) == 0 and f(4, 8, 2, 96) == 0
    assert 0 < f(1, 8, 8, 64) < f(64, 32, 8, 128) < f(1024, 32, 8, 128)
    assert g(0, 8, 2, 1, 128) == 0 and g(4, 8, 2, 0, 128) == 0 and g(4, 8, 3, 1, 128) == 0
    assert 0 < g(1, 16, 16, 1, 64) < g(64, 16, 16, 1, 64) < g(64, 16, 16, 5, 64)
    assert g(1 << 14, 8, 8, 1, 64) == g(1024, 8, 8, 1, 64)       # larger batches run in turns


def test_binding_refuses(fa):
    t = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(fa.FAError):
        fa.decode_shared(t, t[None], t[None], i[None], i, i, i)          # not CUDA tensors
    with pytest.raises(fa.FAError):
        fa.decode_cross(t[None], t[None], t[None])


def test_stream_argument(fa):
    """A stream of another device is refused; the calls keep their signatures."""
    import inspect
    for f in (fa.fwd_cross, fa.fwd_varlen_cross, fa.bwd_cross, fa.bwd_varlen_cross, fa.decode_shared, fa.decode_cross,
              fa.cache_collect, fa.cache_compact):
        assert inspect.signature(f).parameters["stream"].default is None

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    class OnGpu(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 0)

    q = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16).as_subclass(OnGpu)
    for call in (lambda: fa.decode_cross(q, q, q, stream=Stream()), lambda: fa.decode_cross(q=q, k=q, v=q, stream=Stream()),
                 lambda: fa.decode_cross(q, q, q, None, None, None, None, True, None, Stream())):
        with pytest.raises(fa.FAError, match="stream"):
            call()
