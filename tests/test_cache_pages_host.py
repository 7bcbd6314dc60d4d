"""Refusals of the cache-page calls, before any launch (no GPU needed), and the definition the GPU tests use."""
import pytest
import torch

from cache_plain import Cache, batch

P = 1 << 20   # a 256-byte aligned fake device address; never dereferenced
Q = 1 << 24   # another, 16 MiB on


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_75_b200 as fa
    return fa


def fork(fa, **kw):
    a = dict(k=P, v=P, ks=0, vs=0, eb=2, bt=P, sl=P, S=4, par=P, N=4, fp=P, fc=P, cap=100, bto=Q, slo=Q, fco=Q, np=100, Hkv=8,
             d=128, ps=16, maxp=10)
    a.update(kw)
    return fa.library().fa_cache_fork(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), -1), (dict(N=-1), -1), (dict(cap=-1), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(eb=4), -1), (dict(eb=1), -1),
    (dict(ks=P, vs=P), -1), (dict(eb=1, ks=P), -1), (dict(np=0), -1), (dict(Hkv=0), -1), (dict(maxp=0), -1),
    (dict(d=96), -2), (dict(ps=32), -2), (dict(S=8193), -2), (dict(N=8193), -2), (dict(np=1 << 30), -2),
    (dict(bt=0), -1), (dict(sl=0), -1), (dict(par=0), -1), (dict(fp=0), -1), (dict(fc=0), -1), (dict(bto=0), -1),
    (dict(slo=0), -1), (dict(fco=0), -1), (dict(k=P + 8), -3), (dict(bt=P + 2), -3), (dict(fco=Q + 1), -3),
    (dict(eb=1, ks=P + 2, vs=P), -3), (dict(bto=P), -1), (dict(bto=P + 40), -1), (dict(slo=P), -1),
    (dict(fco=P), -1)])
def test_fork_rejects(fa, kw, status):
    assert fork(fa, **kw) == status


def append(fa, **kw):
    a = dict(kn=P, vn=P, cu=P, S=4, T=9, k=P, v=P, bt=P, sl=P, fp=P, fc=P, cap=100, slo=Q, fco=Q, np=100, Hkv=8, d=128, ps=16,
             maxp=10)
    a.update(kw)
    return fa.library().fa_cache_append(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), -1), (dict(T=-1), -1), (dict(cap=-2), -1), (dict(S=0), -1), (dict(kn=0), -1), (dict(cu=0), -1), (dict(k=0), -1),
    (dict(bt=0), -1), (dict(sl=0), -1), (dict(fp=0), -1), (dict(fc=0), -1), (dict(slo=0), -1), (dict(fco=0), -1),
    (dict(d=80), -2), (dict(ps=8), -2), (dict(S=9000), -2), (dict(T=(1 << 30) + 5), -2), (dict(vn=P + 8), -3),
    (dict(cu=P + 1), -3), (dict(slo=P), -1), (dict(fco=P), -1), (dict(np=0), -1)])
def test_append_rejects(fa, kw, status):
    assert append(fa, **kw) == status


def test_collect_rejects(fa):
    def call(**kw):
        a = dict(bt=P, sl=P, S=4, maxp=10, np=100, ps=16, fp=P, fc=P, ws=P, wsb=1 << 20)
        a.update(kw)
        return fa.library().fa_cache_collect(*a.values(), None)
    for kw, status in ((dict(S=-1), -1), (dict(bt=0), -1), (dict(sl=0), -1), (dict(fp=0), -1), (dict(fc=0), -1),
                       (dict(np=0), -1), (dict(maxp=0), -1), (dict(ps=32), -2), (dict(S=65536), -2),
                       (dict(np=1 << 28), -2), (dict(fc=P + 2), -3), (dict(ws=0), -4), (dict(wsb=8), -4),
                       (dict(ws=P + 16), -3)):
        assert call(**kw) == status, kw
    assert fa.cache_collect_workspace_bytes(0) == 0
    assert fa.cache_collect_workspace_bytes(100) == 256
    assert fa.cache_collect_workspace_bytes(70000) == 8960


def test_compact_rejects(fa):
    def call(**kw):
        a = dict(k=P, v=P, ks=0, vs=0, eb=2, bt=P, sl=P, S=4, bto=Q, fp=P, fc=P, np=100, Hkv=8, d=128, ps=16, maxp=10,
                 ws=P, wsb=1 << 20)
        a.update(kw)
        return fa.library().fa_cache_compact(*a.values(), None)
    for kw, status in ((dict(S=-1), -1), (dict(k=0), -1), (dict(eb=3), -1), (dict(eb=1), -1), (dict(bto=0), -1),
                       (dict(fp=0), -1), (dict(d=96), -2), (dict(ps=1), -2), (dict(S=70000), -2), (dict(v=P + 4), -3),
                       (dict(bto=P + 4), -1), (dict(ws=0), -4), (dict(wsb=100), -4), (dict(ws=P + 128), -3)):
        assert call(**kw) == status, kw
    assert fa.cache_compact_workspace_bytes(100) == 256 + 256 + 3 * 512
    assert fa.cache_compact_workspace_bytes(-1) == 0


def test_copy_rejects(fa):
    def call(**kw):
        a = dict(k=P, v=P, ks=0, vs=0, eb=2, src=P, dst=P, n=3, np=100, Hkv=8, d=128, ps=16)
        a.update(kw)
        return fa.library().fa_cache_copy_pages(*a.values(), None)
    for kw, status in ((dict(n=-1), -1), (dict(src=0), -1), (dict(dst=0), -1), (dict(k=0), -1), (dict(d=32), -2),
                       (dict(ps=64), -2), (dict(dst=P + 2), -3), (dict(eb=1, ks=P), -1)):
        assert call(**kw) == status, kw
    assert call(n=0, src=0) == 0


def test_binding_refuses(fa):
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(fa.FAError):
        fa.cache_collect(t, t[:, 0], t[0], t[0, :1])          # not CUDA tensors
    assert fa.status_string(fa.FA_ERR_PAGES) != "unknown status"


def test_definition():
    """The definition itself on a case small enough to follow: 20 tokens, forked twice, one goes on."""
    b = batch([20], 6, 1, 64, seed=1)
    c = Cache(b["k"], b["v"], b["table"], [20], b["free"])
    out = torch.full((2, b["table"].shape[1]), -1, dtype=torch.int32)
    lens, short = c.fork([0, 0], out)
    first, last = b["table"][0, :2].tolist()
    low = min(b["free"])
    assert lens == [20, 20] and not short
    assert out[0, :2].tolist() == [first, last] and out[1, :2].tolist() == [first, low]
    assert torch.equal(c.k[low, :4], b["k"][last, :4]) and torch.equal(c.k[low, 4:], b["k"][low, 4:])
    c.table, c.lens = out, lens
    new = torch.ones((1, 1, 64), dtype=torch.bfloat16)
    lens, _ = c.append(new, new, [0, 0, 1])
    assert lens == [20, 21] and torch.equal(c.k[low, 4], new[0]) and torch.equal(c.k[last], b["k"][last])
    assert sorted(c.collect() + sorted(c.in_use())) == list(range(6))
    moved = torch.full_like(out, -1)
    free = c.compact(moved)
    assert free == [5, 4, 3] and sorted(set(moved[:, :2].flatten().tolist())) == [0, 1, 2]
