"""A decoding step as a serving loop would record it: the beams fork, each gets its new token, the batch decodes on what it shares, all
in one graph that is replayed on changed parents, lengths and tokens; and forks with too few free pages."""
import math

import pytest
import torch

from cache_plain import Cache, batch, pages_of
from cross_plain import attend, check

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (6, 2, 64)])
def test_fork_append_and_decode_in_one_graph(fa, Hq, Hkv, d):
    """Four slots that all continue slots of one prompt of 100 tokens (6 whole pages)."""
    n, prompt = 4, 100
    b = batch([prompt + 30] * n, 80, Hkv, d, seed=1, width=16, share=6)
    held = torch.zeros((80, PAGE), dtype=torch.bool)
    held[b["table"][:, :pages_of(prompt + 30)].flatten().long()] = True
    for t in (b["k"], b["v"]):
        t[~held] = math.nan                            # what no slot holds may be anything
    k, v, table = b["k"].cuda(), b["v"].cuda(), b["table"].cuda()
    lens, parents, cu = i32(b["lens"]), i32(list(range(n))), i32(list(range(n + 1)))
    free, count = i32(b["free"]), i32([len(b["free"])])
    kn, vn, q = (torch.zeros((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    table2 = torch.full_like(table, -1)
    lens2, lens3, count2, count3 = i32([0] * n), i32([0] * n), i32([0]), i32([0])
    groups, prefix = i32([0, n]), i32([prompt])
    ws = torch.empty(fa.decode_shared_workspace_bytes(n, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((n, Hq), device="cuda")

    def step():
        fa.cache_fork(k, v, table, lens, parents, free, count, table2, lens2, count2)
        fa.cache_append(kn, vn, cu, k, v, table2, lens2, free, count2, lens3, count3)
        fa.decode_shared(q, k, v, table2, lens3, groups, prefix, out=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(2)
    for ps, ls in (([0, 1, 2, 3], [130] * 4), ([2, 2, 0, 2], [101, 130, 112, 129]), ([1, 1, 1, 1], [130, 111, 100, 104]),
                   ([3, -1, 3, 0], [112, 127, 128, 113])):
        new = [torch.randn(t.shape, generator=g).to(torch.bfloat16) for t in (kn, vn, q)]
        for t, x in zip((kn, vn, q), new):
            t.copy_(x)
        k.copy_(b["k"]), v.copy_(b["v"]), parents.copy_(i32(ps)), lens.copy_(i32(ls)), table2.fill_(-1)
        # an empty slot shares nothing, and no more is shared than the shortest slot has
        graph.replay()
        torch.cuda.synchronize()
        assert fa.check_device_error() == 0
        c = Cache(b["k"], b["v"], b["table"], ls, b["free"])
        want = torch.full((n, 16), -1, dtype=torch.int32)
        got, short = c.fork(ps, want)
        assert not short
        c.table, c.lens = want, got
        c.lens, short = c.append(new[0], new[1], list(range(n + 1)))
        assert not short and lens3.tolist() == c.lens and torch.equal(table2.cpu(), c.table)
        assert count3.tolist() == [len(c.free)]
        for s in range(n):
            row = c.table[s, :pages_of(c.lens[s])].long()
            keys, values = (t[row].flatten(0, 1)[:c.lens[s]] for t in (c.k, c.v))
            ref = attend(new[2][s:s + 1], keys, values, d ** -0.5)
            check(o[s:s + 1], ref["o"], f"O of slot {s}")
            check(lse[s:s + 1].t(), ref["lse"], f"LSE of slot {s}")


@pytest.mark.parametrize("left", range(6))
def test_fork_with_few_free_pages(fa, left):
    """Four slots need a page; as many as there are get one, in slot order, the others come out empty."""
    lens, parents = [5, 20, 32], [0, 0, 1, 2, 1, 0, 1]
    b = batch(lens, 14, 2, 64, seed=4)
    b["free"] = b["free"][len(b["free"]) - left:]
    k, v = b["k"].cuda(), b["v"].cuda()
    table_out = torch.full((7, b["table"].shape[1]), -9, dtype=torch.int32, device="cuda")
    lens_out, count_out = i32([-9] * 7), i32([-9])
    fa.cache_fork(k, v, b["table"].cuda(), i32(lens), i32(parents), i32(b["free"] + [-1]), i32([left]), table_out, lens_out,
                  count_out)
    assert fa.check_device_error() == (fa.FA_ERR_PAGES if left < 4 else 0)
    c = Cache(b["k"], b["v"], b["table"], lens, b["free"])
    want = torch.full_like(table_out, -9).cpu()
    ref, short = c.fork(parents, want)
    assert short == (left < 4) and ref.count(0) == max(0, 4 - left)
    assert lens_out.tolist() == ref and torch.equal(table_out.cpu(), want) and count_out.tolist() == [len(c.free)]
    assert torch.equal(k.cpu().view(torch.int16), c.k.view(torch.int16)) and torch.equal(v.cpu().view(torch.int16), c.v.view(torch.int16))
