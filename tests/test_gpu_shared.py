"""Decode with shared prefixes (fa_decode_shared) and decode against encoder states (fa_decode_cross) against the
definition in 64 bits, within the bounds cross_plain.py derives (the parts' results are joined in fp32)."""
import math

import pytest
import torch

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
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def pages_of(n):
    return (n + PAGE - 1) // PAGE


class Batch:
    """Sequences of `lens` tokens; those of groups[g] (first, count) share the whole pages of their first prefix[g]
    tokens.  Every slot that no sequence holds is NaN, table entries behind the lengths are out of range."""

    def __init__(self, lens, groups, prefix, Hq, Hkv, d, seed, spare=3, width=1):
        g = torch.Generator().manual_seed(seed)
        S = len(lens)
        shared = [0] * S
        owner = list(range(S))
        for (first, count), p in zip(groups, prefix):
            for s in range(first, first + count):
                shared[s], owner[s] = min([p] + lens[first:first + count]) // PAGE, first
        total = spare + sum(pages_of(n) - (0 if owner[s] == s else shared[s]) for s, n in enumerate(lens))
        ids = torch.randperm(total, generator=g).tolist()
        width = max([width] + [pages_of(n) for n in lens])
        self.table = torch.full((S, width), 1 << 30, dtype=torch.int32)
        self.k = torch.full((total, PAGE, Hkv, d), math.nan, dtype=torch.bfloat16)
        self.v = self.k.clone()
        self.q = torch.randn((S, Hq, d), generator=g).to(torch.bfloat16)
        self.rows = []
        for s, n in enumerate(lens):
            first = 0 if owner[s] == s else shared[s]
            row = self.table[owner[s], :first].tolist() + [ids.pop() for _ in range(pages_of(n) - first)]
            self.table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
            for c in range(first, len(row)):
                fill = min(PAGE, n - c * PAGE)
                self.k[row[c], :fill] = torch.randn((fill, Hkv, d), generator=g).to(torch.bfloat16)
                self.v[row[c], :fill] = torch.randn((fill, Hkv, d), generator=g).to(torch.bfloat16)
            self.rows.append(row)
        self.lens, self.groups, self.prefix = lens, groups, prefix

    def cu(self):
        """Offsets that cover the groups, with groups of no shared token between them."""
        cu, pl, at = [], [], 0
        for (first, count), p in zip(self.groups, self.prefix):
            if first > at:
                cu.append(at)
                pl.append(0)
            cu.append(first)
            pl.append(p)
            at = first + count
        cu.append(at)
        return cu, pl

    def keys(self, s):
        n = self.lens[s]
        row = torch.tensor(self.rows[s], dtype=torch.long)
        return self.k[row].flatten(0, 1)[:n], self.v[row].flatten(0, 1)[:n]

    def run(self, fa, **kw):
        cu, pl = self.cu()
        return fa.decode_shared(self.q.cuda(), self.k.cuda(), self.v.cuda(), self.table.cuda(), i32(self.lens), i32(cu), i32(pl),
                                **kw)

    def check(self, o, lse, scale=None, z=None, only=None):
        scale = scale or self.q.shape[-1] ** -0.5
        for s in only or range(len(self.lens)):
            k, v = self.keys(s)
            want = attend(self.q[s:s + 1], k, v, scale, z=z)
            check(o[s:s + 1], want["o"], f"O of sequence {s}")
            check(lse[s:s + 1].t(), want["lse"], f"LSE of sequence {s}")


CASES = [
    # lens, groups (first, count), prefix
    ([1], [], []),
    ([0], [], []),
    ([0, 5, 0], [], []),
    ([17, 300, 129, 128], [], []),
    ([40, 41], [(0, 2)], [40]),
    ([40, 41], [(0, 2)], [15]),
    ([16, 200, 33], [(0, 3)], [500]),
    ([0, 200, 33], [(0, 3)], [500]),
    ([100, 0, 90, 300, 310, 33], [(0, 1), (2, 3)], [64, 80]),
    ([150 + i for i in range(9)], [(0, 9)], [144]),
    ([1030 + 3 * i for i in range(20)], [(0, 20)], [1024]),
    ([300] * 70, [(0, 33), (33, 37)], [272, 299]),
    ([2000 + i % 7 for i in range(24)] + [1, 700], [(0, 24)], [1999]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (3, 3, 64), (7, 1, 128), (10, 2, 64), (40, 1, 64), (96, 1, 128), (128, 1, 64)])
def test_shared(fa, case, Hq, Hkv, d):
    lens, groups, prefix = CASES[case]
    b = Batch(lens, groups, prefix, Hq, Hkv, d, seed=case + Hq)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (16, 16, 64), (24, 8, 64), (20, 4, 128), (8, 1, 128), (64, 32, 64), (160, 160, 64)])
def test_shared_heads(fa, Hq, Hkv, d):
    """Numbers of KV heads that share the SMs unevenly, more of them than SMs among them."""
    b = Batch([500, 260, 259, 1200, 31], [(0, 3)], [250], Hq, Hkv, d, seed=Hq)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse)


def test_shared_is_decode_paged(fa):
    """The same batch through fa_decode_paged, which shares nothing: equal within both calls' bounds."""
    b = Batch([900 + 11 * i for i in range(16)], [(0, 16)], [890], 32, 8, 128, seed=2)
    o, lse = b.run(fa)
    o2, lse2 = fa.decode_paged(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), i32(b.lens))
    assert fa.check_device_error() == 0
    b.check(o, lse)
    b.check(o2, lse2)


def test_shared_sinks_and_scale(fa):
    b = Batch([300, 260, 0, 900], [(0, 2)], [256], 8, 2, 128, seed=3)
    z = torch.tensor([0.5, -3.0, -math.inf, 12.0, 1.0, 0.0, 40.0, -80.0])
    o, lse = b.run(fa, sinks=z.cuda(), scale=0.2)
    assert fa.check_device_error() == 0
    b.check(o, lse, scale=0.2, z=z)


def test_shared_many_sequences(fa):
    """1,024 sequences: one group of 700 on one page, the rest by themselves."""
    lens = [17 + (i * 13) % 40 for i in range(1024)]
    b = Batch(lens, [(100, 700)], [16], 4, 2, 64, seed=4)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse, only=range(0, 1024, 7))
    b = Batch([20] * 1024, [(2 * i, 2) for i in range(512)], [16] * 512, 128, 1, 64, seed=5)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse, only=range(0, 1024, 37))


def test_shared_long(fa):
    """One sequence of 60,000 tokens, and a long prefix for two sequences of very different lengths."""
    b = Batch([60001], [], [], 8, 8, 64, seed=6)
    o, lse = b.run(fa)
    b.check(o, lse)
    b = Batch([30000, 15010], [(0, 2)], [15000], 8, 2, 128, seed=7)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse)


def test_shared_growing_scores(fa):
    """Keys whose scores rise along the sequence: every block raises the maximum."""
    b = Batch([700, 650], [(0, 2)], [640], 4, 2, 128, seed=8)
    for s in range(2):
        for c, page in enumerate(b.rows[s]):
            if s == 0 or c >= 40:
                b.k[page] = (b.k[page].float() * 0.1 + b.q[0, 0].float() * (0.02 * c)).to(torch.bfloat16)
    o, lse = b.run(fa, scale=0.5)
    assert fa.check_device_error() == 0
    for s in range(2):
        k, v = b.keys(s)
        want = attend(b.q[s:s + 1], k, v, 0.5)
        # scores of up to ~100: fp32 sums of 128 products err by 2^-24 * 128 * sum |q k| scale; LSE and, through the
        # weights, O by as much more
        e = 2.0 ** -24 * 128 * 0.5 * torch.einsum("hd,jhd->hj", b.q[s].double().abs(), k.double().abs().repeat_interleave(2, 1)).max()
        ref, tol = want["o"]
        check(o[s:s + 1], (ref, tol + 2 * e * v.double().abs().max()), "O")
        ref, tol = want["lse"]
        check(lse[s:s + 1].t(), (ref, tol + e), "LSE")


def test_shared_repeats_exactly(fa):
    b = Batch([400 + 5 * i for i in range(30)], [(0, 30)], [390], 32, 8, 128, seed=9)
    a = [t.clone() for t in b.run(fa)]
    c = b.run(fa)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_shared_errors(fa):
    """Device-side input errors: reported, bounded, and the rest computed."""
    b = Batch([100, 90, 300], [(0, 2)], [80], 8, 2, 64, seed=10)
    for cu in ([0, 5], [2, 0], [-1, 2]):
        o, lse = fa.decode_shared(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), i32(b.lens), i32(cu), i32([80]))
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        b.check(o, lse)                                 # no group: every sequence by itself
    o, lse = fa.decode_shared(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), i32(b.lens), i32([0, 2]), i32([-1]))
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    b.check(o, lse)
    o, lse = fa.decode_shared(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.table.cuda(), i32([-3, 90, 300]), i32([0, 2]), i32([80]))
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    b.check(o, lse, only=[1, 2])
    bad = b.table.clone()
    bad[2, 1] = -4
    o, lse = fa.decode_shared(b.q.cuda(), b.k.cuda(), b.v.cuda(), bad.cuda(), i32(b.lens), i32([0, 2]), i32([80]))
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    b.check(o, lse, only=[0, 1])


def test_shared_captured(fa):
    """Recorded in a graph with fork and append, as a decoding loop would, and replayed on changed lengths."""
    b = Batch([200, 210, 330], [(0, 2)], [192], 8, 2, 128, seed=11, width=40)
    dev = [t.cuda() for t in (b.q, b.k, b.v, b.table)]
    lens, cu, pl = i32(b.lens), i32([0, 2]), i32([192])
    ws = torch.empty(fa.decode_shared_workspace_bytes(3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(dev[0]), torch.empty((3, 8), device="cuda")

    def step():
        fa.decode_shared(*dev, lens, cu, pl, out=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cut, prefix in ((0, 192), (8, 100), (150, 192), (200, 0)):
        b.lens = [200 - cut, 210 - cut, 330 - cut]
        lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        pl.fill_(prefix)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.check_device_error() == 0
        b.check(o, lse)


def test_two_calls_at_once(fa):
    """Two streams, each with its own workspace."""
    bs = [Batch([500 + 9 * i for i in range(12)], [(0, 12)], [490], 8, 2, 64, seed=20 + j) for j in range(2)]
    args = [[t.cuda() for t in (b.q, b.k, b.v, b.table)] + [i32(b.lens), i32([0, 12]), i32([490])] for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [None, None]
    for _ in range(5):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                out[j] = fa.decode_shared(*args[j])
    torch.cuda.synchronize()
    assert fa.check_device_error() == 0
    for b, (o, lse) in zip(bs, out):
        b.check(o, lse)


def test_cache_then_shared(fa):
    """The operators as they are used together: a prompt is appended, forked into samples, each sample appends its own
    tokens, the batch decodes on the shared prompt, a sample leaves, the cache is compacted, the rest decodes again."""
    g = torch.Generator().manual_seed(12)
    Hq, Hkv, d, P, W, n = 8, 2, 128, 64, 16, 6
    k, v = (torch.full((P, PAGE, Hkv, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    free, count = torch.arange(P - 1, -1, -1, dtype=torch.int32, device="cuda"), i32([P])
    hist_k = [torch.randn((100, Hkv, d), generator=g).to(torch.bfloat16)]
    hist_v = [torch.randn((100, Hkv, d), generator=g).to(torch.bfloat16)]
    table, lens = torch.full((1, W), -1, dtype=torch.int32, device="cuda"), i32([0])
    lens2, count2 = i32([0]), i32([0])
    fa.cache_append(hist_k[0].cuda(), hist_v[0].cuda(), i32([0, 100]), k, v, table, lens, free, count, lens2, count2)
    ftable, flens, fcount = torch.full((n, W), -1, dtype=torch.int32, device="cuda"), i32([0] * n), i32([0])
    fa.cache_fork(k, v, table, lens2, i32([0] * n), free, count2, ftable, flens, fcount)
    new = [1, 20, 40, 3, 12, 13]
    kn, vn = (torch.randn((sum(new), Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    lens3, count3 = i32([0] * n), i32([0])
    fa.cache_append(kn.cuda(), vn.cuda(), i32(cu), k, v, ftable, flens, free, fcount, lens3, count3)
    q = torch.randn((n, Hq, d), generator=g).to(torch.bfloat16)

    def keys(s):
        return torch.cat([hist_k[0], kn[cu[s]:cu[s + 1]]]), torch.cat([hist_v[0], vn[cu[s]:cu[s + 1]]])

    def verify(o, lse, seqs):
        for i, s in enumerate(seqs):
            want = attend(q[s:s + 1], *keys(s), d ** -0.5)
            check(o[i:i + 1], want["o"], f"O {s}")
            check(lse[i:i + 1].t(), want["lse"], f"LSE {s}")
    o, lse = fa.decode_shared(q.cuda(), k, v, ftable, lens3, i32([0, n]), i32([100]))
    assert fa.check_device_error() == 0 and lens3.tolist() == [100 + x for x in new]
    verify(o, lse, range(n))
    stay = [0, 2, 3, 5]
    parents, m = i32(stay), len(stay)
    t2, l2, c2 = torch.full((m, W), -1, dtype=torch.int32, device="cuda"), i32([0] * m), i32([0])
    fa.cache_fork(k, v, ftable, lens3, parents, free, count3, t2, l2, c2)
    t3, f3, c3 = torch.full((m, W), -1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda"), i32([0])
    fa.cache_compact(k, v, t2, l2, t3, f3, c3)
    # 6 shared pages, and of each its page of the prompt's last 4 tokens and what follows
    live = 6 + sum(pages_of(4 + new[s]) for s in stay)
    assert c3.tolist() == [P - live] and t3.max().item() == live - 1
    o, lse = fa.decode_shared(q[stay].cuda(), k, v, t3, l2, i32([0, m]), i32([100]))
    assert fa.check_device_error() == 0
    verify(o, lse, stay)


# ---------------------------------------------------------------- fa_decode_cross
def cross(fa, B, Hq, Hkv, Nq, Nk, d, lens, seed, only=None):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Nq, Hq, d), generator=g).to(torch.bfloat16)
    k, v = (torch.randn((B, Nk, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens or []):
        k[b, n:], v[b, n:] = math.nan, math.nan
    o, lse = fa.decode_cross(q.cuda(), k.cuda(), v.cuda(), i32(lens))
    assert fa.check_device_error() == 0
    for b in only or range(B):
        n = Nk if lens is None else lens[b]
        want = attend(q[b], k[b, :n], v[b, :n], d ** -0.5)
        check(o[b], want["o"], f"O {b}")
        check(lse[b], want["lse"], f"LSE {b}")


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,d,lens", [
    (1, 1, 1, 1, 1, 64, None), (1, 4, 4, 1, 0, 128, None), (3, 16, 16, 1, 300, 64, [300, 0, 17]), (2, 32, 8, 1, 129, 128, [128, 129]),
    (2, 14, 2, 5, 1000, 64, [999, 1]), (1, 8, 1, 2, 5000, 128, [4999]), (4, 8, 8, 3, 260, 128, [1, 2, 256, 257]),
    (2, 6, 2, 100, 700, 64, [700, 650]), (2, 24, 8, 43, 333, 128, [332, 200]), (1, 8, 1, 33, 400, 64, None),
    (1, 16, 1, 70, 2000, 128, [1990]), (9, 5, 1, 13, 77, 64, [0, 1, 15, 16, 17, 64, 65, 76, 77]),
])
def test_cross(fa, B, Hq, Hkv, Nq, Nk, d, lens):
    cross(fa, B, Hq, Hkv, Nq, Nk, d, lens, seed=Nk + Nq)


def test_cross_large_batch(fa):
    """2,500 sequences run as several launches on one workspace."""
    cross(fa, 2500, 4, 2, 1, 30, 64, [(7 * i) % 31 for i in range(2500)], 1, only=list(range(0, 2500, 61)) + [1023, 1024, 2499])


def test_cross_is_fwd_cross(fa):
    g = torch.Generator().manual_seed(2)
    q = torch.randn((3, 40, 8, 128), generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn((3, 1500, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    lens = i32([1500, 3, 800])
    o, lse = fa.decode_cross(q, k, v, lens)
    o2, lse2 = fa.fwd_cross(q, k, v, lens, split_keys=False)
    assert fa.check_device_error() == 0
    # both round P and O to bf16 their own way: |v| < 6, weights sum to one
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * 6
    assert (lse - lse2).abs().max() <= 2.0 ** -10


def test_cross_bad_length(fa):
    """As fa_fwd_cross: the sequence is skipped, its rows left as they were, and reported."""
    t = torch.ones((3, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.ones((3, 40, 2, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(t, 5.0), torch.full((3, 2, 1), 5.0, device="cuda")
    fa.decode_cross(t, k, k, i32([-1, 41, 40]), out=o, lse=lse)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert (o[:2] == 5).all() and (lse[:2] == 5).all() and (o[2] == 1).all()


def test_a_stream_passed_owns_the_workspace(fa):
    """The call's workspace is not handed out to the caller's stream while the given one still needs it."""
    b = Batch([500 + 9 * i for i in range(12)], [(0, 12)], [490], 8, 2, 64, seed=23)
    dev = [t.cuda() for t in (b.q, b.k, b.v, b.table)] + [i32(b.lens), i32([0, 12]), i32([490])]
    need = fa.decode_shared_workspace_bytes(12, 8, 2, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    o, lse = fa.decode_shared(*dev, stream=side)
    trash = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (need, need) + (o.nbytes, lse.nbytes) * 2]
    torch.cuda.synchronize()
    assert fa.check_device_error() == 0 and len(trash) == 6
    b.check(o, lse)


def test_stream_forms(fa):
    """By position, by name, none: one result."""
    q, k = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((2, 5, 8, 64), (2, 300, 2, 64)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [fa.decode_cross(q, k, k), fa.decode_cross(q, k, k, None, None, None, None, True, None, side),
           fa.decode_cross(q, k, k, stream=side), fa.decode_cross(q=q, k=k, v=k, stream=side)]
    torch.cuda.synchronize()
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
