"""The cache-page operators (fa_cache_*) against their definition, entry by entry (cache_plain.py).  They move
values and compute none, so every comparison is exact."""
import pytest
import torch

from cache_plain import Cache, batch, pages_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


class Dev:
    """The batch on the GPU, with free_pages as the operators take it."""

    def __init__(self, b):
        self.k, self.v = b["k"].cuda(), b["v"].cuda()
        self.scales = {} if b["ks"] is None else {"k_scale": b["ks"].cuda(), "v_scale": b["vs"].cuda()}
        self.table, self.lens = b["table"].cuda(), i32(b["lens"])
        P = self.k.shape[0]
        self.free = i32(b["free"] + [-7] * (P - len(b["free"])))
        self.count = i32([len(b["free"])])
        self.count_out = i32([-5])

    def same_cache(self, c):
        return same(self.k, c.k) and same(self.v, c.v) and (
            not self.scales or (same(self.scales["k_scale"], c.ks) and same(self.scales["v_scale"], c.vs)))


def run_fork(fa, b, parents, stream=None):
    d, n = Dev(b), len(parents)
    table_out = torch.full((n, b["table"].shape[1]), -9, dtype=torch.int32, device="cuda")
    lens_out = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    for _ in range(2):        # a repeated call gives the same
        fa.cache_fork(d.k, d.v, d.table, d.lens, i32(parents), d.free, d.count, table_out, lens_out, d.count_out,
                      stream=stream, **d.scales)
    return d, table_out, lens_out


def check_fork(fa, b, parents, err=0):
    d, table_out, lens_out = run_fork(fa, b, parents)
    assert fa.check_device_error() == err
    c = Cache(b["k"], b["v"], b["table"], b["lens"], b["free"], b["ks"], b["vs"])
    want = torch.full_like(table_out, -9).cpu()
    lens, _ = c.fork(parents, want)
    assert torch.equal(table_out.cpu(), want)
    assert lens_out.tolist() == lens
    assert d.count_out.tolist() == [len(c.free)]
    assert d.same_cache(c)


@pytest.mark.parametrize("lens,parents", [
    ([5], [0]), ([5], [0, 0, 0]), ([16], [0, 0]), ([17, 40, 0, 33], [1, 1, 0, 3, 3, 3, 2, -1, 0]),
    ([1, 15, 16, 31, 32], [4, 3, 2, 1, 0, 0, 1, 2, 3, 4]), ([100, 0], [-1, -1]), ([7, 8, 9], []),
    ([300 + 7 * i for i in range(40)], [3 * i % 40 for i in range(40)] + [5] * 30),
])
@pytest.mark.parametrize("Hkv,d,fp8", [(8, 128, False), (1, 64, False), (3, 64, True), (5, 128, True)])
def test_fork(fa, lens, parents, Hkv, d, fp8):
    pages = sum(map(pages_of, lens)) + len(parents) + 3
    check_fork(fa, batch(lens, pages, Hkv, d, seed=len(parents), fp8=fp8), parents)


def test_fork_many_slots(fa):
    lens = [1 + (i * 37) % 50 for i in range(700)]
    parents = [(i * 11) % 350 for i in range(2000)]
    check_fork(fa, batch(lens, sum(map(pages_of, lens)) + 2100, 1, 64, seed=3), parents)


def test_fork_runs_out_of_pages(fa):
    # five slots need a page and three are left: in slot order, the last two come out empty
    b = batch([5, 20, 32], 6 + 0, 2, 64, seed=4)
    b["free"] = b["free"][-1:]
    assert len(b["free"]) == 1
    parents = [0, 0, 1, 2, 1, 2, 0]
    check_fork(fa, b, parents, err=fa.FA_ERR_PAGES)
    b["free"] = []
    check_fork(fa, b, parents, err=fa.FA_ERR_PAGES)


def test_fork_bad_inputs(fa):
    b = batch([5, 20, 32], 12, 2, 64, seed=5)
    # a parent out of range: an empty slot, reported; the others as usual
    for bad in (3, -2, 1 << 30):
        d, table_out, lens_out = run_fork(fa, b, [0, bad, 1, 1])
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        assert lens_out.tolist() == [5, 0, 20, 20]
        assert torch.all(table_out[1] == -9)
        assert d.count_out.tolist() == [len(b["free"]) - 1]
    # lengths no row can hold
    for bad in (-1, b["table"].shape[1] * 16 + 1):
        c = dict(b, lens=[5, bad, 32])
        _, _, lens_out = run_fork(fa, c, [1, 0, 0])
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        assert lens_out.tolist() == [0, 5, 5]
    # a page number out of range is never followed; nothing but the fork's own page is written
    c = dict(b, table=b["table"].clone())
    c["table"][1, 1] = 99
    d, _, lens_out = run_fork(fa, c, [1, 1])
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert same(d.k, b["k"]) and same(d.v, b["v"])
    # a free list naming a page that does not exist: the slot that would get it stays empty
    c = dict(b, free=[1000] + b["free"][:-1][:0])
    d, _, lens_out = run_fork(fa, c, [0, 0])
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert lens_out.tolist() == [5, 0] and same(d.k, b["k"])


def run_append(fa, b, new, seed=0, dtype=torch.bfloat16):
    d = Dev(b)
    g = torch.Generator().manual_seed(seed + 100)
    T, (Hkv, hd) = sum(new), b["k"].shape[2:]
    kn = torch.randn((T, Hkv, hd), generator=g).to(dtype)
    vn = torch.randn((T, Hkv, hd), generator=g).to(dtype)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    lens_out = torch.full((len(new),), -9, dtype=torch.int32, device="cuda")
    for _ in range(2):
        fa.cache_append(kn.cuda(), vn.cuda(), i32(cu), d.k, d.v, d.table, d.lens, d.free, d.count, lens_out,
                        d.count_out)
    return d, kn, vn, cu, lens_out


def check_append(fa, b, new, err=0):
    d, kn, vn, cu, lens_out = run_append(fa, b, new)
    assert fa.check_device_error() == err
    c = Cache(b["k"], b["v"], b["table"], b["lens"], b["free"])
    lens, short = c.append(kn, vn, cu)
    assert short == (err == fa.FA_ERR_PAGES)
    assert lens_out.tolist() == lens
    assert torch.equal(d.table.cpu(), c.table)
    if not short:
        assert d.count_out.tolist() == [len(c.free)]
    assert d.same_cache(c)
    return d, c


@pytest.mark.parametrize("old,new", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([15], [2]), ([0, 3, 16, 31], [16, 13, 17, 0]),
    ([5, 0, 700], [300, 1000, 1]), ([33] * 70, [1] * 70), (list(range(300)), [i % 5 for i in range(300)]),
    ([0] * 9, [0, 0, 1, 0, 0, 64, 0, 0, 3]),
])
@pytest.mark.parametrize("Hkv,d", [(8, 128), (1, 64), (3, 64)])
def test_append(fa, old, new, Hkv, d):
    pages = sum(pages_of(a + n) for a, n in zip(old, new)) + 3
    width = max(pages_of(a + n) for a, n in zip(old, new)) + 1
    check_append(fa, batch(old, pages, Hkv, d, seed=len(old), width=width), new)


def test_append_runs_out_of_pages(fa):
    # 4 free pages: slot 0 takes 2, slot 1 would need 3, slot 2 needs none, slot 3 would need 1
    b = batch([10, 0, 3, 16], 7, 2, 64, seed=6, width=8)
    assert len(b["free"]) == 4
    d, c = check_append(fa, b, [30, 40, 2, 1], err=fa.FA_ERR_PAGES)
    assert d.count_out.tolist() == [2]


def test_append_bad_inputs(fa):
    b = batch([10, 20, 30], 16, 2, 64, seed=7, width=4)
    # past the row's width, and lengths out of range: left as they were, reported
    for lens, new, want in (([10, 20, 30], [1, 45, 1], [11, 20, 31]), ([10, -4, 30], [1, 1, 1], [11, -4, 31]),
                            ([10, 1000, 30], [1, 1, 1], [11, 1000, 31])):
        d, kn, vn, cu, lens_out = run_append(fa, dict(b, lens=lens), new)
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        assert lens_out.tolist() == want
    # offsets that descend or leave the tensor
    for cu in ([0, 3, 2, 4], [0, 1, 2, 9], [-1, 1, 2, 4]):
        d = Dev(b)
        kn = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
        lens_out = torch.zeros_like(d.lens)
        fa.cache_append(kn, kn, i32(cu), d.k, d.v, d.table, d.lens, d.free, d.count, lens_out, d.count_out)
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    # a free count out of range counts as none
    for count in (-1, 17):
        d = Dev(b)
        d.count.fill_(count)
        lens_out = torch.zeros_like(d.lens)
        fa.cache_append(kn, kn, i32([0, 0, 0, 4]), d.k, d.v, d.table, d.lens, d.free, d.count, lens_out, d.count_out)
        assert fa.check_device_error() in (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_PAGES)
        assert lens_out.tolist() == [10, 20, 30]


@pytest.mark.parametrize("lens,pages", [([], 40), ([0, 0], 33), ([1], 1), ([16 * 31], 31), ([16 * 32], 32),
                                        ([5, 0, 600, 33], 100), ([900, 16, 17], 20000), ([64] * 400, 70000)])
def test_collect(fa, lens, pages):
    b = batch(lens, pages, 1, 64, seed=8, share=2) if lens else None
    table = b["table"] if lens else torch.zeros((0, 3), dtype=torch.int32)
    free = torch.full((pages,), -3, dtype=torch.int32, device="cuda")
    count = i32([-1])
    fa.cache_collect(table.cuda(), i32(lens), free, count)
    assert fa.check_device_error() == 0
    want = Cache(b["k"], b["v"], table, lens).collect() if lens else list(range(pages - 1, -1, -1))
    assert count.tolist() == [len(want)]
    assert free.tolist() == want + [-3] * (pages - len(want))


@pytest.mark.parametrize("lens,pages,Hkv,d,fp8,share", [
    ([16 * 3], 3, 8, 128, False, 0), ([1], 9, 2, 64, False, 0), ([0, 0], 33, 1, 64, False, 0),
    ([5, 0, 600, 33], 100, 2, 64, True, 0), ([300, 500, 200, 77], 90, 3, 128, False, 9),
    ([64] * 200, 9000, 1, 64, False, 0), ([700, 16, 17], 20000, 1, 64, True, 1),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(fa, lens, pages, Hkv, d, fp8, share, in_place):
    b = batch(lens, pages, Hkv, d, seed=9, share=share, fp8=fp8)
    dev = Dev(b)
    table_out = dev.table if in_place else torch.full_like(dev.table, -9)
    before = table_out.clone()
    free = torch.full((pages,), -3, dtype=torch.int32, device="cuda")
    fa.cache_compact(dev.k, dev.v, dev.table, dev.lens, table_out, free, dev.count_out, **dev.scales)
    assert fa.check_device_error() == 0
    c = Cache(b["k"], b["v"], b["table"], lens, (), b["ks"], b["vs"])
    want = before.cpu()
    left = c.compact(want)
    assert torch.equal(table_out.cpu(), want)
    assert dev.count_out.tolist() == [len(left)]
    assert free.tolist() == left + [-3] * (pages - len(left))
    assert dev.same_cache(c)


def test_collect_and_compact_bad_inputs(fa):
    b = batch([20, 40], 12, 1, 64, seed=10)
    b["table"][0, 1] = 12
    b["table"][1, 0] = -1
    good = {int(b["table"][0, 0]), int(b["table"][1, 1]), int(b["table"][1, 2])}
    d = Dev(b)
    free = torch.full((12,), -3, dtype=torch.int32, device="cuda")
    fa.cache_collect(d.table, d.lens, free, d.count_out)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert free.tolist()[:9] == [p for p in range(11, -1, -1) if p not in good]
    table_out = torch.full_like(d.table, -9)
    fa.cache_compact(d.k, d.v, d.table, d.lens, table_out, free, d.count_out)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert d.count_out.tolist() == [9]
    assert table_out[0, 1].item() == 12 and table_out[1, 0].item() == -1
    assert sorted([table_out[0, 0].item(), table_out[1, 1].item(), table_out[1, 2].item()]) == [0, 1, 2]


@pytest.mark.parametrize("lens,pages,width", [
    ([16 * 700, 0, 16 * 257, 16 * 256 + 1], 1500, 700), ([40] * 128, 32768, 256), ([40] * 129, 32768, 256),
    ([16 * 300] * 3, 32769, 300), ([33] * 500, 3000, 513), ([33] * 40, 3000, 768), ([700] * 64, 3000, 512),
])
def test_many_table_entries(fa, lens, pages, width):
    b = batch(lens, pages, 1, 64, seed=14, width=width)
    dev = Dev(b)
    free = torch.full((pages,), -3, dtype=torch.int32, device="cuda")
    c = Cache(b["k"], b["v"], b["table"], lens)
    want = c.collect()
    fa.cache_collect(dev.table, dev.lens, free, dev.count_out)
    assert fa.check_device_error() == 0
    assert dev.count_out.tolist() == [len(want)]
    assert free.tolist() == want + [-3] * (pages - len(want))
    table_out = torch.full_like(dev.table, -9)
    free.fill_(-3)
    fa.cache_compact(dev.k, dev.v, dev.table, dev.lens, table_out, free, dev.count_out)
    assert fa.check_device_error() == 0
    want_table = torch.full_like(b["table"], -9)
    left = c.compact(want_table)
    assert torch.equal(table_out.cpu(), want_table)
    assert free.tolist() == left + [-3] * (pages - len(left))
    assert dev.same_cache(c)


@pytest.mark.parametrize("pages", [12, 40000])
def test_bad_entries_and_lengths_are_not_in_use(fa, pages):
    b = batch([20, 40, 16], 12, 1, 64, seed=15)
    b["table"][0, 1] = pages
    b["table"][1, 0] = -1
    lens = i32([20, 40, 16 * b["table"].shape[1] + 1])     # the last cannot be: read as 0
    used = {int(b["table"][0, 0]), int(b["table"][1, 1]), int(b["table"][1, 2])}
    free = torch.full((pages,), -3, dtype=torch.int32, device="cuda")
    count = i32([-1])
    fa.cache_collect(b["table"].cuda(), lens, free, count)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert free.tolist() == [p for p in range(pages - 1, -1, -1) if p not in used] + [-3] * 3
    assert count.tolist() == [pages - 3]


@pytest.mark.parametrize("Hkv,d,fp8", [(8, 128, False), (1, 64, True)])
def test_copy_pages(fa, Hkv, d, fp8):
    b = batch([1], 60, Hkv, d, seed=11, fp8=fp8)
    dev = Dev(b)
    src, dst = [3, 3, 9, -1, 20, 5], [4, 59, 0, -1, 21, 5]
    fa.cache_copy_pages(dev.k, dev.v, i32(src), i32(dst), **dev.scales)
    assert fa.check_device_error() == 0
    c = Cache(b["k"], b["v"], b["table"], [1], (), b["ks"], b["vs"])
    for s, t in zip(src, dst):
        if s >= 0:
            c._copy(s, t, 16)
    assert dev.same_cache(c)


def test_copy_pages_refuses_entries(fa):
    b = batch([1], 60, 2, 64, seed=12)
    dev = Dev(b)
    # 1: its destination is a source; 2: written again later; 4, 5: out of range; 0, 3, 6 go through
    src, dst = [3, 10, 30, 31, 60, 7, 40], [4, 3, 50, 50, 8, -1, 41]
    fa.cache_copy_pages(dev.k, dev.v, i32(src), i32(dst))
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    c = Cache(b["k"], b["v"], b["table"], [1])
    for i in (0, 3, 6):
        c._copy(src[i], dst[i], 16)
    assert dev.same_cache(c)


def test_captured_and_on_another_stream(fa):
    """A step recorded once and replayed with other lengths, parents and offsets in the same buffers."""
    lens = [33, 50, 7]
    b = batch(lens, 40, 2, 64, seed=13, width=8)
    d = Dev(b)
    parents, cu = i32([0, 1, 2, 2]), i32([0, 1, 2, 3, 4])
    kn = torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16)
    table2 = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    lens2, lens3 = i32([0] * 4), i32([0] * 4)
    count2, count3 = i32([0]), i32([0])
    free = d.free.clone()
    ws = torch.empty(fa.cache_collect_workspace_bytes(40), dtype=torch.uint8, device="cuda")

    def step():
        fa.cache_fork(d.k, d.v, d.table, d.lens, parents, d.free, d.count, table2, lens2, count2)
        fa.cache_append(kn, kn, cu, d.k, d.v, table2, lens2, d.free, count2, lens3, count3)
        fa.cache_collect(table2, lens3, free, d.count_out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ps, ls in (([2, 2, 2, 1], [33, 50, 7]), ([0, 0, -1, 0], [16, 1, 2]), ([1, 0, 1, 2], [31, 47, 16])):
        d.k.copy_(b["k"]), d.v.copy_(b["v"])
        parents.copy_(i32(ps)), d.lens.copy_(i32(ls))
        table2.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.check_device_error() == 0
        c = Cache(b["k"], b["v"], b["table"], ls, b["free"])
        want = torch.full((4, 8), -1, dtype=torch.int32)
        new, _ = c.fork(ps, want)
        c.table, c.lens = want, new
        c.lens, _ = c.append(kn.cpu(), kn.cpu(), [0, 1, 2, 3, 4])
        assert lens3.tolist() == c.lens and torch.equal(table2.cpu(), c.table)
        assert count3.tolist() == [len(c.free)] and d.same_cache(c)
        left = c.collect()
        assert d.count_out.tolist() == [len(left)] and free.tolist()[:len(left)] == left
