"""Pages that do not exist, in the free list or in a table's used entries: the slot they belong to is left out by fa_cache_append and
comes out empty of fa_cache_fork, so that no table names such a page for tokens that a length counts; the others go on."""
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


def append(fa, b, new, bad_slots):
    """Appends `new` tokens; every slot but bad_slots as defined, those with their length and table row as they were."""
    g = torch.Generator().manual_seed(3)
    kn, vn = (torch.randn((sum(new), 2, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    k, v, table = b["k"].cuda(), b["v"].cuda(), b["table"].cuda()
    lens_out, count_out = i32([-9] * len(new)), i32([-9])
    fa.cache_append(kn.cuda(), vn.cuda(), i32(cu), k, v, table, i32(b["lens"]), i32(b["free"]), i32([len(b["free"])]), lens_out,
                    count_out)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    # the definition with a page of its own for every number that does not exist
    pages = b["k"].shape[0]
    names = sorted({p for p in b["free"] + b["table"].flatten().tolist() if not 0 <= p < pages})
    real = {p: pages + i for i, p in enumerate(names)}
    grow = torch.zeros((len(names),) + b["k"].shape[1:], dtype=torch.bfloat16)
    t = b["table"].clone().apply_(lambda p: real.get(p, p))
    c = Cache(torch.cat([b["k"], grow]), torch.cat([b["v"], grow]), t, b["lens"], [real.get(p, p) for p in b["free"]])
    want, short = c.append(kn, vn, cu)
    assert not short
    lens, rows = lens_out.tolist(), table.cpu()
    for s, n in enumerate(new):
        old = b["lens"][s]
        if s in bad_slots:
            assert lens[s] == old and torch.equal(rows[s], b["table"][s]), s
            continue
        assert lens[s] == want[s], s
        used = pages_of(want[s])
        assert torch.equal(rows[s, :used], c.table[s, :used]), s
        row = rows[s, :used].long()
        assert torch.equal(k.cpu()[row].flatten(0, 1)[:want[s]], c.k[row].flatten(0, 1)[:want[s]]), s
        assert torch.equal(v.cpu()[row].flatten(0, 1)[:want[s]], c.v[row].flatten(0, 1)[:want[s]]), s


@pytest.mark.parametrize("bad", [99, 64, -1, 1 << 30])
def test_append_and_a_free_list_with_bad_pages(fa, bad):
    b = batch([10, 16, 40, 300], 64, 2, 64, seed=2, width=60)
    # in slot order: slot 0 takes 1 page, 1 takes 1, 2 takes 4, 3 takes 19
    new = [20, 3, 60, 300]
    for place, slot in ((0, 0), (1, 1), (2, 2), (5, 2), (6, 3), (20, 3)):
        free = list(b["free"])
        free[-1 - place] = bad
        append(fa, dict(b, free=free), new, {slot})
    free = list(b["free"])
    free[-1], free[-4] = bad, bad
    append(fa, dict(b, free=free), new, {0, 2})


@pytest.mark.parametrize("bad", [64, -7])
def test_append_and_a_last_page_that_does_not_exist(fa, bad):
    b = batch([10, 16, 40, 300], 64, 2, 64, seed=2, width=60)
    for slot, entry in ((0, 0), (2, 2), (3, 18)):
        table = b["table"].clone()
        table[slot, entry] = bad
        append(fa, dict(b, table=table), [20, 3, 1, 0 if slot != 3 else 5], {slot})


def test_append_of_nothing_leaves_a_bad_page_alone(fa):
    """A slot that gets no token is not looked at."""
    b = batch([10, 16], 8, 2, 64, seed=2, width=4)
    b["table"][0, 0] = 99
    k, v, lens_out, count = b["k"].cuda(), b["v"].cuda(), i32([0, 0]), i32([0])
    one = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    fa.cache_append(one, one, i32([0, 0, 1]), k, v, b["table"].cuda(), i32([10, 16]), i32(b["free"]), i32([len(b["free"])]),
                    lens_out, count)
    assert fa.check_device_error() == 0 and lens_out.tolist() == [10, 17]


@pytest.mark.parametrize("entry", [0, 1, 600])
@pytest.mark.parametrize("bad", [99999, -1])
def test_fork_of_a_table_with_bad_pages(fa, entry, bad):
    b = batch([5, 16 * 601 + 3, 32], 700, 2, 64, seed=5)
    b["table"][1, entry] = bad
    d = [b["k"].cuda(), b["v"].cuda()]
    table_out, lens_out = torch.full((5, b["table"].shape[1]), -9, dtype=torch.int32, device="cuda"), i32([-9] * 5)
    count_out = i32([0])
    fa.cache_fork(*d, b["table"].cuda(), i32(b["lens"]), i32([0, 1, 2, 1, 0]), i32(b["free"]), i32([len(b["free"])]), table_out,
                  lens_out, count_out)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    assert lens_out.tolist() == [5, 0, 32, 0, 5]
    assert (table_out[[1, 3]] == -9).all()
    rows = table_out.cpu()
    assert rows[0, 0] == b["table"][0, 0] and torch.equal(rows[2, :2], b["table"][2, :2])
    # the last slot's page is the second taken: the fourth slot's came before it
    fresh = b["free"][-2]
    assert rows[4, 0] == fresh and torch.equal(d[0][fresh, :5].cpu(), b["k"][b["table"][0, 0], :5])
