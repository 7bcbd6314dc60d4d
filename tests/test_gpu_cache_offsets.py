"""fa_cache_append with offsets that descend or leave the tensor: the sequences that are right are appended to, every other place of
the cache, the tables and the lengths stays as it was."""
import pytest
import torch

from cache_plain import Cache, batch

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


def right(cu, total):
    """The sequences whose tokens lie behind those of the ones before, as (first, last + 1); None for the others."""
    out, end = [], 0
    for a, e in zip(cu, cu[1:]):
        good = end <= a <= e <= total
        out.append((a, e) if good else None)
        end = e if good else end
    return out


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("lens,cu,total", [
    ([10, 20, 30], [0, 3, 2, 4], 4), ([10, 20, 30], [0, 1, 2, 9], 4), ([10, 20, 30], [-1, 1, 2, 4], 4),
    ([10, 20, 30], [0, 9, 2, 4], 4), ([10, 20, 30], [0, 4, 0, 4], 4), ([0, 16, 5, 31], [0, 40, 20, 20, 60], 60),
    ([0, 16, 5, 31], [30, 60, 0, 30, 50], 60), ([10, 20], [0, -2 ** 31, 4], 4), ([10, 20], [2 ** 31 - 1, -2 ** 31, 4], 4),
    ([7] * 600, [0] + [(i * 5) % 1500 for i in range(600)], 1500),
])
def test_bad_offsets(fa, lens, cu, total):
    g = torch.Generator().manual_seed(total)
    kn, vn = (torch.randn((total, 2, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    b = batch(lens, 1000, 2, 64, seed=1, width=110)
    k, v, table = b["k"].cuda(), b["v"].cuda(), b["table"].cuda()
    free, count, count_out = i32(b["free"]), i32([len(b["free"])]), i32([-5])
    lens_out = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    fa.cache_append(kn.cuda(), vn.cuda(), i32(cu), k, v, table, i32(lens), free, count, lens_out, count_out)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    # the definition on the right ones alone: their tokens packed, none for the others
    parts = right(cu, total)
    assert None in parts
    at, packed = [0], []
    for p in parts:
        packed += range(*p) if p else ()
        at.append(len(packed))
    c = Cache(b["k"], b["v"], b["table"], lens, b["free"])
    want, short = c.append(kn[packed], vn[packed], at)
    assert not short
    assert lens_out.tolist() == want
    assert torch.equal(table.cpu(), c.table) and count_out.tolist() == [len(c.free)]
    assert same(k, c.k) and same(v, c.v)
