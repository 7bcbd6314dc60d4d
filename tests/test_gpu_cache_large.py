"""A cache of more than 2^31 elements (4.6 GB each for K and V), its pages taken from the far end: the offsets pass 32 bits in append,
fork, copy, the decodes and compaction."""
import pytest
import torch

from cross_plain import attend, check

pytestmark = pytest.mark.gpu
P, PAGE, Hq, Hkv, D = 140000, 16, 16, 8, 128


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_far_pages(fa):
    assert P * PAGE * Hkv * D > 1 << 31
    k, v = (torch.zeros((P, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)
    prompt, n = 70, 3
    pk, pv = rand(prompt, Hkv, D), rand(prompt, Hkv, D)
    free, count = i32(list(range(P - 60, P))), i32([60])           # taken from the end: P-1, P-2, ...
    table, lens, count2 = torch.full((1, 8), -1, dtype=torch.int32, device="cuda"), i32([0]), i32([0])
    fa.cache_append(pk.cuda(), pv.cuda(), i32([0, prompt]), k, v, table, i32([0]), free, count, lens, count2)
    assert table[0, :5].tolist() == [P - 1, P - 2, P - 3, P - 4, P - 5]
    tables, lens3, count3 = torch.full((n, 8), -1, dtype=torch.int32, device="cuda"), i32([0] * n), i32([0])
    fa.cache_fork(k, v, table, lens, i32([0] * n), free, count2, tables, lens3, count3)
    new = [1, 20, 9]
    nk, nv = rand(sum(new), Hkv, D), rand(sum(new), Hkv, D)
    lens4, count4 = i32([0] * n), i32([0])
    fa.cache_append(nk.cuda(), nv.cuda(), i32([0, 1, 21, 30]), k, v, tables, lens3, free, count3, lens4, count4)
    assert fa.check_device_error() == 0 and lens4.tolist() == [prompt + x for x in new]
    q = rand(n, Hq, D)

    def verify(tb):
        for call in (lambda: fa.decode_shared(q.cuda(), k, v, tb, lens4, i32([0, n]), i32([prompt])),
                     lambda: fa.decode_paged(q.cuda(), k, v, tb, lens4)):
            o, lse = call()
            assert fa.check_device_error() == 0
            for s, (a, b) in enumerate(((0, 1), (1, 21), (21, 30))):
                want = attend(q[s:s + 1], torch.cat([pk, nk[a:b]]), torch.cat([pv, nv[a:b]]), D ** -0.5)
                check(o[s:s + 1], want["o"], f"O {s}")
                check(lse[s:s + 1].t(), want["lse"], f"LSE {s}")
    verify(tables)
    # copies across the border, both ways
    far, near = tables[0, :3].tolist(), [5, 6, 7]
    fa.cache_copy_pages(k, v, i32(far), i32(near))
    fa.cache_copy_pages(k, v, i32(near), i32([P - 100, P - 101, P - 102]))
    assert fa.check_device_error() == 0
    for a, b, c in zip(far, near, (P - 100, P - 101, P - 102)):
        assert torch.equal(k[a], k[b]) and torch.equal(v[a], v[b]) and torch.equal(k[a], k[c]) and torch.equal(v[a], v[c])
    out, fr, ct = torch.full_like(tables, -1), torch.zeros(P, dtype=torch.int32, device="cuda"), i32([0])
    fa.cache_compact(k, v, tables, lens4, out, fr, ct)
    assert fa.check_device_error() == 0
    live = P - ct.item()
    assert out.max().item() == live - 1 and 0 < live < 20
    verify(out)
