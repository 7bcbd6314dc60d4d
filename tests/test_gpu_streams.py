"""A stream passed to a call owns what the call allocates: memory that the caller's stream takes afterwards is other memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


def rand(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def late(fa, call, sizes):
    """call(stream=side) with `side` busy for some milliseconds, and memory of `sizes` taken and filled meanwhile."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    out = call(stream=side)
    trash = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes * 2]
    torch.cuda.synchronize()
    assert fa.check_device_error() == 0 and len(trash) == 2 * len(sizes)
    return out


@pytest.mark.parametrize("packed", [False, True])
def test_backward(fa, packed):
    B, N, H, d = 2, 300, 4, 64
    q, k, v, do = (rand(B, N, H, d, seed=s) for s in range(4))
    if packed:
        cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
        q, k, v, do = (t.flatten(0, 1) for t in (q, k, v, do))
        o, lse = fa.fwd_varlen(q, k, v, cu, N, causal=True)

        def call(**kw):
            return fa.bwd_varlen(q, k, v, o, do, lse, cu, N, causal=True, **kw)
    else:
        o, lse = fa.fwd(q, k, v, causal=True)

        def call(**kw):
            return fa.bwd(q, k, v, o, do, lse, causal=True, **kw)
    want = call()
    got = late(fa, call, [fa.bwd_workspace_bytes(B * N, H, d), q.nbytes])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    # dQ is summed in 32 bits in any order: at most a step of its rounding to bf16 (2^-8 to either side)
    assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()


def test_decode_and_fp8(fa):
    S, H, Hkv, d, P = 9, 8, 2, 128, 400
    q, kc, vc = rand(S, H, d, seed=5), rand(P, 16, Hkv, d, seed=6), rand(P, 16, Hkv, d, seed=7)
    table = torch.randperm(P, generator=torch.Generator().manual_seed(8))[:S * 40].view(S, 40).int().cuda()
    lens = torch.tensor([40 * 16 - 7 * i for i in range(S)], dtype=torch.int32, device="cuda")
    need = fa.decode_workspace_bytes(S, H, d, 16, 40)
    for call in (lambda **kw: fa.decode_paged(q, kc, vc, table, lens, **kw),
                 lambda **kw: fa.decode_paged_noalloc(q, kc, vc, table, lens, **kw)):
        want = call()
        got = late(fa, call, [need, q.nbytes, S * H * 4])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = [rand(1, 500, h, d, seed=9 + h) for h in (8, 2, 3)]
    x[2] = x[2][:, :, :2].contiguous()
    want = fa.fwd_fp8(fa.fp8_prepare(*x), causal=True)

    def prefill(stream):
        return fa.fwd_fp8(fa.fp8_prepare(*x, stream=stream), causal=True, stream=stream)
    got = late(fa, prefill, [fa.fp8_workspace_bytes(1, 500, 2), x[0].nbytes // 2, x[1].nbytes // 2, x[0].nbytes])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
