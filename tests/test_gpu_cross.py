"""Cross attention (fa_fwd_cross, fa_fwd_varlen_cross and their backward) against the definition in 64 bits, within the
bounds cross_plain.py derives."""
import math

import pytest
import torch

from cross_plain import attend, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


def rand(shape, g):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def poison(x, keep):
    """NaN into the rows of x outside keep."""
    mask = torch.ones(x.shape[0], dtype=torch.bool)
    mask[keep] = False
    x[mask] = math.nan
    return x


def dense(fa, B, Hq, Hkv, Nq, Nk, d, lens=None, out_dtype=torch.bfloat16, seed=0, scale=None, split=False):
    """One forward and backward; rows behind the visible keys hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q, do = rand((B, Nq, Hq, d), g), rand((B, Nq, Hq, d), g)
    k, v = rand((B, Nk, Hkv, d), g), rand((B, Nk, Hkv, d), g)
    scale = scale or d ** -0.5
    for b, n in enumerate(lens or []):
        k[b, n:], v[b, n:] = math.nan, math.nan
    Q, K, V, DO, L = q.cuda(), k.cuda(), v.cuda(), do.cuda(), i32(lens)
    o, lse = fa.fwd_cross(Q, K, V, L, scale, out_dtype=out_dtype, split_keys=split)
    ob = o if o.dtype == torch.bfloat16 else fa.fwd_cross(Q, K, V, L, scale)[0]
    dk, dv = torch.full_like(K, math.nan), torch.full_like(V, math.nan)
    dq, dk, dv = fa.bwd_cross(Q, K, V, ob, DO, lse, L, scale, dk=dk, dv=dv)
    assert fa.check_device_error() == 0
    for b in range(B):
        n = Nk if lens is None else lens[b]
        want = attend(q[b], k[b, :n], v[b, :n], scale, do[b])
        what = f"B={B} Hq={Hq} Hkv={Hkv} Nq={Nq} Nk={Nk} d={d} sequence {b}"
        check(o[b], want["o"], what + " O")
        check(lse[b], want["lse"], what + " LSE")
        check(dq[b], want["dq"], what + " dQ")
        check(dk[b, :n], want["dk"], what + " dK")
        check(dv[b, :n], want["dv"], what + " dV")
        assert (dk[b, n:] == 0).all() and (dv[b, n:] == 0).all()


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,d,lens", [
    (1, 1, 1, 1, 1, 128, None),
    (1, 2, 2, 1, 1000, 64, None),
    (1, 4, 2, 130, 3, 128, None),
    (2, 4, 4, 64, 128, 64, [128, 127]),
    (3, 8, 2, 129, 257, 128, [257, 0, 1]),
    (2, 6, 2, 300, 500, 64, [129, 500]),
    (2, 5, 1, 257, 640, 128, [640, 385]),
    (1, 7, 1, 513, 200, 64, [199]),
    (4, 2, 2, 40, 130, 128, [2, 128, 64, 130]),
    (2, 2, 1, 3, 5, 64, [0, 0]),
])
@pytest.mark.parametrize("split", [False, True, None])
def test_dense(fa, B, Hq, Hkv, Nq, Nk, d, lens, split):
    dense(fa, B, Hq, Hkv, Nq, Nk, d, lens, seed=Nq + Nk, split=split)


def test_many_sequences(fa):
    """More sequences than are ordered by cost; empty ones among them."""
    dense(fa, 130, 2, 1, 20, 150, 64, [(37 * i) % 151 for i in range(130)], seed=2)
    packed(fa, [(11 * i) % 40 for i in range(140)], [(29 * i) % 170 for i in range(140)], 2, 2, 128, seed=3)


def test_fp32_output_and_scale(fa):
    dense(fa, 2, 4, 2, 150, 260, 128, [260, 90], out_dtype=torch.float32, seed=4, scale=0.3)


def packed(fa, nq, nk, Hq, Hkv, d, seed, gap=0):
    """Sequences with `gap` rows of NaN before, between and behind them."""
    g = torch.Generator().manual_seed(seed)

    def offsets(lens):
        # offsets cannot leave holes between sequences: rows before the first and behind the last one only
        cu = [gap]
        for n in lens:
            cu.append(cu[-1] + n)
        return cu, cu[-1] + gap
    cq, Tq = offsets(nq)
    ck, Tk = offsets(nk)
    q, do, k, v = rand((Tq, Hq, d), g), rand((Tq, Hq, d), g), rand((Tk, Hkv, d), g), rand((Tk, Hkv, d), g)
    for x, c in ((q, cq), (do, cq), (k, ck), (v, ck)):
        poison(x, slice(c[0], c[-1]))
    Q, K, V, DO = q.cuda(), k.cuda(), v.cuda(), do.cuda()
    args = (i32(cq), i32(ck), max(nq), max(nk))
    mark = 7.0
    o, dq = torch.full_like(Q, mark), torch.full_like(Q, mark)
    dk, dv = torch.full_like(K, mark), torch.full_like(V, mark)
    lse = torch.full((Hq, Tq), mark, device="cuda")
    fa.fwd_varlen_cross(Q, K, V, *args, out=o, lse=lse)
    fa.bwd_varlen_cross(Q, K, V, o, DO, lse, *args, dq=dq, dk=dk, dv=dv)
    assert fa.check_device_error() == 0
    for s in range(len(nq)):
        a, b, c, e = cq[s], cq[s + 1], ck[s], ck[s + 1]
        want = attend(q[a:b], k[c:e], v[c:e], d ** -0.5, do[a:b])
        what = f"packed {nq} {nk} sequence {s}"
        check(o[a:b], want["o"], what + " O")
        check(lse[:, a:b], want["lse"], what + " LSE")
        check(dq[a:b], want["dq"], what + " dQ")
        check(dk[c:e], want["dk"], what + " dK")
        check(dv[c:e], want["dv"], what + " dV")
    # rows of no sequence are left as they were
    for x, c in ((o, cq), (dq, cq), (dk, ck), (dv, ck), (lse.t(), cq)):
        assert (x[:c[0]] == mark).all() and (x[c[-1]:] == mark).all()


@pytest.mark.parametrize("nq,nk", [
    ([1], [1]), ([5, 0, 130, 1], [7, 40, 0, 300]), ([128, 256, 60], [128, 1, 129]), ([0, 0, 3], [9, 0, 2]),
    ([257, 31, 90, 200], [65, 513, 127, 64]),
])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("gap", [0, 3])
def test_packed(fa, nq, nk, Hq, Hkv, d, gap):
    packed(fa, nq, nk, Hq, Hkv, d, sum(nq) + sum(nk), gap)


@pytest.mark.parametrize("split", [False, True])
def test_large_scores(fa, split):
    """Scores of several hundred: one key takes nearly all the weight, and the conditional rescale runs often.  The
    scores' fp32 sums err by 2^-24 d sum |q k| scale there; inputs whose products are whole numbers make them exact."""
    g = torch.Generator().manual_seed(11)
    B, H, Nq, Nk, d = 1, 2, 140, 700, 64
    q = torch.randint(-3, 4, (B, Nq, H, d), generator=g).to(torch.bfloat16)
    k = torch.randint(-3, 4, (B, Nk, H, d), generator=g).to(torch.bfloat16)
    v = rand((B, Nk, H, d), g)
    o, lse = fa.fwd_cross(q.cuda(), k.cuda(), v.cuda(), scale=1.0, split_keys=split)
    assert fa.check_device_error() == 0
    want = attend(q[0], k[0], v[0], 1.0)
    check(o[0], want["o"], "O")
    # LSE of scores up to 300 in fp32: 300 * 2^-23 more from each of three roundings
    ref, tol = want["lse"]
    check(lse[0], (ref, tol + 3 * 300 * 2.0 ** -23), "LSE")


def test_bad_lengths(fa):
    """Offsets or lengths that do not fit: the sequence is skipped and reported, the others are computed."""
    g = torch.Generator().manual_seed(3)
    q, k, v = rand((3, 20, 2, 64), g), rand((3, 40, 2, 64), g), rand((3, 40, 2, 64), g)
    for bad, split in ((-1, False), (41, False), (-1, True), (41, True)):
        o = torch.full((3, 20, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        _, lse = fa.fwd_cross(q.cuda(), k.cuda(), v.cuda(), i32([40, bad, 17]), out=o, split_keys=split)
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        assert (o[1] == 5.0).all()
        check(o[2], attend(q[2], k[2, :17], v[2, :17], 0.125)["o"], "O")
        dk = torch.full_like(k, 5.0).cuda()
        dq, _, dv = fa.bwd_cross(q.cuda(), k.cuda(), v.cuda(), o, o, torch.zeros_like(lse), i32([40, bad, 17]), dk=dk)
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        assert (dk[1] == 5.0).all() and (dq[1] == 0).all()
    qp, kp = q.view(60, 2, 64).cuda(), k.view(120, 2, 64).cuda()
    # (offsets of queries, of keys, the sequence that still fits)
    for cq, ck, good in (([0, 20, 10, 60], [0, 40, 80, 120], 0), ([0, 20, 40, 60], [0, 40, 121, 120], 0),
                         ([0, 20, 40, 60], [-4, 40, 80, 120], 2)):
        o = torch.full((60, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        fa.fwd_varlen_cross(qp, kp, kp, i32(cq), i32(ck), 45, 45, out=o)     # (10 to 60 is too long, too)
        assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
        rows, keys = slice(cq[good], cq[good + 1]), slice(ck[good], ck[good + 1])
        check(o[rows], attend(qp[rows].cpu(), kp[keys].cpu(), kp[keys].cpu(), 0.125)["o"], "O")


def test_grouped_heads_equal_repeated(fa):
    """dK, dV of shared heads are the sums over the query heads that read them."""
    g = torch.Generator().manual_seed(5)
    q, do = rand((2, 90, 6, 128), g).cuda(), rand((2, 90, 6, 128), g).cuda()
    k, v = rand((2, 200, 2, 128), g).cuda(), rand((2, 200, 2, 128), g).cuda()
    o, lse = fa.fwd_cross(q, k, v, split_keys=False)
    kr, vr = k.repeat_interleave(3, 2).contiguous(), v.repeat_interleave(3, 2).contiguous()
    o2, lse2 = fa.fwd_cross(q, kr, vr, split_keys=False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _, dk, dv = fa.bwd_cross(q, k, v, o, do, lse)
    _, dk2, dv2 = fa.bwd_cross(q, kr, vr, o2, do, lse2)
    assert fa.check_device_error() == 0
    for a, b in ((dk, dk2), (dv, dv2)):
        parts = b.float().view(2, 200, 2, 3, 128)
        # three parts rounded to bf16 each, one sum rounded
        assert ((a.float() - parts.sum(3)).abs() <= 2.0 ** -8 * (parts.abs().sum(3) + a.float().abs()) * 1.01 + 1e-6).all()


def test_gradients_against_differences(fa):
    """Directional derivatives of sum(dO O), taken from the kernel's own forward in fp32, against its gradients."""
    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, Nq, Nk, d = 1, 4, 2, 60, 150, 64
    q, do = rand((B, Nq, Hq, d), g), rand((B, Nq, Hq, d), g)
    k, v = rand((B, Nk, Hkv, d), g), rand((B, Nk, Hkv, d), g)
    want = attend(q[0], k[0], v[0], d ** -0.5, do[0])
    o, lse = fa.fwd_cross(q.cuda(), k.cuda(), v.cuda())
    grads = fa.bwd_cross(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse)

    def f(x, y, z):
        """sum(dO O) of the definition at perturbed inputs: the kernel takes bf16 inputs, whose steps are coarser than a
        difference needs."""
        return (attend(x[0], y[0], z[0], d ** -0.5)["o"][0] * do[0].double()).sum().item()
    h = 1e-4
    for i, (name, x) in enumerate((("dq", q), ("dk", k), ("dv", v))):
        u = torch.randn(x.shape, generator=g, dtype=torch.float64)
        args = [q.double(), k.double(), v.double()]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * u, args[i] - h * u
        num = (f(*hi) - f(*lo)) / (2 * h)
        got = (grads[i].double().cpu() * u).sum().item()
        # the gradient's own bound, weighted by |u|, and h^2 times the third derivative along u (|u k| scale <~ 10)
        assert abs(got - num) <= (want[name][1] * u[0].abs()).sum().item() + h * h * 1e3 * abs(num) + 1e-3


def test_captured_and_replayed(fa):
    """A forward and backward recorded in a graph, replayed on new values in the same tensors."""
    g = torch.Generator().manual_seed(8)
    shapes = {"q": (2, 70, 4, 128), "k": (2, 300, 2, 128), "v": (2, 300, 2, 128), "do": (2, 70, 4, 128)}
    dev = {n: torch.zeros(s, dtype=torch.bfloat16, device="cuda") for n, s in shapes.items()}
    lens = i32([300, 300])
    ws = torch.empty(fa.bwd_workspace_bytes(140, 4, 128), dtype=torch.uint8, device="cuda")
    out = {"o": torch.empty_like(dev["q"]), "lse": torch.empty((2, 4, 70), device="cuda"), "dq": torch.empty_like(dev["q"]),
           "dk": torch.empty_like(dev["k"]), "dv": torch.empty_like(dev["k"])}

    def step():
        fa.fwd_cross(dev["q"], dev["k"], dev["v"], lens, out=out["o"], lse=out["lse"])
        fa.bwd_cross(dev["q"], dev["k"], dev["v"], out["o"], dev["do"], out["lse"], lens, dq=out["dq"], dk=out["dk"],
                     dv=out["dv"], workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([300, 300], [129, 0], [1, 256]):
        host = {name: rand(s, g) for name, s in shapes.items()}
        for name, x in host.items():
            dev[name].copy_(x)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.check_device_error() == 0
        for b in range(2):
            want = attend(host["q"][b], host["k"][b, :n[b]], host["v"][b, :n[b]], 128 ** -0.5, host["do"][b])
            for name in ("o", "lse", "dq"):
                check(out[name][b], want[name], name)
            for name in ("dk", "dv"):
                check(out[name][b, :n[b]], want[name], name)


def test_long_keys(fa):
    """20,000 keys, a handful of queries."""
    dense(fa, 1, 2, 1, 5, 20000, 128, [19990], seed=9)
