"""The cross-attention calls at the ends of their ranges: longest lengths given as 0, batches without queries or without keys."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def run(fa, q, k, cq, ck, mq, mk):
    """Forward and backward into tensors that hold fives; -> (o, lse, dq, dk, dv), the calls' error words."""
    T, Hq, d = q.shape
    o, dq, dk, dv = torch.full_like(q, 5), torch.full_like(q, 5), torch.full_like(k, 5), torch.full_like(k, 5)
    lse = torch.full((Hq, T), 5.0, device="cuda")
    fa.fwd_varlen_cross(q, k, k, i32(cq), i32(ck), mq, mk, out=o, lse=lse)
    errors = [fa.check_device_error()]
    fa.bwd_varlen_cross(q, k, k, q, q, torch.zeros_like(lse), i32(cq), i32(ck), mq, mk, dq=dq, dk=dk, dv=dv)
    return (o, lse, dq, dk, dv), errors + [fa.check_device_error()]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mq,mk", [(0, 30), (20, 0), (0, 0)])
@pytest.mark.parametrize("seqs", [2, 130])
def test_longest_lengths_of_zero(fa, d, mq, mk, seqs):
    """Every sequence is longer: all are skipped and reported, dQ is zeros, the rest as it was."""
    q, k = rand(20 * seqs, 4, d), rand(30 * seqs, 2, d)
    got, errors = run(fa, q, k, [20 * i for i in range(seqs + 1)], [30 * i for i in range(seqs + 1)], mq, mk)
    assert errors == [fa.FA_ERR_INVALID_ARG] * 2
    o, lse, dq, dk, dv = got
    assert (dq == 0).all() and all((t == 5).all() for t in (o, lse, dk, dv))


@pytest.mark.parametrize("seqs", [3, 130])
def test_no_queries(fa, seqs):
    """Keys' gradients are zeros; a sequence that does not fit is skipped and reported; rows of no sequence stay."""
    q, k = rand(0, 4, 64), rand(30 * seqs + 7, 2, 64)
    ck = [3 + 30 * i for i in range(seqs + 1)]
    got, errors = run(fa, q, k, [0] * (seqs + 1), ck, 0, 30)
    assert errors == [0, 0]
    for t in got[3:]:
        assert (t[:3] == 5).all() and (t[3:ck[-1]] == 0).all() and (t[ck[-1]:] == 5).all()
    ck[-1] = 30 * seqs + 8                                  # the last one leaves the tensor (and is too long)
    got, errors = run(fa, q, k, [0] * (seqs + 1), ck, 0, 33)
    assert errors[1] == fa.FA_ERR_INVALID_ARG
    for t in got[3:]:
        assert (t[3:ck[-2]] == 0).all() and (t[ck[-2]:] == 5).all()
    # dense: lengths that the stored keys cannot hold
    k = rand(3, 30, 2, 64)
    dk, dv = torch.full_like(k, 5), torch.full_like(k, 5)
    q = rand(3, 0, 4, 64)
    fa.bwd_cross(q, k, k, q, q, torch.zeros((3, 4, 0), device="cuda"), i32([30, 31, 0]), dk=dk, dv=dv)
    assert fa.check_device_error() == fa.FA_ERR_INVALID_ARG
    for t in (dk, dv):
        assert (t[0] == 0).all() and (t[1] == 5).all() and (t[2] == 0).all()


def test_sequences_within_the_longest_still_run(fa):
    """max_seqlen_k = 0 is right for a sequence without keys; max_seqlen_q = 0 for one without queries."""
    q, k = rand(40, 4, 128), rand(30, 2, 128)
    got, errors = run(fa, q, k, [0, 40, 40], [0, 0, 0], 40, 0)
    assert errors == [0, 0]
    assert (got[0] == 0).all() and torch.isneginf(got[1]).all() and (got[2] == 0).all() and (got[3] == 5).all()
    got, errors = run(fa, q, k, [0, 0, 40], [0, 30, 30], 40, 30)
    assert errors == [0, 0]
    assert (got[3] == 0).all() and (got[0] == 0).all()
    o = fa.fwd_varlen_cross(q, k, k, i32([0, 40]), i32([0, 30]), 40, 30)[0]
    check(o, attend(q.cpu(), k.cpu(), k.cpu(), 128 ** -0.5)["o"], "O")
