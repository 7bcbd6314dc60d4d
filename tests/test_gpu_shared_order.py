"""decode_shared where a CTA goes from shares of many rows to few and back, against the definition in 64 bits."""
import random

import pytest
import torch

from test_gpu_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


@pytest.mark.parametrize("Hq,Hkv,d", [(24, 8, 64), (24, 8, 128), (160, 160, 64), (96, 32, 128), (40, 1, 64)])
@pytest.mark.parametrize("seed", range(4))
def test_many_rows_and_few_in_turn(fa, Hq, Hkv, d, seed):
    """Groups of a few and of many sequences: items of up to 32 rows before and behind larger ones, with one block and with many.
    160 KV heads leave one CTA for all of a head's items."""
    rng = random.Random(seed)
    groups, prefix, lens = [], [], []
    for count in rng.sample([5, 16, 7, 2, 11, 30], 4):
        groups.append((len(lens), count))
        prefix.append(rng.choice([100, 128, 300, 700, 1500]))
        lens += [prefix[-1] + rng.choice([0, 1, 17, 128, rng.randint(1, 400)]) for _ in range(count)]
    b = Batch(lens, groups, prefix, Hq, Hkv, d, seed=seed)
    for _ in range(3):
        o, lse = b.run(fa)
        assert fa.check_device_error() == 0
    b.check(o, lse)


@pytest.mark.parametrize("S", [1, 55, 56, 57, 128, 129])
def test_rows_at_the_borders_of_the_combine(fa, S):
    """440 to 456 rows, and few and many: joined by a block's eight warps or by one."""
    b = Batch([700 + 3 * (i % 50) for i in range(S)], [(0, S)] if S > 1 else [], [300] if S > 1 else [], 8, 2, 64, seed=S)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse)
