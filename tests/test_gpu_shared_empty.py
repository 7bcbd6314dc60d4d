"""decode_shared and decode_cross on batches with sequences without keys: first, in the middle, last, in runs longer than a warp,
against the definition in 64 bits."""
import pytest
import torch

from test_gpu_shared import Batch, cross

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import exact_io_aware_75_b200 as fa
    return fa


PLACES = {
    "first": [0] * 40 + [300, 5, 129],
    "middle": [300] + [0] * 70 + [7] + [0] * 33 + [128, 200],
    "last": [31, 500, 90] + [0] * 65,
    "every other": [0, 140] * 20,
    "one in many": [0] * 31 + [900] + [0] * 32 + [1] + [0] * 31,
    "none": [0] * 70,
}


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (40, 1, 64), (160, 1, 128), (160, 160, 64)])
def test_cross(fa, place, Hq, Hkv, d):
    """4, 40, 128 (two tokens of 64 heads) and 160 rows: each of the kernel's forms."""
    lens = PLACES[place]
    heads = min(Hq, 128 * Hkv)
    cross(fa, len(lens), heads, Hkv, 1 if Hq < 128 else 2, 900, d, lens, seed=3)


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (40, 1, 64), (64, 64, 128)])
def test_shared(fa, place, Hq, Hkv, d):
    """The same with a group behind them whose own parts are empty too (its tokens are all shared)."""
    lens = PLACES[place] + [64] * 12 + [80, 64]
    n = len(PLACES[place])
    b = Batch(lens, [(n, 14)], [64], Hq, Hkv, d, seed=4)
    o, lse = b.run(fa)
    assert fa.check_device_error() == 0
    b.check(o, lse)
