"""fwd_cross of tensors without heads: refused as an argument error (no GPU needed)."""
import pytest
import torch


class OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def gpu(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16).as_subclass(OnGpu)


@pytest.mark.parametrize("Hq,Hkv", [(0, 2), (0, 0), (4, 0), (5, 2)])
@pytest.mark.parametrize("split", [None, False, True])
def test_heads(Hq, Hkv, split, monkeypatch):
    import exact_io_aware_75_b200 as fa
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(fa, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(fa, "_sm_count", lambda device: 148)
    q, k = gpu(2, 3, Hq, 64), gpu(2, 5, Hkv, 64)
    with pytest.raises(fa.FAError):
        fa.fwd_cross(q, k, k, out=gpu(2, 3, Hq, 64), return_lse=False, split_keys=split)
