"""The stream argument of every call that allocates or launches: a stream of another device is refused, and the call, with what
it allocates, runs inside the stream that was passed (no GPU needed)."""
import contextlib
import inspect

import pytest
import torch


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_75_b200 as fa
    return fa


class OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)


class Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device = torch.device("cuda", index)


CALLS = ["fwd", "fwd_varlen", "fwd_paged", "fp8_prepare", "fwd_fp8", "bwd", "bwd_varlen", "decode_paged", "decode_paged_fp8",
         "decode_paged_noalloc", "fwd_cross", "fwd_varlen_cross", "bwd_cross", "bwd_varlen_cross", "decode_shared", "decode_cross",
         "cache_fork", "cache_append", "cache_copy_pages", "cache_collect", "cache_compact"]


def arguments(fa, name):
    """Something for every argument without a default; the first a tensor on a GPU (or the operands of the FP8 prefill)."""
    t = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16).as_subclass(OnGpu)
    first, *rest = [p for p in inspect.signature(getattr(fa, name)).parameters.values() if p.default is p.empty]
    return [dict(q8=t, k8=t, vt8=t) if first.name == "prep" else t] + [t] * len(rest)


def test_all_calls_are_here(fa):
    taking = [n for n, f in vars(fa).items() if inspect.isfunction(f) and not n.startswith("_")
              and "stream" in inspect.signature(f).parameters]
    assert sorted(taking) == sorted(CALLS + ["check_device_error", "selftest_watchdog"])


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(fa, name):
    with pytest.raises(fa.FAError, match="a stream of cuda:1"):
        getattr(fa, name)(*arguments(fa, name), stream=Stream(1))


@pytest.mark.parametrize("name", CALLS)
def test_the_call_runs_inside_the_stream(fa, name, monkeypatch):
    inside, seen = [], []

    @contextlib.contextmanager
    def enter(stream):
        inside.append(stream)
        yield
        inside.pop()
    need = fa._need
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(fa, "_need", lambda *a: (seen.append(list(inside)), need(*a))[1])
    st = Stream(0)
    with pytest.raises(Exception):          # (no GPU, and arguments of one shape for all)
        getattr(fa, name)(*arguments(fa, name), stream=st)
    assert seen and all(s == [st] for s in seen)


@pytest.mark.parametrize("name", ["check_device_error", "selftest_watchdog"])
def test_the_error_word_is_the_streams_devices(fa, name, monkeypatch):
    """Each device has its own error word: the one of the stream's device is read, whichever device is current."""
    inside, seen = [], []

    @contextlib.contextmanager
    def enter(device):
        inside.append(device)
        yield
        inside.pop()

    class Library:
        def __getattr__(self, _):
            return lambda *a: seen.append(list(inside)) or 0
    monkeypatch.setattr(torch.cuda, "device", enter)
    monkeypatch.setattr(fa, "_lib", Library())
    assert getattr(fa, name)(stream=Stream(1)) == 0
    assert seen == [[torch.device("cuda", 1)]]
