"""The Python calls of the speculative decoding step without a GPU: a library that only records, CPU
tensors that say they are on device 0, and streams and devices that note what is done under them."""
import contextlib

import pytest
import torch

from distillation_ce_tvd_gb300 import binding, speculative

BF16 = torch.bfloat16
HERE, SIDE = object(), object()


class Recorder:
    def __init__(self):
        self.calls, self.made, self.now, self.device = [], [], HERE, 0

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 4096
        return lambda *a: self.calls.append((name, self.now, self.device, a)) or 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()

    @contextlib.contextmanager
    def under(stream):
        before, r.now = r.now, stream
        yield
        r.now = before

    @contextlib.contextmanager
    def on(device):
        before, r.device = r.device, device
        yield
        r.device = before
    empty = torch.empty

    def noted(*a, **kw):
        x = empty(*a, **kw)
        r.made.append((r.now, r.device, x))
        return x
    monkeypatch.setattr(binding, "load", lambda: r)
    monkeypatch.setattr(binding, "_library", lambda: r)
    monkeypatch.setattr(binding, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: r.now)
    monkeypatch.setattr(torch.cuda, "Stream", object)
    monkeypatch.setattr(torch, "empty", noted)
    return r


def cache(index=0):
    c = object.__new__(binding.KVCache)
    c.k = c.v = torch.zeros((4, 8, 2, 64), dtype=BF16)
    c.k_scale = c.v_scale = c.ref = None
    c.device, c.index, c.n_heads, c.head_dim = torch.device("cpu"), index, 2, 64
    return c


I32 = dict(dtype=torch.int32)
PAGES = (torch.zeros((2, 2), **I32), torch.tensor([3, 5], **I32))
STARTS = torch.tensor([0, 2, 5], **I32)


def write(c, **kw):
    k = torch.zeros((5, 2, 64), dtype=BF16)
    return binding.fct_kv_cache_write(c, k, k.clone(), torch.zeros(5, dtype=torch.int64), **kw)


def move(c, **kw):
    return binding.fct_kv_cache_move(c, *PAGES, torch.zeros((2, 3), **I32), torch.zeros(2, **I32), **kw)


def attend(c, **kw):
    return binding.fct_tree_attention(torch.zeros((5, 4, 64), dtype=BF16), c, *PAGES, STARTS, **kw)


def verify(c, **kw):
    z = torch.zeros((5, 10))
    return binding.fct_spec_verify(z, torch.zeros(5, dtype=torch.int64), torch.zeros(5, **I32), STARTS,
                                   torch.zeros(5), torch.ones((2, 10)), max_depth=2, **kw)


CALLS = [write, move, attend, verify]


@pytest.mark.parametrize("call", CALLS)
def test_what_a_call_allocates_belongs_to_its_stream(lib, call):
    call(cache())
    assert [c[1] for c in lib.calls] == [HERE] and all(now is HERE for now, _, _ in lib.made)
    made = len(lib.made)
    assert made == {write: 0, move: 0, attend: 3, verify: 3}[call]
    call(cache(), stream=SIDE)
    assert [c[1] for c in lib.calls] == [HERE, SIDE] and lib.now is HERE
    assert len(lib.made) == 2 * made and all(now is SIDE for now, _, _ in lib.made[made:])


def test_the_new_context_lengths_are_computed_on_the_calls_stream(lib):
    # they depend on what verification writes there
    class Watch(torch.overrides.TorchFunctionMode):
        sums = []

        def __torch_function__(self, f, types, args=(), kwargs=None):
            if getattr(f, "__name__", "") in ("add", "__add__", "gt", "__gt__"):
                self.sums.append(lib.now)
            return f(*args, **(kwargs or {}))
    z = torch.zeros((5, 10))
    args = ([cache(), cache()], *PAGES, z, torch.zeros(5, dtype=torch.int64), torch.zeros(5, **I32),
            STARTS, torch.zeros(5), torch.ones((2, 10)))
    for stream in (None, SIDE):
        lib.calls.clear()
        Watch.sums.clear()
        with Watch():
            speculative.commit(*args, max_depth=2, stream=stream)
        want = HERE if stream is None else SIDE
        assert [c[:2] for c in lib.calls] == [("fct_spec_verify", want)] + [("fct_kv_cache_move", want)] * 2
        assert len(Watch.sums) >= 3 and all(x is want for x in Watch.sums)
