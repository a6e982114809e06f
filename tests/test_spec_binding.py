"""The Python calls of the speculative decoding step without a GPU: a library that only records, CPU
tensors that say they are on device 0, and streams and devices that note what is done under them."""
import contextlib

import pytest
import torch

from distillation_ce_tvd_gb300 import binding, speculative, vocab_parallel

BF16 = torch.bfloat16


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device_index = handle, 0


HERE, SIDE = Stream(0), Stream(64)


class Recorder:
    def __init__(self):
        self.calls, self.made, self.marked, self.asked = [], [], [], []
        self.now, self.device = HERE, 0

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: self.asked.append(self.device) or 4096
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
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: r.marked.append((s, self)))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: r.now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: r.device)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
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
    # the results are marked as used by the caller's stream
    assert [s for s, _ in lib.marked] == [HERE] * {write: 0, move: 0, attend: 2, verify: 3}[call]


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


@pytest.mark.parametrize("call", CALLS)
def test_a_call_runs_on_its_tensors_device(lib, call):
    lib.device = 1                      # the tensors say 0
    call(cache())
    assert [c[2] for c in lib.calls] == [0] and all(d == 0 for _, d, _ in lib.made)
    assert lib.asked == [0] * (call is attend) and lib.device == 1
    other = Stream(128)
    other.device_index = 1
    with pytest.raises(ValueError):
        call(cache(), stream=other)


def loss_calls():
    z, t = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int64)
    row, one = torch.zeros(4), torch.ones(1)
    signs = torch.zeros((4, 16), dtype=torch.uint8)
    h, w = torch.zeros((4, 8), dtype=BF16), torch.zeros((16, 8), dtype=BF16)
    b = binding
    return {
        "forward": lambda **k: b.fused_ce_tvd_forward(z, z, t, **k),
        "backward": lambda **k: b.fused_ce_tvd_backward(z, z, t, row, row, row, one, row, **k),
        "forward_backward": lambda **k: b.fused_ce_tvd_forward_backward(z, z, t, one, row, **k),
        "ce_forward": lambda **k: b.ce_forward(z, t, **k),
        "ce_backward": lambda **k: b.ce_backward(z, t, row, row, **k),
        "ce_forward_backward": lambda **k: b.ce_forward_backward(z, t, row, **k),
        "mean_upstream": lambda **k: b.fused_ce_tvd_mean_upstream(t, **k),
        "mean_loss": lambda **k: b.fused_ce_tvd_mean_loss(row, row, t, **k),
        "vp_lse": lambda **k: b.fused_ce_tvd_vp_lse(z, z, t, 0, **k),
        "vp_backward": lambda **k: b.fused_ce_tvd_vp_backward(z, z, t, 0, 8, row, row, row, one, one, **k),
        "linear": lambda **k: b.fused_linear_ce_tvd_forward_backward(h, w, h, w, t, one, row, **k),
        "gemm": lambda **k: b.fct_gemm_bf16(h, w, **k),
    }


@pytest.mark.parametrize("name", sorted(loss_calls()))
def test_so_it_does_in_the_loss_calls(lib, name):
    # zero-filled gradients and broadcast upstream values too
    class Watch(torch.overrides.TorchFunctionMode):
        made = []

        def __torch_function__(self, f, types, args=(), kwargs=None):
            if getattr(f, "__name__", "") in ("empty_like", "zeros", "contiguous", "expand", "to"):
                self.made.append(lib.now)
            return f(*args, **(kwargs or {}))
    call = loss_calls()[name]
    Watch.made.clear()
    with Watch():
        call(stream=SIDE)
    assert len(lib.calls) == 1 and lib.calls[0][1] is SIDE
    assert all(now is SIDE for now, _, _ in lib.made) and all(now is SIDE for now in Watch.made)
    assert len(lib.made) + len(Watch.made) > 0


def test_the_vocabulary_shards_partials_are_exchanged_on_the_steps_stream(lib):
    z, t, one = torch.zeros((4, 16)), torch.zeros(4, dtype=torch.int64), torch.ones(1)
    seen = []

    def exchange(part):
        seen.append(lib.now)
        return torch.stack([part, part])

    class Watch(torch.overrides.TorchFunctionMode):
        def __torch_function__(self, f, types, args=(), kwargs=None):
            if getattr(f, "__name__", "") == "stack":
                seen.append(lib.now)
            return f(*args, **(kwargs or {}))
    vocab_parallel.step(z[:, :8], z[:, :8], t, 0, 16, one, one, exchange, stream=SIDE)
    assert seen == [SIDE] * 2 and all(c[1] is SIDE for c in lib.calls) and len(lib.calls) == 5
    with Watch():
        vocab_parallel.forward_backward_local(z, z, t, 2, one, one, stream=SIDE)
    assert seen == [SIDE] * 4 and all(c[1] is SIDE for c in lib.calls) and len(lib.calls) == 13


@pytest.mark.parametrize("call", CALLS)
def test_the_status_word_and_the_workspace_are_checked(lib, monkeypatch, call):
    good = torch.zeros(1, **I32)
    call(cache(), dev_status=good)
    for bad in (good.long(), good.float(), good[:0]):
        with pytest.raises(ValueError):
            call(cache(), dev_status=bad)
    far = torch.zeros(4096, dtype=torch.uint8)
    if call is attend:
        call(cache(), workspace=far)
        with pytest.raises(ValueError):
            call(cache(), workspace=torch.zeros((64, 128), dtype=torch.uint8)[:, ::2])
    # on another device
    where = {id(good): -1, id(far): 1}
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: where.get(id(self), 0))
    with pytest.raises(ValueError):
        call(cache(), dev_status=good)
    if call is attend:
        with pytest.raises(ValueError):
            call(cache(), workspace=far)
    assert len(lib.calls) == 1 + (call is attend)


def test_a_mask_without_words_is_not_a_chain(lib):
    # its address is null, which the library takes for no mask
    for n in (1, 5):
        q, mask = torch.zeros((n, 4, 64), dtype=BF16), torch.zeros((n, 1), dtype=torch.int64)
        args = (cache(), PAGES[0][:1], PAGES[1][:1], torch.tensor([0, n], **I32))
        lib.calls.clear()
        binding.fct_tree_attention(q, *args, mask)
        with pytest.raises(ValueError):
            binding.fct_tree_attention(q, *args, mask[:, :0])
        assert len(lib.calls) == 1
