"""Distillation from a teacher's top logits without a GPU: refusals of the C ABI and of the binding,
the workspaces' sizes, and the plain forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import top_util as tu
from distillation_ce_tvd_gb300 import autograd, binding

OK, INVALID, UNSUPPORTED, ALIGN, CUDA = 0, 1, 2, 3, 4
MB = 1 << 20


def at(i):
    """Addresses far apart, never followed."""
    return 0x7F0000000000 + i * (1 << 34)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def lists(**kw):
    f = dict(values=at(1), ld_values=16, index=at(2), ld_index=16, rest_lse=at(3), K=16)
    f.update(kw)
    reserved = f.pop("reserved", (0, 0))
    return ctypes.byref(binding._TopList(*f.values(), (ctypes.c_int64 * 2)(*reserved)))


def change(args, edits):
    a = list(args)
    for i, v in edits.items():
        a[i] = v
    return a


SELECT = [at(0), 1000, 1, 8, 1000, 16, at(1), 16, at(2), 16, at(3), None, None]


@pytest.mark.parametrize("edits,want", [
    ({3: 0}, OK), ({3: -1}, INVALID), ({0: None}, INVALID), ({1: 999}, INVALID), ({2: 2}, UNSUPPORTED),
    ({4: 0}, INVALID), ({4: -5}, INVALID), ({4: 1 << 31, 1: 1 << 31}, UNSUPPORTED), ({5: 0}, INVALID),
    ({5: 1025, 7: 2000, 9: 2000}, UNSUPPORTED), ({6: None}, INVALID), ({7: 15}, INVALID),
    ({8: None}, INVALID), ({9: 15}, INVALID), ({10: None}, INVALID), ({0: at(0) + 1}, ALIGN),
    ({2: 0, 0: at(0) + 2}, ALIGN), ({6: at(1) + 2}, ALIGN), ({8: at(2) + 1}, ALIGN),
    ({10: at(3) + 2}, ALIGN), ({11: at(4) + 2}, ALIGN), ({6: at(0)}, INVALID),
    ({8: at(1) + 64}, INVALID), ({10: at(2)}, INVALID), ({1: 1 << 60}, UNSUPPORTED)])
def test_selection_is_checked(lib, edits, want):
    assert lib.fct_top_logits(*change(SELECT, edits)) == want


FWD = [at(0), 1000, 1, at(4), None, 8, 1000, -100, at(5), at(6), at(7), at(8), at(9), at(10), None,
       None]
BWD = [at(0), 1000, 1, at(4), None, 8, 1000, -100, at(7), at(8), at(9), at(10), at(11), at(12), 1,
       at(13), 1000, None, None]
BOTH = [at(0), 1000, 1, at(4), None, 8, 1000, -100, at(11), at(12), 1, at(5), at(6), at(7), at(8),
        at(9), at(10), at(13), 1000, None, None]
CALLS = {"fused_ce_tvd_top_forward": FWD, "fused_ce_tvd_top_backward": BWD,
         "fused_ce_tvd_top_forward_backward": BOTH}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("edits,want", [
    ({5: 0}, OK), ({5: -1}, INVALID), ({0: None}, INVALID), ({1: 999}, INVALID), ({2: 2}, UNSUPPORTED),
    ({3: None}, INVALID), ({3: at(4) + 4}, ALIGN), ({6: 0}, INVALID),
    ({1: (1 << 23) + 1, 6: (1 << 23) + 1}, UNSUPPORTED), ({0: at(0) + 1}, ALIGN)])
def test_losses_are_checked(lib, name, edits, want):
    args = change(CALLS[name], edits)
    args[4] = lists()
    assert getattr(lib, name)(*args) == want


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("edit,want", [
    (dict(values=None), INVALID), (dict(index=None), INVALID), (dict(K=0), INVALID),
    (dict(K=1025, ld_values=2000, ld_index=2000), UNSUPPORTED), (dict(ld_values=15), INVALID),
    (dict(ld_index=15), INVALID), (dict(values=at(1) + 2), ALIGN), (dict(index=at(2) + 2), ALIGN),
    (dict(rest_lse=at(3) + 1), ALIGN), (dict(reserved=(1, 0)), INVALID)])
def test_lists_are_checked(lib, name, edit, want):
    args = list(CALLS[name])
    args[4] = lists(**edit)
    assert getattr(lib, name)(*args) == want
    args[4] = None
    assert getattr(lib, name)(*args) == INVALID


def test_what_overlaps_is_refused(lib):
    for name, args in CALLS.items():
        out = 13 if name.endswith("top_forward") else 15 if name.endswith("top_backward") else 17
        for other in (at(4), at(1), at(2), at(3)):
            a = change(args, {out: other})
            a[4] = lists()
            assert getattr(lib, name)(*a) == INVALID, (name, other)
    a = change(FWD, {8: at(6)})
    a[4] = lists()
    assert lib.fused_ce_tvd_top_forward(*a) == INVALID
    for name, grad in (("fused_ce_tvd_top_backward", 15), ("fused_ce_tvd_top_forward_backward", 17)):
        a = change(CALLS[name], {grad: at(0) + 2000})   # neither apart nor in place
        a[4] = lists()
        assert getattr(lib, name)(*a) == INVALID
        a = change(CALLS[name], {grad: at(0), grad + 1: 1008})
        a[4] = lists()
        assert getattr(lib, name)(*a) == INVALID
        a = change(CALLS[name], {10 if grad == 17 else 14: 2})
        a[4] = lists()
        assert getattr(lib, name)(*a) == INVALID


LFWD = [at(0), 64, at(14), 64, 64, at(4), None, 8, 1000, -100, at(5), at(6), at(7), at(8), at(9),
        at(10), at(15), 64 * MB, None, None]
LBWD = [at(0), 64, at(14), 64, 64, at(4), None, 8, 1000, -100, at(7), at(8), at(9), at(10), at(11),
        at(12), 1, at(13), 64, at(16), 64, 1, at(15), 64 * MB, 0, None, None]
CFWD = [at(0), 64, at(14), 64, 64, at(4), 8, 1000, -100, at(5), at(7), at(15), 64 * MB, None, None]
CBWD = [at(0), 64, at(14), 64, 64, at(4), 8, 1000, -100, at(7), at(11), 1, at(13), 64, at(16), 64, 1,
        at(15), 64 * MB, 0, None, None]
LINEAR = {"fused_linear_ce_tvd_top_forward": (LFWD, 7, 16), "fused_linear_ce_tvd_top_backward": (LBWD, 7, 22),
          "fused_linear_ce_forward": (CFWD, 6, 11), "fused_linear_ce_backward": (CBWD, 6, 17)}


@pytest.mark.parametrize("name", LINEAR)
def test_linear_calls_are_checked(lib, name):
    args, bt, ws = LINEAR[name]

    def call(edits):
        a = change(args, edits)
        if bt == 7:
            a[6] = lists()
        return getattr(lib, name)(*a)
    big = (1 << 31) - 1023
    for edits, want in [
            ({bt: -1}, INVALID), ({bt + 1: 0}, INVALID), ({4: 0}, INVALID), ({0: None}, INVALID),
            ({2: None}, INVALID), ({5: None}, INVALID), ({1: 63}, INVALID), ({3: 56}, INVALID),
            ({1: 68}, ALIGN), ({3: 68}, ALIGN), ({0: at(0) + 2}, ALIGN), ({2: at(14) + 8}, ALIGN),
            ({bt: big}, UNSUPPORTED), ({bt + 1: big}, UNSUPPORTED), ({ws: None}, INVALID),
            ({ws: at(15) + 64}, ALIGN), ({ws + 1: 100}, INVALID), ({ws: at(0)}, INVALID)]:
        assert call(edits) == want, edits
    if name.endswith("backward"):
        kind = ws - 1
        assert call({kind: 3}) == UNSUPPORTED and call({ws + 2: -1}) == INVALID
        assert call({kind - 5: 2}) == INVALID            # grad_stride
        assert call({kind - 3: 63}) == INVALID and call({kind - 1: 63}) == INVALID
        assert call({kind - 2: at(13)}) == INVALID       # the gradients overlap
        assert call({kind: 0, kind - 2: at(16) + 2}) == ALIGN
        assert call({bt: 0, kind - 2: None}) == OK
    else:
        assert call({bt: 0}) == OK


def test_workspace_sizes(lib):
    f, b = (binding.fused_linear_ce_tvd_top_forward_workspace_size,
            binding.fused_linear_ce_tvd_top_backward_workspace_size)
    assert f(0, 10) == f(10, 0) == f(10, 10, 1025) == f(10, 10, -1) == f(1 << 31, 10) == 0
    assert b(0, 10, 8) == b(10, 0, 8) == b(10, 10, 0) == b(10, 10, 8, 0, -1) == 0
    assert f(8192, 151936) >= 8192 * (2 * 594 * 8 + 8) and f(100, 1000, 64) > f(100, 1000, 0)
    whole = b(4096, 151936, 2048, 0, 151936)
    assert whole >= 4096 * 151936 * 2 and b(4096, 151936, 2048, 0, 1024) < whole / 8
    assert b(4096, 151936, 2048) == b(4096, 151936, 2048, 0, (1 << 28) // 4096)
    assert f((1 << 31) - 1024, (1 << 31) - 1024) > 0


def test_status_bits_and_limits():
    assert binding.FCT_DEV_BAD_LIST == 0x10 and binding.FCT_TOP_MAX == 1024


def test_the_binding_wants_cuda_tensors():
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    v, i = torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    h = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.fct_top_logits(x, 3)
    with pytest.raises(ValueError):
        binding.fused_ce_tvd_top_forward(x, t, v, i)
    with pytest.raises(ValueError):
        binding.fused_ce_tvd_top_forward_backward(student=x, target=t, top_values=v, top_index=i,
                                                  rest_lse=None, grad_ce=1.0, grad_tvd=1.0)
    with pytest.raises(ValueError):
        binding.fused_linear_ce_forward(h, h, t)
    with pytest.raises(ValueError):
        autograd.fused_linear_ce_loss(h, h, t)


def test_plain_forms():
    """The comparison's own forms: closed forms, and autograd for the gradient."""
    v, i, rest = tu.top_ref(torch.tensor([1.0, 3.0, 3.0, -math.inf, 2.0]), 2)
    assert (v, i) == ([3.0, 3.0], [1, 2]) and abs(rest - math.log(math.e + math.e ** 2)) < 1e-12
    assert tu.top_ref(torch.tensor([-math.inf, 4.0]), 3) == ([4.0, -math.inf, -math.inf], [1, -1, -1],
                                                             -math.inf)
    s, target, values, index, rests, gce, gtvd = tu.make(5, 40, 6, torch.float64, 3)
    for r in (0, 1, 3, 4):
        x = s[r].clone().requires_grad_()
        used = index[r] >= 0
        p = torch.softmax(x, 0)
        q = torch.softmax(torch.cat([values[r][used].double(), rests[r:r + 1].double()]), 0)
        mine = p[index[r][used].long()]
        ce = -torch.log_softmax(x, 0)[target[r]]
        tvd = 0.5 * ((mine - q[:-1]).abs().sum() + (1 - mine.sum() - q[-1]).abs())
        (gce[r].double() * ce + gtvd[r].double() * tvd).backward()
        want = tu.row_ref(s[r], int(target[r]), values[r], index[r], float(rests[r]), float(gce[r]),
                          float(gtvd[r]))
        assert abs(want["ce"] - ce.item()) < 1e-12 and abs(want["tvd"] - tvd.item()) < 1e-12
        assert torch.allclose(want["grad"], x.grad, rtol=0, atol=1e-12)
