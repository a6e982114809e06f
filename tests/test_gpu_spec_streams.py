"""The speculative decoding calls with ``stream=`` on the GPU: a side stream that is busy when the
call is made, while the current stream allocates and writes."""
import pytest
import torch

import test_gpu_tree_attention as attention
import test_gpu_verify as verification
from distillation_ce_tvd_gb300 import binding, speculative

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 100_000_000      # cycles, some 50 ms


def busy_side_stream():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    return side


def fill(sizes):
    """Memory of these sizes, written on the current stream."""
    return [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]


@pytest.mark.parametrize("raw", [False, True])
def test_attention_without_a_workspace(raw):
    c = attention.case([3000, 77, 640], [9, 2, 30], 8, 2, 128, 16, seed=16)
    want, want_lse, _ = attention.run(c)
    torch.cuda.synchronize()
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (c["q"], binding.KVCache(c["k"], c["v"]), c["table"].to(DEV),
            torch.tensor(c["contexts"], **i32), torch.tensor(c["starts"], **i32), c["mask"].to(DEV))
    need = binding.fct_tree_attention_workspace_size(41, 8, 2, 128)
    side = busy_side_stream()
    out, lse = binding.fct_tree_attention(*args, stream=side.cuda_stream if raw else side)
    junk = fill([need, out.numel() * 2, lse.numel() * 4])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    del junk


def test_verification_outputs():
    c = verification.case([6] * 8, 3000, torch.float32, True, seed=1)
    want, _ = verification.run(c, 5)
    args = [c[x].to(DEV) for x in ("target", "tokens", "parent")] \
        + [torch.tensor(c["starts"], dtype=torch.int32, device=DEV)] \
        + [c[x].to(DEV) for x in ("uniform", "noise", "draft")]
    side = busy_side_stream()
    got = binding.fct_spec_verify(*args, max_depth=5, stream=side)
    junk = fill([x.numel() * x.element_size() for x in got])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    del junk


def test_the_default_streams_handles():
    c = attention.case([50], [3], 4, 2, 64, 16, seed=2)
    want, _, _ = attention.run(c)
    for handle in (0, 1):
        torch.cuda.synchronize()
        assert torch.equal(attention.run(c, stream=handle)[0], want)


@pytest.mark.parametrize("raw", [False, True])
def test_commit(raw):
    # the new context lengths wait for verification
    c = verification.case([6] * 8, 3000, torch.float32, True, seed=1)
    want, _ = verification.run(c, 5)
    i32 = dict(dtype=torch.int32, device=DEV)
    pool = torch.zeros((16, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    table, context = torch.arange(16, **i32).view(8, 2), torch.arange(8, **i32)
    args = [c[x].to(DEV) for x in ("target", "tokens", "parent")] \
        + [torch.tensor(c["starts"], dtype=torch.int32, device=DEV)] \
        + [c[x].to(DEV) for x in ("uniform", "noise", "draft")]
    side = busy_side_stream()
    out, path, count, lengths = speculative.commit(
        [binding.KVCache(pool, pool.clone())], table, context, *args, max_depth=5,
        stream=side.cuda_stream if raw else side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.cpu(), b) for a, b in zip((out, path, count), want))
    assert torch.equal(lengths.cpu(), torch.arange(8, dtype=torch.int32) + 1 + want[2])
    assert 0 < int(want[2].sum())


def test_the_loss_from_hidden_states():
    # its workspace and the zero-filled weight gradient
    gen = torch.Generator(device=DEV).manual_seed(4)
    h, w, ht, wt = (torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16) * 0.1
                    for s in ((256, 64), (2048, 64), (256, 128), (2048, 128)))
    target = torch.randint(0, 2048, (256,), generator=gen, device=DEV)
    args = (h, w, ht, wt, target, 1 / 256, 1 / 256)
    want = binding.fused_linear_ce_tvd_forward_backward(*args, chunk_rows=64)
    need = binding.fused_linear_ce_tvd_workspace_size(2048, 64)
    side = busy_side_stream()
    got = binding.fused_linear_ce_tvd_forward_backward(*args, chunk_rows=64, stream=side)
    junk = fill([need] + [x.numel() * x.element_size() for x in got])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk
