"""The speculative decoding calls with ``stream=`` on the GPU: a side stream that is busy when the
call is made, while the current stream allocates and writes."""
import pytest
import torch

import test_gpu_tree_attention as attention
import test_gpu_verify as verification
from distillation_ce_tvd_gb300 import binding

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
    side = torch.cuda.Stream()
    got, st = verification.run(c, 5, stream=side)
    torch.cuda.synchronize()
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_default_streams_handles():
    c = attention.case([50], [3], 4, 2, 64, 16, seed=2)
    want, _, _ = attention.run(c)
    for handle in (0, 1):
        torch.cuda.synchronize()
        assert torch.equal(attention.run(c, stream=handle)[0], want)
