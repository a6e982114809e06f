"""Indexing helpers of the speculative decoding step, on the CPU, and what writing makes of them."""
import pytest
import torch

from distillation_ce_tvd_gb300 import binding, speculative

I32 = dict(dtype=torch.int32)
NONE = speculative.NO_SLOT


def slots(table, context, start, n, page=4):
    return speculative.node_slots(torch.tensor(table, **I32), torch.tensor(context, **I32),
                                  torch.tensor(start, **I32), n, page).tolist()


def test_slots_across_pages_and_requests_without_nodes():
    assert slots([[7, 3], [1, -1], [5, 6]], [3, 0, 4], [0, 2, 2, 4], 4) == [31, 12, 24, 25]


def test_positions_outside_the_table_have_no_slot():
    assert slots([[7, 3], [1, 2]], [7, 10 ** 6], [0, 2, 4], 4) == [15, NONE, NONE, NONE]
    assert slots([[7, 3], [1, 2]], [-1, -9], [0, 3, 4], 4) == [NONE, 28, 29, NONE]


def test_entries_without_a_page_have_no_slot():
    assert slots([[7, -1]], [3], [0, 2], 2) == [31, NONE]


def test_nodes_of_no_request_have_no_slot():
    assert slots([[7, 3]], [0], [0, 2], 4) == [28, 29, NONE, NONE]
    assert slots([[7, 3]], [0], [1, 3], 3) == [NONE, 28, 29]
    empty = speculative.node_slots(torch.zeros((0, 3), **I32), torch.zeros(0, **I32),
                                   torch.zeros(1, **I32), 2, 4)
    assert empty.tolist() == [NONE, NONE]


def test_no_slot_is_past_any_pool():
    # pools hold fewer than 2^62 / 8 vectors of 8 elements
    assert NONE >= 2 ** 62 and NONE < 2 ** 63


@pytest.mark.gpu
def test_writing_skips_and_reports_nodes_without_a_slot():
    i32 = dict(dtype=torch.int32, device="cuda:0")
    pool = torch.zeros((4, 4, 1, 64), dtype=torch.bfloat16, device="cuda:0")
    cache = binding.KVCache(pool, pool.clone())
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda:0")
    at = speculative.node_slots(torch.tensor([[2, 3], [1, -1]], **i32), torch.tensor([7, 3], **i32),
                                torch.tensor([0, 2, 4], **i32), 4, 4)
    st = torch.zeros(1, **i32)
    binding.fct_kv_cache_write(cache, x, x, at, dev_status=st)
    assert st.item() == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert cache.k.sum((1, 2, 3)).tolist() == [0, 64, 0, 64]
    assert bool((cache.k[3, 3] == 1).all()) and bool((cache.k[1, 3] == 1).all())
