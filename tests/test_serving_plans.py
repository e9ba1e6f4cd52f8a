"""Plans of sequences that have outgrown their page table."""
import pytest
import torch

lg = pytest.importorskip("epilogue_scaled_gemm_amd")


def test_nodes_past_the_page_table_have_no_slot():
    table = torch.tensor([[3, 1], [2, -1], [0, 4]], dtype=torch.int32)
    ctx = torch.tensor([6, 3, 2 ** 31 - 2], dtype=torch.int32)
    off = torch.tensor([0, 4, 6, 8], dtype=torch.int32)
    got = lg.node_slots(table, ctx, off, 4)
    # positions 6, 7 and two past the table; 3 and one on an entry of -1; far past it
    assert got.tolist() == [1 * 4 + 2, 1 * 4 + 3, -1, -1, 2 * 4 + 3, -1, -1, -1]
    assert got.dtype == torch.int32


def test_an_empty_plan_has_no_slots():
    table = torch.zeros(2, 3, dtype=torch.int32)
    zero = torch.zeros(2, dtype=torch.int32)
    assert lg.node_slots(table, zero, torch.zeros(3, dtype=torch.int32), 16).tolist() == []
