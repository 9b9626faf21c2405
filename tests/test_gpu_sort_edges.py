"""GPU: the expert sort at the ends of its range."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def plan_of(lib, idx, E, align, capacity):
    T, R = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.full((E,), -9, **i32), torch.full((E + 1,), -9, **i32),
           torch.full((lib.sort_rows_bound(T, R, E, align, capacity),), -9, **i32),
           torch.full((T, R), -9, **i32))
    lib.moe_sort(idx, E, *out, lib.workspace(lib.sort_ws_bytes(T, E, R)), align=align,
                 capacity=capacity, flags=lib.MOE_CHECK)
    return out


def test_limit_under_an_expert_that_takes_nearly_all(lib):
    """2^31 - 32 slots, a row an expert: the hot expert's first row plus the rank of its last slots
    is past 2^31, and those slots have no row like the others that the limit leaves out."""
    T, R, E, align = 2 ** 26 - 1, 32, 1024, 4096
    idx = torch.full((T, R), E - 1, dtype=torch.int32, device="cuda")
    idx.view(-1)[:E] = torch.arange(E, device="cuda").int()
    counts, offsets, row_slot, slot_row = plan_of(lib, idx, E, align, 1)
    assert (counts == 1).all()
    first = torch.arange(E + 1, device="cuda").int() * align
    assert torch.equal(offsets, first)
    flat = slot_row.view(-1)
    assert torch.equal(flat[:E], first[:E])
    for part in flat[E:].split(2 ** 28):
        assert (part == -1).all()
    rows = row_slot.view(E, align)
    assert torch.equal(rows[:, 0], torch.arange(E, device="cuda").int()) and (rows[:, 1:] == -1).all()


def test_one_expert_whose_rows_end_near_2_to_the_31(lib):
    """2^31 - 2 slots in tiles of three rows: the end of the plan is 2^31 - 2 as well."""
    T, R, align = 2 ** 30 - 1, 2, 3
    idx = torch.zeros((T, R), dtype=torch.int32, device="cuda")
    counts, offsets, row_slot, slot_row = plan_of(lib, idx, 1, align, 0)
    n = T * R
    assert counts.tolist() == [n] and offsets.tolist() == [0, n]
    for of in (row_slot, slot_row.view(-1)):
        for at in range(0, n, 2 ** 28):
            part = of[at:at + 2 ** 28]
            assert torch.equal(part, torch.arange(at, at + part.numel(), device="cuda").int())
