"""What the SwiGLU quantizer does with a buffer that no plan was written to: the number of rows in use
that it reads there is checked like every other entry of a plan."""
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc

pytestmark = pytest.mark.gpu

INVALID = 1  # ARC_ERR_INVALID_ARG


def _sections(T, k, E, rows_in_use):
    """A plan buffer whose places are those of rows_in_use = S (all slots, expert 0), but for the total."""
    plan = arc.expert_plan(torch.zeros(T, k, dtype=torch.int32, device="cuda"), E)
    plan.offsets[E] = rows_in_use
    return plan


# a CTA for each row (few rows, wide rows), and lane groups (many narrow rows); without and with appended blocks
@pytest.mark.parametrize("T,k,E,F,r", [(16, 2, 4, 64, 0), (3, 1, 2, 2048, 32), (4801, 1, 5, 96, 0),
                                       (2400, 2, 5, 512, 64)])
@pytest.mark.parametrize("total", ["negative", "one too many", "huge"])
def test_a_total_outside_the_slots_is_reported(T, k, E, F, r, total):
    S = T * k
    n = {"negative": -5, "one too many": S + 1, "huge": 0x7F7F7F7F}[total]
    plan = _sections(T, k, E, n)
    gu = torch.ones(S, 2 * F, dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(r, dtype=torch.int32, device="cuda") if r else None
    size = (S * arc.kpad(F + r) // 2 + 255) // 256 * 256 + arc.lib().arc_expert_sf_bytes(T, k, E, F + r)
    out = arc.ExpertMXFP4(torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda"), S, F + r)
    assert arc.last_device_status() == 0
    arc.quantize_swiglu_experts_mxfp4(gu, plan, idx, out=out)
    assert arc.last_device_status() == INVALID
    assert (out.buf == 0xA5).all()  # treated as no row
    assert arc.last_device_status() == 0


@pytest.mark.parametrize("T,k,E,F", [(16, 2, 4, 64), (4801, 1, 5, 96)])
def test_totals_at_the_ends_of_the_range_are_fine(T, k, E, F):
    gu = torch.ones(T * k, 2 * F, dtype=torch.bfloat16, device="cuda")
    for expert in (0, -1):  # every slot a row, none
        plan = arc.expert_plan(torch.full((T, k), expert, dtype=torch.int32, device="cuda"), E)
        arc.quantize_swiglu_experts_mxfp4(gu, plan)
        assert arc.last_device_status() == 0
