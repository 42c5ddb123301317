"""The router weights' gradient adds up no longer fp32 chains than its comment says, whatever shape the
kernel takes its rows in.

Bound. A lane keeps one sum for each of its four vectors of a round, so a sum has 8 products a round: at
most three rounds (24 products) where few lanes take a row, 8 ceil(d / 1024) where the whole warp does. Two
additions join the four sums, five shuffles the lanes: (max(24, 8 ceil(d / 1024)) + 7) half-steps of fp32
times the sum of magnitudes.
"""
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc

pytestmark = pytest.mark.gpu


def _bound(d):
    return (max(24, 8 * -(-d // 1024)) + 7) * 2.0 ** -24


# many slots, whose rows few lanes take in several rounds, and few
@pytest.mark.parametrize("T,k,d", [(6001, 1, 264), (2400, 2, 264), (3001, 2, 520), (2501, 1, 1024), (700, 4, 1536),
                                   (40, 2, 264), (9, 3, 4104), (25, 1, 8192)])
@pytest.mark.parametrize("lead", [0, 1])
def test_a_large_first_product_swallows_few_small_ones(T, k, d, lead):
    # one product of 2^24, then ones: each one that is added to a sum of 2^24 is lost (a tie, to even),
    # so the error counts the products of the longest chain. lead: which vector begins large.
    plan = arc.expert_plan(torch.zeros(T, k, dtype=torch.int32, device="cuda"), 1)
    rows = torch.ones(T * k, d, dtype=torch.bfloat16, device="cuda")
    rows[:, 8 * lead] = 2.0 ** 24
    dy, w = torch.ones(T, d, dtype=torch.bfloat16, device="cuda"), torch.ones(T, k, device="cuda")
    _, d_w = arc.combine_experts_grad(dy, rows, w, plan)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    exact = 2.0 ** 24 + d - 1
    assert ((d_w.double() - exact).abs() <= _bound(d) * exact).all(), (d_w.double() - exact).abs().max().item()


@pytest.mark.parametrize("T,k,d", [(6001, 1, 264), (3001, 2, 520), (2501, 3, 1032), (33, 2, 4104)])
def test_random_rows_stay_within_the_bound(T, k, d):
    gen = torch.Generator(device="cuda").manual_seed(d)
    rows, dy = (torch.randn(n, d, generator=gen, device="cuda").bfloat16() for n in (T * k, T))
    ids = torch.randint(0, 7, (T, k), generator=gen, device="cuda")
    plan = arc.expert_plan(ids, 7)
    _, d_w = arc.combine_experts_grad(dy, rows, torch.ones(T, k, device="cuda"), plan)
    prod = dy.double().repeat_interleave(k, 0) * rows.double()[plan.row_of_slot.long()]
    assert ((d_w.double().view(-1) - prod.sum(1)).abs() <= _bound(d) * prod.abs().sum(1)).all()
