"""A mixture-of-experts layer beside a shared expert on a second stream, joined by events, eager and captured:
calls that may begin before the kernel in front of them ends still wait for what the other stream makes, and
what both streams read may be written again after the join.
"""
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc
import workloads as W
from tests._experts import make_ids
from tests._helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,d,F", [(300, 2, 6, 512, 256), (4, 4, 40, 256, 128), (5000, 2, 4, 256, 128)])
def test_shared_expert_on_a_second_stream(T, k, E, d, F):
    x, add = to_dev(W.matrix_bf16(31, 1, T, d, 1.0)), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.from_numpy(make_ids(31, T, k, E)).cuda()
    weights = torch.rand(T, k, device="cuda")
    wgu = to_dev(W.matrix_bf16(31, 2, E * 2 * F, d, 0.05)).view(E, 2 * F, d)
    wd = to_dev(W.matrix_bf16(31, 3, E * d, F, 0.05)).view(E, d, F)
    q = [arc.pack_weight_experts_mxfp4(w) for w in (wgu, wd)]
    side = torch.cuda.Stream()

    def layer(parallel):
        main = torch.cuda.current_stream()
        plan = arc.expert_plan(ids, E)
        if parallel:  # right behind the plan, which both streams read
            side.wait_stream(main)
        with torch.cuda.stream(side if parallel else main):
            rows16 = arc.dispatch_experts(x, plan)
            back = arc.dispatch_experts_grad(rows16, plan)
            shared = arc.gemm_bf16(arc.silu_mul_bf16(arc.gemm_bf16(x, wgu[0])), wd[0])
        gu = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan), q[0], plan)
        rows = arc.gemm_experts_mxfp4(arc.quantize_swiglu_experts_mxfp4(gu, plan), q[1], plan)
        if parallel:
            main.wait_stream(side)
        y = arc.combine_experts(rows, weights, plan, add=shared)
        d_rows, d_w = arc.combine_experts_grad(y, rows, weights, plan)
        return y, back, shared, d_w, arc.dispatch_experts_grad(d_rows, plan)

    layer(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(True)
    for turn in range(6):
        gen = torch.Generator(device="cuda").manual_seed(turn)
        torch.cuda.synchronize()
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        ids.copy_(torch.from_numpy(make_ids(turn, T, k, E, ("skewed", "one", "repeat")[turn % 3])))
        want = [t.clone() for t in layer(False)]
        torch.cuda.synchronize()
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)
        for _ in range(3):
            for got, ref in zip(layer(True), want):
                assert torch.equal(got, ref)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0


def test_plan_written_again_while_its_readers_run():
    # one plan buffer and one row buffer for a sequence of layers on one stream: each call that writes them
    # waits for the calls that read what was there
    T, k, E, d = 3000, 4, 16, 512
    ids = [torch.from_numpy(make_ids(40 + i, T, k, E)).cuda() for i in range(8)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(T, d, device="cuda", generator=gen).bfloat16() for _ in range(8)]
    w = torch.full((T, k), 0.25, device="cuda")
    plan = arc.expert_plan(ids[0], E)
    rows = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    ys = []
    for _ in range(4):
        for i in range(8):
            arc.expert_plan(ids[i], E, out=plan)
            arc.dispatch_experts(x[i], plan, out=rows)
            ys.append(arc.combine_experts(rows, w, plan))
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    for j, y in enumerate(ys):  # four equal rows, a quarter of each: the token
        assert torch.equal(y, x[j % 8]), j
