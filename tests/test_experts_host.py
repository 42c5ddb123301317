"""Host-side checks of the mixture-of-experts calls (no GPU): sizes, NULL pointers, leading
dimensions, alignment and limits are refused before any launch; the binding refuses tensors that do
not fit the call."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc

INVALID, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 6
P = ctypes.c_void_p
A = P(0x10000)  # never dereferenced: the checks return first
ODD = P(0x10008)


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_scaled_arc_b200 import _build

    _build.build()
    return arc.lib()


def _each(fn, good, cases):
    """fn(*good) with one argument (or several) replaced returns the status given."""
    for change, status in cases:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert fn(*args) == status, (change, status)


def test_size_queries(L):
    pad = lambda n: (n + 63) // 64 * 64  # noqa: E731
    for T, k, E in [(1, 1, 1), (1, 8, 128), (4096, 2, 8), (1000, 6, 512)]:
        S = T * k
        assert L.arc_expert_plan_bytes(T, k, E) == 4 * (2 * pad(E + 1) + 3 * pad(S))
        for ka in (32, 256, 4224):
            places = (S + 127 * min(E, S)) // 128 * 128
            assert L.arc_expert_sf_bytes(T, k, E, ka) == places * 8 * ((pad(ka) + 255) // 256)
    for bad in [(0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1025, 2000), (1, 1, 513), (1 << 28, 2, 4)]:
        assert L.arc_expert_plan_bytes(*bad) == 0 and L.arc_expert_sf_bytes(*bad, 64) == 0
    # every group a row longer than whole blocks: the places are the most that any routing needs
    counts = [129] * 7
    assert (sum(counts) + 127 * 7) // 128 == sum((c + 127) // 128 for c in counts)


def test_plan_checks(L):
    size = L.arc_expert_plan_bytes(16, 4, 8)
    _each(L.arc_expert_plan, [A, 4, 4, 16, 4, 8, A, size, None], [
        ({0: None}, INVALID), ({6: None}, INVALID), ({1: 2}, INVALID), ({2: 3}, INVALID), ({3: 0}, INVALID),
        ({4: 0}, INVALID), ({5: 0}, INVALID), ({5: 513}, UNSUPPORTED), ({3: 1 << 28}, UNSUPPORTED),
        ({4: 1025, 2: 1025}, UNSUPPORTED), ({0: P(0x10002)}, ALIGN), ({1: 8, 0: P(0x10004)}, ALIGN),
        ({6: ODD}, ALIGN), ({7: size - 1}, WORKSPACE)])


def test_move_checks(L):
    dispatch = [A, 64, 64, A, 16, 4, 8, A, 64, None]
    bad = [({0: None}, INVALID), ({3: None}, INVALID), ({7: None}, INVALID), ({1: 56}, INVALID), ({8: 56}, INVALID),
           ({2: 60}, INVALID), ({1: 68}, INVALID), ({8: 68}, INVALID), ({2: 0}, INVALID), ({4: -1}, INVALID),
           ({6: 600}, UNSUPPORTED), ({0: ODD}, ALIGN), ({7: ODD}, ALIGN), ({3: P(0x10004)}, ALIGN)]
    _each(L.arc_dispatch_experts_bf16, dispatch, bad)
    _each(L.arc_dispatch_experts_grad_bf16, dispatch, bad)
    _each(L.arc_combine_experts_bf16, [A, 64, 64, A, 4, A, 16, 4, 8, A, 64, A, 64, None], [
        ({0: None}, INVALID), ({3: None}, INVALID), ({5: None}, INVALID), ({11: None}, INVALID), ({4: 3}, INVALID),
        ({10: 56}, INVALID), ({10: 68}, INVALID), ({1: 32}, INVALID), ({12: 32}, INVALID), ({2: 12}, INVALID),
        ({3: P(0x10002)}, ALIGN), ({9: ODD}, ALIGN), ({11: ODD}, ALIGN), ({8: 513}, UNSUPPORTED)])
    _each(L.arc_combine_experts_grad_bf16, [A, 64, A, 64, 64, A, 4, A, 16, 4, 8, A, 64, A, 4, None], [
        ({0: None}, INVALID), ({2: None}, INVALID), ({5: None}, INVALID), ({7: None}, INVALID), ({11: None}, INVALID),
        ({13: None}, INVALID), ({6: 3}, INVALID), ({14: 3}, INVALID), ({12: 56}, INVALID), ({12: 68}, INVALID),
        ({1: 32}, INVALID), ({13: P(0x10002)}, ALIGN), ({11: ODD}, ALIGN), ({0: ODD}, ALIGN)])


def test_quantizer_checks(L):
    good = [A, 128, 64, A, 32, A, 16, 4, 8, A, A, None]
    both = [({0: None}, INVALID), ({5: None}, INVALID), ({9: None}, INVALID), ({10: None}, INVALID), ({2: 48}, INVALID),
            ({4: 16}, INVALID), ({4: 96}, INVALID), ({4: -32}, INVALID), ({3: None}, INVALID), ({7: 0}, INVALID),
            ({8: 513}, UNSUPPORTED), ({2: 1 << 21, 1: 1 << 22}, UNSUPPORTED), ({0: ODD}, ALIGN), ({1: 132}, ALIGN),
            ({9: ODD}, ALIGN), ({10: ODD}, ALIGN), ({5: ODD}, ALIGN)]
    _each(L.arc_quantize_act_experts_mxfp4, good, both + [({1: 32}, INVALID)])
    _each(L.arc_quantize_swiglu_experts_mxfp4, good, both + [({1: 64}, INVALID)])  # gate and up: 2 F columns
    _each(L.arc_pack_weight_experts_mxfp4, [A, 8, 128, 64, 64, A, 32, A, A, None], [
        ({1: 0}, INVALID), ({2: 0}, INVALID), ({0: None}, INVALID), ({7: None}, INVALID), ({8: None}, INVALID),
        ({3: 48}, INVALID), ({6: 16}, INVALID), ({4: 32}, INVALID), ({1: 513}, UNSUPPORTED),
        ({2: 1 << 30}, UNSUPPORTED), ({2: 100, 0: None}, INVALID), ({2: 100, 8: ODD}, ALIGN), ({0: ODD}, ALIGN)])


def test_product_checks(L):
    _each(L.arc_gemm_experts_mxfp4, [A, A, A, A, A, 16, 4, 8, 64, 64, A, 64, None], [
        ({i: None}, INVALID) for i in (0, 1, 2, 3, 4, 10)] + [
        ({i: ODD}, ALIGN) for i in (0, 1, 2, 3, 4, 10)] + [
        ({8: 12}, INVALID), ({8: 0}, INVALID), ({9: 0}, INVALID), ({11: 56}, INVALID), ({11: 68}, INVALID),
        ({5: 0}, INVALID), ({7: 513}, UNSUPPORTED), ({8: 1 << 28, 11: 1 << 28}, UNSUPPORTED),
        ({9: 1 << 25}, UNSUPPORTED)])
    _each(L.arc_gemm_experts_bf16, [A, 64, A, 64, A, 16, 4, 8, 64, 64, A, 64, None], [
        ({i: None}, INVALID) for i in (0, 2, 4, 10)] + [({i: ODD}, ALIGN) for i in (0, 2, 4, 10)] + [
        ({9: 60}, INVALID), ({8: 60}, INVALID), ({1: 56}, INVALID), ({1: 68}, INVALID), ({3: 56}, INVALID),
        ({3: 68}, INVALID), ({11: 56}, INVALID), ({11: 68}, INVALID), ({6: 0}, INVALID), ({7: 600}, UNSUPPORTED)])


def test_binding_refuses_cpu_tensors_and_wrong_plans():
    buf = torch.zeros(2 * 64 + 3 * 64, dtype=torch.int32)
    plan = arc.ExpertPlan(buf, 16, 4, 8)
    assert plan.offsets.shape == (9,) and plan.blocks.shape == (9,)
    assert plan.row_of_slot.shape == plan.slot_of_row.shape == plan.sf_row.shape == (64,)
    for bad in (buf[:-1], buf.long(), torch.zeros(640, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="ExpertPlan"):
            arc.ExpertPlan(bad, 16, 4, 8)
    x, rows = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    w = torch.zeros(16, 4)
    calls = [lambda: arc.expert_plan(torch.zeros(16, 4, dtype=torch.int32), 8), lambda: arc.dispatch_experts(x, plan),
             lambda: arc.dispatch_experts_grad(rows, plan), lambda: arc.combine_experts(rows, w, plan),
             lambda: arc.combine_experts_grad(x, rows, w, plan), lambda: arc.quantize_act_experts_mxfp4(x, plan),
             lambda: arc.quantize_swiglu_experts_mxfp4(rows, plan),
             lambda: arc.pack_weight_experts_mxfp4(torch.zeros(8, 64, 64, dtype=torch.bfloat16)),
             lambda: arc.gemm_experts_bf16(rows, torch.zeros(8, 64, 64, dtype=torch.bfloat16), plan),
             lambda: arc.gemm_experts_mxfp4(arc.ExpertMXFP4(torch.zeros(1 << 16, dtype=torch.uint8), 64, 64),
                                            arc.ExpertWeightMXFP4(buf, buf, 8, 64, 64), plan)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    with pytest.raises(ValueError, match="int32 or int64"):
        arc.expert_plan(torch.zeros(16, 4), 8)
    with pytest.raises(ValueError, match="gate"):
        arc.quantize_swiglu_experts_mxfp4(torch.zeros(64, 63, dtype=torch.bfloat16), plan)
    with pytest.raises(ValueError, match="experts, N, K"):
        arc.gemm_experts_bf16(rows, rows, plan)
    with pytest.raises(ValueError, match="depths"):
        arc.gemm_experts_mxfp4(arc.ExpertMXFP4(buf, 64, 64), arc.ExpertWeightMXFP4(buf, buf, 8, 64, 128), plan)
