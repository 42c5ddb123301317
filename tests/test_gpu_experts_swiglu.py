"""The SwiGLU quantizer's accuracy as it is stated, and the down product behind it.

The kernel forms silu(g) u in fp32 as g r u with r = 1 / (1 + 2^(-g log2 e)). Its relative error before the one
rounding to bf16, in units of 2^-24:
  the exponent's rounding, and log2 e's own (2^-26.1 of it): max(-g, 0) (1 + 0.23); for g > 0 the factor
    e^-g / (1 + e^-g) makes of g (1 + 0.23) at most 0.35, and of the 2^x below at most half
  2^x, two ulp: 4
  1 + 2^x: 1
  the reciprocal, one ulp: 2
  two products: 2
together (1.25 max(-g, 0) + 9) 2^-24. Where silu(g) u in 64 bits lies farther than that from a rounding
border, its bf16 value is the kernel's, and codes and scale bytes are the oracle's bit for bit.
"""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc
import oracle as O
import workloads as W
from tests._experts import bf16, f64, make_ids, plan_of
from tests._helpers import to_bits, to_dev
from tests.test_gpu_experts import _check_coded, _coded_out, _values

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a bf16 step, relative


def _product(gate_bits, up_bits):
    g, u = (O.bf16_bits_to_f32(b).astype(np.float64) for b in (gate_bits, up_bits))
    with np.errstate(over="ignore"):
        return g, g / (1 + np.exp(-g)) * u


def _act(gate_bits, up_bits):
    """bf16 bits of silu(gate) up from 64 bits, and whether the kernel's may differ from them."""
    g, v = _product(gate_bits, up_bits)
    bits = to_bits(torch.from_numpy(v).to(torch.float32).to(torch.bfloat16))
    near = np.abs(O.bf16_bits_to_f32(bits).astype(np.float64))
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-300))) - 7)
    off = np.abs(np.abs(np.abs(v) - near) - step / 2)
    # (a 32-bit copy of v that lies on a border itself can round the other way: 2^-24 more)
    return bits, (off <= (1.25 * np.maximum(-g, 0) + 10) * 2.0 ** -24 * np.abs(v)) | (np.abs(g) > 87)


def _clear_of_borders(gate_bits, up_bits):
    return np.where(_act(gate_bits, up_bits)[1], 0, gate_bits).astype(np.uint16)


def test_every_gate_from_87_down_to_2_60th():
    # all 17 thousand bf16 gates between, 32 neighbours a block, with all channels appended: the
    # residuals' codes show more of act than the primary ones
    bits = np.arange(0x2180, 0x42AE + 1)  # 2^-60 .. 87
    gates = np.concatenate([bits, bits | 0x8000]).astype(np.uint16)
    K = 2048
    gates = np.concatenate([gates, np.zeros(-gates.size % K, np.uint16)]).reshape(-1, K)
    S = len(gates)
    rng = np.random.default_rng(11)
    ups = to_bits(bf16(rng.uniform(0.25, 4.0, gates.shape) * rng.choice([-1.0, 1.0], gates.shape)))
    act, close = _act(gates, ups)
    # few are set aside. A border is at least 2^-8 of the value away from the next: 2 x 119 half-steps of fp32
    # of 2^16. And silu(g) u is g u / 2 to 32 bits for gates below 2^-24, a product of two significands of 8
    # bits: of its 16 (or 15) bits the lower 8 (or 7) are those of a border itself in 1 case of 128, at most.
    assert close.mean() < 2 * 119 / 2 ** 16 + 1 / 128
    gates = np.where(close, 0, gates).astype(np.uint16)
    act = _act(gates, ups)[0]
    ids = make_ids(12, S, 1, 3)
    p, plan = plan_of(ids, 3), arc.expert_plan(torch.from_numpy(ids).cuda(), 3)
    idx = rng.permutation(K).astype(np.int32)
    out = _coded_out(plan, 2 * K)
    gu = to_dev(np.concatenate([gates, ups], 1))
    arc.quantize_swiglu_experts_mxfp4(gu, plan, torch.from_numpy(idx).cuda(), out=out)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    _check_coded(out, p, *O.quantize_act_mxfp4(act, idx), 2 * K)


@pytest.mark.parametrize("T,k,E,F,how", [(77, 4, 12, 320, "drop"), (3, 2, 5, 64, "skewed"), (300, 2, 3, 1056, "repeat"),
                                         (2500, 2, 4, 256, "drop")])
def test_coded_rows_read_back_through_a_unit_matrix(T, k, E, F, how):
    # weights of ones on the diagonal: the product's row is the coded row's values, exactly
    S, ids = T * k, make_ids(F, T, k, E, how)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    ub = W.matrix_bf16(13, 2, S, F, 1.0)
    gb = _clear_of_borders(W.matrix_bf16(13, 1, S, F, 3.0), ub)
    q = arc.quantize_swiglu_experts_mxfp4(to_dev(np.concatenate([gb, ub], 1)), plan)
    w = torch.eye(F, dtype=torch.bfloat16, device="cuda").repeat(E, 1, 1)
    y = arc.gemm_experts_mxfp4(q, arc.pack_weight_experts_mxfp4(w), plan)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    act = _act(gb, ub)[0][: p["used"]]
    np.testing.assert_array_equal(f64(y)[: p["used"]],
                                  _values(*O.quantize_act_mxfp4(act, np.zeros(0, np.int32)))[:, :F])


@pytest.mark.parametrize("T,k,E,F,N,r,how", [(77, 4, 12, 320, 264, 32, "drop"), (1, 8, 64, 512, 520, 64, "skewed"),
                                             (400, 2, 3, 1056, 200, 0, "skewed"), (3000, 2, 4, 256, 264, 32, "drop")])
def test_down_product_behind_the_quantizer(T, k, E, F, N, r, how):
    # every result within one rounding and the sum's error of the coded rows' product in 64 bits
    S, ids = T * k, make_ids(F + N, T, k, E, how)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    ub = W.matrix_bf16(14, 2, S, F, 1.0, col_mult=W.outlier_multipliers(14, 0, F, max(1, F // 64), 10.0, 60.0))
    gb = _clear_of_borders(W.matrix_bf16(14, 1, S, F, 2.0), ub)
    act = _act(gb, ub)[0][: p["used"]]
    idx = O.calibrate(act, r) if r else np.zeros(0, np.int32)
    di = torch.from_numpy(idx).cuda() if r else None
    wb = W.matrix_bf16(14, 3, E * N, F, 0.05)
    q = arc.quantize_swiglu_experts_mxfp4(to_dev(np.concatenate([gb, ub], 1)), plan, di)
    y = f64(arc.gemm_experts_mxfp4(q, arc.pack_weight_experts_mxfp4(to_dev(wb).view(E, N, F), di), plan))
    assert arc.last_device_status() == 0
    a = _values(*O.quantize_act_mxfp4(act, idx))
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if hi > lo:
            w = _values(*O.pack_weight_mxfp4(wb[e * N:(e + 1) * N], idx))
            ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
            assert (np.abs(y[lo:hi] - ref) <= HALF * np.abs(ref) + (F + r) * 2.0 ** -23 * mag).all(), e


@pytest.mark.parametrize("T,k,E,d,F,how", [(77, 4, 12, 512, 320, "drop"), (700, 2, 3, 1024, 512, "skewed")])
def test_layers_rows_away_from_borders(T, k, E, d, F, how):
    # gate|up product, SwiGLU quantizer, down product: rows of which no act lies near a rounding border are
    # the formula's; with up to 85 half-steps of fp32 either side of a border (gates from -60 on) a row of 512
    # has one with a probability of at most 512 * 2 * 85 / 2^16, on average (gates near -3) a tenth of that
    ids = make_ids(15, T, k, E, how)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    used = p["used"]
    x = to_dev(W.matrix_bf16(15, 1, T, d, 1.0))
    wgu = to_dev(W.matrix_bf16(15, 2, E * 2 * F, d, 0.1)).view(E, 2 * F, d)
    wdb = W.matrix_bf16(15, 3, E * d, F, 0.05)
    gu = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan), arc.pack_weight_experts_mxfp4(wgu), plan)
    q = arc.quantize_swiglu_experts_mxfp4(gu, plan)
    y = f64(arc.gemm_experts_mxfp4(q, arc.pack_weight_experts_mxfp4(to_dev(wdb).view(E, d, F)), plan))
    assert arc.last_device_status() == 0
    gub = to_bits(gu)[:used]
    act, close = _act(gub[:, :F], gub[:, F:])
    clear = ~close.any(1)
    assert clear.mean() > 0.5
    none = np.zeros(0, np.int32)
    a = _values(*O.quantize_act_mxfp4(act, none))
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if hi > lo:
            w = _values(*O.pack_weight_mxfp4(wdb[e * d:(e + 1) * d], none))
            ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
            fine = np.abs(y[lo:hi] - ref) <= HALF * np.abs(ref) + F * 2.0 ** -23 * mag
            assert fine[clear[lo:hi]].all(), e


@pytest.mark.parametrize("T,k,E,F,r,how", [(77, 4, 12, 320, 32, "drop"), (1, 2, 8, 128, 0, "skewed"),
                                           (2500, 2, 5, 256, 64, "drop"), (40, 3, 512, 64, 32, "skewed")])
def test_act_of_the_bf16_form_coded_by_a_plan_of_the_sorted_rows(T, k, E, F, r, how):
    # sorted rows sorted again, one choice each, stay where they are: quantize_act_experts_mxfp4 then codes
    # arc_silu_mul_bf16's act into the places that the layer's own plan names
    S, ids = T * k, make_ids(F + r, T, k, E, how)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    gu = bf16(np.random.default_rng(F).standard_normal((S, 2 * F)))
    act = arc.silu_mul_bf16(gu)
    idx = torch.randperm(F, generator=torch.Generator().manual_seed(F))[:r].int().cuda() if r else None
    at = plan.slot_of_row.long()
    again = arc.expert_plan(torch.where(at >= 0, torch.from_numpy(ids).cuda().reshape(-1)[at], -1)[:, None], E)
    for name in ("offsets", "blocks", "slot_of_row", "sf_row"):
        want = getattr(plan, name)
        if name == "slot_of_row":
            want = torch.where(at >= 0, torch.arange(S, device="cuda"), -1).int()
        assert torch.equal(getattr(again, name), want), name
    out = _coded_out(again, F + r)
    arc.quantize_act_experts_mxfp4(act, again, idx, out=out)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    ab = to_bits(act)[: p["used"]]
    _check_coded(out, p, *O.quantize_act_mxfp4(ab, idx.cpu().numpy() if r else np.zeros(0, np.int32)), F + r)
    # and the product takes the rows with the layer's own plan
    w = arc.pack_weight_experts_mxfp4(to_dev(W.matrix_bf16(16, 3, E * 64, F, 0.1)).view(E, 64, F), idx)
    used = p["used"]
    assert torch.equal(arc.gemm_experts_mxfp4(out, w, plan)[:used], arc.gemm_experts_mxfp4(out, w, again)[:used])
