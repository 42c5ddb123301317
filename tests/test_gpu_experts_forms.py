"""Kernel forms of the expert operators that only many narrow rows or very wide rows reach: tokens and
gradients moved by groups of 1 to 16 lanes with four vectors each, gradients whose rows few lanes take in
several rounds, and quantizers whose rows take several rounds of a CTA's warps.

Tolerances as in test_gpu_experts.py: one rounding to bf16, n 2^-24 of the sum of magnitudes for a sum of n
fp32 terms; copies, codes and scale bytes exact.
"""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc
import oracle as O
import workloads as W
from tests._experts import make_ids, plan_of
from tests._helpers import to_bits, to_dev
from tests.test_gpu_experts import _check_coded, _coded_out
from tests.test_gpu_experts_swiglu import _act, _clear_of_borders

pytestmark = pytest.mark.gpu

HALF, F32 = 2.0 ** -8, 2.0 ** -24

# 148 SMs x 16 warps of groups (combine, gradients) and x 32 (dispatch) from: groups of 1, 2, 4, 8 and 16
# lanes; choices that are more than a group's lanes, odd ones, slots without an expert, a partly filled last warp
MANY = [(151601, 2, 5, 8, "drop"), (75801, 3, 6, 40, "drop"), (37901, 8, 32, 128, "repeat"), (18950, 9, 12, 72, "drop"),
        (37999, 5, 7, 104, "drop"), (18977, 5, 7, 136, "drop"), (20011, 3, 9, 264, "drop"),
        (20003, 5, 7, 512, "skewed"), (9601, 1, 3, 488, "one")]


@pytest.mark.parametrize("tokens,k,experts,d,how", MANY)
@pytest.mark.parametrize("pad", [0, 24])
def test_many_narrow_rows(tokens, k, experts, d, how, pad):
    S = tokens * k
    ids = make_ids(tokens + d, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), arc.expert_plan(torch.from_numpy(ids).cuda(), experts)
    used = p["used"]
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    slot, row = (torch.from_numpy(p[n]).cuda() for n in ("slot_of_row", "row_of_slot"))
    has = (row >= 0)[:, None]

    def mat(rows, fill=None):
        m = torch.randn(rows, d + pad, generator=gen, device="cuda").bfloat16()
        return (m if fill is None else m.fill_(fill))[:, :d]

    def by_slot(rows):
        return torch.where(has, rows[row.clamp(min=0)].double(), 0.0).view(tokens, k, d)

    x, out = mat(tokens), mat(S, float("nan"))
    arc.dispatch_experts(x, plan, out=out)
    assert torch.equal(out[:used], x[slot[:used] // k]) and torch.isnan(out[used:]).all()

    rows, add = mat(S), mat(tokens)
    rows[used:] = float("nan")
    w = torch.randn(tokens, k + 1, generator=gen, device="cuda")[:, :k]
    w[~has.view(tokens, k)] = float("nan")
    terms, wt = by_slot(rows), torch.where(has.view(tokens, k), w.double(), 0.0)[:, :, None]

    def check(y, ref, mag, what):
        assert ((y.double() - ref).abs() <= HALF * ref.abs() + (k + 2) * 2 * F32 * mag).all(), what

    y = mat(tokens, float("nan"))
    check(arc.dispatch_experts_grad(rows, plan, out=y), terms.sum(1), terms.abs().sum(1), "dispatch gradient")
    terms = terms * wt
    ref, mag = terms.sum(1), terms.abs().sum(1)
    y = mat(tokens, float("nan"))
    check(arc.combine_experts(rows, w, plan, out=y), ref, mag, "combine")
    y = mat(tokens, float("nan"))
    arc.combine_experts(rows, w, plan, add=add, out=y)
    check(y, ref + add.double(), mag + add.double().abs(), "combine + add")
    y.copy_(add)
    want = arc.combine_experts(rows, w, plan, add=add)
    assert torch.equal(arc.combine_experts(rows, w, plan, add=y, out=y), want)
    del terms

    dy, d_rows, d_w = mat(tokens), mat(S, float("nan")), torch.full((tokens, k + 1), -7.0, device="cuda")
    arc.combine_experts_grad(dy, rows, w, plan, d_rows=d_rows, d_weights=d_w[:, :k])
    ref = dy[slot[:used] // k].double() * w.reshape(-1)[slot[:used]].double()[:, None]
    assert ((d_rows[:used].double() - ref).abs() <= (HALF + 2 * F32) * ref.abs()).all()
    assert torch.isnan(d_rows[used:]).all() and (d_w[:, k] == -7.0).all()
    prod = dy.double()[:, None, :] * by_slot(rows)
    tol = (max(24, 8 * -(-d // 1024)) + 7) * F32 * prod.abs().sum(2)
    assert ((d_w[:, :k].double() - prod.sum(2)).abs() <= tol).all()
    assert (d_w[:, :k][~has.view(tokens, k)] == 0).all()
    arc.combine_experts_grad(dy, rows, w, plan, d_rows=rows)
    assert torch.equal(rows[:used], d_rows[:used])
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0


# blocks of 32 channels over warps that take 32 each: 257 blocks in two rounds of five warps (the last
# segment one block), 448 in two of seven, 529 and 513 in three of six, 1025 in five of seven
WIDE = [(5, 2, 3, 8224, 0, "drop"), (5, 2, 3, 8224, 64, "drop"), (3, 2, 8, 14336, 128, "skewed"),
        (4, 3, 5, 16928, 96, "drop"), (1, 8, 64, 16416, 2048, "skewed"), (2, 40, 16, 32800, 32, "repeat")]


def _late_channels(rng, K, r):
    """r outlier channels, half of them in the last segments; the last channel and the first among them."""
    late = K - 1 - rng.choice(min(K // 2, 4096), r // 2, replace=False)
    early = rng.choice(K // 2, r - r // 2, replace=False)
    idx = np.concatenate([late, early]).astype(np.int32)
    idx[0], idx[-1] = K - 1, 0
    return rng.permutation(idx).astype(np.int32)


@pytest.mark.parametrize("tokens,k,experts,K,r,how", WIDE)
@pytest.mark.parametrize("source", ["tokens", "swiglu"])
def test_wide_rows_are_coded_in_rounds(tokens, k, experts, K, r, how, source):
    ids = make_ids(K + r, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), arc.expert_plan(torch.from_numpy(ids).cuda(), experts)
    idx = _late_channels(np.random.default_rng(K + r), K, r) if r else np.zeros(0, np.int32)
    di = torch.from_numpy(idx).cuda() if r else None
    mult = np.ones(K, np.float32)
    mult[idx] = 40.0
    n = tokens if source == "tokens" else tokens * k
    xb = W.matrix_bf16(21, 1, n, K, 1.0, col_mult=mult)
    out = _coded_out(plan, K + r)
    if source == "tokens":
        arc.quantize_act_experts_mxfp4(to_dev(xb), plan, di, out=out)
        c, s = O.quantize_act_mxfp4(xb, idx)
        token = p["slot_of_row"][: p["used"]] // k
        c, s = c[token], s[token]
    else:
        gb = _clear_of_borders(W.matrix_bf16(21, 2, n, K, 2.0), xb)
        arc.quantize_swiglu_experts_mxfp4(to_dev(np.concatenate([gb, xb], 1)), plan, di, out=out)
        c, s = O.quantize_act_mxfp4(_act(gb, xb)[0][: p["used"]], idx)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    _check_coded(out, p, c, s, K + r)


def test_wide_rows_repeat_bit_for_bit_and_through_the_product():
    # the coded rows of two rounds in a product, against 64 bits
    T, k, E, K, N, r = 40, 2, 3, 8224, 136, 96
    ids = make_ids(22, T, k, E)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    idx = _late_channels(np.random.default_rng(22), K, r)
    di = torch.from_numpy(idx).cuda()
    xb, wb = W.matrix_bf16(22, 1, T, K, 1.0), W.matrix_bf16(22, 2, E * N, K, 0.02)
    w = arc.pack_weight_experts_mxfp4(to_dev(wb).view(E, N, K), di)
    ys = [arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(to_dev(xb), plan, di), w, plan) for _ in range(2)]
    assert torch.equal(*ys) and arc.last_device_status() == 0
    ca, sa = O.quantize_act_mxfp4(xb, idx)
    y = O.bf16_bits_to_f32(to_bits(ys[0])).astype(np.float64)
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        cw, sw = O.pack_weight_mxfp4(wb[e * N:(e + 1) * N], idx)
        token = p["slot_of_row"][lo:hi] // k
        ref = O.gemm_mxfp4_f64(ca[token], sa[token], cw, sw)
        mag = O.gemm_mxfp4_f64(ca[token] & 0x77, sa[token], cw & 0x77, sw)  # the codes without their signs
        assert (np.abs(y[lo:hi] - ref) <= HALF * np.abs(ref) + (K + r) * 2 * F32 * mag).all(), e
