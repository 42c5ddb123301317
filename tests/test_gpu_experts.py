"""Mixture-of-experts operators on the GPU: the plan, tokens into sorted order and back with their
gradients, the MXFP4 quantizers that write sorted rows, the experts' products in MXFP4 and BF16, and
a whole layer of them.

Tolerances. A bf16 result is one rounding, at most 2^-8 of its value; sums of n fp32 terms add at
most n 2^-24 of the sum of magnitudes (n 2^-23 for tensor-core sums, which may cut instead of round).
Plans, copies, codes and scale bytes are exact.
"""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc
import oracle as O
import workloads as W
from tests._experts import bf16, f64, make_ids, plan_of, sf_canonical, sf_places
from tests._helpers import to_bits, to_dev

pytestmark = pytest.mark.gpu

BF16_HALF_STEP, F32_HALF_STEP = 2.0 ** -8, 2.0 ** -24


def _plan(ids, experts, dtype=torch.int32):
    return arc.expert_plan(torch.from_numpy(ids).cuda().to(dtype), experts)


def _status_ok():
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0


# ------------------------------------------------------------------------------------------ plan


@pytest.mark.parametrize("tokens,k,experts,how", [
    (1, 1, 1, "skewed"), (1, 8, 128, "skewed"), (3, 2, 5, "drop"), (130, 3, 7, "drop"), (257, 4, 256, "skewed"),
    (1000, 8, 512, "skewed"), (513, 8, 16, "one"), (4099, 6, 61, "drop"), (16384, 8, 64, "skewed"),
    (2, 1024, 33, "repeat"), (5000, 1, 3, "repeat"), (4096, 1, 2, "repeat"), (40001, 8, 512, "drop")])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_plan_is_the_stable_sort(tokens, k, experts, how, dtype):
    ids = make_ids(tokens + experts, tokens, k, experts, how)
    want = plan_of(ids, experts)
    p = _plan(ids, experts, dtype)
    for name in ("offsets", "blocks", "row_of_slot", "slot_of_row", "sf_row"):
        np.testing.assert_array_equal(getattr(p, name).cpu().numpy(), want[name], err_msg=name)


def test_plan_of_strided_ids_and_of_ids_beyond_int32():
    wide = torch.full((70, 9), 5, dtype=torch.int64, device="cuda")
    wide[:, :4] = torch.from_numpy(make_ids(3, 70, 4, 10)).cuda()
    wide[3, 1] = 2 ** 32 + 2  # its low half is an expert's number
    wide[5, 0] = -2 ** 40
    ids = wide[:, :4]
    p = arc.expert_plan(ids, 10)
    ref = ids.cpu().numpy()
    want = plan_of(np.where((ref < 0) | (ref > 9), -1, ref), 10)
    np.testing.assert_array_equal(p.row_of_slot.cpu().numpy(), want["row_of_slot"])


def test_plan_without_any_row():
    p = arc.expert_plan(torch.full((9, 2), -1, dtype=torch.int32, device="cuda"), 4)
    assert p.offsets.tolist() == [0] * 5 and p.blocks.tolist() == [0] * 5
    for v in (p.row_of_slot, p.slot_of_row, p.sf_row):
        assert v.tolist() == [-1] * 18


# ------------------------------------------------------------------------------------------ rows

MOVES = [(1, 8, 128, 4096, "skewed"), (5, 2, 4, 8, "drop"), (67, 3, 9, 264, "drop"), (300, 8, 32, 1032, "repeat"),
         (33, 40, 64, 72, "skewed"), (1023, 1, 5, 2048, "one"), (129, 6, 61, 4104, "drop"), (9, 3, 512, 8, "drop"),
         (5000, 2, 8, 1032, "drop")]


def _inputs(tokens, k, experts, d, how, pad=0):
    ids = make_ids(tokens * 7 + d, tokens, k, experts, how)
    rng = np.random.default_rng(d)
    p = plan_of(ids, experts)

    def mat(rows):
        return bf16(rng.standard_normal((rows, d + pad)))[:, :d]

    return ids, p, mat, rng


def _poisoned(rows, d, pad=0):
    return torch.full((rows, d + pad), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :d]


@pytest.mark.parametrize("tokens,k,experts,d,how", MOVES)
@pytest.mark.parametrize("pad", [0, 24])
def test_dispatch_copies_and_leaves_the_rest(tokens, k, experts, d, how, pad):
    ids, p, mat, _ = _inputs(tokens, k, experts, d, how, pad)
    x = mat(tokens)
    out = _poisoned(tokens * k, d, pad)
    arc.dispatch_experts(x, _plan(ids, experts), out=out)
    got = to_bits(out.contiguous())
    used = p["used"]
    np.testing.assert_array_equal(got[:used], to_bits(x.contiguous())[p["slot_of_row"][:used] // k])
    assert torch.isnan(out[used:]).all()


def _by_slot(rows, p):
    """Sorted rows [S, d] by slot, zero where the slot has none."""
    out = np.zeros(rows.shape)
    has = p["row_of_slot"] >= 0
    out[has] = rows[p["row_of_slot"][has]]
    return out


@pytest.mark.parametrize("tokens,k,experts,d,how", MOVES)
@pytest.mark.parametrize("pad", [0, 24])
def test_dispatch_gradient_and_combine(tokens, k, experts, d, how, pad):
    ids, p, mat, rng = _inputs(tokens, k, experts, d, how, pad)
    rows, add = mat(tokens * k), mat(tokens)
    rows[p["used"]:] = float("nan")  # behind the last row: not read
    weights = torch.rand(tokens, k + 3, generator=torch.Generator().manual_seed(d)).cuda()[:, :k]
    weights[torch.from_numpy(p["row_of_slot"].reshape(tokens, k) < 0).cuda()] = float("nan")  # not used
    plan = _plan(ids, experts)
    by_slot = _by_slot(f64(rows), p).reshape(tokens, k, d)
    w = np.where(p["row_of_slot"].reshape(tokens, k) >= 0, f64(weights), 0.0)[:, :, None]
    for name, terms, base in (("dispatch gradient", by_slot, None), ("combine", by_slot * w, None),
                              ("combine + add", by_slot * w, add)):
        out = _poisoned(tokens, d, pad)
        if name == "dispatch gradient":
            arc.dispatch_experts_grad(rows, plan, out=out)
        else:
            arc.combine_experts(rows, weights, plan, add=base, out=out)
        ref, mag = terms.sum(1), np.abs(terms).sum(1)
        if base is not None:
            ref, mag = ref + f64(base), mag + np.abs(f64(base))
        tol = BF16_HALF_STEP * np.abs(ref) + (k + 2) * F32_HALF_STEP * 2 * mag
        assert (np.abs(f64(out) - ref) <= tol).all(), name


def test_combine_into_its_addend():
    ids, p, mat, _ = _inputs(50, 3, 6, 520, "drop")
    rows, y = mat(150), mat(50)
    plan = _plan(ids, 6)
    w = torch.rand(50, 3, device="cuda")
    want = arc.combine_experts(rows, w, plan, add=y)
    arc.combine_experts(rows, w, plan, add=y, out=y)
    assert torch.equal(want, y)


@pytest.mark.parametrize("tokens,k,experts,d,how", MOVES)
@pytest.mark.parametrize("pad", [0, 24])
def test_combine_gradients(tokens, k, experts, d, how, pad):
    ids, p, mat, _ = _inputs(tokens, k, experts, d, how, pad)
    rows, dy = mat(tokens * k), mat(tokens)
    rows[p["used"]:] = float("nan")
    weights = torch.rand(tokens, k, generator=torch.Generator().manual_seed(d)).cuda()
    plan = _plan(ids, experts)
    d_rows, d_w = _poisoned(tokens * k, d, pad), torch.full((tokens, k + 1), -7.0, device="cuda")
    arc.combine_experts_grad(dy, rows, weights, plan, d_rows=d_rows, d_weights=d_w[:, :k])
    used, slot = p["used"], p["slot_of_row"]
    ref = f64(dy)[slot[:used] // k] * f64(weights).reshape(-1)[slot[:used]][:, None]
    assert (np.abs(f64(d_rows)[:used] - ref) <= (BF16_HALF_STEP + 2 * F32_HALF_STEP) * np.abs(ref)).all()
    assert torch.isnan(d_rows[used:]).all() and (d_w[:, k] == -7.0).all()
    prod = np.repeat(f64(dy), k, axis=0) * _by_slot(f64(rows), p)
    # a lane adds up at most three rounds of four vectors of 8 values, or d / 32 of them and a vector's
    # rest where 32 lanes share the row; five shuffles join the lanes
    tol = (max(d / 32 + 8, 96) + 5) * F32_HALF_STEP * np.abs(prod).sum(1)
    assert (np.abs(f64(d_w[:, :k]).reshape(-1) - prod.sum(1)) <= tol).all()
    # the rows' gradient in the rows' own place
    want = d_rows.clone()
    arc.combine_experts_grad(dy, rows, weights, plan, d_rows=rows)
    assert torch.equal(want[:used], rows[:used])


def test_gradients_against_differences():
    # d/ds of <g, combine(rows + s e)> and <g, combine with weights + s e> along random directions:
    # the combine is linear in each, so a difference over s = 1 is the derivative. All values are
    # small whole numbers and halves, exact in bf16 and in every sum.
    T, k, E, d = 40, 3, 7, 64
    ids = make_ids(5, T, k, E, "drop")
    plan = _plan(ids, E)
    rng = np.random.default_rng(1)

    def whole(*shape):
        return torch.from_numpy(rng.integers(-2, 3, shape).astype(np.float32)).cuda()

    rows, e_rows, g = (whole(n, d).bfloat16() for n in (T * k, T * k, T))
    w, e_w = whole(T, k), whole(T, k)
    d_rows, d_w = arc.combine_experts_grad(g, rows, w, plan)
    y = arc.combine_experts(rows, w, plan).double()
    used = plan_of(ids, E)["used"]
    dy = (arc.combine_experts(rows + e_rows, w, plan).double() - y) * g.double()
    assert dy.sum() == (d_rows.double() * e_rows.double())[:used].sum()
    dy = (arc.combine_experts(rows, w + e_w, plan).double() - y) * g.double()
    assert dy.sum() == (d_w.double() * e_w.double()).sum()
    # dispatch: <g_rows, dispatch(x)> is linear in x, its gradient the summed rows of g_rows
    x, g_rows = whole(T, d).bfloat16(), whole(T * k, d).bfloat16()
    sent = arc.dispatch_experts(x, plan)[:used].double()
    d_x = arc.dispatch_experts_grad(g_rows, plan).double()
    assert (sent * g_rows[:used].double()).sum() == (d_x * x.double()).sum()


# ----------------------------------------------------------------------------------- quantization


def _x_bits(seed, rows, K):
    mult = W.outlier_multipliers(seed, 0, K, max(1, K // 64), 10.0, 80.0)
    return W.matrix_bf16(seed, 1, rows, K, 1.0, col_mult=mult)


def _check_coded(q, p, codes_ref, sc_ref, k_aug):
    """codes_ref, sc_ref: by sorted row in use."""
    used, kp = p["used"], O.kpad(k_aug)
    codes = q.codes.view(-1, kp // 2).cpu().numpy()
    np.testing.assert_array_equal(codes[:used], codes_ref)
    assert (codes[used:] == 0xA5).all()
    sf, ncols = q.sf.cpu().numpy(), (kp + 255) // 256 * 8
    places = sf_places(len(p["slot_of_row"]), len(p["offsets"]) - 1)
    assert sf.size == places * ncols
    got = sf_canonical(sf, p["sf_row"][:used], ncols, places)
    np.testing.assert_array_equal(got[:, : kp // 32], sc_ref)
    # columns behind K_pad and places without a row are left as they were
    assert (got[:, kp // 32:] == 0xA5).all()
    rest = np.setdiff1d(np.arange(places), p["sf_row"][:used])
    assert (sf_canonical(sf, rest, ncols, places) == 0xA5).all()


def _coded_out(plan, k_aug):
    at = (plan.slots * O.kpad(k_aug) // 2 + 255) // 256 * 256
    n = at + arc.lib().arc_expert_sf_bytes(plan.tokens, plan.k, plan.experts, k_aug)
    out = arc.ExpertMXFP4(torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"), plan.slots, k_aug)
    assert out.sf_at == at
    return out


QUANTS = [(1, 8, 16, 64, 0, "skewed"), (1, 2, 4, 4096, 64, "skewed"), (37, 3, 5, 96, 32, "drop"),
          (130, 2, 8, 1056, 128, "repeat"), (300, 1, 3, 512, 512, "one"), (9, 40, 64, 288, 0, "skewed"),
          (200, 4, 64, 2048, 96, "drop"), (5, 2, 3, 32, 32, "drop"),
          # many narrow rows (lane groups of 8, 4, 1, 16 and 2)
          (5003, 3, 8, 256, 0, "drop"), (4801, 1, 5, 96, 0, "skewed"), (4737, 5, 4, 32, 0, "repeat"),
          (4750, 1, 2, 480, 0, "drop"), (4799, 2, 512, 64, 0, "skewed"),
          # with appended blocks, and of a whole warp
          (4751, 2, 8, 512, 96, "drop"), (4803, 1, 4, 64, 64, "skewed"), (4740, 3, 5, 736, 160, "repeat"),
          (4738, 40, 64, 32, 32, "skewed"), (4757, 1, 3, 1024, 0, "drop")]


@pytest.mark.parametrize("tokens,k,experts,K,r,how", QUANTS)
def test_token_quantizer_matches_the_oracle(tokens, k, experts, K, r, how):
    ids = make_ids(K + r, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), _plan(ids, experts)
    xb = _x_bits(61, tokens, K)
    idx = O.calibrate(xb, r) if r else np.zeros(0, np.int32)
    big = torch.full((tokens, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, :K] = to_dev(xb)
    out = _coded_out(plan, K + r)
    arc.quantize_act_experts_mxfp4(big[:, :K], plan, torch.from_numpy(idx).cuda() if r else None, out=out)
    _status_ok()
    c, s = O.quantize_act_mxfp4(xb, idx)
    token = p["slot_of_row"][: p["used"]] // k
    _check_coded(out, p, c[token], s[token], K + r)


def _bf16_bits(v):
    """bf16 bits of 64-bit values, and how far (relative) each lies from a rounding border."""
    bits = to_bits(torch.from_numpy(v).to(torch.float32).to(torch.bfloat16))  # right away from a border
    near = O.bf16_bits_to_f32(bits).astype(np.float64)
    ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(near), 1e-300))) - 7)
    off = np.abs(np.abs(np.abs(v) - np.abs(near)) - ulp / 2)
    return bits, off / np.maximum(np.abs(v), 1e-300)


@pytest.mark.parametrize("tokens,k,experts,F,r,how", QUANTS)
def test_swiglu_quantizer_matches_the_formula(tokens, k, experts, F, r, how):
    # silu(gate) * up in 64 bits, rounded to bf16, coded by the oracle. |gate| <= 60; there the kernel's
    # fp32 product is off by at most 2^-18.5 (half an ulp of 60 log2 e, times ln 2) + 60 2^-26.2 (log2 e
    # itself) + 4 2^-23 (2^x, reciprocal, products) < 2^-17.9: gates with a product within 2^-17 of a
    # rounding border (one value in 250) are set to zero, so that the rounding is the formula's.
    ids = make_ids(F + r + 1, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), _plan(ids, experts)
    S = tokens * k
    gb = np.where(np.abs(O.bf16_bits_to_f32(_x_bits(62, S, F))) <= 60, _x_bits(62, S, F), 0).astype(np.uint16)
    ub = _x_bits(63, S, F)

    def product(gate):
        g, u = O.bf16_bits_to_f32(gate).astype(np.float64), O.bf16_bits_to_f32(ub).astype(np.float64)
        return g / (1 + np.exp(-g)) * u

    gb = np.where(_bf16_bits(product(gb))[1] < 2.0 ** -17, 0, gb).astype(np.uint16)
    ab = _bf16_bits(product(gb))[0][: p["used"]]
    gu = torch.full((S, 2 * F + 8), float("nan"), dtype=torch.bfloat16, device="cuda")[:, : 2 * F]
    gu[: p["used"]] = to_dev(np.concatenate([gb, ub], axis=1))[: p["used"]]
    idx = O.calibrate(ab, r) if r else np.zeros(0, np.int32)
    out = _coded_out(plan, F + r)
    arc.quantize_swiglu_experts_mxfp4(gu, plan, torch.from_numpy(idx).cuda() if r else None, out=out)
    _status_ok()
    c, s = O.quantize_act_mxfp4(ab, idx)
    _check_coded(out, p, c, s, F + r)


def test_swiglu_quantizer_at_the_ends_of_the_range():
    # gates of the largest magnitudes and zeros of both signs, each a block of its own, times one:
    # far above zero the result is the gate, far below it is a zero with the gate's sign
    gates = [-3e38, -1000.0, -200.0, -120.0, -89.0, -88.0, -0.0, 0.0, 88.0, 89.0, 120.0, 200.0, 1000.0, 3e38]
    F = 32 * len(gates)
    gu = torch.ones(1, 2 * F, dtype=torch.bfloat16, device="cuda")
    gu[0, :F] = torch.tensor(gates).repeat_interleave(32)
    plan = arc.expert_plan(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    q = arc.quantize_swiglu_experts_mxfp4(gu, plan)
    _status_ok()
    g = gu[0, :F].float().cpu()
    act = torch.where(g > 0, g, -torch.zeros_like(g)).to(torch.bfloat16)
    c, s = O.quantize_act_mxfp4(to_bits(act)[None], np.zeros(0, np.int32))
    np.testing.assert_array_equal(sf_canonical(q.sf.cpu().numpy(), np.zeros(1, int), F // 32, 128), s)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), c)


def test_token_quantizer_special_values():
    # all-zero blocks and rows, signed zeros, subnormal maxima, the largest magnitudes, saturation
    T, K = 12, 256
    v = np.random.default_rng(5).standard_normal((T, K)).astype(np.float32)
    v[0] = 0.0
    v[1, :32] = -0.0
    v[2, 5] = -0.0
    v[3, 32:64] = np.float32(2.0 ** -130)
    v[4, 64:96] = np.float32(3.0e38)
    v[5, 96] = 7.9
    v[6] = np.float32(2.0 ** -133)
    xb = (v.view(np.uint32) >> 16).astype(np.uint16)
    ids = make_ids(1, T, 2, 5)
    p, plan = plan_of(ids, 5), _plan(ids, 5)
    idx = np.arange(0, 64, dtype=np.int32)[::-1].copy()
    out = _coded_out(plan, K + 64)
    arc.quantize_act_experts_mxfp4(to_dev(xb), plan, torch.from_numpy(idx).cuda(), out=out)
    _status_ok()
    c, s = O.quantize_act_mxfp4(xb, idx)
    token = p["slot_of_row"] // 2
    _check_coded(out, p, c[token], s[token], K + 64)


@pytest.mark.parametrize("E,N,K,r", [(1, 8, 32, 0), (3, 128, 256, 32), (5, 200, 96, 32), (2, 264, 512, 0)])
def test_weights_are_packed_expert_by_expert(E, N, K, r):
    wb = W.matrix_bf16(64, 2, E * N, K, 0.02)
    idx = O.calibrate(_x_bits(64, 32, K), r) if r else np.zeros(0, np.int32)
    big = torch.zeros(E, N, K + 8, dtype=torch.bfloat16, device="cuda")
    big[:, :, :K] = to_dev(wb).view(E, N, K)
    di = torch.from_numpy(idx).cuda() if r else None
    for w in (to_dev(wb).view(E, N, K), big[:, :, :K]):
        q = arc.pack_weight_experts_mxfp4(w, di)
        _status_ok()
        kp = O.kpad(K + r)
        per = arc.mxfp4_sf_bytes(N, K + r)
        for e in range(E):
            c, s = O.pack_weight_mxfp4(wb[e * N:(e + 1) * N], idx)
            np.testing.assert_array_equal(q.codes.view(E, N, kp // 2)[e].cpu().numpy(), c)
            np.testing.assert_array_equal(q.sf[e * per:(e + 1) * per].cpu().numpy(), O.sf_swizzle(s))


# --------------------------------------------------------------------------------------- products


def _values(codes, scales):
    """MXFP4 values in 64 bits."""
    rows, half = codes.shape
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    c = np.stack([codes & 15, codes >> 4], 2).reshape(rows, 2 * half)
    v = np.where(c & 8, -grid[c & 7], grid[c & 7])
    return v * np.exp2(np.repeat(scales.astype(np.float64) - 127, 32, axis=1))


def _check_product(y, a, w_of, p, N, K, pad_value=None):
    """y [S, N] against sorted rows a (64 bits, rows in use) times the experts' weights."""
    yv = f64(y)
    used = p["used"]
    for e in range(len(p["offsets"]) - 1):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if hi == lo:
            continue
        w = w_of(e)
        ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
        tol = BF16_HALF_STEP * np.abs(ref) + K * 2 * F32_HALF_STEP * mag
        bad = np.argwhere(~(np.abs(yv[lo:hi] - ref) <= tol))
        assert len(bad) == 0, (e, lo, hi, len(bad), bad[:3], yv[lo:hi][tuple(bad[0])], ref[tuple(bad[0])])
    assert np.isnan(yv[used:]).all()  # rows behind the last one: as they were


# few rows for each expert, ragged groups, whole tiles and pairs of them, groups that end inside a
# pair's first or second half, experts without rows
PRODUCTS = [(1, 2, 8, 64, 8, 0, "skewed"), (1, 8, 64, 512, 264, 32, "skewed"), (37, 3, 5, 96, 200, 32, "drop"),
            (64, 4, 32, 1056, 520, 0, "skewed"), (300, 1, 3, 224, 256, 32, "one"), (257, 2, 4, 512, 768, 64, "drop"),
            (600, 2, 2, 4096, 264, 128, "repeat"), (900, 3, 7, 320, 1032, 0, "skewed"),
            (129, 1, 1, 256, 256, 32, "one"), (1500, 2, 5, 1024, 520, 96, "drop"), (40, 6, 512, 128, 72, 0, "drop"),
            (65, 1, 1, 64, 8, 0, "one"), (257, 1, 1, 32, 128, 0, "one"), (33, 2, 2, 288, 384, 0, "one"),
            # the most experts with tiles of 256 rows, shallow and deep
            (2101, 8, 512, 64, 8, 0, "skewed"), (2101, 8, 512, 1056, 40, 32, "drop")]


@pytest.mark.parametrize("tokens,k,experts,K,N,r,how", PRODUCTS)
def test_mxfp4_product(tokens, k, experts, K, N, r, how):
    ids = make_ids(K + N, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), _plan(ids, experts)
    xb, wb = _x_bits(65, tokens, K), W.matrix_bf16(65, 2, experts * N, K, 0.02)
    idx = O.calibrate(xb, r) if r else np.zeros(0, np.int32)
    di = torch.from_numpy(idx).cuda() if r else None
    a = arc.quantize_act_experts_mxfp4(to_dev(xb), plan, di)
    w = arc.pack_weight_experts_mxfp4(to_dev(wb).view(experts, N, K), di)
    y = _poisoned(tokens * k, N, 8)
    arc.gemm_experts_mxfp4(a, w, plan, out=y)
    _status_ok()
    av = _values(*O.quantize_act_mxfp4(xb, idx))[p["slot_of_row"][: p["used"]] // k]

    def w_of(e):
        return _values(*O.pack_weight_mxfp4(wb[e * N:(e + 1) * N], idx))

    _check_product(y, av, w_of, p, N, K + r)


@pytest.mark.parametrize("tokens,k,experts,K,N,r,how", PRODUCTS)
def test_bf16_product(tokens, k, experts, K, N, r, how):
    ids = make_ids(K + N, tokens, k, experts, how)
    p, plan = plan_of(ids, experts), _plan(ids, experts)
    K = K + r + 8  # lengths that are no multiple of a pipeline stage
    xb, wb = W.matrix_bf16(66, 1, tokens, K, 1.0), W.matrix_bf16(66, 2, experts * N, K, 0.02)
    rows = _poisoned(tokens * k, K, 16)
    arc.dispatch_experts(to_dev(xb), plan, out=rows)
    y = _poisoned(tokens * k, N, 8)
    arc.gemm_experts_bf16(rows, to_dev(wb).view(experts, N, K), plan, out=y)
    _status_ok()
    av = O.bf16_bits_to_f32(xb).astype(np.float64)[p["slot_of_row"][: p["used"]] // k]
    _check_product(y, av, lambda e: O.bf16_bits_to_f32(wb[e * N:(e + 1) * N]).astype(np.float64), p, N, K)


def test_bf16_product_of_eight_channels():
    rows = torch.ones(3, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2, 8, 8, dtype=torch.bfloat16, device="cuda")
    w[1] = 2
    plan = arc.expert_plan(torch.tensor([[1], [0], [1]], device="cuda"), 2)
    assert arc.gemm_experts_bf16(rows, w, plan).tolist() == [[8.0] * 8, [16.0] * 8, [16.0] * 8]


def test_neighbours_in_a_tile_do_not_meet():
    # rows and experts of NaN and infinity lie in the same tiles as finite ones: they reach their own
    # results alone
    T, E, K, N = 300, 3, 192, 200
    ids = make_ids(21, T, 1, E)
    p, plan = plan_of(ids, E), _plan(ids, E)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.randn(E, N, K, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want = arc.gemm_experts_bf16(arc.dispatch_experts(x, plan), w, plan)
    want4 = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan), arc.pack_weight_experts_mxfp4(w), plan)
    x[5], x[17, 3], x[200] = float("nan"), float("inf"), 3e38
    w[1] = float("nan")
    w[2, 7] = float("inf")
    rows = arc.dispatch_experts(x, plan)
    got = arc.gemm_experts_bf16(rows, w, plan)
    fine = np.ones((T, N), bool)
    fine[p["row_of_slot"][[5, 17, 200]]] = False
    fine[p["expert"] == 1] = False
    fine[p["expert"] == 2, 7] = False
    fine = torch.from_numpy(fine).cuda()
    assert torch.equal(got[fine], want[fine])
    assert torch.isnan(got[plan.row_of_slot[5]]).all()
    assert torch.isnan(got[torch.from_numpy(p["expert"] == 1).cuda()]).all()
    # MXFP4: codes of such rows are not specified, other rows keep their results
    wq = arc.pack_weight_experts_mxfp4(torch.where(torch.isfinite(w), w, torch.full_like(w, 3e38)))
    got = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan), wq, plan)
    # (an expert with a changed weight keeps its other features: one scale block is one feature's)
    assert torch.equal(got[fine], want4[fine])


def test_gpu_refusals():
    plan = arc.expert_plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(3, 64, 64, dtype=torch.bfloat16, device="cuda")
    wt = torch.zeros(4, 2, device="cuda")
    a, q = arc.quantize_act_experts_mxfp4(x, plan), arc.pack_weight_experts_mxfp4(w)
    refused = [
        lambda: arc.dispatch_experts(x[:3], plan), lambda: arc.dispatch_experts(x.float(), plan),
        lambda: arc.dispatch_experts(x.t().contiguous().t(), plan), lambda: arc.dispatch_experts(x, plan, out=rows[:4]),
        lambda: arc.dispatch_experts_grad(rows[:7], plan), lambda: arc.combine_experts(rows, wt.half(), plan),
        lambda: arc.combine_experts(rows, wt[:, :1], plan), lambda: arc.combine_experts(rows, wt, plan, add=rows),
        lambda: arc.combine_experts_grad(rows, rows, wt, plan), lambda: arc.combine_experts(rows, wt.cpu(), plan),
        lambda: arc.quantize_act_experts_mxfp4(rows, plan), lambda: arc.quantize_swiglu_experts_mxfp4(x, plan),
        lambda: arc.quantize_act_experts_mxfp4(x, plan, torch.arange(32, device="cuda")),
        lambda: arc.quantize_act_experts_mxfp4(x, plan, out=arc.ExpertMXFP4(a.buf[:-1], 8, 64)),
        lambda: arc.gemm_experts_bf16(rows, w[:2], plan), lambda: arc.gemm_experts_bf16(rows, w[:, :, :32], plan),
        lambda: arc.gemm_experts_bf16(rows, torch.zeros(6, 64, 64, dtype=torch.bfloat16, device="cuda")[::2], plan),
        lambda: arc.gemm_experts_mxfp4(arc.ExpertMXFP4(a.buf[:-1], 8, 64), q, plan),
        lambda: arc.gemm_experts_mxfp4(a, arc.ExpertWeightMXFP4(q.codes[:-1], q.sf, 3, 64, 64), plan),
        lambda: arc.gemm_experts_mxfp4(a, arc.ExpertWeightMXFP4(q.codes, q.sf[:-1], 3, 64, 64), plan),
        lambda: arc.expert_plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 4, out=plan)]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    for call in (lambda: arc.dispatch_experts(x[:, :60], plan),
                 lambda: arc.expert_plan(plan.offsets[:2].view(2, 1), 513),
                 lambda: arc.gemm_experts_bf16(rows, w[:, :60].contiguous(), plan),
                 lambda: arc.quantize_act_experts_mxfp4(x, plan, torch.arange(16, dtype=torch.int32, device="cuda")),
                 lambda: arc.expert_plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 3)):
        with pytest.raises(arc.ArcError):
            call()
    _status_ok()


def test_products_repeat_bit_for_bit():
    ids = make_ids(9, 700, 3, 5)
    plan = _plan(ids, 5)
    xb, wb = _x_bits(67, 700, 1024), W.matrix_bf16(67, 2, 5 * 512, 1024, 0.02)
    w16 = to_dev(wb).view(5, 512, 1024)
    w = arc.pack_weight_experts_mxfp4(w16)
    outs = []
    for _ in range(3):
        a = arc.quantize_act_experts_mxfp4(to_dev(xb), plan)
        rows = arc.dispatch_experts(to_dev(xb), plan)
        outs.append((arc.gemm_experts_mxfp4(a, w, plan), arc.gemm_experts_bf16(rows, w16, plan)))
    for y in outs[1:]:
        assert torch.equal(y[0], outs[0][0]) and torch.equal(y[1], outs[0][1])
