"""The mixture-of-experts operators as they are used: whole layers in MXFP4 and in BF16, a training
step's gradients, captured and replayed graphs, other streams, buffers between canaries, a pipeline
wait that runs out, and tensors beyond 2^31 elements.
"""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_arc_b200 as arc
import oracle as O
import workloads as W
from tests._experts import bf16, f64, make_ids, plan_of
from tests._helpers import to_bits, to_dev

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a bf16 step, relative
TIMEOUT = 5


def _layer_inputs(seed, T, k, E, d, F, how="skewed"):
    ids = make_ids(seed, T, k, E, how)
    mult = W.outlier_multipliers(seed, 0, d, max(1, d // 64), 10.0, 60.0)
    x = to_dev(W.matrix_bf16(seed, 1, T, d, 1.0, col_mult=mult))
    wgu = to_dev(W.matrix_bf16(seed, 2, E * 2 * F, d, 0.05)).view(E, 2 * F, d)
    wd = to_dev(W.matrix_bf16(seed, 3, E * d, F, 0.05)).view(E, d, F)
    weights = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(seed)), 1).cuda()
    return ids, x, wgu, wd, weights


def _mxfp4_layer(x, ids, weights, q, E, idx_up, idx_down, add):
    plan = arc.expert_plan(ids, E)
    gu = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan, idx_up), q["gu"], plan)
    rows = arc.gemm_experts_mxfp4(arc.quantize_swiglu_experts_mxfp4(gu, plan, idx_down), q["d"], plan)
    return arc.combine_experts(rows, weights, plan, add=add), gu, rows, plan


def _bf16_layer(x, ids, weights, wgu, wd, E, add):
    plan = arc.expert_plan(ids, E)
    gu = arc.gemm_experts_bf16(arc.dispatch_experts(x, plan), wgu, plan)
    rows = arc.gemm_experts_bf16(arc.silu_mul_bf16(gu), wd, plan)
    return arc.combine_experts(rows, weights, plan, add=add), gu, rows, plan


def _combined(rows, weights, p, T, k, add):
    out, mag = f64(add), np.abs(f64(add))
    r, w = f64(rows), f64(weights)
    for j in range(k):
        row = p["row_of_slot"].reshape(T, k)[:, j]
        part = np.where(row[:, None] >= 0, w[:, j:j + 1] * r[np.maximum(row, 0)], 0.0)
        out, mag = out + part, mag + np.abs(part)
    return out, mag


@pytest.mark.parametrize("T,k,E,d,F,how", [(1, 2, 8, 256, 128, "skewed"), (77, 4, 12, 512, 320, "drop"),
                                           (700, 2, 3, 1024, 512, "skewed")])
def test_layers_stage_by_stage(T, k, E, d, F, how):
    # every stage against 64 bits, from the values that the stage before it left
    ids, x, wgu, wd, weights = _layer_inputs(71, T, k, E, d, F, how)
    p, used = plan_of(ids, E), plan_of(ids, E)["used"]
    add = to_dev(W.matrix_bf16(72, 1, T, d, 1.0))
    dev_ids = torch.from_numpy(ids).cuda()
    r = 32
    iu = arc.calibrate_outliers(x, r)
    idn = torch.arange(0, 2 * r, 2, dtype=torch.int32, device="cuda")
    q = {"gu": arc.pack_weight_experts_mxfp4(wgu, iu), "d": arc.pack_weight_experts_mxfp4(wd, idn)}

    def coded(bits, idx, pack=False):
        c, s = (O.pack_weight_mxfp4 if pack else O.quantize_act_mxfp4)(bits, idx.cpu().numpy())
        grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
        n = np.stack([c & 15, c >> 4], 2).reshape(len(c), -1)
        return np.where(n & 8, -grid[n & 7], grid[n & 7]) * np.exp2(np.repeat(s.astype(float) - 127, 32, axis=1))

    def check(y, a, ws, depth, what):
        yv = f64(y)
        for e in range(E):
            lo, hi = p["offsets"][e], p["offsets"][e + 1]
            if hi > lo:
                w = ws(e)
                ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
                assert (np.abs(yv[lo:hi] - ref) <= HALF * np.abs(ref) + depth * 2.0 ** -23 * mag).all(), (what, e)

    token = p["slot_of_row"][:used] // k
    y, gu, rows, _ = _mxfp4_layer(x, dev_ids, weights, q, E, iu, idn, add)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    xb, gb, db = to_bits(x), to_bits(wgu), to_bits(wd)
    check(gu, coded(xb, iu)[token], lambda e: coded(gb[e], iu, True), d + r, "gate|up")
    # the fused SwiGLU coding, read back through the product with a unit matrix, is the act's coding
    # up to one bf16 step of act: compared through the down product within that step's reach
    act = to_bits(arc.silu_mul_bf16(gu[:used].contiguous() if used else gu[:1]))
    a = coded(act, idn)
    yv = f64(rows)
    for e in range(E):
        lo, hi = p["offsets"][e], p["offsets"][e + 1]
        if hi > lo:
            w = coded(db[e], idn, True)
            # a bf16 step of act moves its code by at most one of E2M1's steps, half the value (or X/2)
            ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
            err = np.abs(yv[lo:hi] - ref)
            assert (err <= 0.5 * mag + HALF * np.abs(ref)).all()
            # and hardly any is moved (a rounding border lies within 2^-21 of one value in 2^12)
            close = err <= HALF * np.abs(ref) + (F + r) * 2.0 ** -23 * mag
            assert close.mean() > 0.5, close.mean()
    ref, mag = _combined(rows, weights, p, T, k, add)
    assert (np.abs(f64(y) - ref) <= HALF * np.abs(ref) + (k + 2) * 2.0 ** -23 * mag).all()

    y, gu, rows, _ = _bf16_layer(x, dev_ids, weights, wgu, wd, E, add)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    check(gu, f64(x)[token], lambda e: f64(wgu[e]), d, "bf16 gate|up")
    check(rows, f64(arc.silu_mul_bf16(gu))[:used], lambda e: f64(wd[e]), F, "bf16 down")
    ref, mag = _combined(rows, weights, p, T, k, add)
    assert (np.abs(f64(y) - ref) <= HALF * np.abs(ref) + (k + 2) * 2.0 ** -23 * mag).all()


def test_training_step_gradients_against_autograd():
    # y = combine(dispatch(x) W_e^T, w): gradients of x, the weights' rows and the router weights
    # against autograd of the formula in 64 bits
    T, k, E, d, N = 150, 3, 5, 128, 192
    ids = make_ids(81, T, k, E, "drop")
    p = plan_of(ids, E)
    rng = np.random.default_rng(2)
    x, w = bf16(rng.standard_normal((T, d))), bf16(0.1 * rng.standard_normal((E * N, d))).view(E, N, d)
    g = bf16(rng.standard_normal((T, N)))
    wt = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(3)), 1).cuda()
    plan = arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    rows = arc.dispatch_experts(x, plan)
    out = arc.gemm_experts_bf16(rows, w, plan)
    y = arc.combine_experts(out, wt, plan)
    d_out, d_wt = arc.combine_experts_grad(g, out, wt, plan)
    d_rows = arc.gemm_experts_bf16(d_out, w.transpose(1, 2).contiguous(), plan)  # [E, d, N]: rows times W_e
    d_x = arc.dispatch_experts_grad(d_rows, plan)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    x64, wt64 = x.double().cpu().requires_grad_(), wt.double().cpu().requires_grad_()
    w64, y64 = w.double().cpu(), torch.zeros(T, N, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                y64[t] = y64[t] + wt64[t, j] * (w64[e] @ x64[t])
    (y64 * g.double().cpu()).sum().backward()
    # roundings on the way, each at most 2^-8 of a term: product and sum for y; d_out, product and sum
    # for d_x; the product alone for d_wt. The terms' magnitudes bound what they can move.
    mag_y, mag_x = np.zeros((T, N)), np.zeros((T, d))
    mag_w = np.zeros((T, k))
    aw, ax, ag, at = np.abs(f64(w)), np.abs(f64(x)), np.abs(f64(g)), f64(wt)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                mag_y[t] += at[t, j] * (aw[e] @ ax[t])
                mag_x[t] += at[t, j] * (ag[t] @ aw[e])
                mag_w[t, j] = ag[t] @ (aw[e] @ ax[t])
    assert (np.abs(f64(y) - y64.detach().numpy()) <= 2.1 * HALF * mag_y).all()
    assert (np.abs(f64(d_x) - x64.grad.numpy()) <= 3.1 * HALF * mag_x).all()
    assert (np.abs(f64(d_wt) - wt64.grad.numpy()) <= 1.1 * HALF * mag_w).all()
    assert p["used"] < T * k and (d_wt.cpu().numpy().reshape(-1)[p["row_of_slot"] < 0] == 0).all()


def test_captured_layers_replay_on_new_inputs():
    # two graphs of different layers, replayed in turn with new inputs in place; a replay's routing,
    # and with it the number of tiles, differs from the captured one
    graphs = []
    for seed, (T, k, E, d, F) in ((91, (200, 2, 6, 256, 128)), (92, (3, 4, 40, 512, 256))):
        ids, x, wgu, wd, weights = _layer_inputs(seed, T, k, E, d, F)
        iu = arc.calibrate_outliers(x, 32)
        q = {"gu": arc.pack_weight_experts_mxfp4(wgu, iu), "d": arc.pack_weight_experts_mxfp4(wd)}
        dev_ids, add = torch.from_numpy(ids).cuda(), torch.zeros_like(x)

        def run(x=x, dev_ids=dev_ids, weights=weights, q=q, E=E, iu=iu, add=add, wgu=wgu, wd=wd):
            y, _, rows, plan = _mxfp4_layer(x, dev_ids, weights, q, E, iu, None, add)
            z = _bf16_layer(x, dev_ids, weights, wgu, wd, E, add)[0]
            return y, z, *arc.combine_experts_grad(y, rows, weights, plan)

        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        graphs.append((g, outs, run, x, dev_ids, weights, T, k, E))
    for turn in range(3):
        for g, outs, run, x, dev_ids, weights, T, k, E in graphs:
            gen = torch.Generator(device="cuda").manual_seed(turn)
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            weights.copy_(torch.rand(weights.shape, generator=gen, device="cuda"))
            dev_ids.copy_(torch.from_numpy(make_ids(turn, T, k, E, ("one", "skewed", "repeat")[turn])))
            g.replay()
        for g, outs, run, *_ in graphs:
            torch.cuda.synchronize()
            for got, want in zip(outs, run()):
                assert torch.equal(got, want)
    assert arc.last_device_status() == 0


def test_calls_on_two_streams_at_once():
    T, k, E, d, F = 400, 2, 6, 512, 256
    ids, x, wgu, wd, weights = _layer_inputs(95, T, k, E, d, F)
    dev_ids, add = torch.from_numpy(ids).cuda(), torch.zeros_like(x)
    q = {"gu": arc.pack_weight_experts_mxfp4(wgu), "d": arc.pack_weight_experts_mxfp4(wd)}
    want = _mxfp4_layer(x, dev_ids, weights, q, E, None, None, add)[0]
    want16 = _bf16_layer(x, dev_ids, weights, wgu, wd, E, add)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        # one layer with the streams given call by call, the other under the stream as current one
        p = arc.expert_plan(dev_ids, E, stream=s1)
        a = arc.quantize_act_experts_mxfp4(x, p, stream=s1)
        gu = arc.gemm_experts_mxfp4(a, q["gu"], p, stream=s1)
        a2 = arc.quantize_swiglu_experts_mxfp4(gu, p, stream=s1)
        rows = arc.gemm_experts_mxfp4(a2, q["d"], p, stream=s1)
        got.append((arc.combine_experts(rows, weights, p, add=add, stream=s1), want))
        with torch.cuda.stream(s2):
            got.append((_bf16_layer(x, dev_ids, weights, wgu, wd, E, add)[0], want16))
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    for y, w in got:
        assert torch.equal(y, w)


MARGIN, CANARY = 4096, 0xA5


def _guarded(nbytes):
    full = torch.full((nbytes + 2 * MARGIN,), CANARY, dtype=torch.uint8, device="cuda")
    return full, full[MARGIN:MARGIN + nbytes]


def _untouched(full, what):
    torch.cuda.synchronize()
    edge = torch.cat([full[:MARGIN], full[-MARGIN:]])
    assert (edge == CANARY).all(), what


@pytest.mark.parametrize("T,k,E,K,N,r,how", [(1, 1, 1, 32, 8, 0, "one"), (5, 3, 17, 96, 264, 32, "drop"),
                                             (131, 2, 3, 544, 200, 64, "skewed"), (400, 2, 2, 256, 520, 0, "repeat")])
def test_only_the_outputs_are_written(T, k, E, K, N, r, how):
    S = T * k
    ids = torch.from_numpy(make_ids(97, T, k, E, how)).cuda()
    x, gu = to_dev(W.matrix_bf16(97, 1, T, K, 1.0)), to_dev(W.matrix_bf16(97, 2, S, 2 * K, 1.0))
    w = to_dev(W.matrix_bf16(97, 3, E * N, K, 0.05)).view(E, N, K)
    idx = arc.calibrate_outliers(x, r) if r else None
    weights = torch.rand(T, k, device="cuda")
    f, b = _guarded(arc.lib().arc_expert_plan_bytes(T, k, E))
    plan = arc.expert_plan(ids, E, out=arc.ExpertPlan(b.view(torch.int32), T, k, E))
    _untouched(f, "plan")
    guards = []

    def mat(rows, cols, dtype=torch.bfloat16):
        f, b = _guarded(rows * cols * dtype.itemsize)
        guards.append(f)
        return b.view(dtype).view(rows, cols)

    rows = arc.dispatch_experts(x, plan, out=mat(S, K))
    arc.dispatch_experts_grad(rows, plan, out=mat(T, K))
    arc.combine_experts(rows, weights, plan, out=mat(T, K))
    arc.combine_experts_grad(x, rows, weights, plan, d_rows=mat(S, K), d_weights=mat(T, k, torch.float32))
    for q, src in ((arc.quantize_act_experts_mxfp4, x), (arc.quantize_swiglu_experts_mxfp4, gu)):
        kp = (K + r + 63) // 64 * 64
        n = (S * kp // 2 + 255) // 256 * 256 + arc.lib().arc_expert_sf_bytes(T, k, E, K + r)
        a = q(src, plan, idx, out=arc.ExpertMXFP4(mat(1, n, torch.uint8).view(-1), S, K + r))
    kp = (K + r + 63) // 64 * 64
    wc, ws = mat(E * N, kp // 2, torch.uint8), mat(1, E * arc.mxfp4_sf_bytes(N, K + r), torch.uint8)
    wq = arc.pack_weight_experts_mxfp4(w, idx, out=arc.ExpertWeightMXFP4(wc, ws.view(-1), E, N, K + r))
    arc.gemm_experts_mxfp4(a, wq, plan, out=mat(S, N))
    arc.gemm_experts_bf16(rows, w, plan, out=mat(S, N))
    wide = mat(S, N + 24)
    wide.view(torch.uint8).fill_(CANARY)
    arc.gemm_experts_mxfp4(a, wq, plan, out=wide[:, :N])
    assert (wide.view(torch.uint8).view(S, -1)[:, 2 * N:] == CANARY).all()
    for i, f in enumerate(guards):
        _untouched(f, i)
    assert arc.last_device_status() == 0


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("T,E", [(6, 8), (600, 2)])
def test_withheld_load_times_out_and_recovers(kind, T, E):
    ids, x, wgu, _, _ = _layer_inputs(98, T, 2, E, 512, 256)
    plan = arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    if kind == "mxfp4":
        a, w = arc.quantize_act_experts_mxfp4(x, plan), arc.pack_weight_experts_mxfp4(wgu)
    else:
        a = arc.dispatch_experts(x, plan)

    def run():
        return arc.gemm_experts_mxfp4(a, w, plan) if kind == "mxfp4" else arc.gemm_experts_bf16(a, wgu, plan)

    good = run()
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    arc.set_wait_limit_ns(50_000_000)  # 50 ms
    try:
        arc.debug_inject(1)
        run()
        assert arc.last_device_status() == TIMEOUT
    finally:
        arc.set_wait_limit_ns(2_000_000_000)
    again = run()
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    assert torch.equal(again, good)


def test_outlier_channel_out_of_range_is_reported():
    x = to_dev(W.matrix_bf16(99, 1, 4, 128, 1.0))
    plan = arc.expert_plan(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 2)
    idx = torch.arange(32, dtype=torch.int32, device="cuda")
    idx[7] = 128
    arc.quantize_act_experts_mxfp4(x, plan, idx)
    assert arc.last_device_status() == 1  # ARC_ERR_INVALID_ARG
    assert arc.last_device_status() == 0


@pytest.mark.parametrize("fill", [0x7F7F7F7F, -5, 33])
def test_a_buffer_without_a_plan_is_reported(fill):
    # the kernels check a plan's entries against their buffers: nothing is written outside (canaries
    # above), outputs that depend on a place stay as they were
    T, k, E, K, N = 16, 2, 4, 64, 64
    plan = arc.ExpertPlan(torch.full((2 * 64 + 3 * 64,), fill, dtype=torch.int32, device="cuda"), T, k, E)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(T * k, K, dtype=torch.bfloat16, device="cuda")
    w16, wt = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda"), torch.ones(T, k, device="cuda")
    w = arc.pack_weight_experts_mxfp4(w16)
    full, y = _guarded(T * k * N * 2)
    y = y.view(torch.bfloat16).view(T * k, N)
    calls = [lambda: arc.dispatch_experts(x, plan, out=y), lambda: arc.combine_experts(rows, wt, plan),
             lambda: arc.dispatch_experts_grad(rows, plan),
             lambda: arc.combine_experts_grad(x, rows, wt, plan, d_rows=y),
             lambda: arc.quantize_act_experts_mxfp4(x, plan), lambda: arc.gemm_experts_bf16(rows, w16, plan, out=y)]
    good = arc.quantize_act_experts_mxfp4(x, arc.expert_plan(torch.zeros(T, k, dtype=torch.int32, device="cuda"), E))
    calls.append(lambda: arc.gemm_experts_mxfp4(good, w, plan, out=y))
    for i, call in enumerate(calls):
        call()
        assert arc.last_device_status() == 1, i  # ARC_ERR_INVALID_ARG
    arc.quantize_swiglu_experts_mxfp4(torch.zeros(T * k, 2 * K, dtype=torch.bfloat16, device="cuda"), plan)
    _untouched(full, "outputs")
    assert (full == CANARY).all()
    arc.last_device_status()


@pytest.mark.slow
def test_sorted_rows_beyond_2_31_elements():
    T, k, E, d = 70000, 8, 9, 4096  # 2.3e9 elements
    ids = make_ids(5, T, k, E)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    np.testing.assert_array_equal(plan.row_of_slot.cpu().numpy(), p["row_of_slot"])
    x = torch.randn(T, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    rows = arc.dispatch_experts(x, plan)
    at = torch.cat([torch.arange(5), torch.randint(0, T * k, (4000,)), torch.arange(T * k - 5, T * k)]).cuda()
    assert torch.equal(rows[at], x[(plan.slot_of_row[at] // k).long()])
    w = torch.full((T, k), 0.125, device="cuda")  # eight equal rows: the token itself, exactly
    assert torch.equal(arc.combine_experts(rows, w, plan), x)
    d_rows, d_w = arc.combine_experts_grad(x, rows, w, plan, d_rows=rows)
    norm = (x.double() ** 2).sum(1, keepdim=True)
    assert ((d_w.double() - norm).abs() <= (d / 32 + 8) * 2.0 ** -24 * norm).all()
    assert torch.equal(arc.dispatch_experts_grad(d_rows, plan), x)


@pytest.mark.slow
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_product_beyond_2_31_outputs(kind):
    T, k, E, K, N = 40000, 2, 3, 64, 28672  # 2.3e9 outputs
    ids = make_ids(6, T, k, E)
    p, plan = plan_of(ids, E), arc.expert_plan(torch.from_numpy(ids).cuda(), E)
    # values that MXFP4 and bf16 both hold exactly, and whose sums fp32 does
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-2, 3, (T, K), generator=gen, device="cuda").bfloat16()
    w = torch.randint(-2, 3, (E, N, K), generator=gen, device="cuda").bfloat16()
    if kind == "mxfp4":
        y = arc.gemm_experts_mxfp4(arc.quantize_act_experts_mxfp4(x, plan), arc.pack_weight_experts_mxfp4(w), plan)
    else:
        y = arc.gemm_experts_bf16(arc.dispatch_experts(x, plan), w, plan)
    torch.cuda.synchronize()
    assert arc.last_device_status() == 0
    at = np.r_[0:3, 30000:30003, T * k - 3:T * k]
    for row in at:
        e, t = p["expert"][row], p["slot_of_row"][row] // k
        assert torch.equal(y[row].float(), (w[e].float() @ x[t].float()).bfloat16().float()), row
