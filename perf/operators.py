"""Cases of the mixture-of-experts operators: tokens sorted by expert and back (with gradients), and
the experts' products in MXFP4 (quantisation included) and in BF16.

A slot is one (token, choice) pair, slot = token * k + choice. The plan sorts the slots stably by
expert: row i of a sorted tensor belongs to slot slot_of_row[i], expert e owns rows
offsets[e] .. offsets[e+1]. MXFP4 scale bytes of a sorted operand are stored in 128-row blocks that
begin anew with every expert: expert e's blocks start at blocks[e], row i's scales are at row
sf_row[i]. Kinds:

  dispatch       plan from the expert ids, then the tokens' rows copied into sorted order
  dispatch_grad  gradient of the tokens: the sum of each token's row gradients
  combine        each token's sorted rows summed with its router weights
  combine_grad   gradients of the sorted rows and of the router weights
  up             plan, tokens quantised to MXFP4 into sorted order (r residual channels appended),
                 product with each expert's packed weights
  down           silu(gate) * up of the sorted rows, rounded to bf16, quantised to MXFP4 with r
                 residual channels, product with each expert's packed weights
  bf16           product of sorted bf16 rows with each expert's bf16 weights
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a decoding sequence reaches its experts: launch latency
        {"name": "dispatch one token", "kind": "dispatch", "tokens": 1, "k": 8, "experts": 128, "d": 4096},
        # a training batch of a model with many small experts
        {"name": "dispatch batch", "kind": "dispatch", "tokens": 8192, "k": 8, "experts": 64, "d": 2048},
        # its way back, at odd sizes
        {"name": "dispatch gradient", "kind": "dispatch_grad", "tokens": 4099, "k": 6, "experts": 61, "d": 4104},
        {"name": "combine one token", "kind": "combine", "tokens": 1, "k": 8, "experts": 128, "d": 4096},
        # a long prompt through a model with few large experts
        {"name": "combine prompt", "kind": "combine", "tokens": 16384, "k": 2, "experts": 8, "d": 4096},
        {"name": "combine gradient", "kind": "combine_grad", "tokens": 4096, "k": 8, "experts": 128, "d": 2048},
        # four sequences decode one token each: few rows for each expert, the weights' bytes count
        {"name": "up decode", "kind": "up", "tokens": 4, "k": 8, "experts": 64, "d": 2048, "n": 2048, "r": 64},
        # a prompt of 4096 tokens through eight experts of the 4096 -> 28672 gate|up projection
        {"name": "up prompt", "kind": "up", "tokens": 4096, "k": 2, "experts": 8, "d": 4096, "n": 28672, "r": 128},
        # a short ragged prompt through many experts: groups that end inside tiles
        {"name": "down ragged", "kind": "down", "tokens": 509, "k": 4, "experts": 32, "d": 1056, "n": 2040, "r": 32},
        # the 14336 -> 4096 down projection of the same prompt
        {"name": "down prompt", "kind": "down", "tokens": 4096, "k": 2, "experts": 8, "d": 14336, "n": 4096, "r": 128},
        # the BF16 form of the experts, for one token and for a batch
        {"name": "bf16 one token", "kind": "bf16", "tokens": 1, "k": 2, "experts": 8, "d": 2048, "n": 8192},
        {"name": "bf16 batch", "kind": "bf16", "tokens": 4096, "k": 4, "experts": 16, "d": 2048, "n": 8192},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "up", "down", "bf16"])
    e = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, e))
    if kind in ("up", "down", "bf16"):
        step = 8 if kind == "bf16" else 32
        d = step * _log_int(rng, 256 // step, 8192 // step)
        n = 8 * _log_int(rng, 32, 2048)
        while e * n * d > 8 * 4096 * 14336:  # the weights fit the listed cases' room
            e, n, d = max(k, e // 2), max(256, n // 16 * 8), max(256, d // 2 // step * step)
        tokens = _log_int(rng, 1, min(16384, max(2, (1 << 38) // (k * n * d))))
        case = {"kind": kind, "tokens": tokens, "k": k, "experts": e, "d": d, "n": n}
        if kind != "bf16":
            case["r"] = 32 * rng.randint(0, min(8, d // 32))
        return case
    d = 8 * _log_int(rng, 16, 1024)
    tokens = _log_int(rng, 1, max(2, min(32768, (1 << 27) // (k * d))))
    return {"kind": kind, "tokens": tokens, "k": k, "experts": e, "d": d}


# --------------------------------------------------------------------------------------------
# The plan and the MXFP4 format in elementary operations
# --------------------------------------------------------------------------------------------


def _plan_views(buf, slots, experts):
    """The sections of a plan's int32 buffer; each begins at a multiple of 64 values."""
    sizes = [("offsets", experts + 1), ("blocks", experts + 1), ("row_of_slot", slots), ("slot_of_row", slots),
             ("sf_row", slots)]
    starts = [sum((n + 63) // 64 * 64 for _, n in sizes[:i]) for i in range(len(sizes) + 1)]
    if buf is None:
        return starts[-1]
    return {name: buf[at:at + n] for (name, n), at in zip(sizes, starts)}


def _plan(ids, experts):
    """offsets, blocks, row_of_slot, slot_of_row and sf_row of the slots sorted stably by expert."""
    flat = ids.reshape(-1).long()
    slots = flat.numel()
    order = torch.argsort(flat, stable=True)
    counts = (flat[None, :] == torch.arange(experts, device=flat.device)[:, None]).sum(1)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    blocks = torch.nn.functional.pad(((counts + 127) // 128).cumsum(0), (1, 0))
    rows = torch.arange(slots, device=flat.device)
    expert = flat[order]
    buf = torch.zeros(_plan_views(None, slots, experts), dtype=torch.int32, device=flat.device)
    p = _plan_views(buf, slots, experts)
    p["offsets"][:] = offsets
    p["blocks"][:] = blocks
    p["row_of_slot"][order] = rows.int()
    p["slot_of_row"][:] = order
    p["sf_row"][:] = 128 * blocks[expert] + rows - offsets[expert]
    return dict(p, buf=buf)


def _expert_of_row(p):
    rows = torch.arange(p["slot_of_row"].numel(), device=p["offsets"].device)
    return (rows[:, None] >= p["offsets"][None, 1:-1]).sum(1) if p["offsets"].numel() > 2 else rows * 0


def _kpad(k):
    return (k + 63) // 64 * 64


def _e2m1(q):
    """The nearest E2M1 value (ties to even, saturating at 6) of q."""
    a = q.abs()
    a = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(a.clamp(max=6), q)


def _pow2(e):
    """2^e of whole numbers -127 <= e <= 127, put together from its bits: exactly."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).int().view(torch.float32)


def _mx_parts(x):
    """E2M1 values [rows, K] and scale exponents [rows, K/32] of x in MXFP4."""
    rows, k = x.shape
    b = x.float().view(rows, k // 32, 32)
    amax = b.abs().amax(2)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    q = _e2m1(b * _pow2(-e)[:, :, None])
    return torch.where(amax[:, :, None] > 0, q, torch.zeros_like(q)).view(rows, k), e


def _mx(x, idx, weight):
    """MXFP4 values of x with its appended channels: the residuals, or for weights the channels again."""
    q, e = _mx_parts(x)
    rows, k = x.shape
    v = (q.view(rows, k // 32, 32) * _pow2(e)[:, :, None]).view(rows, k)
    if idx is None:
        return v, q, e
    tail = x.float()[:, idx.long()] - (0 if weight else v[:, idx.long()])
    tq, te = _mx_parts(tail)
    tv = (tq.view(rows, -1, 32) * _pow2(te)[:, :, None]).view(rows, -1)
    return torch.cat([v, tv], 1), torch.cat([q, tq], 1), torch.cat([e, te], 1)


def _packed(w, idx, experts):
    """Codes [E * N, K_pad/2] and scale bytes (512-byte atoms, anew for every expert) of w [E * N, K]."""
    _, q, e = _mx(w, idx, True)
    rows, k = q.shape
    n, kp = rows // experts, _kpad(k)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    code = torch.nn.functional.pad(code, (0, kp - k))
    codes = code[:, 0::2] + 16 * code[:, 1::2]
    sb = (e + 127).to(torch.uint8).view(experts, n, k // 32)
    sb = torch.nn.functional.pad(sb, (0, (kp + 127) // 128 * 4 - k // 32, 0, -n % 128))
    sb = sb.view(experts, -1, 4, 32, sb.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return codes.contiguous(), sb.reshape(-1).contiguous()


def _weights(s):
    """The values [E, N, K_pad] that the packed experts stand for."""
    experts, n, kp = s["experts"], s["n"], _kpad(s["k_aug"])
    c = torch.stack([s["w_codes"] & 15, s["w_codes"] >> 4], 2).view(experts, n, kp // 32, 32)
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=c.device)[(c & 7).int()]
    v = torch.where(c >= 8, -mag, mag)
    atoms = (kp + 127) // 128
    sb = s["w_sf"].view(experts, -1, atoms, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(experts, -1, 4 * atoms)
    sb = sb[:, :n, : kp // 32].int()
    return (v * _pow2(sb - 127)[:, :, :, None]).view(experts, n, kp)


def _product(a, w, p, cap):
    """Rows of a [S, K] times their expert's w [E, N, K], as one padded batched product."""
    e = _expert_of_row(p)
    at = e * cap + torch.arange(a.shape[0], device=a.device) - p["offsets"].long()[e]
    pad = torch.zeros(w.shape[0] * cap, w.shape[2], dtype=a.dtype, device=a.device)
    pad[at, : a.shape[1]] = a
    y = torch.bmm(pad.view(w.shape[0], cap, w.shape[2]), w.transpose(1, 2))
    return y.view(w.shape[0] * cap, w.shape[1])[at]


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    t, k, e, d, kind = case["tokens"], case["k"], case["experts"], case["d"], case["kind"]
    # router scores: some experts are more popular than others
    scores = torch.randn(t, e, generator=g, device=dev) + 0.5 * torch.randn(e, generator=g, device=dev)
    top, ids = torch.topk(scores, k, dim=1)
    s = {"kind": kind, "tokens": t, "k": k, "experts": e, "d": d, "ids": ids.int().contiguous()}
    s["weights"] = torch.softmax(top, 1).contiguous()
    p = s["plan"] = _plan(s["ids"], e)
    # the longest group, which the plain form's padded product needs
    s["cap"] = int((p["offsets"][1:] - p["offsets"][:-1]).max())
    slots = t * k
    if kind == "dispatch":
        s["x"] = normal(t, d)
    elif kind == "dispatch_grad":
        s["d_rows"] = normal(slots, d)
    elif kind == "combine":
        s["rows"] = normal(slots, d)
    elif kind == "combine_grad":
        s["rows"], s["dy"] = normal(slots, d), normal(t, d)
    elif kind == "bf16":
        s["n"] = case["n"]
        s["rows"], s["w"] = normal(slots, d), normal(e, case["n"], d, scale=0.02)
    else:
        n, r = case["n"], case["r"]
        # a hundredth of the channels are 20 to 80 times larger, as activations have them
        mult = torch.ones(d, device=dev)
        loud = torch.randperm(d, generator=g, device=dev)[: max(1, d // 100)]
        mult[loud] = 20 * 4 ** torch.rand(loud.numel(), generator=g, device=dev)
        if kind == "up":
            s["x"] = (normal(t, d).float() * mult).to(torch.bfloat16)
        else:
            s["gu"] = normal(slots, 2 * d)
            s["gu"][:, d:] = (s["gu"][:, d:].float() * mult).to(torch.bfloat16)
        s["idx"] = torch.argsort(mult, descending=True, stable=True)[:r].int().contiguous() if r else None
        s["n"], s["k_aug"] = n, d + r
        s["w_codes"], s["w_sf"] = _packed(normal(e * n, d, scale=0.02), s["idx"], e)
    return s


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------


def _silu_mul(gu, d):
    g, u = gu[:, :d].float(), gu[:, d:].float()
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import nvfp4_block_scaled_arc_b200 as arc

    kind = s["kind"]
    if kind == "dispatch":
        plan = arc.expert_plan(s["ids"], s["experts"])
        rows = arc.dispatch_experts(s["x"], plan)
        return {"rows": rows, "offsets": plan.offsets, "row_of_slot": plan.row_of_slot, "slot_of_row": plan.slot_of_row}
    if kind == "up":
        plan = arc.expert_plan(s["ids"], s["experts"])
        a = arc.quantize_act_experts_mxfp4(s["x"], plan, s["idx"])
        w = arc.ExpertWeightMXFP4(s["w_codes"], s["w_sf"], s["experts"], s["n"], s["k_aug"])
        return arc.gemm_experts_mxfp4(a, w, plan)
    # the plan that the forward pass or the layer's first product made
    plan = arc.ExpertPlan(s["plan"]["buf"], s["tokens"], s["k"], s["experts"])
    if kind == "dispatch_grad":
        return arc.dispatch_experts_grad(s["d_rows"], plan)
    if kind == "combine":
        return arc.combine_experts(s["rows"], s["weights"], plan)
    if kind == "combine_grad":
        return arc.combine_experts_grad(s["dy"], s["rows"], s["weights"], plan)
    if kind == "down":
        a = arc.quantize_swiglu_experts_mxfp4(s["gu"], plan, s["idx"])
        w = arc.ExpertWeightMXFP4(s["w_codes"], s["w_sf"], s["experts"], s["n"], s["k_aug"])
        return arc.gemm_experts_mxfp4(a, w, plan)
    return arc.gemm_experts_bf16(s["rows"], s["w"], plan)


def _run_plain(s):
    kind, t, k = s["kind"], s["tokens"], s["k"]
    if kind == "dispatch":
        p = _plan(s["ids"], s["experts"])
        return {"rows": s["x"][(p["slot_of_row"] // k).long()], "offsets": p["offsets"],
                "row_of_slot": p["row_of_slot"], "slot_of_row": p["slot_of_row"]}
    if kind == "up":
        p = _plan(s["ids"], s["experts"])
        a = _mx(s["x"], s["idx"], False)[0][(p["slot_of_row"] // k).long()]
        return _product(a, _weights(s), p, s["cap"]).to(torch.bfloat16)
    p = s["plan"]
    if kind == "dispatch_grad":
        return s["d_rows"].float()[p["row_of_slot"].long()].view(t, k, -1).sum(1).to(torch.bfloat16)
    if kind == "combine":
        rows = s["rows"].float()[p["row_of_slot"].long()].view(t, k, -1)
        return (rows * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)
    if kind == "combine_grad":
        at = p["slot_of_row"].long()
        dy = s["dy"].float()[at // k]
        d_rows = (dy * s["weights"].view(-1)[at][:, None]).to(torch.bfloat16)
        dots = (dy * s["rows"].float()).sum(1)
        return d_rows, dots[p["row_of_slot"].long()].view(t, k)
    if kind == "down":
        a = _mx(_silu_mul(s["gu"], s["d"]), s["idx"], False)[0]
        return _product(a, _weights(s), p, s["cap"]).to(torch.bfloat16)
    return _product(s["rows"].float(), s["w"].float(), p, s["cap"]).to(torch.bfloat16)


# --------------------------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------------------------

_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _block_values(x):
    """MXFP4 values of x [rows, K] (64 bits): nearest grid value, ties to the even code."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    v = x.reshape(-1, 32)
    top = v.abs().amax(1, keepdim=True)
    # 2^(floor(log2 top) - 2): the exponent field of a double is floor(log2) + 1023
    step = (((top.view(torch.int64) >> 52) - 2).clamp(min=1023 - 127) << 52).view(torch.float64)
    q = (v.abs() / step)[:, :, None]
    code = (q > mid[0::2]).sum(2) + (q >= mid[1::2]).sum(2)
    return (torch.sign(v) * grid[code] * step).view(x.shape)


def _augmented(x, idx):
    v = _block_values(x)
    return v if idx is None else torch.cat([v, _block_values(x[:, idx.long()] - v[:, idx.long()])], 1)


def exact(case, seed):
    if 2.0 * case["tokens"] * case["k"] * case.get("n", 0) * case["d"] > 1e13:
        return None
    s = prepare(case, seed)
    kind, t, k, n_e = s["kind"], s["tokens"], s["k"], s["experts"]
    flat = s["ids"].reshape(-1).cpu()
    lists = [torch.nonzero(flat == e).view(-1) for e in range(n_e)]
    slots = torch.cat(lists).to("cuda")  # slots by expert, each expert's in ascending order
    bounds = [0]
    for v in lists:
        bounds.append(bounds[-1] + v.numel())
    row_of = torch.empty_like(slots)
    row_of[slots] = torch.arange(slots.numel(), device=slots.device)
    if kind == "dispatch":
        return {"rows": s["x"].double()[slots // k], "offsets": None, "row_of_slot": None, "slot_of_row": None}
    if kind in ("dispatch_grad", "combine"):
        rows = s["d_rows" if kind == "dispatch_grad" else "rows"]
        out = torch.zeros(t, s["d"], dtype=torch.float64, device=rows.device)
        for j in range(k):
            part = rows[row_of[torch.arange(t, device=rows.device) * k + j]].double()
            out += part if kind == "dispatch_grad" else part * s["weights"][:, j:j + 1].double()
        return out
    if kind == "combine_grad":
        dy = s["dy"].double()
        w = s["weights"].double().view(-1)
        d_w = torch.empty(t, k, dtype=torch.float64, device=dy.device)
        for j in range(k):
            d_w[:, j] = (dy * s["rows"][row_of[torch.arange(t, device=dy.device) * k + j]].double()).sum(1)
        return dy[slots // k] * w[slots][:, None], d_w
    n, order = s["n"], torch.arange(slots.numel(), device=slots.device)
    if kind == "bf16":
        a = s["rows"].double()
    elif kind == "up":
        a, order = _augmented(s["x"].double(), s["idx"]), slots // k
    else:
        gate, up = s["gu"][:, : s["d"]].double(), s["gu"][:, s["d"]:].double()
        a = _augmented((gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double(), s["idx"])
    grid = torch.tensor(_GRID, dtype=torch.float64, device="cuda")
    out = torch.empty(slots.numel(), n, dtype=torch.float64, device="cuda")
    for e in range(n_e):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        if kind == "bf16":
            w = s["w"][e].double()
        else:
            ka, per = s["k_aug"], s["w_sf"].numel() // n_e
            c = s["w_codes"][e * n:(e + 1) * n].long()
            w = torch.empty(n, 2 * c.shape[1], dtype=torch.float64, device=c.device)
            w[:, 0::2], w[:, 1::2] = (grid[h & 7] * (1 - 2 * (h >> 3)) for h in (c & 15, c >> 4))
            m = torch.arange(n, device=c.device)[:, None]
            kb = torch.arange(ka // 32, device=c.device)[None, :]
            atom = m // 128 * ((_kpad(ka) + 127) // 128) + kb // 4
            byte = s["w_sf"][e * per + atom * 512 + m % 32 * 16 + m // 32 % 4 * 4 + kb % 4]
            w = w[:, :ka] * torch.exp2(byte.double() - 127).repeat_interleave(32, 1)
        out[lo:hi] = a[order[lo:hi]] @ w.T
    return out


def work(case):
    t, k, d, kind = case["tokens"], case["k"], case["d"], case["kind"]
    slots = t * k
    if kind == "dispatch":
        return {"bytes": 2 * d * (t + slots) + 12 * slots, "flops": 0}
    if kind == "dispatch_grad":
        return {"bytes": 2 * d * (t + slots) + 4 * slots, "flops": slots * d}
    if kind == "combine":
        return {"bytes": 2 * d * (t + slots) + 8 * slots, "flops": 2 * slots * d}
    if kind == "combine_grad":
        return {"bytes": 2 * d * (t + 2 * slots) + 12 * slots, "flops": 3 * slots * d}
    n = case["n"]
    used = min(case["experts"], slots)  # every expert that has a row is read
    if kind == "bf16":
        return {"bytes": 2 * slots * (d + n) + 2 * used * n * d, "flops": 2 * slots * n * d}
    kp = _kpad(d + case["r"])
    inputs = 2 * t * d if kind == "up" else 4 * slots * d
    return {"bytes": inputs + used * n * kp * 17 // 32 + 2 * slots * n, "flops": 2 * slots * n * (d + case["r"])}
