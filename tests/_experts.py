"""Plain forms of the mixture-of-experts operators for the tests: numpy in 64 bits, and the oracle's
MXFP4 coding."""
import numpy as np
import torch

import oracle as O


def plan_of(ids: np.ndarray, experts: int) -> dict:
    """The plan of ids [T, k], by lists."""
    flat = ids.reshape(-1)
    slots = flat.size
    lists = [np.flatnonzero(flat == e) for e in range(experts)]
    counts = np.array([len(v) for v in lists])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    blocks = np.concatenate([[0], np.cumsum((counts + 127) // 128)])
    slot_of_row = np.full(slots, -1)
    row_of_slot = np.full(slots, -1)
    sf_row = np.full(slots, -1)
    expert = np.full(slots, -1)
    for e, v in enumerate(lists):
        rows = offsets[e] + np.arange(len(v))
        slot_of_row[rows], row_of_slot[v], expert[rows] = v, rows, e
        sf_row[rows] = 128 * blocks[e] + np.arange(len(v))
    return dict(offsets=offsets, blocks=blocks, row_of_slot=row_of_slot, slot_of_row=slot_of_row, sf_row=sf_row,
                expert=expert, used=int(offsets[-1]))


def make_ids(seed: int, tokens: int, k: int, experts: int, how: str = "skewed") -> np.ndarray:
    """Expert ids [T, k]. skewed: distinct per token, popular experts; drop: a third lies outside
    [0, experts); one: every slot the same expert; repeat: experts may repeat within a token."""
    rng = np.random.default_rng(seed)
    if how == "one":
        return np.full((tokens, k), experts // 2, np.int32)
    if how == "repeat":
        return rng.integers(0, experts, (tokens, k)).astype(np.int32)
    score = rng.standard_normal((tokens, experts)) + rng.standard_normal(experts)
    ids = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    if how == "drop":
        out = rng.random((tokens, k)) < 1 / 3
        ids[out] = rng.choice([-1, experts, experts + 7, -2 ** 31, 2 ** 31 - 1], out.sum())
    return ids


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def sf_places(slots: int, experts: int) -> int:
    """Places of the scale layout."""
    return (slots + 127 * min(experts, slots)) // 128 * 128


def sf_canonical(sf: np.ndarray, sf_row: np.ndarray, ncols: int, places: int) -> np.ndarray:
    """Scale bytes [rows, ncols] of the rows at places sf_row."""
    m = sf_row[:, None].astype(np.int64)
    kb = np.arange(ncols)[None, :]
    return sf[(kb // 8 * places + m) * 8 + kb % 8]
