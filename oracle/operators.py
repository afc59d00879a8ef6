"""Oracle of the operators around the paged cache, in float64 on the CPU: head norm and rotation of
new rows, attention over a list of keys, and the sampled token of a row of logits.  Loops over
sequences, rows and tokens; nothing is blocked or fused."""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import torch

from .model import attention_explicit, block_mask, rmsnorm, rope_rotate


def norm_rope(x: torch.Tensor, gain: Optional[torch.Tensor], eps: float, pos: torch.Tensor,
              theta: float) -> torch.Tensor:
    """x [n, heads, hd] of rows at positions pos [n]: RMSNorm of each head times gain (None: no
    norm), then the rotation."""
    x = x.double()
    if gain is not None:
        x = rmsnorm(x, eps) * gain.double()
    return rope_rotate(x, pos[:, None], theta)


def block_causal_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_size: int) -> torch.Tensor:
    """q [m, Hq, hd] at the last m of the keys k, v [n, Hkv, hd]: [m, Hq, hd]."""
    m = q.shape[0]
    mask = block_mask(m, k.shape[0] - m, block_size)
    o = attention_explicit(q.double().transpose(0, 1), k.double().transpose(0, 1), v.double().transpose(0, 1), mask)
    return o.transpose(0, 1)


def paged_rows(pool: torch.Tensor, pages: List[int], n: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """The first n K and V rows [n, Hkv, hd] (float64) behind a list of pages of a pool
    [n_pages, 2, Hkv, 64, hd]."""
    rows = torch.stack([pool[pages[j // 64], :, :, j % 64].double() for j in range(n)]) if n else \
        torch.zeros(0, *pool[0, :, :, 0].shape, dtype=torch.float64)
    return rows[:, 0], rows[:, 1]


def sample_token(x: torch.Tensor, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0,
                 min_p: float = 0.0) -> Tuple[int, float]:
    """(token, probability) of one row of logits x [vocab]."""
    v = [float(t) for t in x.double()]
    v = [-math.inf if math.isnan(t) else t for t in v]
    top = max(v)
    if top == -math.inf:
        return -1, 0.0
    if not temperature > 0:
        return v.index(top), 1.0
    if top == math.inf:
        w = [1.0 if t == top else 0.0 for t in v]
    else:
        w = [math.exp((t - top) / temperature) if t > -math.inf else 0.0 for t in v]
    order = sorted((i for i in range(len(v)) if v[i] > -math.inf), key=lambda i: (-v[i], i))
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        limit = top_p * math.fsum(w[i] for i in order)
        kept, before = [], 0.0
        for i in order:
            if kept and not before < limit:
                break
            kept.append(i)
            before = math.fsum((before, w[i]))
        order = kept
    if min_p > 0:
        order = [i for i in order if w[i] >= min(min_p, 1.0)]
    total = math.fsum(w[i] for i in order)
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    run = 0.0
    for i in sorted(order):
        run = math.fsum((run, w[i]))
        if run > u * total:
            return i, w[i] / total
    raise AssertionError("unreachable: u < 1")
