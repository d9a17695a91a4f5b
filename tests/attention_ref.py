"""Attention over a key/value cache in 64 bits, from the definition: a plain
implementation for the tests, and the error bounds that the kernels' arithmetic
allows."""
from __future__ import annotations

import math

import torch

# A bf16 value has 8 significant bits: neighbours are 2^-7 of a power of two apart, and
# rounding to nearest is off by at most 2^-8 of the value.
BF16 = 2.0 ** -8
F32 = 2.0 ** -24


def visible(pos, t, window, sinks):
    """[rows, keys]: whether a query at position t sees position pos."""
    seen = pos[None, :] <= t[:, None]
    if window:
        seen &= (pos[None, :] > t[:, None] - window) | (pos[None, :] < sinks)
    return seen


def attention(q, k, v, lens, *, slots=None, cu_q=None, window=0, sinks=0, scale=None, prefix_ids=None,
              prefix_slots=None, prefix_lens=None, rounded=None):
    """(out, bound, weights): out f64 [rows, q_heads, d]; `bound` what each value
    may be off by; weights {b: f64 [kv_heads, len]} summed over the rows."""
    T, Hq, D = q.shape
    Hk = k.shape[2]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    # prefill and prefixes multiply probabilities rounded to bf16, decode nearly exact ones
    rounded = cu_q is not None or prefix_ids is not None if rounded is None else rounded
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    weights, weight_rel = {}, {}
    for b, L in enumerate(lens.tolist()):
        r0, r1 = (b, b + 1) if cu_q is None else (int(cu_q[b]), int(cu_q[b + 1]))
        slot = b if slots is None else int(slots[b])
        P = 0
        pid = -1 if prefix_ids is None else int(prefix_ids[b])
        if pid >= 0:
            P = int(prefix_lens[pid])
        kk, vv = k[slot, :L].double(), v[slot, :L].double()
        if P:
            ps = int(prefix_slots[pid])
            kk, vv = torch.cat([k[ps, :P].double(), kk]), torch.cat([v[ps, :P].double(), vv])
        weights[b] = torch.zeros(Hk, L, dtype=torch.float64, device=q.device)
        n = P + L
        if n == 0 or r1 == r0:
            continue
        t = torch.arange(n - (r1 - r0), n, device=q.device)
        mask = visible(torch.arange(n, device=q.device), t, window, sinks)
        used = mask.any(0)
        kk, vv = torch.where(used[:, None, None], kk, 0.0), torch.where(used[:, None, None], vv, 0.0)
        for h in range(Hk):
            qq = q[r0:r1, h * G:(h + 1) * G].double()                      # [r, G, D]
            s = torch.einsum("rgd,nd->rgn", qq, kk[:, h]) * scale
            size = torch.einsum("rgd,nd->rgn", qq.abs(), kk[:, h].abs()) * abs(scale)
            s = s.masked_fill(~mask[:, None], -math.inf)
            m = s.amax(-1, keepdim=True)
            e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            l = e.sum(-1, keepdim=True)
            p = torch.where(l > 0, e / l, 0.0)
            out[r0:r1, h * G:(h + 1) * G] = torch.einsum("rgn,nd->rgd", p, vv[:, h])
            amount = torch.einsum("rgn,nd->rgd", p, vv[:, h].abs())
            # One rounding of the result to bf16, and where p is rounded one of each p.  In f32: a product sum of D
            # terms is off by (D + 2) 2^-24 of its terms' sizes, which exp() turns into a
            # relative error of p -- of the score's and of the sum's, hence twice -- and a
            # few more roundings: the exponential, the sum, the division.
            rel = 2 * (D + 2) * F32 * float((size * mask[:, None]).amax()) + 64 * F32
            bound[r0:r1, h * G:(h + 1) * G] = ((2 if rounded else 1) * BF16 * (1 + BF16 / 2) + 4 * rel) * amount
            weights[b][h] = p.sum((0, 1))[P:]
            weight_rel[b] = max(weight_rel.get(b, 0.0), 2 * rel)
    return out, bound, (weights, weight_rel)


def hide_unseen(k, v, lens, fill, *, rows=None, slots=None, window=0, sinks=0, prefix_ids=None, prefix_slots=None,
                prefix_lens=None):
    """Overwrite with `fill` every cached value that no query of the call sees."""
    used = torch.zeros(k.shape[:2], dtype=torch.bool, device=k.device)
    for b, L in enumerate(lens.tolist()):
        slot = b if slots is None else int(slots[b])
        P = 0
        pid = -1 if prefix_ids is None else int(prefix_ids[b])
        if pid >= 0:
            P = int(prefix_lens[pid])
        n, r = P + L, 1 if rows is None else int(rows[b])
        if n == 0 or r == 0:
            continue
        seen = visible(torch.arange(n, device=k.device), torch.arange(n - r, n, device=k.device), window, sinks).any(0)
        used[slot, :L] |= seen[P:]
        if P:
            used[int(prefix_slots[pid]), :P] |= seen[:P]
    k[~used] = fill
    v[~used] = fill


def assert_close(out, ref, bound, what=""):
    err = (out.double() - ref).abs()
    assert torch.isfinite(out.float()).all(), what + ": non-finite output"
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 1e-30, "%s: %.3e beyond its bound (largest error %.3e)" % (what, worst, err.max().item())


def evict(weights, lens, src, budget, sinks, recent):
    """Kept places of each (request, head), by sorting: [[list of int]]."""
    kept = []
    for s in src.tolist():
        n = int(lens[s])
        rows = []
        for h in range(weights.shape[1]):
            w = weights[s, h, :n].tolist()

            def rank(j):
                if j < sinks or j >= n - recent:
                    return (0, 0.0, j)
                return (1, -math.inf if math.isnan(w[j]) else -w[j], 0 if math.isnan(w[j]) else 1, j)
            order = sorted(range(n), key=rank)
            rows.append(sorted(order[:min(n, budget)]))
        kept.append(rows)
    return kept
