"""A decoder layer's seven linears chained as one decode step.

Page: "BitDelta: serving 14 Zen models from one GPU cluster", section
"Serving architecture": every linear of a variant's forward pass runs as the
fused multi-variant linear against the shared base weights.  This module
chains one layer's projections the way a decoder layer feeds them, with the
glue between them in plain torch:

    q, k, v = L_q(h), L_k(h), L_v(h)
    o       = L_o(attend(q, k, v))   (without an ``attend``, q stands in for the
                                 attention output: the attention arithmetic is
                                 not part of the method)
    h1      = h + o
    a       = silu(L_gate(h1)) * L_up(h1)
    h2      = h1 + L_down(a)

All tokens of the batch keep their variant through the layer, so the batch is
grouped once (``bd.group``) and every projection runs through
``bd.linear_grouped`` on that grouping.

``CachedAttention`` is an ``attend`` on a key/value cache: it appends the step's
keys and values (plain torch) and runs the library's attention on them, decode
or prefill, with shared prefixes, a window, and eviction to a budget.  Rotating
q and k by position, where a model does, is its caller's.
"""
from __future__ import annotations

NAMES = ("q", "k", "v", "o", "gate", "up", "down")


def chained_layer(bd, lin: dict, h, V: int, ws, bufs: dict, path: str = "auto", keep: bool = False,
                  attend=None):
    """One layer on the hidden states ``h`` [M, hidden] (bf16).

    ``lin`` maps each name in ``NAMES`` to a dict with ``wb`` (bf16 [N, K]),
    ``alphas`` (f32 [V]) and ``ptrs`` (from ``bd.bits_pointer_array``);
    ``bufs`` maps each name to a preallocated bf16 output [M, N].  The batch
    must already be grouped in ``ws``.  ``attend``: None, or a function of the q, k
    and v projections that gives the attention output [M, q_heads * head_dim].
    Returns h2, and with ``keep`` also the
    dict of every projection's input and output."""
    import torch

    def proj(name, x):
        L = lin[name]
        bd.linear_grouped(x, L["wb"], L["alphas"], L["ptrs"], V, bufs[name], ws, path=path)
        return bufs[name]

    q = proj("q", h)
    proj("k", h)
    proj("v", h)
    mixed = q if attend is None else attend(q, bufs["k"], bufs["v"])
    o = proj("o", mixed)
    h1 = h + o
    g = proj("gate", h1)
    u = proj("up", h1)
    a = torch.nn.functional.silu(g) * u
    d = proj("down", a)
    h2 = h1 + d
    if not keep:
        return h2
    return h2, {"q": (h, q), "k": (h, bufs["k"]), "v": (h, bufs["v"]), "o": (mixed, o), "h1": h1,
                "gate": (h1, g), "up": (h1, u), "down": (a, d)}


class CachedAttention:
    """One layer's key/value cache and the attention on it.

    k, v : bf16 [slots, capacity, kv_heads, head_dim]; lens : int32 [slots], the
    keys of every slot; weights : f32 [slots, kv_heads, capacity], what decode
    steps gave each key (None unless ``weigh``).  All on the device: a decode
    step can be captured in a CUDA graph.  A shared prefix lies in a slot of its
    own, filled by ``prefill`` like any other."""

    def __init__(self, bd, slots: int, capacity: int, q_heads: int, kv_heads: int, head_dim: int, tokens: int,
                 batch: int, window: int = 0, sinks: int = 0, weigh: bool = False, device="cuda"):
        import torch
        self.bd, self.torch = bd, torch
        self.heads = (q_heads, kv_heads, head_dim)
        self.mask = {"window": window, "sinks": sinks}
        shape = (slots, capacity, kv_heads, head_dim)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.lens = torch.zeros(slots, dtype=torch.int32, device=device)
        self.weights = torch.zeros(slots, kv_heads, capacity, device=device) if weigh else None
        self.ws = bd.attn_workspace(tokens, batch, q_heads, kv_heads, head_dim, capacity if weigh else 0, device)
        self.evict_ws = bd.evict_workspace(batch, kv_heads, capacity, device)

    def _append(self, k, v, slots, at):
        _, hk, d = self.heads
        self.k[slots, at] = k.view(-1, hk, d)
        self.v[slots, at] = v.view(-1, hk, d)
        if self.weights is not None:
            self.weights[slots, :, at] = 0

    def decode(self, q, k, v, slots, prefix_ids=None, prefix_slots=None):
        """One token for each request: its slot in ``slots`` (int32 [M]); requests
        may name shared prefixes by their index in ``prefix_slots``."""
        hq, _, d = self.heads
        to = slots.long()
        self._append(k, v, to, self.lens[to].long())
        self.lens[to] += 1
        lens = self.lens[to]
        plens = None if prefix_slots is None else self.lens[prefix_slots.long()]
        out = self.bd.attn_decode_prefix(q.view(-1, hq, d), self.k, self.v, lens, prefix_ids, prefix_slots, plens,
                                         self.ws, slots=slots, weights=self.weights, **self.mask)
        return out.view(-1, hq * d)

    def prefill(self, q, k, v, slots, cu_q, prefix_ids=None, prefix_slots=None):
        """The next tokens of some requests: rows ``cu_q[b]`` to ``cu_q[b + 1]`` are
        the request's in slot ``slots[b]``."""
        torch = self.torch
        hq, _, d = self.heads
        rows = torch.arange(q.shape[0], device=q.device)
        of = torch.searchsorted(cu_q[1:].contiguous(), rows.to(torch.int32), right=True)
        to = slots.long()
        self._append(k, v, to[of], self.lens[to].long()[of] + rows - cu_q.long()[of])
        self.lens[to] += cu_q[1:] - cu_q[:-1]
        plens = None if prefix_slots is None else self.lens[prefix_slots.long()]
        out = self.bd.attn_prefill(q.view(-1, hq, d), self.k, self.v, cu_q, self.lens[to], self.ws, slots=slots,
                                   prefix_ids=prefix_ids, prefix_slots=prefix_slots, prefix_lens=plens, **self.mask)
        return out.view(-1, hq * d)

    def evict(self, src, dst, budget: int, recent: int) -> None:
        """Move requests from slots ``src`` to the free slots ``dst`` with at most
        ``budget`` keys a head; the mask's first tokens stay."""
        self.bd.cache_evict(self.k, self.v, self.weights, self.lens, src, dst, budget, self.evict_ws,
                            sinks=self.mask["sinks"], recent=recent)
