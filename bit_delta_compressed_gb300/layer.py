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

import contextlib

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


def _held(name: str):
    """A tensor that stays in its place: what is assigned to it is copied into it."""
    return property(lambda self: getattr(self, name), lambda self, t: getattr(self, name).copy_(t))


class CachedAttention:
    """One layer's key/value cache and the attention on it.

    k, v : bf16 [slots, capacity, kv_heads, head_dim]; lens : int32 [slots], the
    keys of every slot; weights : f32 [slots, kv_heads, capacity], what decode
    steps gave each key (None unless ``weigh``; a prompt's own queries give none).  All on the device: a decode
    step can be captured in a CUDA graph.  A shared prefix lies in a slot of its
    own, filled by ``prefill`` like any other.

    A request whose slot is not there, or has no room for all its new tokens, is
    left as it is: nothing is appended, its rows come out as zeros, and the status
    word of ``ws`` holds ``BD_ERR_SLOT``."""

    k, v, lens, weights = _held("_k"), _held("_v"), _held("_lens"), _held("_weights")

    def __init__(self, bd, slots: int, capacity: int, q_heads: int, kv_heads: int, head_dim: int, tokens: int,
                 batch: int, window: int = 0, sinks: int = 0, weigh: bool = False, device="cuda"):
        import torch
        self.bd, self.torch = bd, torch
        self.heads = (q_heads, kv_heads, head_dim)
        self.mask = {"window": window, "sinks": sinks}
        # Behind the cache's places lies one more key, and a slot that is always full: what
        # has no place of its own goes there, so that no index leaves its tensor (on a GPU
        # that ends the context) and no step waits for the host.
        shape = (slots, capacity, kv_heads, head_dim)
        self.rows_k = torch.zeros(slots * capacity + 1, kv_heads, head_dim, dtype=torch.bfloat16, device=device)
        self.rows_v = torch.zeros_like(self.rows_k)
        self._k, self._v = self.rows_k[:-1].view(shape), self.rows_v[:-1].view(shape)
        self.slot_lens = torch.zeros(slots + 1, dtype=torch.int32, device=device)
        self.slot_lens[-1] = capacity
        self._lens = self.slot_lens[:-1]
        self._weights = None
        if weigh:
            self.slot_weights = torch.zeros(slots + 1, kv_heads, capacity, device=device)
            self._weights = self.slot_weights[:-1]
            self.zero = torch.zeros((), device=device)
        self.ws = bd.attn_workspace(tokens, batch, q_heads, kv_heads, head_dim, capacity if weigh else 0, device)
        self.evict_ws = bd.evict_workspace(batch, kv_heads, capacity, device)

    def _slots(self, slots):
        """Places in ``slot_lens``: those of no slot (-1 and ``slots``) are the one behind."""
        return slots.clamp(-1, self.lens.shape[0]).long()

    def _append(self, k, v, place):
        """Rows of k and v become the keys at ``place``, counted through all slots (-1: the one behind)."""
        _, hk, d = self.heads
        self.rows_k[place] = k.view(-1, hk, d)
        self.rows_v[place] = v.view(-1, hk, d)
        if self.weights is not None:
            capacity = self.k.shape[1]
            # (a number would be copied from the host, which the capture of a graph refuses)
            self.slot_weights[place // capacity, :, place % capacity] = self.zero

    @contextlib.contextmanager
    def _given_back(self, to, have):
        """The lengths before the step, if its attention call is refused."""
        try:
            yield
        except Exception:
            self.slot_lens[to] = have
            raise

    def _prefix_lens(self, prefix_slots):
        return None if prefix_slots is None else self.slot_lens[self._slots(prefix_slots)]

    def decode(self, q, k, v, slots, prefix_ids=None, prefix_slots=None):
        """One token for each request: its slot in ``slots`` (int32 [M], none twice); requests
        may name shared prefixes by their index in ``prefix_slots``."""
        torch, capacity = self.torch, self.k.shape[1]
        hq, _, d = self.heads
        to = self._slots(slots)
        have = self.slot_lens[to]
        self._append(k, v, torch.where(have < capacity, torch.add(have, to, alpha=capacity), -1))
        lens = have + 1                           # beyond a full slot's capacity: the call below reports it
        self.slot_lens[to] = lens.clamp_max(capacity)
        with self._given_back(to, have):
            out = self.bd.attn_decode_prefix(q.view(-1, hq, d), self.k, self.v, lens, prefix_ids, prefix_slots,
                                             self._prefix_lens(prefix_slots), self.ws, slots=slots, weights=self.weights,
                                             **self.mask)
        return out.view(-1, hq * d)

    def prefill(self, q, k, v, slots, cu_q, prefix_ids=None, prefix_slots=None):
        """The next tokens of some requests: rows ``cu_q[b]`` to ``cu_q[b + 1]`` are
        the request's in slot ``slots[b]``.  Rows of no request are not written."""
        torch, capacity = self.torch, self.k.shape[1]
        hq, _, d = self.heads
        T = q.shape[0]
        to = self._slots(slots)
        have = self.slot_lens[to]
        # requests from the first whose offsets do not ascend on are not served (as the
        # library's call has it), nor those whose tokens the slot has no room for
        steady = cu_q.clamp(0, T).cummax(0).values
        served = (steady == cu_q).cumprod(0, dtype=torch.int32)[1:]
        lens = have + (cu_q[1:] - cu_q[:-1]) * served
        fits = (lens <= capacity) & (served > 0)
        # a request's first place less its first row; far below zero for rows that are appended nowhere
        start = torch.where(fits, torch.add(have, to, alpha=capacity) - cu_q[:-1], -1 << 40)
        start = torch.nn.functional.pad(start, (1, 1), value=-1 << 40)
        row = torch.arange(T, dtype=torch.int32, device=q.device)
        self._append(k, v, (start[torch.searchsorted(steady, row, right=True)] + row).clamp_min_(-1))
        self.slot_lens[to] = torch.where(fits, lens, have)
        with self._given_back(to, have):
            out = self.bd.attn_prefill(q.view(-1, hq, d), self.k, self.v, cu_q, lens, self.ws, slots=slots,
                                       prefix_ids=prefix_ids, prefix_slots=prefix_slots,
                                       prefix_lens=self._prefix_lens(prefix_slots), **self.mask)
        return out.view(-1, hq * d)

    def evict(self, src, dst, budget: int, recent: int, sinks: int | None = None) -> None:
        """Move requests from slots ``src`` to the free slots ``dst`` with at most
        ``budget`` keys a head, the first ``sinks`` and the last ``recent`` among them.

        ``sinks``: how many of the mask's first tokens are own keys of these requests:
        all of them (None) without a prefix, max(0, mask's - P) behind one of P keys --
        the rest lie in the prefix, and own keys kept in their stead would take the
        places of heavier ones.

        A kept key stands at its new place from then on, nearer to the keys to come
        than it was.  So that none comes back into the window, it has to lie among
        the keys that stay: ``recent`` >= window - 1 (the next query sees itself and
        as many before it)."""
        window = self.mask["window"]
        if window > 0 and recent < window - 1:
            raise ValueError("recent must be at least window - 1 (%d): keys that left the window would come back into it"
                             % (window - 1))
        self.bd.cache_evict(self.k, self.v, self.weights, self.lens, src, dst, budget, self.evict_ws,
                            sinks=self.mask["sinks"] if sinks is None else sinks, recent=recent)
