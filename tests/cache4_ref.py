"""The 4-bit cache from its definition, in 64 bits and byte by byte: what a cache stands
for, what it stands for after a write, and the bounds of the attention on it."""
from __future__ import annotations

import torch

from tests import attention_ref

CODES = 184                                   # scales up to 240
NAN_CODE = 255


def scale_table(device):
    table = [c / 8 * 2.0 ** -14 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 15) for c in range(248)]
    return torch.tensor(table + [float("inf")] + [float("nan")] * 7, dtype=torch.float64, device=device)   # exponent 31, as in f16


def quantise(x):
    """(n + 8 int64 [.., D], scale codes int64 [.., D / 32]) of bf16 values [.., D]."""
    x = x.double().unflatten(-1, (-1, 32))
    odd = ~torch.isfinite(x).all(-1)
    table = scale_table(x.device)[:CODES].contiguous()
    want = (torch.where(odd[..., None], 0.0, x).abs().amax(-1) / 7).clamp_max(240.0)
    above = torch.searchsorted(table, want).clamp(0, CODES - 1)
    below = (above - 1).clamp_min(0)
    up, down = table[above] - want, want - table[below]
    code = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    s = table[code][..., None]
    n = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0).round().clamp(-7, 7)
    n = torch.where(odd[..., None], 0.0, n)   # whatever they are: the scale makes NaN of them
    return (n + 8).long().flatten(-2), torch.where(odd, NAN_CODE, code)


def as_held(x):
    """What a cache stands for once x has been written."""
    n, code = quantise(x)
    return ((n - 8).double().unflatten(-1, (-1, 32)) * scale_table(x.device)[code][..., None]).flatten(-2)


def spots(d, j, which):
    """Where dims 0 .. d - 1 of token j of a block lie, keys (0) or values (1): the two bytes
    of their unit and the field, and the scale's byte."""
    e = torch.arange(d)
    if which == 0:
        return j * (d // 2) + e // 8 * 4 + e % 2 * 2, e % 8 // 2, 16 * d + j * (d // 32) + e // 32
    return 8 * d + j // 2 * d + e // 4 * 4 + j % 2 * 2, e % 4, 16 * d + d // 2 + e // 32 * 16 + j


def held(cache):
    """What a cache [slots, heads, blocks, 17 d] stands for: k, v f64 [slots, tokens, heads, d]."""
    d, dev = cache.shape[-1] // 17, cache.device
    table, result = scale_table(dev), []
    for which in (0, 1):
        tokens = []
        for j in range(16):
            byte, field, code = (t.to(dev) for t in spots(d, j, which))
            low, high = cache[..., byte].long(), cache[..., byte + 1].long()
            unit = torch.where(field < 2, low + 256 * high, high + 256 * low)
            n = torch.where(field % 2 == 0, unit // 64, unit // 4) % 16 - 8
            tokens.append(n * table[cache[..., code].long()])
        result.append(torch.stack(tokens, -2).flatten(2, 3).transpose(1, 2))
    return result


def put(cache, slot, place, k, v):
    """Writes one token, k and v [heads, d], as the definition has it; on the CPU."""
    d, block, j = cache.shape[-1] // 17, place // 16, place % 16
    for which, x in ((0, k), (1, v)):
        n, code = quantise(x)
        byte, field, _ = spots(d, j, which)
        unit = torch.zeros(x.shape[0], d * 16 // 64, 4, dtype=torch.long)
        order = torch.argsort(byte * 4 + field)          # dims by unit, then by field
        unit[:] = n[:, order].unflatten(1, (-1, 4))
        plain = unit[..., 0] << 6 | unit[..., 1] << 2
        turned = unit[..., 2] << 6 | unit[..., 3] << 2
        word = plain | (turned & 255) << 8 | turned >> 8
        at = byte[order].unflatten(0, (-1, 4))[:, 0]
        cache[slot, :, block, at] = (word & 255).to(torch.uint8)
        cache[slot, :, block, at + 1] = (word >> 8).to(torch.uint8)
        scales = spots(d, j, which)[2][::32]
        cache[slot, :, block, scales] = code.to(torch.uint8)


def write(cache, k, v, lens, slots, cu_q=None):
    """The cache, on the CPU, after a write of rows k, v [T, heads, d]."""
    cache = cache.cpu().clone()
    k, v = k.cpu(), v.cpu()
    ends = list(range(len(lens) + 1)) if cu_q is None else [int(x) for x in cu_q]
    for b, (length, slot) in enumerate(zip(lens, slots)):
        for row in range(ends[b], ends[b + 1]):
            put(cache, slot, length - ends[b + 1] + row, k[row], v[row])
    return cache


def hide(cache, used):
    """Overwrites with 0xFF (scales that are NaN) the tokens that are not `used` [slots, tokens]."""
    d = cache.shape[-1] // 17
    for j in range(16):
        at = torch.cat([torch.cat([byte, byte + 1, code]) for byte, _, code in (spots(d, j, 0), spots(d, j, 1))]).unique().to(cache.device)
        slot, block = (~used.unflatten(1, (-1, 16))[:, :, j]).nonzero(as_tuple=True)
        cache[slot[:, None, None], torch.arange(cache.shape[1], device=cache.device)[:, None], block[:, None, None], at] = 255


def hide_unseen(cache, lens, *, rows=None, slots=None, window=0, sinks=0):
    """Overwrites every token that no query of the call sees."""
    used = torch.zeros(cache.shape[0], cache.shape[2] * 16, dtype=torch.bool, device=cache.device)
    for b, n in enumerate(lens.tolist()):
        r = 1 if rows is None else int(rows[b])
        if n and r:
            pos = torch.arange(n, device=cache.device)
            used[b if slots is None else int(slots[b]), :n] |= attention_ref.visible(pos, pos[n - r:], window, sinks).any(0)
    hide(cache, used)


def attention(q, cache, lens, **how):
    """(out, bound) of attention on what the cache stands for.

    Decode multiplies probabilities rounded to f16, in the sum that divides as in the product, so the
    result is off by 2 x 2^-11 of the sum of |p v| for them; that sum is at most `bound` / 2^-8 of the bf16 cache's
    bound, which counts one bf16 rounding of it.  Probabilities below 2^-14 lose bits, 2^-25 each at most
    where the largest one is 2^6 or more: 2^-31 of it, and so of the sum, for each key.

    A prompt call of few rows is served by the same arithmetic, row by row: 2 x 2^-11 is less than the bf16 rounding of
    the probabilities that its bound counts, and the last term is added."""
    k, v = held(cache)
    out, bound, _ = attention_ref.attention(q, k, v, lens, **how)
    keys = lens.double()[:, None, None]
    if how.get("cu_q") is None:
        bound = bound * (1 + 2 * 2.0 ** -11 * (1 + 2.0 ** -11) / attention_ref.BF16)
    else:
        keys = lens.max() if lens.numel() else 0
    largest = torch.nan_to_num(v.abs(), nan=0.0).amax() if v.numel() else 0.0
    return out, bound + keys * 2.0 ** -31 * largest
