"""64-bit references of the KV-cache and attention calls, and the error bounds
their results are held to.  Plain numpy / torch on the CPU, loops where they are
clearest; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

GRANULE, GROUP = 16, 64
# half a step of a type relative to the value (rounding to nearest), and half its least step
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def block_bytes(heads, dim, block):
    return heads * (block // GRANULE) * 2 * (GRANULE * dim // 2 + GRANULE * 4 * (dim // GROUP))


def layout(past, new, req_ids, T, block, table, free, head):
    """The outputs of lora_kv_layout as a dict of numpy arrays, request by request; free None: the table is complete."""
    R, width = table.shape
    table = table.copy()
    cu, kv_len = [0], []
    pos, slots, ids = (np.full(T, -1, dtype=np.int64) for _ in range(3))
    at, dry, taken, err = head, False, 0, 0
    for r in range(R):
        p, n = int(past[r]), int(new[r])
        rows = max(n, 0)
        bad = p < 0 or n < 0 or p + n > width * block
        start, end = cu[-1], min(cu[-1] + rows, T)
        cut = cu[-1] + rows > T and rows > 0
        before, after = -(-p // block), -(-(p + n) // block)
        need = 0 if bad or free is None else after - before
        dry = dry or (need > 0 and at + need > len(free))
        failed = bad or cut or (need > 0 and dry)
        err |= 32 if bad or cut else (16 if failed else 0)
        if not failed and need:
            table[r, before:after] = free[at:at + need]
            taken = at + need - head
        at += need
        kv_len.append(0 if failed else p + n)
        cu.append(end)
        if failed:
            continue
        for i in range(n):
            page = table[r, (p + i) // block]
            pos[start + i] = p + i
            slots[start + i] = page * block + (p + i) % block if page >= 0 else -1
            err |= 8 if page < 0 else 0
            ids[start + i] = -1 if req_ids is None else req_ids[r]
    return {"table": table, "cu": np.array(cu), "kv_len": np.array(kv_len), "positions": pos, "slots": slots, "ids": ids,
            "head": head + taken, "err": err}


def rotate(x, pos, freq, mscale, interleaved):
    """x [T, H, D] (any type) rotated in 64 bits."""
    x = x.double().cpu().clone()
    n = 0 if freq is None else freq.numel()
    if n == 0:
        return x
    ang = pos.double().cpu()[:, None] * freq.double().cpu()[None, :]
    c, s = (ang.cos() * mscale)[:, None], (ang.sin() * mscale)[:, None]
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    u, v = x[..., a], x[..., b]
    x[..., a], x[..., b] = u * c - v * s, v * c + u * s
    return x


def quantise(x):
    """codes [T, H, D] and fp16 (step, low) [T, H, D/64] of values x (held in their row type), every rounding from the exact value."""
    x = x.double().cpu().numpy()
    T, H, D = x.shape
    g = x.reshape(T, H, D // GROUP, GROUP)
    with np.errstate(all="ignore"):
        low = g.min(-1).astype(np.float32).astype(np.float16)
        step = ((g.max(-1) - g.min(-1)) / 15).astype(np.float32).astype(np.float16)
        s = step.astype(np.float64)[..., None]
        n = np.where(s > 0, np.rint((g - low.astype(np.float64)[..., None]) / np.where(s > 0, s, 1)), 0)
        n = np.clip(np.nan_to_num(n, nan=0.0), 0, 15)
    return n.reshape(T, H, D).astype(np.uint8), step, low


def value(codes, step, low):
    """What codes stand for, n * step + low rounded once to fp32."""
    with np.errstate(all="ignore"):
        n = codes.astype(np.float64) * np.repeat(step.astype(np.float64), GROUP, -1) + np.repeat(low.astype(np.float64), GROUP, -1)
        return n.astype(np.float32)


class Cache:
    """A host copy of a cache: pages [N, page_bytes] uint8."""

    def __init__(self, pages, heads, dim, block):
        self.b, self.heads, self.dim, self.block = pages, heads, dim, block
        self.half = GRANULE * dim // 2 + GRANULE * 4 * (dim // GROUP)

    def _where(self, slot, h, which):
        page, off = slot // self.block, slot % self.block
        g = (h * (self.block // GRANULE) + off // GRANULE) * 2 * self.half + which * self.half
        row = off % GRANULE
        codes = slice(g + row * self.dim // 2, g + (row + 1) * self.dim // 2)
        p = g + GRANULE * self.dim // 2 + row * 4 * (self.dim // GROUP)
        return page, codes, slice(p, p + 4 * (self.dim // GROUP))

    def write(self, slot, h, which, codes, step, low):
        page, c, p = self._where(slot, h, which)
        self.b[page, c] = codes[0::2] | (codes[1::2] << 4)
        self.b[page, p] = np.stack([step, low], -1).astype(np.float16).reshape(-1).view(np.uint8)

    def read(self, slot, h, which):
        """(codes [D], step [D/64], low [D/64])."""
        page, c, p = self._where(slot, h, which)
        codes = np.empty(self.dim, dtype=np.uint8)
        codes[0::2], codes[1::2] = self.b[page, c] & 15, self.b[page, c] >> 4
        par = self.b[page, p].copy().view(np.float16).reshape(-1, 2)
        return codes, par[:, 0], par[:, 1]


def cached_kv(cache, table, n, h):
    """float64 k, v [n, D] of the first n tokens of a request with block list `table`, and per token the largest step of k."""
    k, v, step = np.zeros((n, cache.dim)), np.zeros((n, cache.dim)), np.zeros(n)
    for j in range(n):
        slot = int(table[j // cache.block]) * cache.block + j % cache.block
        for which, out in ((0, k), (1, v)):
            c, s, lo = cache.read(slot, h, which)
            out[j] = c.astype(np.float64) * np.repeat(s.astype(np.float64), GROUP) + np.repeat(lo.astype(np.float64), GROUP)
            if which == 0:
                step[j] = s.astype(np.float64).max()
    return k, v, step


def attend_row(q, k, v, scale):
    """softmax(scale q k^T) v in 64 bits -> (out [D], lse, sum p |v| / sum p)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1])
    s = (k @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    return p @ v / p.sum(), m + math.log(p.sum()), p @ np.abs(v) / p.sum()


def row_bound(q, k, scale, step=None):
    """Bound of the error of one fp32 score: D products and sums, each off by at most 2^-24 of the sum of magnitudes (with slack
    for the order of sums and a truncating accumulator, 2^-22), on codes offset by up to 128 steps where `step` is given."""
    if k.shape[0] == 0:
        return 0.0
    mag = np.abs(k) + (0 if step is None else 144 * step[:, None])
    return float((mag @ np.abs(q)).max() * abs(scale) * (k.shape[1] + 16) * 2.0 ** -22)


def out_bound(o, absv, delta, dtype, p_half):
    """Error bound of a row of outputs: each weight is off by a factor within p_half + delta (its rounding, its score, the
    exponential's 2^-21), numerator and denominator alike, and the result is rounded to `dtype`."""
    rel = 2 * (p_half + math.expm1(2 * delta) + 2.0 ** -21) + 64 * 2.0 ** -24
    return HALF[dtype] * np.abs(o) * (1 + 2.0 ** -6) + rel * absv + TINY[dtype]
