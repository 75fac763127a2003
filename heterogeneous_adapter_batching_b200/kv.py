"""KV cache of a served model in the pages of a lora_pool, and the metadata of a
step (device tensors only; every computation goes through the C-ABI calls in
_binding).

Page "Multi-LoRA Serving in Production" (llms.blog), section "Unified Paging
Architecture": KV-cache tensors and adapter weights share one pool of pages;
page "LoRA Adapters at Serve Time with vLLM Multi-LoRA", section "The Inference
Mechanism: A Worked Scenario": KV blocks are allocated per request, and every
step batches requests with adapters of their own."""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _binding as B


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """(inverse frequencies [rot_dim / 2] fp32 on the host, mscale) for lora_rope and lora_kv_append.

    scaling: None, or {"kind": ..., "factor": s, ...} for contexts s times as long as the model was trained on:
      "linear"   every position divided by s
      "ntk"      base raised to base * s^(rot_dim / (rot_dim - 2)): the slowest pair slowed by s, the fastest not at all
      "yarn"     pairs that turn fewer than beta_slow (1) times over original_max_position tokens slowed by s, those that
                 turn more than beta_fast (32) times kept, a ramp in the pair index between; mscale = 0.1 ln s + 1
      "bands"    pairs with wavelengths above original_max_position / low_freq_factor (1) slowed by s, below
                 original_max_position / high_freq_factor (4) kept, interpolated in between
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim is a positive even number")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = base ** (-i / rot_dim)
    if scaling is None:
        return f.float(), 1.0
    kind, s = scaling["kind"], float(scaling["factor"])
    if not 0.0 < s < math.inf:
        raise ValueError("factor is a positive number")
    if kind == "linear":
        return (f / s).float(), 1.0
    if kind == "ntk":
        if rot_dim == 2:
            raise ValueError("one pair has no slowest one beside the fastest")
        return ((base * s ** (rot_dim / (rot_dim - 2))) ** (-i / rot_dim)).float(), 1.0
    n = float(scaling["original_max_position"])
    if kind == "yarn":
        def pair(turns):   # the (fractional) pair that turns so many times over n tokens
            return rot_dim * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(scaling.get("beta_fast", 32.0))), 0)
        hi = min(math.ceil(pair(scaling.get("beta_slow", 1.0))), rot_dim - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return (f * (1 - ramp) + f / s * ramp).float(), 0.1 * math.log(s) + 1.0 if s > 1 else 1.0
    if kind == "bands":
        low, high = scaling.get("low_freq_factor", 1.0), scaling.get("high_freq_factor", 4.0)
        if not low < high:
            raise ValueError("low_freq_factor lies below high_freq_factor")
        keep = ((n * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return (f * keep + f / s * (1 - keep)).float(), 1.0
    raise ValueError(f"unknown scaling {kind!r}")


class KVCache:
    """A 4-bit KV cache in pages of `pool` (lora_pool_alloc_pages) and the device tensors of a step.

    One block of `block_tokens` tokens of one layer lives in a page; a model keeps one KVCache per layer (on one pool or
    several).  A request is a row of the block table: begin() runs lora_kv_layout over the rows' lengths, handing
    out reserved pages; append() and attend() (or prompt_attend()) are the layer's calls; free() gives the pages of
    finished rows back to the pool.  past_len says where the new tokens go: a row whose past has become shorter (drafts
    that were rejected, a step repeated after an error) fills the blocks it holds again before it takes any.  block_table
    and held go together: what clears a row is free().

    The calls of a step may be captured in a graph and replayed: every tensor keeps its place, reserve() and free()
    between replays included.  Steps of one KVCache follow one another on one stream (they share its workspace).
    Requests that bring more than max_q_len tokens in a step go through prompt_attend(); a step that mixes both kinds
    lists one kind behind the other and names the requests of each call (first, last).  prompt_attend() is for prompts
    from their first token on; a chunk over a cached past reads it back with lora_kv_gather for lora_prompt_attend."""

    def __init__(self, pool: B.Pool, q_heads: int, kv_heads: int, head_dim: int, block_tokens: int, max_requests: int,
                 max_len: int, max_tokens: int, max_q_len: int = 1, dtype=torch.bfloat16):
        page_bytes = B.PAGE_ROWS * pool.width * 2
        need = B.lora_kv_block_bytes(kv_heads, head_dim, block_tokens)
        if need == 0 or need > page_bytes:
            raise ValueError(f"a block needs {need} bytes, a page of the pool has {page_bytes}")
        self.pool, self.q_heads, self.kv_heads, self.head_dim = pool, q_heads, kv_heads, head_dim
        self.block_tokens, self.max_q_len, self.dtype = block_tokens, max_q_len, dtype
        n = B.lora_pool_num_pages(pool)
        self.pages = pool.buf.view(-1).view(torch.uint8)[:n * page_bytes].view(n, page_bytes)
        dev = self.device = pool.buf.device
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)  # noqa: E731
        self.block_table = i32(max_requests, -(-max_len // block_tokens)).fill_(-1)
        self.cu_new, self.kv_len = i32(max_requests + 1), i32(max_requests)
        self.positions, self.slots, self.ids = i32(max_tokens), i32(max_tokens), i32(max_tokens)
        # pages in reserve: free_list[head:], so that its end, which lora_kv_layout is told, never moves; held: blocks of each row
        self.free_list = i32(n)
        self._state, self._next = i32(1 + max_requests), i32(1 + max_requests)
        self.head, self._next_head, self.held = self._state[:1].fill_(n), self._next[:1].fill_(n), self._state[1:]
        self.rows, self._views = 0, None
        self.err = i32(1)
        self.ws = torch.empty(B.lora_kv_attend_workspace_size(q_heads, kv_heads, head_dim, max_q_len), dtype=torch.uint8,
                              device=dev)

    def reserve(self, n: int) -> None:
        """Take n pages of the pool for the steps to come.  Synchronises the device.  What is left of them when the object
        goes, free_list[head:], goes back through lora_pool_free_page_list."""
        torch.cuda.synchronize(self.device)
        ids = B.lora_pool_alloc_pages(self.pool, n)
        kept = self.free_list[int(self.head.item()):]
        both = torch.cat([kept, ids.to(self.device)])
        self.free_list[self.free_list.numel() - both.numel():] = both
        self.head.fill_(self.free_list.numel() - both.numel())
        torch.cuda.synchronize(self.device)

    def begin(self, past_len, new_len, req_ids=None, stream=None) -> None:
        """lora_kv_layout over rows 0 .. R-1 of the block table (past_len, new_len, req_ids [R] int32 on the device;
        past_len is not this object's kv_len, which the call writes)."""
        R = past_len.numel()
        table, cu_new, kv_len, held, held_out, state, after = self._slices(R)
        B.lora_kv_layout(past_len, new_len, req_ids, self.block_tokens, table, self.free_list, self.head, cu_new, kv_len,
                         self.positions, self.slots, self.ids, self._next_head, err=self.err, stream=stream, held=held,
                         held_out=held_out)
        if stream is None:
            state.copy_(after)
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=self.device)
            with torch.cuda.stream(stream):
                state.copy_(after)
        self.rows = R

    def append(self, q, k, v, inv_freq, q_out, k_out=None, v_out=None, interleaved=False, mscale=1.0, stream=None) -> None:
        T = k.shape[0]
        B.lora_kv_append(q, k, v, self.positions[:T], inv_freq, self.slots[:T], self.pages, self.block_tokens, q_out, k_out,
                         v_out, interleaved=interleaved, mscale=mscale, dtype=self.dtype, err=self.err, stream=stream)

    def _slices(self, R: int):
        """The tensors of a step of R requests; made once, as steps mostly have as many as the last."""
        own = (R, self.block_table, self.cu_new, self.kv_len)
        if self._views is None or any(a is not b for a, b in zip(self._views[0][1:], own[1:])) or self._views[0][0] != R:
            self._views = (own, (self.block_table[:R], self.cu_new[:R + 1], self.kv_len[:R], self.held[:R], self._next[1:1 + R],
                                 self._state[:1 + R], self._next[:1 + R]))
        return self._views[1]

    def _requests(self, first: int, last: Optional[int]):
        """(block table, row starts, lengths) of requests first .. last - 1 of the step; None if there are none."""
        if first == 0 and last is None:
            return self._slices(self.rows)[:3]
        last = self.rows if last is None else last
        if not 0 <= first <= last <= self.rows:
            raise ValueError(f"requests {first} .. {last} of a step of {self.rows}")
        return (self.block_table[first:last], self.cu_new[first:last + 1], self.kv_len[first:last]) if first < last else None

    def attend(self, q, out, scale: Optional[float] = None, lse=None, stream=None, first: int = 0,
               last: Optional[int] = None) -> None:
        """Attention of the new tokens of requests first .. last - 1 (all of the step) over the cache.  q, out and lse hold
        the rows of the whole step; those of other requests are left alone."""
        r = self._requests(first, last)
        if r:
            B.lora_kv_attend(q, self.pages, self.block_tokens, self.kv_heads, *r, self.max_q_len,
                             self.head_dim ** -0.5 if scale is None else scale, out, self.ws, lse=lse, err=self.err, stream=stream)

    def prompt_attend(self, q, k, v, out, scale: Optional[float] = None, lse=None, stream=None, first: int = 0,
                      last: Optional[int] = None) -> None:
        """Attention among the step's own rows for requests first .. last - 1 (all of the step), rows as in attend().  A
        request whose past is not empty sets LORA_DEV_ERR_BAD_LENGTH and its rows are left alone."""
        r = self._requests(first, last)
        if r:
            B.lora_prompt_attend_whole(q, k, v, r[1], r[2], self.head_dim ** -0.5 if scale is None else scale, out, lse=lse,
                                       err=self.err, stream=stream)

    def free(self, rows) -> None:
        """Return the pages of finished requests' rows to the pool and clear the rows.  Synchronises the device."""
        torch.cuda.synchronize(self.device)
        done = torch.zeros(self.block_table.shape[0], dtype=torch.bool)
        done[rows] = True                     # a row that is named twice is freed once
        held = self.block_table[done.to(self.device)].flatten().cpu()
        B.lora_pool_free_page_list(self.pool, held[held >= 0])
        self.block_table[done.to(self.device)] = -1
        self.held[done.to(self.device)] = 0
        torch.cuda.synchronize(self.device)
