"""The attention-side operators of a multi-LoRA serving step, as cases to measure.

The adapter branch leaves query, key and value rows in fp32; the page pool has
pages for a KV cache.  The operators here take a step from there:

  layout   block tables, slot maps, positions and per-token adapter ids built
           on the GPU from request lengths (lora_kv_layout)
  rope     rotary positions of query and key rows (lora_rope)
  append   rotary positions, then keys and values written to cache pages in
           4 bits (lora_kv_append), and the written tokens read back
           (lora_kv_gather)
  attend   attention of one or a few new tokens per request over the paged
           4-bit cache (lora_kv_attend)
  prompt   causal attention over packed prompts of different lengths with
           grouped heads (lora_prompt_attend)

`own` chooses between the framework's entry points and the plain forms below.

The 4-bit cache.  A block of `block` tokens (a multiple of 16) lives in one
page: [kv head][block / 16 granules][granule].  A granule holds 16 tokens of
one head: K codes [16][D/2] bytes, K parameters [16][D/64] pairs of fp16
(step, low), V codes, V parameters.  Byte j of a code row holds dimension 2j in
its low half and 2j + 1 in its high half; a group of 64 dimensions shares one
pair, and a code n stands for n * step + low.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64            # dimensions that share a (step, low) pair
GRANULE = 16          # tokens of one head stored together
WORKSPACE_BYTES = 32 << 20
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a running batch: every request brings one token
        {"name": "layout decode 64", "op": "layout", "requests": 64, "rows": 64, "block": 16, "chunk": 1, "max_past": 8192},
        # a large mixed step: most requests decode, some bring prompt chunks, padded to a captured graph's rows
        {"name": "layout mixed 1024", "op": "layout", "requests": 1024, "rows": 16384, "block": 64, "chunk": 509, "max_past": 32768},
        # q and k of 16 decoding requests, 8B head layout, straight from the fp32 projections
        {"name": "rope decode 16", "op": "rope", "tokens": 16, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
         "interleaved": False, "src": "fp32", "dtype": "bf16", "max_pos": 131072, "factor": 8.0},
        # a prompt batch, 7B layout (one kv head per query head), interleaved pairs over half of each head
        {"name": "rope prompts 7B", "op": "rope", "tokens": 8191, "q_heads": 32, "kv_heads": 32, "head_dim": 128, "rot": 64,
         "interleaved": True, "src": "bf16", "dtype": "bf16", "max_pos": 1000000, "factor": 1.0},
        # decode: one token of each of 256 requests enters the cache
        {"name": "append decode 256", "op": "append", "tokens": 256, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
         "interleaved": False, "src": "fp32", "dtype": "bf16", "max_pos": 32768, "factor": 1.0, "block": 64, "dense": False},
        # prompts: the same for a packed batch of 8101 prompt tokens, with the dense keys and values that prompt attention reads
        {"name": "append prompts", "op": "append", "tokens": 8101, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
         "interleaved": False, "src": "fp32", "dtype": "bf16", "max_pos": 8192, "factor": 1.0, "block": 64, "dense": True},
        # one user with a long context: latency
        {"name": "attend 1 x 32749", "op": "attend", "requests": 1, "q_len": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "block": 64, "dtype": "bf16", "min_len": 32749, "max_len": 32749},
        # a batch of ragged contexts: bandwidth
        {"name": "attend 128 ragged", "op": "attend", "requests": 128, "q_len": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "block": 64, "dtype": "bf16", "min_len": 1, "max_len": 16384},
        # verifying up to 4 drafted tokens per request, small pages
        {"name": "attend drafts fp16", "op": "attend", "requests": 48, "q_len": 4, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "block": 16, "dtype": "fp16", "min_len": 257, "max_len": 4096},
        # many short prompts in one step, small heads
        {"name": "prompt 24 short fp16", "op": "prompt", "requests": 24, "min_len": 1, "max_len": 97, "prefix": 0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 64, "dtype": "fp16", "fused": True},
        # 16 prompts of 128 to 2048 tokens, 8B layout
        {"name": "prompt 16 ragged", "op": "prompt", "requests": 16, "min_len": 128, "max_len": 2048, "prefix": 0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "fused": True},
        # one long prompt
        {"name": "prompt 1 x 8192", "op": "prompt", "requests": 1, "min_len": 8192, "max_len": 8192, "prefix": 0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "fused": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    return rng.choice([(32, 8), (32, 32), (32, 4), (16, 2), (8, 8), (28, 4), (12, 2), (16, 1)])


def draw(rng):
    op = rng.choice(["layout", "rope", "append", "attend", "attend", "prompt", "prompt"])
    if op == "layout":
        requests = _log(rng, 1, 1024)
        return {"op": op, "requests": requests, "rows": requests + _log(rng, 1, 15000), "block": rng.choice([16, 32, 64, 96, 128]),
                "chunk": _log(rng, 1, 700), "max_past": _log(rng, 16, 32768)}
    hq, hkv = _heads(rng)
    dim, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "fp16"])
    if op in ("rope", "append"):
        c = {"op": op, "tokens": _log(rng, 1, 8191), "q_heads": hq, "kv_heads": hkv, "head_dim": dim,
             "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4, "src": rng.choice(["fp32", dtype]),
             "dtype": dtype, "max_pos": _log(rng, 64, 1000000), "factor": rng.choice([1.0, 1.0, 4.0, 16.0])}
        if op == "append":
            c.update({"block": rng.choice([16, 32, 64, 96]), "dense": rng.random() < 0.5})
        return c
    if op == "attend":
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        top = _log(rng, 17, 16384)
        return {"op": op, "requests": _log(rng, 1, max(1, min(256, (1 << 20) * 8 // (top * hkv)))), "q_len": q_len, "q_heads": hq,
                "kv_heads": hkv, "head_dim": dim, "block": rng.choice([16, 32, 64, 96]), "dtype": dtype,
                "min_len": max(q_len, top // rng.choice([1, 4, 64])), "max_len": max(q_len, top)}
    top = _log(rng, 16, 6000)
    return {"op": op, "requests": _log(rng, 1, max(1, min(128, 16384 // top, (1 << 25) // (top * top)))), "min_len": max(1, top // rng.choice([1, 4, 64])),
            "max_len": top, "prefix": rng.choice([0, 0, 1]) * _log(rng, 1, 1500), "q_heads": hq, "kv_heads": hkv, "head_dim": dim,
            "dtype": dtype, "fused": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Per-request lengths, log-uniform between min_len and max_len; the first one is the longest. They belong to the case, not to the seed."""
    r = np.random.default_rng([case["requests"], case["max_len"], 11])
    lo, hi = math.log(case["min_len"]), math.log(case["max_len"])
    n = np.exp(r.uniform(lo, hi, case["requests"])).round().astype(np.int64).clip(case["min_len"], case["max_len"])
    n[0] = case["max_len"]
    return n


def _q_lengths(case):
    n = np.random.default_rng([case["requests"], case["max_len"], 12]).integers(1, case["q_len"] + 1, case["requests"])
    n[0] = case["q_len"]
    return n


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _starts(n):
    return np.concatenate([[0], np.cumsum(n)])


def block_bytes(kv_heads, dim, block):
    return kv_heads * (block // GRANULE) * (GRANULE * dim + GRANULE * 8 * (dim // GROUP))


def _page_views(pages, kv_heads, dim, block):
    """(codes, parameters) views of pages [N, bytes]: uint8 [N, heads, granules, 2, 16, D/2] and fp16 [N, heads, granules, 2, 16, D/64, 2]."""
    half = GRANULE * (dim // 2 + 4 * (dim // GROUP))
    p = pages[:, :block_bytes(kv_heads, dim, block)].unflatten(1, (kv_heads, block // GRANULE, 2, half))
    codes = p[..., :GRANULE * dim // 2].unflatten(-1, (GRANULE, dim // 2))
    params = p[..., GRANULE * dim // 2:].view(torch.float16).unflatten(-1, (GRANULE, dim // GROUP, 2))
    return codes, params


def _scaled_frequencies(rot, base, factor):
    """Inverse frequencies of rotary pairs and the factor on sine and cosine. factor > 1 stretches them for contexts `factor` times
    as long as trained on: slow pairs are slowed by the whole factor, fast ones not at all, with a ramp between (YaRN)."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f.float(), 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return (f * keep + f / factor * (1 - keep)).float(), 0.1 * math.log(factor) + 1.0


def _rows(case, seed, kinds):
    """Fused projection rows [T, heads, D] of the source type and its q, k, v views: unit normal, with a few strong key channels."""
    T, hq, hkv, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    x = torch.randn((T, hq + (len(kinds) - 1) * hkv, dim), generator=_gen(seed), device="cuda")
    x[:, hq:hq + hkv, 3::16] *= 6
    x = x.to(TYPES[case["src"]])
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def prepare(case, seed):
    return {"layout": _prepare_layout, "rope": _prepare_rope, "append": _prepare_append, "attend": _prepare_attend,
            "prompt": _prepare_prompt}[case["op"]](case, seed)


def _layout_lengths(case, seed):
    r = np.random.default_rng([seed, 21])
    n, rows, chunk = case["requests"], case["rows"], case["chunk"]
    new = np.ones(n, dtype=np.int64)
    past = r.integers(0, case["max_past"], n)
    if chunk > 1:
        is_prompt = r.random(n) < 0.06
        new[is_prompt] = r.integers(1, chunk + 1, int(is_prompt.sum()))
        past[is_prompt & (r.random(n) < 0.5)] = 0
        new[r.random(n) < 0.03] = 0                      # finished, not yet replaced
    over = np.cumsum(new) > rows
    new[over] = 0
    return past, new


def _prepare_layout(case, seed):
    past, new = _layout_lengths(case, seed)
    R, T, block = case["requests"], case["rows"], case["block"]
    width = -(-(case["max_past"] + case["chunk"]) // block)
    held = -(-past // block)
    need = -(-(past + new) // block) - held
    r = np.random.default_rng([seed, 22])
    ids = r.permutation(int(held.sum() + need.sum()) + 64).astype(np.int64)
    table = np.full((R, width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < held[:, None]] = ids[:held.sum()]
    free = ids[held.sum():]
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "past": _i32(past), "new": _i32(new), "adapters": _i32(r.integers(-1, 32, R)), "table": _i32(table),
            "free": _i32(free), "head": _i32(np.array([int(r.integers(0, 8))])), "cu": i32(R + 1), "kv_len": i32(R),
            "positions": i32(T), "slots": i32(T), "ids": i32(T), "head_out": i32(1), "err": i32(1)}


def _prepare_rope(case, seed):
    q, k, _ = _rows(case, seed, "qk")
    r = np.random.default_rng([seed, 31])
    f, m = _scaled_frequencies(case["rot"], 10000.0, case["factor"])
    return {"case": case, "q": q, "k": k, "positions": _i32(r.integers(0, case["max_pos"], case["tokens"])), "freq": f.cuda(), "mscale": m,
            "q_out": torch.empty(q.shape, dtype=TYPES[case["dtype"]], device="cuda"),
            "k_out": torch.empty(k.shape, dtype=TYPES[case["dtype"]], device="cuda")}


def _prepare_append(case, seed):
    q, k, v = _rows(case, seed, "qkv")
    r = np.random.default_rng([seed, 32])
    T, block, dim, hkv = case["tokens"], case["block"], case["head_dim"], case["kv_heads"]
    f, m = _scaled_frequencies(case["rot"], 10000.0, case["factor"])
    n_pages = T // block + 9
    slots = (r.permutation(n_pages)[:, None] * block + np.arange(block)[None, :]).reshape(-1)[:T]
    empty = lambda x: torch.empty(x.shape, dtype=TYPES[case["dtype"]], device="cuda")  # noqa: E731
    return {"case": case, "q": q, "k": k, "v": v, "positions": _i32(r.integers(0, case["max_pos"], T)), "freq": f.cuda(), "mscale": m,
            "slots": _i32(slots), "pages": torch.zeros((n_pages, block_bytes(hkv, dim, block)), dtype=torch.uint8, device="cuda"),
            "q_out": empty(q), "k_out": empty(k) if case["dense"] else None, "v_out": empty(v) if case["dense"] else None,
            "k_read": empty(k), "v_read": empty(v), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_attend(case, seed):
    hq, hkv, dim, block = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    lens, q_lens = _lengths(case), _q_lengths(case)
    q_lens = np.minimum(q_lens, lens)
    held = -(-lens // block)
    n_pages = int(held.sum()) + 5
    r = np.random.default_rng([seed, 41])
    table = np.full((case["requests"], int(held.max())), -1, dtype=np.int64)
    table[np.arange(table.shape[1])[None, :] < held[:, None]] = r.permutation(n_pages)[:held.sum()]
    g = _gen(seed)
    # codes of normal values over a 64-wide group: low near -2.4 sigma, step near 4.8 sigma / 15, codes near normal around 7.5
    pages = torch.zeros((n_pages, block_bytes(hkv, dim, block)), dtype=torch.uint8, device="cuda")
    codes, params = _page_views(pages, hkv, dim, block)
    for i in range(0, n_pages, 256):                     # a chunk of pages at a time keeps the temporaries small
        c, p = codes[i:i + 256], params[i:i + 256]
        n = (torch.randn((2, *c.shape), generator=g, device="cuda", dtype=torch.float16) * 3.1 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
        c.copy_(n[0] | (n[1] << 4))
        step = torch.rand(p.shape[:-1], generator=g, device="cuda") * 0.2 + 0.2
        p.copy_(torch.stack([step, step * -7.5 + 0.1 * torch.randn(step.shape, generator=g, device="cuda")], -1))
    T = int(q_lens.sum())
    q = torch.randn((T, hq, dim), generator=g, device="cuda").to(TYPES[case["dtype"]])
    return {"case": case, "q": q, "pages": pages, "table": _i32(table), "cu_q": _i32(_starts(q_lens)), "kv_len": _i32(lens),
            "out": torch.empty_like(q), "ws": torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
            "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prompt_lengths(case):
    q = _lengths(case)
    past = np.random.default_rng([case["requests"], case["max_len"], 51]).integers(0, case["prefix"] + 1, case["requests"])
    return q, q + past


def _prepare_prompt(case, seed):
    hq, hkv, dim, t = case["q_heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    q_len, k_len = _prompt_lengths(case)
    Tq, Tk, g = int(q_len.sum()), int(k_len.sum()), _gen(seed)
    if case["fused"] and Tq == Tk:                       # one projection's rows, q beside k beside v
        x = torch.randn((Tq, hq + 2 * hkv, dim), generator=g, device="cuda").to(t)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q = torch.randn((Tq, hq, dim), generator=g, device="cuda").to(t)
        k, v = (torch.randn((Tk, hkv, dim), generator=g, device="cuda").to(t) for _ in range(2))
    return {"case": case, "q": q, "k": k, "v": v, "cu_q": _i32(_starts(q_len)), "cu_k": _i32(_starts(k_len)),
            "max_q": int(q_len.max()), "max_k": int(k_len.max()), "out": torch.empty((Tq, hq, dim), dtype=t, device="cuda"),
            "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_layout(s):
    import heterogeneous_adapter_batching_b200 as H
    H.lora_kv_layout(s["past"], s["new"], s["adapters"], s["case"]["block"], s["table"], s["free"], s["head"], s["cu"], s["kv_len"],
                     s["positions"], s["slots"], s["ids"], s["head_out"], err=s["err"])
    return {k: s[k] for k in ("table", "cu", "kv_len", "positions", "slots", "ids", "head_out")}


def _own_rope(s):
    import heterogeneous_adapter_batching_b200 as H
    H.lora_rope(s["q"], s["k"], s["positions"], s["freq"], s["q_out"], s["k_out"], interleaved=s["case"]["interleaved"], mscale=s["mscale"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s):
    import heterogeneous_adapter_batching_b200 as H
    block = s["case"]["block"]
    H.lora_kv_append(s["q"], s["k"], s["v"], s["positions"], s["freq"], s["slots"], s["pages"], block, s["q_out"], s["k_out"], s["v_out"],
                     interleaved=s["case"]["interleaved"], mscale=s["mscale"], err=s["err"])
    H.lora_kv_gather(s["pages"], block, s["slots"], s["k_read"], s["v_read"], err=s["err"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "k_cached": s["k_read"], "v_cached": s["v_read"]}


def _own_attend(s):
    import heterogeneous_adapter_batching_b200 as H
    c = s["case"]
    H.lora_kv_attend(s["q"], s["pages"], c["block"], c["kv_heads"], s["table"], s["cu_q"], s["kv_len"], c["q_len"], c["head_dim"] ** -0.5,
                     s["out"], s["ws"], err=s["err"])
    return s["out"]


def _own_prompt(s):
    import heterogeneous_adapter_batching_b200 as H
    H.lora_prompt_attend(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["case"]["head_dim"] ** -0.5, s["out"], err=s["err"])
    return s["out"]


_own = {"layout": _own_layout, "rope": _own_rope, "append": _own_append, "attend": _own_attend, "prompt": _own_prompt}


def _plain_layout(s):
    block, table, free = s["case"]["block"], s["table"], s["free"].long()
    past, new = s["past"].long(), s["new"].long()
    ends = new.cumsum(0)
    before = (past + block - 1) // block
    fresh = (past + new + block - 1) // block - before
    first = s["head"].long() + fresh.cumsum(0) - fresh   # a request's first place in the free list
    b = torch.arange(table.shape[1], device="cuda")
    is_new = (b >= before[:, None]) & (b < (before + fresh)[:, None])
    at = (first[:, None] + b - before[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(is_new, free[at], table.long()))
    t = torch.arange(s["case"]["rows"], device="cuda")
    r = torch.searchsorted(ends, t, right=True).clamp(max=past.numel() - 1)
    live = t < ends[-1]
    pos = past[r] + t - (ends - new)[r]
    page = table.long()[r, (pos // block).clamp(0, table.shape[1] - 1)]
    none = torch.full_like(t, -1)
    i32 = torch.int32
    return {"table": table, "cu": torch.cat([ends.new_zeros(1), ends]).to(i32), "kv_len": (past + new).to(i32),
            "positions": torch.where(live, pos, none).to(i32), "slots": torch.where(live, page * block + pos % block, none).to(i32),
            "ids": torch.where(live, s["adapters"].long()[r], none).to(i32), "head_out": (s["head"] + fresh.sum()).to(i32)}


def _rotate(x, positions, freq, mscale, interleaved):
    """Rotates the first 2 * len(freq) dimensions of x [T, H, D], in 64 bits (angles of far positions)."""
    angle = positions.double()[:, None] * freq.double()[None, :]
    c, s = (angle.cos() * mscale)[:, None, :], (angle.sin() * mscale)[:, None, :]
    n, x = freq.numel(), x.double()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1).float()


def _plain_rope(s):
    t, i = TYPES[s["case"]["dtype"]], s["case"]["interleaved"]
    return {"q": _rotate(s["q"], s["positions"], s["freq"], s["mscale"], i).to(t), "k": _rotate(s["k"], s["positions"], s["freq"], s["mscale"], i).to(t)}


def _quantise(x):
    """4-bit codes and (step, low) of x [..., D], in 64 bits (codes next to a border): low is the group's least value, 15 steps reach its greatest."""
    g = x.double().unflatten(-1, (-1, GROUP))
    low = g.amin(-1).half()
    step = ((g.amax(-1) - g.amin(-1)) / 15).half()
    d = step.double()[..., None]
    n = torch.where(d > 0, (g - low.double()[..., None]) / d, torch.zeros_like(g)).round().clamp(0, 15)
    return n.flatten(-2).to(torch.uint8), torch.stack([step, low], -1)


def _plain_append(s):
    c = s["case"]
    t, block = TYPES[c["dtype"]], c["block"]
    q = _rotate(s["q"], s["positions"], s["freq"], s["mscale"], c["interleaved"]).to(t)
    k = _rotate(s["k"], s["positions"], s["freq"], s["mscale"], c["interleaved"]).to(t)
    v = s["v"].to(t)
    codes, params = _page_views(s["pages"], c["kv_heads"], c["head_dim"], block)
    slots = s["slots"].long()
    page, granule, row = slots // block, slots % block // GRANULE, slots % GRANULE
    n, p = _quantise(torch.stack([k, v], 1))             # [T, 2, heads, D]
    codes.permute(0, 2, 4, 3, 1, 5)[page, granule, row] = n[..., 0::2] | (n[..., 1::2] << 4)
    params.permute(0, 2, 4, 3, 1, 5, 6)[page, granule, row] = p
    back = _dequantise(codes.permute(0, 2, 4, 3, 1, 5)[page, granule, row], params.permute(0, 2, 4, 3, 1, 5, 6)[page, granule, row]).to(t)
    return {"q": q, "k": k if c["dense"] else None, "v": v if c["dense"] else None, "k_cached": back[:, 0], "v_cached": back[:, 1]}


def _dequantise(codes, params):
    """fp32 values [..., D] of codes [..., D/2] and (step, low) [..., D/64, 2]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (n * params[..., 0:1].float() + params[..., 1:2].float()).flatten(-2)


def _plain_attend(s):
    c = s["case"]
    codes, params = _page_views(s["pages"], c["kv_heads"], c["head_dim"], c["block"])
    kv_len, cu = s["kv_len"].long(), s["cu_q"].long()
    R, G = kv_len.numel(), c["q_heads"] // c["kv_heads"]
    at = s["table"].long().clamp(min=0)
    x = _dequantise(codes[at], params[at])               # [R, blocks, heads, granules, 2, 16, D]
    k, v = x.permute(4, 0, 2, 1, 3, 5, 6).flatten(3, 5)  # [R, heads, L, D]
    i = torch.arange(c["q_len"], device="cuda")
    q_len = cu[1:] - cu[:-1]
    live = i < q_len[:, None]
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]  # [R, q_len, Hq, D]
    q = q.unflatten(2, (c["kv_heads"], G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    sees = torch.arange(k.shape[2], device="cuda") <= (kv_len - q_len)[:, None, None] + i[:, None]  # [R, q_len, L]
    sees &= live[:, :, None]
    score = (q @ k.transpose(-1, -2)).unflatten(2, (G, c["q_len"])) * c["head_dim"] ** -0.5
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = (p.flatten(2, 3) @ v) / p.sum(-1).clamp(min=1e-30).flatten(2, 3)[..., None]
    o = o.unflatten(2, (G, c["q_len"])).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [R, q_len, Hq, D]
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    return o[r, t - cu[r]].to(s["q"].dtype)


def _plain_prompt(s):
    c = s["case"]
    cu_q, cu_k, G = s["cu_q"].long(), s["cu_k"].long(), c["q_heads"] // c["kv_heads"]
    q_len, k_len = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    q = s["q"].float()[(cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].unflatten(2, (c["kv_heads"], G)).permute(0, 2, 3, 1, 4)
    at = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    k, v = (x.float()[at].transpose(1, 2)[:, :, None] for x in (s["k"], s["v"]))   # [R, heads, 1, L, D]
    p = (q @ k.transpose(-1, -2)).mul_(c["head_dim"] ** -0.5)                       # [R, heads, G, Lq, Lk]
    sees = (j <= (k_len - q_len)[:, None, None] + i[:, None]) & (i < q_len[:, None])[:, :, None]
    p.masked_fill_(~sees[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    t = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(cu_q[1:], t, right=True)
    return o[r, t - cu_q[r]].to(s["q"].dtype)


_plain = {"layout": _plain_layout, "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "prompt": _plain_prompt}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "layout":
        past, new = _layout_lengths(case, 0)
        fresh = int((-(-(past + new) // case["block"]) - -(-past // case["block"])).sum())
        # lengths, adapters and each request's last block in; starts, lengths, fresh blocks (list and table) and three row maps out
        return {"bytes": 24 * case["requests"] + 8 * fresh + 12 * case["rows"], "flops": 0}
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op in ("rope", "append"):
        T, src, dst = case["tokens"], 4 if case["src"] == "fp32" else 2, 2
        b = T * 4 + T * (hq + hkv) * dim * (src + dst)
        f = T * (hq + hkv) * case["rot"] * 3
        if op == "append":
            cached = block_bytes(hkv, dim, GRANULE) // GRANULE
            b += T * (4 + hkv * dim * src) - (0 if case["dense"] else T * hkv * dim * dst) + (T * hkv * dim * dst if case["dense"] else 0)
            b += T * (2 * cached + 4 + 2 * hkv * dim * dst)  # written, read back, handed out
            f += T * hkv * dim * 2 * 6
        return {"bytes": b, "flops": f}
    if op == "attend":
        lens, q_lens = _lengths(case), _q_lengths(case)
        q_lens = np.minimum(q_lens, lens)
        pairs = int((q_lens * lens - q_lens * (q_lens - 1) // 2).sum())
        per_token = block_bytes(hkv, dim, GRANULE) // GRANULE
        return {"bytes": int(lens.sum()) * per_token + int(q_lens.sum()) * hq * dim * 4 + 4 * int((-(-lens // case["block"])).sum()),
                "flops": 4 * pairs * hq * dim}
    q, k = _prompt_lengths(case)
    pairs = int((q * k - q * (q - 1) // 2).sum())
    return {"bytes": 4 * hq * dim * int(q.sum()) + 4 * hkv * dim * int(k.sum()), "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"layout": lambda s: None, "rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "prompt": _exact_prompt}[case["op"]](s)


def _turn(x, s):
    """Rotary positions as a product of complex numbers."""
    n = s["freq"].numel()
    a = s["positions"].double()[:, None] * s["freq"].double()
    w = torch.polar(torch.full_like(a, s["mscale"]), a)[:, None]
    y = x.double().clone()
    i = torch.arange(n, device="cuda")
    one, two = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + n)
    z = torch.complex(y[..., one], y[..., two]) * w
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rope(s):
    return {"q": _turn(s["q"], s), "k": _turn(s["k"], s)}


def _through_cache(x):
    """What 4 bits keep of values x [T, H, D]."""
    out = torch.empty_like(x)
    for g in range(x.shape[-1] // GROUP):
        y = x[..., g * GROUP:(g + 1) * GROUP]
        low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        step, low = ((high - low) / 15).to(torch.float16).double(), low.to(torch.float16).double()
        n = torch.clamp(torch.round((y - low) / torch.where(step == 0, torch.ones_like(step), step)), 0, 15)
        out[..., g * GROUP:(g + 1) * GROUP] = torch.where(step == 0, torch.zeros_like(n), n) * step + low
    return out


def _exact_append(s):
    t = TYPES[s["case"]["dtype"]]
    q, k, v = _turn(s["q"], s), _turn(s["k"], s), s["v"].double()
    dense = s["case"]["dense"]
    return {"q": q, "k": k if dense else None, "v": v if dense else None,
            "k_cached": _through_cache(k.float().to(t).double()), "v_cached": _through_cache(v.float().to(t).double())}


def _softmax_rows(q, k, v, first, scale):
    """out [H, n, D] of queries q [H, n, D] over k, v [L, D]; query i sees keys 0 .. first + i."""
    a = (q @ k.T) * scale
    a.masked_fill_(torch.arange(k.shape[0], device="cuda")[None, :] > first + torch.arange(q.shape[1], device="cuda")[:, None], -math.inf)
    return torch.softmax(a, -1) @ v


def _exact_attend(s):
    c = s["case"]
    block, dim, hkv, G = c["block"], c["head_dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    half = GRANULE * (dim // 2 + 4 * (dim // GROUP))
    cu, lens, table = s["cu_q"].tolist(), s["kv_len"].tolist(), s["table"].long()
    if sum(lens) * hkv > 1 << 24 or len(lens) * hkv > 3000:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        pages = s["pages"][table[r, :-(-n // block)]].reshape(-1, hkv, block // GRANULE, 2, half)
        for h in range(hkv):
            x = pages[:, h].reshape(-1, 2, half)         # granules of the request in order
            kv = []
            for i in range(2):
                byte = x[:, i, :GRANULE * dim // 2].reshape(-1, dim // 2).int()
                par = x[:, i, GRANULE * dim // 2:].contiguous().view(torch.float16).reshape(-1, dim // GROUP, 2).double()
                n4 = torch.empty((byte.shape[0], dim), dtype=torch.float64, device="cuda")
                n4[:, 0::2], n4[:, 1::2] = (byte % 16).double(), (byte // 16).double()
                kv.append((n4 * par[..., 0].repeat_interleave(GROUP, 1) + par[..., 1].repeat_interleave(GROUP, 1))[:n])
            q = s["q"][cu[r]:cu[r + 1], h * G:(h + 1) * G].double().transpose(0, 1)
            out[cu[r]:cu[r + 1], h * G:(h + 1) * G] = _softmax_rows(q, *kv, n - (cu[r + 1] - cu[r]), dim ** -0.5).transpose(0, 1)
    return out


def _exact_prompt(s):
    c = s["case"]
    cu_q, cu_k, G = s["cu_q"].tolist(), s["cu_k"].tolist(), c["q_heads"] // c["kv_heads"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for r in range(len(cu_q) - 1):
        a, b, u, w = cu_q[r], cu_q[r + 1], cu_k[r], cu_k[r + 1]
        for h in range(c["kv_heads"]):
            q = s["q"][a:b, h * G:(h + 1) * G].double().transpose(0, 1)
            o = _softmax_rows(q, s["k"][u:w, h].double(), s["v"][u:w, h].double(), (w - u) - (b - a), c["head_dim"] ** -0.5)
            out[a:b, h * G:(h + 1) * G] = o.transpose(0, 1)
    return out
