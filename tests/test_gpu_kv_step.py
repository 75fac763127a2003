"""GPU: the calls of a serving step run together, as a program would: adapters and
KV blocks in one pool, request lengths -> ids, plan and block tables, projections
with their adapters, rotary positions and the cache, attention; prompts first,
then decoding, drafts, and a prompt in two chunks."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import _kv as K
from tests import _util as U

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
D, HQ, HK, DIM, BLOCK = 256, 4, 2, 64, 48


@pytest.fixture(scope="module")
def H():
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


class Model:
    """Query, key and value projections of one layer with adapters; the q layer's pool holds the KV blocks too."""

    def __init__(self, H, seed):
        wl = W.random_small(seed=seed, T=64, d_in=D, d_out=D, S=5, ranks=(4, 16, 33), p_none=0.0)
        self.wl, self.H = wl, H
        self.q = U.make_layer(wl, max_tokens=512, shared_pool=True, extra_pages=60)
        self.kv = []
        for s in (1, 2):
            w = W.random_small(seed=seed + s, T=64, d_in=D, d_out=HK * DIM, S=5, ranks=(4, 16, 33), p_none=0.0)
            self.kv.append(U.make_layer(w, max_tokens=512))
        g = torch.Generator()
        g.manual_seed(seed)
        self.base = [(torch.randn((D, n), generator=g) / 16).cuda() for n in (HQ * DIM, HK * DIM, HK * DIM)]

    def project(self, X, cache):
        """fp32 rows q, k, v of X [T, D] (bf16) with the step's adapter ids, as views of one buffer each."""
        T = X.shape[0]
        ys = [X.float() @ w for w in self.base]
        layers = [self.q, *self.kv]
        self.q.plan(cache.ids[:T])
        self.H.apply_multi(layers, X, ys, None, ws=self.q.ws, err=self.q.err)
        return [y.view(T, -1, DIM) for y in ys]


class Reference:
    """Per request: cached k and v as the cache holds them, and dense ones, in 64 bits, from the device's projections."""

    def __init__(self, R):
        self.k, self.v = [np.zeros((0, HK, DIM))] * R, [np.zeros((0, HK, DIM))] * R
        self.step = [np.zeros((0, HK))] * R
        self.dense_k, self.dense_v = [np.zeros((0, HK, DIM))] * R, [np.zeros((0, HK, DIM))] * R

    def add(self, r, k, v, pos, freq):
        kr = K.rotate(k, pos, freq, 1.0, False).float().to(BF)
        vr = v.float().cpu().to(BF)
        for name, x in (("k", kr), ("v", vr)):
            c, s, lo = K.quantise(x)
            val = c.astype(np.float64) * np.repeat(s.astype(np.float64), 64, -1) + np.repeat(lo.astype(np.float64), 64, -1)
            getattr(self, name)[r] = np.concatenate([getattr(self, name)[r], val])
            if name == "k":
                self.step[r] = np.concatenate([self.step[r], s.astype(np.float64).max(-1)])
            d = "dense_" + name
            getattr(self, d)[r] = np.concatenate([getattr(self, d)[r], x.double().numpy()])


def check_rows(out, q, ref, r, first, n, dense=False, split=None):
    """Rows first .. first + n of out are the last n tokens of request r.  dense: keys as computed; split: the first `split` from
    the cache, the rest as computed."""
    k, v = (ref.dense_k[r], ref.dense_v[r]) if dense else (ref.k[r], ref.v[r])
    if split is not None:   # what lora_kv_gather hands out is rounded to bf16
        bf = lambda x: torch.from_numpy(x).float().to(BF).double().numpy()  # noqa: E731
        k, v = (np.concatenate([bf(c[:split]), d[split:]]) for c, d in ((ref.k[r], ref.dense_k[r]), (ref.v[r], ref.dense_v[r])))
    L = k.shape[0]
    p_half = K.HALF[BF] if dense or split is not None else 2.0 ** -11
    for i in range(n):
        m = L - n + i + 1
        for h in range(HQ):
            g = h // (HQ // HK)
            qv = q[first + i, h].double().cpu().numpy()
            o, _, absv = K.attend_row(qv, k[:m, g], v[:m, g], DIM ** -0.5)
            step = None if dense or split is not None else ref.step[r][:m, g]
            delta = K.row_bound(qv, k[:m, g], DIM ** -0.5, step)
            x = out[first + i, h].double().cpu().numpy()
            assert (np.abs(x - o) <= K.out_bound(o, absv, delta, BF, p_half)).all(), (r, i, h)


def test_prompts_then_decoding_then_drafts(H):
    model = Model(H, 70)
    R, lens = 5, np.array([1, 37, 100, 48, 130])
    adapters = i32([3, 0, -1, 4, 2])
    cache = H.KVCache(model.q.pool_a, HQ, HK, DIM, BLOCK, max_requests=R, max_len=400, max_tokens=340, max_q_len=3)
    adapter_pages, _ = H.lora_pool_usage(model.q.pool_a)
    before = [model.q.page_rows(int(p)).clone() for p in model.q.page_table.cpu().flatten() if p >= 0]
    cache.reserve(20)
    freq, _ = H.rope_frequencies(DIM)
    f, ref = freq.cuda(), Reference(R)
    gen = torch.Generator()
    gen.manual_seed(1)
    past = np.zeros(R, dtype=int)

    def step(new, prompt):
        nonlocal past
        T = int(new.sum())
        cache.begin(i32(past), i32(new), adapters)
        X = torch.randn((T, D), generator=gen).to(BF).cuda()
        q, k, v = model.project(X, cache)
        ids = cache.ids[:T].cpu().numpy()
        assert np.array_equal(ids, np.repeat(adapters.cpu().numpy(), new)) and (cache.ids[T:] == -1).all()
        qo, ko, vo = (torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v))
        cache.append(q, k, v, f, qo, ko if prompt else None, vo if prompt else None)
        out = torch.empty_like(qo)
        cache.prompt_attend(qo, ko, vo, out) if prompt else cache.attend(qo, out)
        torch.cuda.synchronize()
        assert int(cache.err.item()) == 0 and int(model.q.err.item()) == 0
        at = 0
        for r in range(R):
            n = int(new[r])
            ref.add(r, k[at:at + n], v[at:at + n], torch.arange(past[r], past[r] + n), freq)
            check_rows(out, qo, ref, r, at, n, dense=prompt)
            at += n
        past = past + new

    step(lens, True)
    for _ in range(3):
        step(np.ones(R, dtype=int), False)
    step(np.array([3, 1, 0, 2, 3]), False)
    # the adapters' pages were never touched, and the blocks go back to the pool
    after = [model.q.page_rows(int(p)) for p in model.q.page_table.cpu().flatten() if p >= 0]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    used = int((cache.block_table >= 0).sum())
    assert used == int((-(-past // BLOCK)).sum()) and cache.free_list[int(cache.head.item()):].numel() == 20 - used
    cache.free(list(range(R)))
    assert H.lora_pool_usage(model.q.pool_a) == (adapter_pages, 20 - used) and (cache.block_table == -1).all()


def test_a_prompt_in_two_chunks(H):
    """The second chunk attends to the first through the cache (lora_kv_layout without a free list, lora_kv_gather) and to itself."""
    model = Model(H, 80)
    cache = H.KVCache(model.q.pool_a, HQ, HK, DIM, BLOCK, max_requests=2, max_len=400, max_tokens=300)
    cache.reserve(12)
    freq, _ = H.rope_frequencies(DIM)
    f, ref = freq.cuda(), Reference(2)
    gen = torch.Generator()
    gen.manual_seed(2)
    first, second = np.array([70, 49]), np.array([90, 3])
    adapters = i32([1, 2])
    for past, new in ((np.zeros(2, int), first), (first, second)):
        T = int(new.sum())
        cache.begin(i32(past), i32(new), adapters)
        q, k, v = model.project(torch.randn((T, D), generator=gen).to(BF).cuda(), cache)
        qo, ko, vo = (torch.empty(x.shape, dtype=BF, device="cuda") for x in (q, k, v))
        cache.append(q, k, v, f, qo, ko, vo)
        at = 0
        for r in range(2):
            n = int(new[r])
            ref.add(r, k[at:at + n], v[at:at + n], torch.arange(past[r], past[r] + n), freq)
            at += n
    # the prefix out of the cache, in front of each request's new rows
    n = int(first.sum())
    cu, kl, pos, slots = i32(np.zeros(3)), i32(np.zeros(2)), i32(np.zeros(n)), i32(np.zeros(n))
    H.lora_kv_layout(i32([0, 0]), i32(first), None, BLOCK, cache.block_table, None, None, cu, kl, pos, slots)
    kp, vp = (torch.empty((n, HK, DIM), dtype=BF, device="cuda") for _ in range(2))
    H.lora_kv_gather(cache.pages, BLOCK, slots, kp, vp, err=cache.err)
    cat = lambda p, x: torch.cat([p[:70], x[:90], p[70:], x[90:]])  # noqa: E731
    out = torch.empty_like(qo)
    H.lora_prompt_attend(qo, cat(kp, ko), cat(vp, vo), i32([0, 90, 93]), i32([0, 160, 160 + 52]), DIM ** -0.5, out, err=cache.err)
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0
    check_rows(out, qo, ref, 0, 0, 90, split=70)
    check_rows(out, qo, ref, 1, 90, 3, split=49)


def test_a_decode_step_as_one_graph(H):
    """layout, append and attention captured together and replayed step after step; lengths and rows change in place."""
    R = 3
    buf = torch.empty((40 * 16, 256), dtype=BF, device="cuda")
    cache = H.KVCache(H.lora_pool_create(buf, 256), HQ, HK, DIM, BLOCK, max_requests=R, max_len=200, max_tokens=R)
    cache.reserve(10)
    freq, _ = H.rope_frequencies(DIM)
    f, ref = freq.cuda(), Reference(R)
    past, new = i32([0] * R), i32([1] * R)
    y = torch.zeros((R, HQ + 2 * HK, DIM), device="cuda")
    qo, out = (torch.empty((R, HQ, DIM), dtype=BF, device="cuda") for _ in range(2))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        H.lora_kv_layout(past, i32([0] * R), None, BLOCK, cache.block_table, cache.free_list, cache.head, cache.cu_new, cache.kv_len,
                         cache.positions, cache.slots, cache.ids, cache._next_head)
        H.lora_kv_attend(qo, cache.pages, BLOCK, HK, cache.block_table, cache.cu_new, cache.kv_len, 1, 0.1, out, cache.ws)
    torch.cuda.synchronize()
    heads = [cache.head, cache._next_head]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.lora_kv_layout(past, new, None, BLOCK, cache.block_table, cache.free_list, heads[0], cache.cu_new, cache.kv_len,
                         cache.positions, cache.slots, cache.ids, heads[1], err=cache.err)
        heads[0].copy_(heads[1])
        cache.append(y[:, :HQ], y[:, HQ:HQ + HK], y[:, HQ + HK:], f, qo)
        cache.rows = R
        cache.attend(qo, out)
        past.add_(new)
    gen = torch.Generator()
    gen.manual_seed(3)
    for t in range(60):                      # over a block's end
        y.copy_(torch.randn(y.shape, generator=gen))
        g.replay()
        torch.cuda.synchronize()
        for r in range(R):
            ref.add(r, y[r:r + 1, HQ:HQ + HK], y[r:r + 1, HQ + HK:], torch.tensor([t]), freq)
            if t in (0, 1, 47, 48, 59):
                check_rows(out, qo, ref, r, r, 1)
    assert int(cache.err.item()) == 0 and cache.free_list[int(heads[0].item()):].numel() == 10 - 2 * R


def test_a_captured_step_of_the_cache_object(H):
    """begin() replayed hands out new pages every time, and goes on after reserve() and free() between replays."""
    R = 2
    buf = torch.empty((40 * 16, 256), dtype=BF, device="cuda")
    pool = H.lora_pool_create(buf, 256)
    cache = H.KVCache(pool, HQ, HK, DIM, 16, max_requests=R, max_len=96, max_tokens=R)
    cache.reserve(2)
    past, new = i32([0] * R), i32([1] * R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.begin(past, i32([0] * R), stream=side)          # a first call outside the graph, on another stream
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.begin(past, new)
        past.add_(new)
    for t in range(96):
        if t == 16:
            cache.reserve(10)
        g.replay()
        if t == 15:
            assert cache.free_list[int(cache.head.item()):].numel() == 0
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0 and cache.slots.tolist() == [16 * int(cache.block_table[r, 5]) + 15 for r in range(R)]
    pages = cache.block_table.flatten().tolist()
    assert min(pages) >= 0 and len(set(pages)) == 12
    cache.free([1, 1])                                    # a row named twice is freed once
    assert H.lora_pool_usage(pool)[1] == 6 and (cache.block_table[1] == -1).all() and cache.block_table[0].tolist() == pages[:6]
    past[0], new[0], past[1] = 96, 0, 0
    cache.reserve(1)
    g.replay()
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0 and int(cache.block_table[1, 0]) in pages[6:] + [p for p in range(40) if p not in pages]


def test_a_cache_without_pages_in_reserve(H):
    """An empty list of free pages is a list that has run dry, not a complete table."""
    buf = torch.empty((8 * 16, 256), dtype=BF, device="cuda")
    cache = H.KVCache(H.lora_pool_create(buf, 256), HQ, HK, DIM, 16, max_requests=1, max_len=32, max_tokens=4)
    cache.begin(i32([0]), i32([3]))
    torch.cuda.synchronize()
    assert int(cache.err.item()) == H.DEV_ERR_NO_PAGES and int(cache.kv_len[0]) == 0 and (cache.slots == -1).all()
    cu, kl, pos, slots, err = i32([0, 0]), i32([9]), i32([9] * 4), i32([9] * 4), i32([0])
    table = i32([[5, 5]])
    H.lora_kv_layout(i32([0]), i32([3]), None, 16, table, i32([]), None, cu, kl, pos, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == H.DEV_ERR_NO_PAGES and table.tolist() == [[5, 5]] and kl.tolist() == [0] and slots.tolist() == [-1] * 4


def test_the_binding_refuses_tensors_that_do_not_fit(H):
    """Every check of the binding, on tensors of the device: nothing runs."""
    z = lambda *n, dtype=BF: torch.zeros(n, dtype=dtype, device="cuda")  # noqa: E731
    q, k, pos, f = z(4, 8, 64), z(4, 2, 64), i32([0] * 4), z(32, dtype=torch.float32)
    pages = z(6, H.lora_kv_block_bytes(2, 64, 16), dtype=torch.uint8)
    slots, table, cu, lens = i32([-1] * 4), i32([[0, 1]]), i32([0, 1]), i32([1])
    ws = z(H.lora_kv_attend_workspace_size(8, 2, 64, 1), dtype=torch.uint8)
    ok = {
        "rope": (lambda **a: H.lora_rope(**a), dict(q=q, k=k, positions=pos, inv_freq=f, q_out=z(4, 8, 64), k_out=z(4, 2, 64))),
        "append": (lambda **a: H.lora_kv_append(**a), dict(q=q, k=k, v=z(4, 2, 64), positions=pos, inv_freq=f, slots=slots, pages=pages,
                                                           block_tokens=16, q_out=z(4, 8, 64), k_out=z(4, 2, 64), v_out=z(4, 2, 64))),
        "gather": (lambda **a: H.lora_kv_gather(**a), dict(pages=pages, block_tokens=16, slots=slots, k_out=z(4, 2, 64), v_out=z(4, 2, 64))),
        "attend": (lambda **a: H.lora_kv_attend(**a), dict(q=q, pages=pages, block_tokens=16, kv_heads=2, block_table=table, cu_q=cu,
                                                           kv_len=lens, max_q_len=1, scale=1.0, out=z(4, 8, 64), ws=ws)),
        "prompt": (lambda **a: H.lora_prompt_attend(**a), dict(q=q, k=k, v=z(4, 2, 64), cu_q=cu, cu_k=cu, scale=1.0, out=z(4, 8, 64))),
    }
    for call, args in ok.values():
        call(**args)
    torch.cuda.synchronize()
    wide = z(4, 8, 128)
    for name, arg, bad in [
            ("rope", "q", q[0]), ("rope", "k", None), ("rope", "k_out", None), ("rope", "k", z(3, 2, 64)), ("rope", "k", z(4, 2, 32)),
            ("rope", "q_out", z(4, 8, 32)), ("rope", "q_out", q.float()), ("rope", "positions", i32([0] * 3)), ("rope", "positions", pos.long()),
            ("rope", "inv_freq", f.double()), ("rope", "q", wide[:, :, ::2]), ("rope", "q", q.cpu()), ("rope", "k", k.cpu()),
            ("append", "q", z(5, 8, 64)), ("append", "q_out", None), ("append", "v", z(4, 3, 64)), ("append", "k", k[0]),
            ("append", "k_out", z(4, 2, 64, dtype=torch.float16)), ("append", "slots", i32([0] * 3)), ("append", "pages", pages[:, :64]),
            ("gather", "k_out", z(3, 2, 64)), ("gather", "v_out", z(4, 2, 64, dtype=torch.float16)), ("gather", "slots", i32([0])),
            ("attend", "out", z(4, 8, 64, dtype=torch.float16)), ("attend", "out", z(3, 8, 64)), ("attend", "cu_q", i32([0])),
            ("attend", "kv_len", i32([])), ("attend", "block_table", i32([0, 1])), ("attend", "ws", ws[:-1]), ("attend", "ws", ws.cpu()),
            ("attend", "q", q[0]), ("attend", "kv_heads", 3),
            ("prompt", "k", z(4, 2, 32)), ("prompt", "v", z(5, 2, 64)), ("prompt", "cu_k", i32([0])), ("prompt", "out", z(4, 4, 64)),
            ("prompt", "q", q.float()), ("prompt", "scale", -1.0)]:
        call, args = ok[name]
        with pytest.raises(H.LoraError):
            call(**{**args, arg: bad})
    with pytest.raises(H.LoraError):
        H.lora_kv_gather(pages, 16, slots, None)
    with pytest.raises(H.LoraError):          # the lengths of the last step are not updated in place
        H.lora_kv_layout(lens, i32([1]), None, 16, table, None, None, cu, lens, pos, slots)
