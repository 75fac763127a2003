"""GPU: steps of a KVCache that do not simply go on: rejected drafts, steps that
are repeated, steps that mix prompts and decoding; no page is lost or used twice."""
import numpy as np
import pytest
import torch

from tests import _kv as K

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def H():
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def make(H, n_pages=40, block=16, max_requests=3, max_len=160, max_tokens=64, hq=4, hk=2, dim=64, **kw):
    buf = torch.empty((n_pages * 16, 256), dtype=BF, device="cuda")
    pool = H.lora_pool_create(buf, 256)
    return H.KVCache(pool, hq, hk, dim, block, max_requests=max_requests, max_len=max_len, max_tokens=max_tokens, **kw)


def accounted(H, cache, reserved):
    """Every page that was reserved is in a row of the table or in the reserve, once."""
    torch.cuda.synchronize()
    held = cache.block_table[cache.block_table >= 0].tolist()
    spare = cache.free_list[int(cache.head.item()):].tolist()
    assert len(set(held + spare)) == len(held) + len(spare) == reserved == H.lora_pool_usage(cache.pool)[1]
    return len(held)


def test_rejected_drafts_lose_no_page(H):
    """A past that becomes shorter across a block's border, again and again."""
    R, reserved = 3, 24
    cache = make(H, max_q_len=4)
    cache.reserve(reserved)
    r = np.random.default_rng(1)
    past = np.array([0, 14, 31])
    cache.begin(i32([0, 0, 0]), i32(past))
    for step in range(60):
        new = r.integers(1, 5, R)
        first = cache.block_table.cpu().numpy().copy()
        cache.begin(i32(past), i32(new))
        accounted(H, cache, reserved)
        table = cache.block_table.cpu().numpy()
        assert (table[first >= 0] == first[first >= 0]).all()          # a row's blocks stay where they are
        at = np.concatenate([[0], np.cumsum(new)])
        slots, pos = cache.slots.cpu().numpy(), cache.positions.cpu().numpy()
        for q in range(R):
            want = past[q] + np.arange(new[q])
            assert (pos[at[q]:at[q + 1]] == want).all()
            assert (slots[at[q]:at[q + 1]] == table[q, want // 16] * 16 + want % 16).all()
        assert cache.kv_len.tolist() == (past + new).tolist() and int(cache.err.item()) == 0
        past = past + r.integers(0, new + 1)                           # how many of them were accepted
        past = np.where(past > 100, past - 40, past)                   # and a request that goes back a long way
    cache.free([0, 1, 2])
    spare = cache.free_list[int(cache.head.item()):].numel()
    assert H.lora_pool_usage(cache.pool)[1] == spare and (cache.held == 0).all()


def test_a_step_repeated_after_an_empty_reserve(H):
    """The request that got its pages keeps them when the step is repeated for the one that got none."""
    cache = make(H, max_requests=2)
    cache.reserve(3)
    past, new = i32([0, 0]), i32([20, 30])
    cache.begin(past, new)
    assert accounted(H, cache, 3) == 2 and int(cache.err.item()) == H.DEV_ERR_NO_PAGES and cache.kv_len.tolist() == [20, 0]
    held = cache.block_table[0].tolist()
    cache.reserve(5)
    cache.err.zero_()
    cache.begin(past, new)
    assert accounted(H, cache, 8) == 4 and int(cache.err.item()) == 0 and cache.kv_len.tolist() == [20, 30]
    assert cache.block_table[0].tolist() == held


def test_a_captured_step_with_drafts(H):
    cache = make(H, max_q_len=4)
    cache.reserve(6)
    past, new = i32([10, 13, 15]), i32([4, 4, 4])
    cache.begin(i32([0, 0, 0]), past.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.begin(past, new)
    for p in ([10, 13, 15], [11, 14, 16], [12, 15, 15], [12, 12, 17]):
        past.copy_(i32(p))
        g.replay()
        accounted(H, cache, 6)
        assert cache.kv_len.tolist() == [x + 4 for x in p] and int(cache.err.item()) == 0
    assert accounted(H, cache, 6) == 5 and cache.held.tolist() == [1, 2, 2]


def layout_held(past, new, T, block, table, free, head, held):
    """The rule, request by request: a request takes pages for the blocks beyond those it holds."""
    table, at, dry, taken, out = table.copy(), head, False, 0, []
    pos, slots, kv_len, err = [], [], [], 0
    for r in range(len(past)):
        p, n = int(past[r]), int(new[r])
        first, after = max(-(-p // block), int(held[r])), -(-(p + n) // block)
        bad = not 0 <= held[r] <= table.shape[1] or p + n > table.shape[1] * block
        need = 0 if bad else max(0, after - first)
        dry = dry or (need > 0 and at + need > len(free))
        failed = bad or (need > 0 and dry)
        err |= 32 if bad else 16 if failed else 0
        if not failed:
            table[r, first:first + need] = free[at:at + need]
            taken = at + need - head if need else taken
        at += need
        out.append(int(held[r]) if failed else max(first, after))
        kv_len.append(0 if failed else p + n)
        pos += [-1 if failed else p + i for i in range(n)]
        slots += [-1 if failed else int(table[r, (p + i) // block]) * block + (p + i) % block for i in range(n)]
    pad = [-1] * (T - len(pos))
    return table, kv_len, pos + pad, slots + pad, out, head + taken, err


@pytest.mark.parametrize("R,block,width", [(1, 16, 4), (40, 16, 9), (300, 32, 6), (1024, 16, 5)])
def test_layout_of_rows_that_hold_more(H, R, block, width):
    r = np.random.default_rng(R)
    held = r.integers(0, width + 1, R)
    past = np.minimum(r.integers(0, width * block + 1, R), held * block)
    past[r.random(R) < 0.1] = 0
    new = np.minimum(r.integers(0, 2 * block, R), width * block - past)
    ids = r.permutation(R * width + 7)
    table = np.full((R, width), -1)
    own = np.arange(width) < held[:, None]
    table[own] = ids[:own.sum()]
    free = ids[own.sum():][:R // 2 + 3]
    if R > 10:
        held[3], held[7] = -1, width + 1
    T = int(new.sum()) + 5
    want = layout_held(past, new, T, block, table, free, 1, held)
    cu, kv, pos, slots, head, out, err, dt = (i32(np.full(n, -7)) for n in (R + 1, R, T, T, 1, R, 1, (R, width)))
    err.zero_()
    dt.copy_(i32(table))
    H.lora_kv_layout(i32(past), i32(new), None, block, dt, i32(free), i32([1]), cu, kv, pos, slots, None, head, err=err, held=i32(held),
                     held_out=out)
    got = (dt.cpu().numpy(), kv.tolist(), pos.tolist(), slots.tolist(), out.tolist(), int(head.item()), int(err.item()))
    assert np.array_equal(got[0], want[0]) and got[1:] == want[1:]


def fill(cache, T, seed, rot=None):
    """Random rows of a step, appended without rotation; -> q, k, v as attention reads them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v = (torch.randn((T, n, cache.head_dim), generator=g, device="cuda").to(BF) for n in (cache.q_heads, cache.kv_heads, cache.kv_heads))
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    cache.append(q, k, v, rot, qo, ko, vo)
    return qo, ko, vo


def want_rows(q, k, v, scale):
    """softmax(scale q k^T) v in 64 bits for the last rows q [n, Hq, D] of k, v [m, Hk, D]."""
    G, n, m = q.shape[1] // k.shape[1], q.shape[0], k.shape[0]
    k, v = (x.double().repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("nhd,mhd->hnm", q.double(), k) * scale
    s.masked_fill_(torch.arange(m, device="cuda") > (m - n) + torch.arange(n, device="cuda")[:, None], -torch.inf)
    return torch.einsum("hnm,mhd->nhd", torch.softmax(s, -1), v)


def near(got, want):
    """Row by row: the output's rounding (2^-8 of each element) and that of the weights (2^-8 in a prompt, rows as long as
    their values' sums; half as much on average, so that a norm stays below)."""
    return bool(((got.double() - want).norm(dim=-1) <= 2.0 ** -7 * want.norm(dim=-1)).all())


def test_a_step_that_mixes_decoding_and_prompts(H):
    """Decoding requests first, prompts behind them: two calls, each for its own requests, nothing flagged."""
    cache = make(H, n_pages=60, max_requests=4, max_tokens=200, max_q_len=2)
    cache.reserve(40)
    cache.begin(i32([0, 0]), i32([37, 50]))
    _, k0, v0 = fill(cache, 87, 1)
    past, new = np.array([37, 50, 0, 0]), np.array([1, 2, 70, 33])
    cache.begin(i32(past), i32(new))
    q, k, v = fill(cache, 106, 2)
    out = torch.full_like(q, 7.0)
    cache.attend(q, out, last=2)
    assert (out[3:] == 7).all()
    cache.prompt_attend(q, k, v, out, first=2)
    again = torch.full_like(q, 7.0)
    cache.prompt_attend(q, k, v, again, first=2)
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0 and (again[:3] == 7).all() and torch.equal(again[3:], out[3:])
    at = [0, 1, 3, 73, 106]
    for r in (2, 3):
        s = slice(at[r], at[r + 1])
        assert near(out[s], want_rows(q[s], k[s], v[s], 64 ** -0.5))
    slots = i32(np.zeros(90))
    H.lora_kv_layout(i32([0, 0]), i32([38, 52]), None, 16, cache.block_table[:2], None, None, i32([0] * 3), i32([0] * 2), i32([0] * 90), slots)
    kc, vc = (torch.empty((90, 2, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    H.lora_kv_gather(cache.pages, 16, slots, kc, vc)
    assert near(out[:1], want_rows(q[:1], kc[:38], vc[:38], 64 ** -0.5)) and near(out[1:3], want_rows(q[1:3], kc[38:], vc[38:], 64 ** -0.5))
    cache.attend(q, out, first=4)                            # no such requests: nothing happens
    cache.prompt_attend(q, k, v, out, first=2, last=2)
    for bad in ((-1, 2), (0, 5), (3, 2)):
        with pytest.raises(ValueError):
            cache.attend(q, out, first=bad[0], last=bad[1])
        with pytest.raises(ValueError):
            cache.prompt_attend(q, k, v, out, first=bad[0], last=bad[1])
    cache.attend(q, out, first=1, last=3)                    # a prompt longer than max_q_len is still refused there
    torch.cuda.synchronize()
    assert int(cache.err.item()) == H.DEV_ERR_BAD_LENGTH


@pytest.mark.parametrize("R", [2, 40])
def test_prompt_attention_refuses_requests_with_a_past(H, R):
    """Their keys are not all among the step's rows: flagged, and their outputs are left alone; the others are as ever."""
    cache = make(H, n_pages=200, max_requests=R, max_tokens=40 * R)
    cache.reserve(150)
    past, new = np.zeros(R, int), 20 + np.arange(R) % 11
    past[1::3] = 17
    cache.begin(i32(np.zeros(R)), i32(past))
    fill(cache, int(past.sum()), 3)
    cache.begin(i32(past), i32(new))
    at = np.concatenate([[0], np.cumsum(new)])
    q, k, v = fill(cache, int(at[-1]), 4)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    cache.prompt_attend(q, k, v, out, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.err.item()) == H.DEV_ERR_BAD_LENGTH
    for r in range(R):
        s = slice(at[r], at[r + 1])
        if past[r]:
            assert (out[s] == 7).all() and (lse[s] == 7).all()
        else:
            assert near(out[s], want_rows(q[s], k[s], v[s], 64 ** -0.5))
    cache.err.zero_()
    out.fill_(7.0)
    cache.prompt_attend(q, k, v, out, first=0, last=1, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0 and (out[at[1]:] == 7).all()
    assert near(out[:at[1]], want_rows(q[:at[1]], k[:at[1]], v[:at[1]], 64 ** -0.5))


def test_prompt_attention_in_a_graph_over_changing_lengths(H):
    cache = make(H, max_tokens=64)
    cache.reserve(20)
    past, new = i32([0, 0]), i32([20, 30])
    cache.begin(past, new)
    q, k, v = fill(cache, 50, 5)
    out = torch.full_like(q, 7.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.begin(past, new)
        cache.prompt_attend(q, k, v, out)
    for a, b, p in ((20, 30, 0), (1, 49, 0), (3, 4, 0), (20, 30, 5)):
        new.copy_(i32([a, b]))
        past.copy_(i32([0, p]))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(cache.err.item()) == (H.DEV_ERR_BAD_LENGTH if p else 0) and (out[a + b:] == 7).all()
        assert near(out[:a], want_rows(q[:a], k[:a], v[:a], 64 ** -0.5))
        rest = out[a:a + b]
        assert (rest == 7).all() if p else near(rest, want_rows(q[a:a + b], k[a:a + b], v[a:a + b], 64 ** -0.5))


def test_steps_of_different_sizes_and_tensors_put_in_place_of_others(H):
    """The slices that a step reuses follow the number of requests, and the object's tensors."""
    cache = make(H, max_tokens=8)
    cache.reserve(20)
    for R in (3, 1, 3, 2):
        cache.begin(i32([0] * R), i32([2] * R))
        assert cache.cu_new[:R + 1].tolist() == [2 * i for i in range(R + 1)] and cache.kv_len[:R].tolist() == [2] * R
        q, k, v = fill(cache, 2 * R, R)
        out = torch.empty_like(q)
        cache.prompt_attend(q, k, v, out)
        for r in range(R):
            s = slice(2 * r, 2 * r + 2)
            assert near(out[s], want_rows(q[s], k[s], v[s], 64 ** -0.5))
    other = torch.full_like(cache.block_table, -1)
    other[0, 0] = 39
    cache.block_table = other
    cache.held.zero_()
    cache.begin(i32([1, 0]), i32([1, 1]))
    torch.cuda.synchronize()
    assert cache.slots[:2].tolist() == [39 * 16 + 1, int(other[1, 0]) * 16] and int(cache.err.item()) == 0


def test_a_step_without_tokens(H):
    """Empty rows go through every call of a step and change nothing."""
    cache = make(H)
    cache.reserve(3)
    cache.begin(i32([0, 0]), i32([5, 6]))
    fill(cache, 11, 1)
    torch.cuda.synchronize()
    before = cache.pages.clone()
    cache.begin(i32([5, 6]), i32([0, 0]))
    f = H.rope_frequencies(64)[0].cuda()
    q, k, v = fill(cache, 0, 2, f)
    out, lse = torch.empty_like(q), torch.empty((0, 4), device="cuda")
    cache.attend(q, out, lse=lse)
    cache.prompt_attend(q, k, v, out, lse=lse)
    H.lora_rope(q, k, cache.positions[:0], f, torch.empty_like(q), torch.empty_like(k))
    H.lora_kv_gather(cache.pages, 16, cache.slots[:0], k, v)
    torch.cuda.synchronize()
    assert int(cache.err.item()) == 0 and torch.equal(cache.pages, before) and cache.kv_len[:2].tolist() == [5, 6]


def test_as_many_rows_as_an_int_counts(H):
    """The last rows of 2^31 - 1: no index turns back, no grid is refused."""
    T = 2 ** 31 - 1
    pos, slots, err = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda"), i32([0])
    table = i32([[3, -1], [5, -1]])
    H.lora_kv_layout(i32([7, 0]), i32([12, 3]), None, 16, table, i32([8, 9]), None, i32([0] * 3), i32([0] * 2), pos, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and pos[:15].tolist() == list(range(7, 19)) + [0, 1, 2]
    assert slots[:15].tolist() == [3 * 16 + i for i in range(7, 16)] + [8 * 16 + i for i in range(3)] + [9 * 16 + i for i in range(3)]
    for x in (pos, slots):                                   # in pieces: a comparison takes as many bytes as rows
        assert all(bool((x[i:i + (1 << 28)] == -1).all()) for i in range(15, T, 1 << 28))
    del slots
    pos[T - 1] = 4
    q = torch.randn((1, 1, 16), device="cuda").to(BF)
    out = torch.empty((T, 1, 16), dtype=BF, device="cuda")
    out[:3], out[T - 3:] = 7.0, 7.0
    f = H.rope_frequencies(16)[0].cuda()
    H.lora_rope(q.expand(T, 1, 16), None, pos, f, out)
    one = torch.empty((1, 1, 16), dtype=BF, device="cuda")
    H.lora_rope(q, None, i32([4]), f, one)
    last = out[T - 3:].clone()
    torch.cuda.synchronize()
    assert (last[:2] == 7).all() and torch.equal(last[2], one[0])
    del out, pos
    torch.cuda.empty_cache()


def test_nobody_overtakes_a_request_that_waits_for_pages(H):
    """Pages that a refused request asked for stay with it: later requests that need any are refused, those that need none are
    served, and what was handed out before it stands.  A request refused for its lengths holds nothing back."""
    past, new = [0, 0, 5, 15, 0, 3], [10, 70, 3, 4, 1, 2]     # needs 1, 5, 0, 1, 1, 0 pages of a list of 4
    table = np.full((6, 5), -1)
    table[2, 0], table[3, 0], table[5, 0] = 40, 41, 42
    T = 101

    def run(past, new):
        d, cu, kv, pos, slots, head, err = i32(table), i32([0] * 7), i32([0] * 6), i32([0] * T), i32([0] * T), i32([0]), i32([0])
        H.lora_kv_layout(i32(past), i32(new), None, 16, d, i32([60, 61, 62, 63]), i32([0]), cu, kv, pos, slots, None, head, err=err)
        return d.cpu().numpy(), kv.tolist(), slots.tolist(), int(head.item()), int(err.item())
    d, kv, slots, head, err = run(past, new)
    assert err == H.DEV_ERR_NO_PAGES and kv == [10, 0, 8, 0, 0, 5] and head == 1
    assert d[0].tolist() == [60, -1, -1, -1, -1] and (d[1:] == table[1:]).all()
    assert slots[:10] == [960 + i for i in range(10)] and slots[10:80] == [-1] * 70 and slots[80:83] == [645, 646, 647]
    assert slots[83:88] == [-1] * 5 and slots[88:90] == [675, 676]
    d, kv, slots, head, err = run(past, [10, 81, 3, 4, 1, 2])   # the second is too long for its row of the table
    assert err == H.DEV_ERR_BAD_LENGTH and kv == [10, 0, 8, 19, 1, 5] and head == 3 and d[3, 1] == 61 and d[4, 0] == 62
