"""GPU: attention of new tokens over the paged 4-bit cache, against a 64-bit
reference that reads the same pages."""
import math

import numpy as np
import pytest
import torch

from tests import _kv as K

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def H():
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def make_cache(seed, lens, hk, dim, block, k_gain=1.0, poison=True):
    """Pages with normal keys and values for requests of these lengths, everything else (page tails too) garbage: codes at random and
    NaN parameters.  -> (pages uint8, table)."""
    r = np.random.default_rng(seed)
    held = [-(-max(int(n), 0) // block) for n in lens]
    n_pages = sum(held) + 2
    width = max(max(held), 1) + 1
    pages = r.integers(0, 256, (n_pages, K.block_bytes(hk, dim, block) + 16), dtype=np.uint8)
    cache = K.Cache(pages, hk, dim, block)
    if poison:
        blocks = pages[:, :K.block_bytes(hk, dim, block)].reshape(n_pages, -1, cache.half)
        blocks[:, :, 16 * dim // 2:] = np.full(16 * 2 * (dim // 64), np.nan, np.float16).view(np.uint8)
    order = r.permutation(n_pages)
    table = np.full((len(lens), width), -1)
    at = 0
    for i, n in enumerate(lens):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
        if n <= 0:
            continue
        kv = torch.from_numpy(r.standard_normal((int(n), 2 * hk, dim)))
        kv[:, :hk] *= k_gain
        c, s, lo = K.quantise(kv.to(FP))
        for j in range(int(n)):
            slot = int(table[i, j // block]) * block + j % block
            for h in range(hk):
                cache.write(slot, h, 0, c[j, h], s[j, h], lo[j, h])
                cache.write(slot, h, 1, c[j, hk + h], s[j, hk + h], lo[j, hk + h])
    return pages, table


def check(H, q, pages, table, q_lens, lens, hq, hk, dim, block, dtype, q0=0, scale=None, max_q=None, lse=True, stream=None, skip=(), err_want=0):
    """Run and compare every row; rows of requests in `skip` and rows outside have to stay as they were."""
    scale = dim ** -0.5 if scale is None else scale
    T = q.shape[0]
    cu = q0 + np.concatenate([[0], np.cumsum(q_lens)])
    qd = q.cuda()
    out = torch.full_like(qd, 7.0)
    ls = torch.full((T, hq), 7.0, device="cuda") if lse else None
    err = i32([0])
    mq = max(1, max(q_lens)) if max_q is None else max_q
    ws = torch.randint(0, 256, (H.lora_kv_attend_workspace_size(hq, hk, dim, mq),), dtype=torch.uint8, device="cuda")
    dev_pages = torch.from_numpy(pages).cuda()
    H.lora_kv_attend(qd, dev_pages, block, hk, i32(table), i32(cu), i32(lens), mq, scale, out, ws, lse=ls, err=err, stream=stream)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    got, gl = out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None
    cache = K.Cache(pages, hk, dim, block)
    seen = np.zeros(T, dtype=bool)
    G = hq // hk
    for r, n in enumerate(lens):
        if r in skip:
            continue
        a, b = cu[r], cu[r + 1]
        if a == b:
            continue
        seen[a:b] = True
        for h in range(hk):
            k, v, step = K.cached_kv(cache, table[r], max(int(n), 0), h)
            for t in range(a, b):
                m = max(0, int(n) - (b - a) + (t - a) + 1)
                for g in range(G):
                    qv = q[t, h * G + g].double().numpy()
                    o, l, absv = K.attend_row(qv, k[:m], v[:m], scale)
                    delta = K.row_bound(qv, k[:m], scale, step[:m])
                    bound = K.out_bound(o, absv, delta, dtype, 2.0 ** -11)
                    x = got[t, h * G + g]
                    assert (np.abs(x - o) <= bound).all(), (r, t, h, g, np.abs(x - o).max(), bound.min())
                    if lse:
                        y = gl[t, h * G + g]
                        assert y == l if m == 0 else abs(y - l) <= delta + 2.0 ** -20 * max(1, abs(l))
    assert (got[~seen] == 7).all() and (gl is None or (gl[~seen] == 7).all())
    return out


def queries(seed, T, hq, dim, dtype, gain=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn((T, hq, dim), generator=g) * gain).to(dtype)


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (8, 2), (7, 1), (12, 2), (16, 1), (3, 3), (33, 1), (64, 1)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_decode_heads(H, hq, hk, dim, dtype):
    lens = [1, 70, 16, 33]
    pages, table = make_cache(hq + dim, lens, hk, dim, 32)
    check(H, queries(hq, 4, hq, dim, dtype), pages, table, [1] * 4, lens, hq, hk, dim, 32, dtype)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63, 64, 65], [127, 128, 129], [1] * 40, [511], [0, 5, 0], [0], [257, 1, 3, 600, 2, 2, 2]])
@pytest.mark.parametrize("block", [16, 96])
def test_decode_lengths(H, lens, block):
    pages, table = make_cache(len(lens) + block, lens, 2, 128, block)
    check(H, queries(1, len(lens), 8, 128, BF), pages, table, [1] * len(lens), lens, 8, 2, 128, block, BF)


@pytest.mark.parametrize("q_lens,lens", [([4], [4]), ([3, 1, 2], [40, 9, 2]), ([5, 0, 8], [100, 30, 8]), ([1, 17], [64, 130]), ([33], [95]),
                                         ([2, 2], [1, 0]), ([6], [3])])
@pytest.mark.parametrize("hq,hk", [(8, 2), (6, 1), (2, 2), (16, 1)])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
def test_several_new_tokens(H, q_lens, lens, hq, hk, dtype, dim):
    """Causal at the end; rows that come before the request's first token attend to nothing."""
    pages, table = make_cache(sum(q_lens), lens, hk, dim, 16)
    check(H, queries(2, sum(q_lens), hq, dim, dtype), pages, table, q_lens, lens, hq, hk, dim, 16, dtype)


@pytest.mark.parametrize("R", [129, 300])
def test_more_requests_than_threads(H, R):
    lens = np.random.default_rng(R).integers(0, 40, R)
    new = np.random.default_rng(R + 1).integers(0, 3, R)
    pages, table = make_cache(R, lens, 1, 64, 16)
    check(H, queries(R, int(new.sum()), 2, 64, BF), pages, table, list(new), list(lens), 2, 1, 64, 16, BF)


def test_max_q_len_above_the_batch(H):
    pages, table = make_cache(1, [50, 9], 2, 128, 16)
    q = queries(3, 3, 8, 128, BF)
    a = check(H, q, pages, table, [2, 1], [50, 9], 8, 2, 128, 16, BF, max_q=2)
    check(H, q, pages, table, [2, 1], [50, 9], 8, 2, 128, 16, BF, max_q=40)
    assert torch.isfinite(a.float()).all()


def test_long_context_is_split_and_joined(H):
    lens = [3001, 5, 1200]
    for dim, dtype in ((128, BF), (64, FP)):
        pages, table = make_cache(7, lens, 1, dim, 64)
        check(H, queries(4, 3, 4, dim, dtype), pages, table, [1] * 3, lens, 4, 1, dim, 64, dtype)


def test_sharp_and_flat_scores(H):
    """Weights that span hundreds of powers of two, one key that takes all, equal keys, scale 0 and a negative scale."""
    lens = [200, 90]
    for gain, scale in ((8.0, None), (60.0, 1.0), (1.0, 0.0), (3.0, -0.2)):
        pages, table = make_cache(int(gain), lens, 1, 128, 16, k_gain=gain)
        check(H, queries(5, 2, 4, 128, FP, 2.0), pages, table, [1, 1], lens, 4, 1, 128, 16, FP, scale=scale)


def test_values_of_many_sizes(H):
    """Steps from fp16's denormals to thousands in one request: large and small tokens side by side."""
    lens = [150]
    pages, table = make_cache(11, lens, 1, 128, 16)
    cache = K.Cache(pages, 1, 128, 16)
    r = np.random.default_rng(3)
    for j in range(150):
        slot = int(table[0, j // 16]) * 16 + j % 16
        c, s, lo = cache.read(slot, 0, 1)
        f = np.float16(2.0 ** r.integers(-20, 10))
        cache.write(slot, 0, 1, c, (s * f).astype(np.float16), (lo * f).astype(np.float16))
    check(H, queries(6, 1, 8, 128, FP), pages, table, [1], lens, 8, 1, 128, 16, FP)
    for j in range(150):                                       # and all steps zero: constant values
        slot = int(table[0, j // 16]) * 16 + j % 16
        c, s, lo = cache.read(slot, 0, 1)
        cache.write(slot, 0, 1, c, np.zeros_like(s), lo)
    check(H, queries(6, 1, 8, 128, FP), pages, table, [1], lens, 8, 1, 128, 16, FP)


def test_later_tokens_that_are_not_finite(H):
    """Rows before a token with NaN parameters do not see it."""
    lens, n = [40], 4
    pages, table = make_cache(12, lens, 1, 128, 16)
    cache = K.Cache(pages, 1, 128, 16)
    for j in (38, 39):
        slot = int(table[0, j // 16]) * 16 + j % 16
        for which in (0, 1):
            c, s, lo = cache.read(slot, 0, which)
            cache.write(slot, 0, which, c, np.full_like(s, np.nan), np.full_like(lo, np.inf))
    q = queries(8, n, 4, 128, BF)
    qd, out, err = q.cuda(), torch.empty((n, 4, 128), dtype=BF, device="cuda"), i32([0])
    ws = torch.empty(H.lora_kv_attend_workspace_size(4, 1, 128, n), dtype=torch.uint8, device="cuda")
    H.lora_kv_attend(qd, torch.from_numpy(pages).cuda(), 16, 1, i32(table), i32([0, n]), i32(lens), n, 0.1, out, ws, err=err)
    got = out.double().cpu().numpy()
    k, v, step = K.cached_kv(cache, table[0], 38, 0)
    for t in range(2):
        for g in range(4):
            qv = q[t, g].double().numpy()
            m = 40 - n + t + 1
            o, _, absv = K.attend_row(qv, k[:m], v[:m], 0.1)
            assert (np.abs(got[t, g] - o) <= K.out_bound(o, absv, K.row_bound(qv, k[:m], 0.1, step[:m]), BF, 2.0 ** -11)).all()
    assert np.isnan(got[2:]).all()


def test_a_key_that_is_not_finite_reaches_only_its_request(H):
    lens = [20, 30]
    pages, table = make_cache(13, lens, 1, 64, 16)
    cache = K.Cache(pages, 1, 64, 16)
    slot = int(table[0, 0]) * 16 + 3
    c, s, lo = cache.read(slot, 0, 0)
    cache.write(slot, 0, 0, c, np.full_like(s, np.nan), lo)
    q = queries(9, 2, 2, 64, BF)
    qd, out = q.cuda(), torch.empty((2, 2, 64), dtype=BF, device="cuda")
    ws = torch.empty(H.lora_kv_attend_workspace_size(2, 1, 64, 1), dtype=torch.uint8, device="cuda")
    H.lora_kv_attend(qd, torch.from_numpy(pages).cuda(), 16, 1, i32(table), i32([0, 1, 2]), i32(lens), 1, 0.1, out, ws)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


def test_rows_outside_strides_and_a_wide_buffer(H):
    """Queries as a column block of wider rows, rows before and behind the batch left alone, outputs strided too."""
    lens, q_lens = [40, 3], [2, 1]
    pages, table = make_cache(14, lens, 2, 64, 16)
    big = queries(10, 9, 14, 64, BF).cuda()
    out = torch.full((9, 20, 64), 7.0, dtype=BF, device="cuda")
    ws = torch.empty(H.lora_kv_attend_workspace_size(8, 2, 64, 2), dtype=torch.uint8, device="cuda")
    args = (torch.from_numpy(pages).cuda(), 16, 2, i32(table), i32([4, 6, 7]), i32(lens), 2, 0.125)
    H.lora_kv_attend(big[:, 3:11], *args, out[:, 5:13], ws)
    ref = check(H, big[4:7, 3:11].cpu().contiguous(), pages, table, q_lens, lens, 8, 2, 64, 16, BF)
    assert torch.equal(out[4:7, 5:13], ref)
    assert (out[:4] == 7).all() and (out[7:] == 7).all() and (out[:, :5] == 7).all() and (out[:, 13:] == 7).all()


@pytest.mark.parametrize("what", ["table", "too many rows", "too long", "rows beyond"])
def test_bad_requests(H, what):
    lens, q_lens = [40, 20, 33], [1, 2, 1]
    pages, table = make_cache(15, lens, 1, 128, 16)
    q = queries(11, 4, 4, 128, BF)
    if what == "table":                                        # a block that is passed over: the request attends to its other blocks
        bad = table.copy()
        bad[0, 1] = pages.shape[0] + 5
        qd, out, err = q.cuda(), torch.full((4, 4, 128), 7.0, dtype=BF, device="cuda"), i32([0])
        ws = torch.empty(H.lora_kv_attend_workspace_size(4, 1, 128, 2), dtype=torch.uint8, device="cuda")
        H.lora_kv_attend(qd, torch.from_numpy(pages).cuda(), 16, 1, i32(bad), i32([0, 1, 3, 4]), i32(lens), 2, 0.1, out, ws, err=err)
        assert int(err.item()) == 8
        k, v, step = K.cached_kv(K.Cache(pages, 1, 128, 16), table[0], 40, 0)
        keep = np.r_[0:16, 32:40]
        for g in range(4):
            qv = q[0, g].double().numpy()
            o, _, absv = K.attend_row(qv, k[keep], v[keep], 0.1)
            got = out[0, g].double().cpu().numpy()
            assert (np.abs(got - o) <= K.out_bound(o, absv, K.row_bound(qv, k, 0.1, step), BF, 2.0 ** -11)).all()
        bad[0, :] = -1                                         # and with no block at all: nothing
        H.lora_kv_attend(qd, torch.from_numpy(pages).cuda(), 16, 1, i32(bad), i32([0, 1, 3, 4]), i32(lens), 2, 0.1, out, ws, err=err)
        assert (out[0] == 0).all() and torch.isfinite(out.float()).all()
    elif what == "too many rows":
        check(H, q, pages, table, q_lens, lens, 4, 1, 128, 16, BF, max_q=1, skip=(1,), err_want=32)
    elif what == "too long":
        check(H, q, pages, table, q_lens, [40, table.shape[1] * 16 + 1, 33], 4, 1, 128, 16, BF, skip=(1,), err_want=32)
    else:
        check(H, q[:3], pages, table, q_lens, lens, 4, 1, 128, 16, BF, skip=(2,), err_want=32)


def test_same_bits_again_other_streams_and_graphs_that_share_a_workspace(H):
    """No result depends on what ran before: repeated, on a side stream, and as two captured graphs over one workspace."""
    a = dict(lens=[700, 33, 90], q_lens=[1, 1, 1])
    b = dict(lens=[5, 1500], q_lens=[1, 1])
    ws = torch.empty(H.lora_kv_attend_workspace_size(8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    calls, outs, firsts = [], [], []
    for i, c in enumerate((a, b)):
        pages, table = make_cache(20 + i, c["lens"], 2, 128, 16)
        q = queries(30 + i, len(c["lens"]), 8, 128, BF).cuda()
        out = torch.empty_like(q)
        args = (q, torch.from_numpy(pages).cuda(), 16, 2, i32(table), i32(np.arange(len(c["lens"]) + 1)), i32(c["lens"]), 1, 0.09, out, ws)
        H.lora_kv_attend(*args)
        torch.cuda.synchronize()
        calls.append(args)
        outs.append(out)
        firsts.append(out.clone())
    side = torch.cuda.Stream()
    graphs = []
    for args, out, first in zip(calls, outs, firsts):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        H.lora_kv_attend(*args, stream=side)
        side.synchronize()
        assert torch.equal(out, first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            H.lora_kv_attend(*args)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, f) for o, f in zip(outs, firsts))


def test_cache_beyond_32_bits(H):
    """Pages above 2^32 bytes."""
    lens, block = [40], 16
    pages, table = make_cache(25, lens, 1, 64, block)
    n = pages.shape[1]
    big = torch.empty((4, (2 << 30) + 4096), dtype=torch.uint8, device="cuda")
    at = [3, 1, 2]
    for i, p in enumerate(at):
        big[p, :n] = torch.from_numpy(pages[table[0, i]]).cuda()
    q = queries(12, 1, 4, 64, BF)
    ws = torch.empty(H.lora_kv_attend_workspace_size(4, 1, 64, 1), dtype=torch.uint8, device="cuda")
    a, b = torch.empty((1, 4, 64), dtype=BF, device="cuda"), torch.empty((1, 4, 64), dtype=BF, device="cuda")
    rest = (i32([0, 1]), i32(lens), 1, 0.1)
    H.lora_kv_attend(q.cuda(), torch.from_numpy(pages).cuda(), block, 1, i32(table), *rest, a, ws)
    H.lora_kv_attend(q.cuda(), big, block, 1, i32([at]), *rest, b, ws)
    assert torch.equal(a, b)
    del big
    torch.cuda.empty_cache()
