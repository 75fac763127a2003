"""GPU: causal attention over packed prompts, against a 64-bit reference."""
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


def rows(seed, T, heads, dim, dtype, gain=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn((T, heads, dim), generator=g) * gain).to(dtype)


def check_rows(got, gl, q, k, v, cu_q, cu_k, scale, dtype, skip=(), step=1):
    """Every `step`-th row of each request and its last one, whole rows; rows outside as they were (7)."""
    G = q.shape[1] // k.shape[1]
    T = q.shape[0]
    seen = np.zeros(T, dtype=bool)
    for r in range(len(cu_q) - 1):
        a, b, c, d = (int(x) for x in (cu_q[r], cu_q[r + 1], cu_k[r], cu_k[r + 1]))
        if r in skip:
            continue
        seen[a:b] = True
        for t in sorted(set(range(a, b, step)) | set(range(max(a, b - 1), b))):
            m = min(max(0, (d - c) - (b - a) + (t - a) + 1), d - c)
            for h in range(k.shape[1]):
                kk, vv = k[c:c + m, h].double().numpy(), v[c:c + m, h].double().numpy()
                for g in range(G):
                    qv = q[t, h * G + g].double().numpy()
                    o, l, absv = K.attend_row(qv, kk, vv, scale)
                    delta = K.row_bound(qv, kk, scale)
                    bound = K.out_bound(o, absv, delta, dtype, K.HALF[dtype])
                    x = got[t, h * G + g]
                    assert (np.abs(x - o) <= bound).all(), (r, t - a, h, g, np.abs(x - o).max(), bound.min())
                    if gl is not None:
                        y = gl[t, h * G + g]
                        assert y == l if m == 0 else abs(y - l) <= delta + 2.0 ** -20 * max(1, abs(l))
    assert (got[~seen] == 7).all() and (gl is None or (gl[~seen] == 7).all())


def run(H, q, k, v, cu_q, cu_k, scale, lse=True, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    ls = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    err = i32([0])
    H.lora_prompt_attend(q.cuda(), k.cuda(), v.cuda(), i32(cu_q), i32(cu_k), scale, out, lse=ls, err=err, stream=stream)
    torch.cuda.synchronize()
    return out, ls, int(err.item())


def check(H, q_lens, k_lens, hq, hk, dim, dtype, seed=0, q0=0, k0=0, tail=0, scale=None, gain=1.0, step=1):
    scale = dim ** -0.5 if scale is None else scale
    cu_q, cu_k = q0 + np.r_[0, np.cumsum(q_lens)], k0 + np.r_[0, np.cumsum(k_lens)]
    q, k, v = (rows(seed + i, int(c[-1]) + tail, n, dim, dtype, gain if i < 2 else 1.0)
               for i, (c, n) in enumerate(((cu_q, hq), (cu_k, hk), (cu_k, hk))))
    out, ls, err = run(H, q, k, v, cu_q, cu_k, scale)
    assert err == 0
    check_rows(out.double().cpu().numpy(), ls.double().cpu().numpy(), q, k, v, cu_q, cu_k, scale, dtype, step=step)
    return out


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (8, 2), (7, 1), (6, 2), (12, 1), (16, 1), (3, 3), (33, 1), (64, 1)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_heads(H, hq, hk, dim, dtype):
    n = [5, 40, 1]
    check(H, n, n, hq, hk, dim, dtype, seed=hq)


@pytest.mark.parametrize("n", [[1], [2], [31], [32], [33], [63, 64, 65], [127], [128], [129], [255, 1, 256, 257], [1] * 50, [0, 3, 0, 0, 9, 0]])
@pytest.mark.parametrize("hq,hk", [(4, 1), (2, 2), (8, 1)])
def test_lengths(H, n, hq, hk):
    check(H, n, n, hq, hk, 128, BF, seed=len(n), step=3)


@pytest.mark.parametrize("dim,dtype", [(64, FP), (128, BF), (128, FP), (64, BF)])
def test_longer_prompts(H, dim, dtype):
    n = [700, 1100, 385]
    check(H, n, n, 4, 2, dim, dtype, seed=dim, step=37)


@pytest.mark.parametrize("q_lens,k_lens", [([1], [200]), ([3, 40], [130, 41]), ([130], [513]), ([5, 5], [2, 0]), ([200], [3]), ([300], [129]), ([2], [0]),
                                           ([260, 0, 1], [400, 77, 128])])
@pytest.mark.parametrize("hq,hk,dim", [(4, 1, 128), (3, 1, 64)])
def test_prefix_and_fewer_keys_than_rows(H, q_lens, k_lens, hq, hk, dim):
    """m > n: a cached prefix; m < n: the first rows attend to nothing."""
    check(H, q_lens, k_lens, hq, hk, dim, BF, seed=sum(q_lens), step=5)


@pytest.mark.parametrize("R", [33, 257, 700])
def test_many_requests(H, R):
    n = np.random.default_rng(R).integers(0, 9, R)
    n[[3, R // 2, R - 1]] = 150, 0, 130
    check(H, list(n), list(n), 4, 2, 64, BF, seed=R, step=3)


def test_rows_outside_the_batch(H):
    check(H, [20, 33], [20, 33], 4, 2, 64, FP, q0=3, k0=11, tail=9)


def test_sharp_and_flat_scores(H):
    for gain, scale in ((6.0, None), (20.0, 1.0), (1.0, 0.0), (2.0, 1e-20)):
        check(H, [150], [150], 4, 1, 128, FP, seed=int(gain), gain=gain, scale=scale, step=7)
        check(H, [150], [150], 4, 1, 64, BF, seed=int(gain), gain=gain, scale=scale, step=7)


def test_rising_scores(H):
    """Every next key scores higher than all before: the running maximum moves at every tile."""
    n, dim = 600, 128
    q = torch.zeros((n, 2, dim))
    q[:, :, 0] = 4.0
    k = rows(1, n, 1, dim, FP).float() * 0.1
    k[:, 0, 0] = torch.linspace(0, 200, n)
    v = rows(2, n, 1, dim, FP)
    q, k = q.to(FP), k.to(FP)
    out, ls, err = run(H, q, k, v, [0, n], [0, n], 0.5)
    check_rows(out.double().cpu().numpy(), ls.double().cpu().numpy(), q, k, v, [0, n], [0, n], 0.5, FP, step=13)
    k[:, 0, 0] = torch.linspace(200, 0, n).to(FP)               # and falling: the first key takes all
    out, ls, err = run(H, q, k, v, [0, n], [0, n], 0.5)
    check_rows(out.double().cpu().numpy(), ls.double().cpu().numpy(), q, k, v, [0, n], [0, n], 0.5, FP, step=13)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_requests_do_not_reach_a_request(H, bad):
    """Rows of neighbours, of the next request in the same tile, and behind the last one hold NaN or infinities."""
    cu = np.array([6, 40, 70, 190])
    q, k, v = (rows(i, 230, n, 128, BF) for i, n in ((1, 4), (2, 1), (3, 1)))
    for x in (q, k, v):
        x[:6], x[40:70], x[190:] = bad, bad, bad
    out, ls, err = run(H, q, k, v, cu, cu, 0.1)
    assert err == 0
    got = out.double().cpu().numpy()
    G = 4
    for a, b in ((6, 40), (70, 190)):
        for t in range(a, b, 3):
            kk, vv = k[a:t + 1, 0].double().numpy(), v[a:t + 1, 0].double().numpy()
            for g in range(G):
                qv = q[t, g].double().numpy()
                o, _, absv = K.attend_row(qv, kk, vv, 0.1)
                assert (np.abs(got[t, g] - o) <= K.out_bound(o, absv, K.row_bound(qv, kk, 0.1), BF, K.HALF[BF])).all()
    assert (got[:6] == 7).all() and (got[190:] == 7).all()


def test_later_keys_that_are_not_finite(H):
    """A key that is not finite does not reach the rows before it."""
    n = 200
    q, k, v = (rows(i, n, m, 64, BF) for i, m in ((1, 2), (2, 1), (3, 1)))
    k[150:] = float("nan")
    out, _, _ = run(H, q, k, v, [0, n], [0, n], 0.1)
    got = out.double().cpu().numpy()
    for t in range(0, 150, 7):
        for g in range(2):
            kk, vv, qv = k[:t + 1, 0].double().numpy(), v[:t + 1, 0].double().numpy(), q[t, g].double().numpy()
            o, _, absv = K.attend_row(qv, kk, vv, 0.1)
            assert (np.abs(got[t, g] - o) <= K.out_bound(o, absv, K.row_bound(qv, kk, 0.1), BF, K.HALF[BF])).all()
    assert np.isnan(got[150:]).all()


def test_views_of_a_fused_projection(H):
    n, hq, hk, dim = 300, 6, 2, 128
    x = rows(5, n, hq + 2 * hk, dim, BF)
    d = x.cuda()
    out = torch.full((n, hq + 4, dim), 7.0, dtype=BF, device="cuda")
    cu = i32([0, 170, 300])
    H.lora_prompt_attend(d[:, :hq], d[:, hq:hq + hk], d[:, hq + hk:], cu, cu, 0.09, out[:, 2:2 + hq])
    ref, _, _ = run(H, x[:, :hq].contiguous(), x[:, hq:hq + hk].contiguous(), x[:, hq + hk:].contiguous(), [0, 170, 300], [0, 170, 300], 0.09, lse=False)
    assert torch.equal(out[:, 2:2 + hq], ref) and (out[:, :2] == 7).all() and (out[:, 2 + hq:] == 7).all()
    # heads as the slower dimension, and one token's rows (whose stride says nothing)
    t = d[:, :hq].transpose(0, 1).contiguous().transpose(0, 1)
    o2 = torch.empty((hq, n, dim), dtype=BF, device="cuda").transpose(0, 1)
    H.lora_prompt_attend(t, d[:, hq:hq + hk], d[:, hq + hk:], cu, cu, 0.09, o2)
    assert torch.equal(o2, ref)
    o3 = torch.empty((1, hq, dim), dtype=BF, device="cuda")
    H.lora_prompt_attend(d[:1, :hq], d[:1, hq:hq + hk], d[:1, hq + hk:], i32([0, 1]), i32([0, 1]), 0.09, o3)
    assert torch.equal(o3[0], d[0, hq + hk:].repeat_interleave(3, 0))


@pytest.mark.parametrize("cu_q,cu_k,skip", [([0, 10, 5, 30], [0, 10, 20, 30], (1, 2)), ([0, 10, 20, 40], [0, 10, 20, 30], (2,)), ([-1, 10, 20, 30], [0, 10, 20, 30], (0,)),
                                            ([0, 10, 20, 30], [0, 10, 40, 30], (1, 2)), ([0, 10, 20, 30], [0, 10, 8, 30], (1,)), ([0, 10, 20, 30], [-2, 10, 20, 30], (0,))])
def test_bad_row_ranges(H, cu_q, cu_k, skip):
    """A request whose range is not one is flagged; the others are as ever."""
    q, k, v = (rows(i, 30, n, 64, BF) for i, n in ((1, 2), (2, 1), (3, 1)))
    out, ls, err = run(H, q, k, v, cu_q, cu_k, 0.2)
    assert err == 32
    got = out.double().cpu().numpy()
    for r in range(3):
        if r in skip:
            continue
        a, b, c, d = cu_q[r], cu_q[r + 1], cu_k[r], cu_k[r + 1]
        if r == 0 and cu_q[1] == 10 and cu_q[2] == 5:
            b = 5                                              # rows 5..9 are claimed twice
        for t in range(a, b):
            m = (d - c) - (cu_q[r + 1] - a) + t - a + 1
            for g in range(2):
                kk, vv, qv = k[c:c + m, 0].double().numpy(), v[c:c + m, 0].double().numpy(), q[t, g].double().numpy()
                o, _, absv = K.attend_row(qv, kk, vv, 0.2)
                assert (np.abs(got[t, g] - o) <= K.out_bound(o, absv, K.row_bound(qv, kk, 0.2), BF, K.HALF[BF])).all()


@pytest.mark.parametrize("R", [9, 400])
def test_row_ranges_that_turn_back_again_and_again(H, R):
    """Every other request is refused; the others name the same rows over and over.  The call ends, says so, and writes those
    rows only."""
    T = 300
    q, k, v = (rows(90 + i, T + 5, n, 64, BF) for i, n in enumerate((2, 1, 1)))
    cu = np.arange(R + 1) % 2 * T
    out, ls, err = run(H, q, k, v, cu, cu, 0.125)
    assert err == H.DEV_ERR_BAD_LENGTH and (out[T:] == 7).all() and (ls[T:] == 7).all()


def test_no_keys_at_all(H):
    q, k = rows(1, 5, 2, 64, BF), torch.empty((0, 1, 64), dtype=BF)
    out, ls, err = run(H, q, k, k, [0, 5], [0, 0], 0.2)
    assert err == 0 and (out == 0).all() and torch.isneginf(ls).all()


def test_same_bits_again_side_stream_and_graph(H):
    n = [300, 5, 129]
    cu = np.r_[0, np.cumsum(n)]
    q, k, v = (rows(i, int(cu[-1]), m, 128, BF) for i, m in ((1, 8), (2, 2), (3, 2)))
    first, _, _ = run(H, q, k, v, cu, cu, 0.09, lse=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, _, _ = run(H, q, k, v, cu, cu, 0.09, lse=False, stream=side)
    assert torch.equal(first, again)
    dq, dk, dv, dc, out = q.cuda(), k.cuda(), v.cuda(), i32(cu), torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.lora_prompt_attend(dq, dk, dv, dc, dc, 0.09, out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
