"""GPU: causal attention over longer packed prompts, every row compared with a
64-bit reference by the norm of its error, which a lost or doubled key shows in."""
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


def rows(seed, T, heads, dim, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, heads, dim), generator=g, device="cuda").to(dtype)


def check(q, k, v, cu_q, cu_k, scale, out, lse, dtype):
    """Allowed: HALF of the outputs' norm for their rounding; for the weights', HALF and independent from key to key, the root of
    the sum of (weight * norm of the value)^2 times HALF (1 / sqrt(3) of that on average); for the scores, 2^-20 of the norms'
    product, the exponential and the sums 2^-20.  One key missing of n alike is an error of 1 / sqrt(n)."""
    G = q.shape[1] // k.shape[1]
    for r in range(len(cu_q) - 1):
        n, m = cu_q[r + 1] - cu_q[r], cu_k[r + 1] - cu_k[r]
        if n == 0:
            continue
        hide = torch.arange(m, device="cuda") > (m - n) + torch.arange(n, device="cuda")[:, None]
        none = hide.all(-1) if m else torch.ones(n, dtype=torch.bool, device="cuda")
        for h in range(q.shape[1]):
            a = q[cu_q[r]:cu_q[r + 1], h].double()
            kk, vv = (x[cu_k[r]:cu_k[r + 1], h // G].double() for x in (k, v))
            s = ((a @ kk.T) * scale).masked_fill(hide, -math.inf)
            l = torch.logsumexp(s, -1) if m else torch.full((n,), -math.inf, device="cuda", dtype=torch.float64)
            p = (s - l.masked_fill(none, 0)[:, None]).exp()
            o = p @ vv
            size = a.norm(dim=-1) * (kk.norm(dim=-1).amax() if m else 0) * abs(scale)
            noise = (p.square() @ vv.square().sum(-1)).sqrt()
            e = (out[cu_q[r]:cu_q[r + 1], h].double() - o).norm(dim=-1)
            allowed = K.HALF[dtype] * (o.norm(dim=-1) + noise) + 2.0 ** -19 * (size + 1) * noise
            assert (e <= allowed).all(), (r, h, int((e - allowed).argmax()), float((e - allowed).max()))
            y = lse[cu_q[r]:cu_q[r + 1], h].double()
            ok = torch.isneginf(y) if bool(none.all()) else torch.where(none, torch.isneginf(y), (y - l).abs() <= 2.0 ** -20 * (size + 1 + l.abs()))
            assert ok.all(), (r, h)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hq,hk,dim", [(4, 2, 128), (8, 1, 64), (7, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("q_lens,past", [([2100, 900, 385], [0, 0, 0]), ([1, 130, 1500], [2000, 700, 64]), ([300] * 40, [0, 5, 200, 129] * 10),
                                         ([700, 0, 256], [-40, 3, 128])])
def test_rows_by_their_norm(H, dtype, hq, hk, dim, q_lens, past):
    """Whole prompts, chunks over a past, more rows than keys, many items of every CTA; and the same bits again."""
    cu_q, cu_k = np.r_[0, np.cumsum(q_lens)], np.r_[0, np.cumsum(np.add(q_lens, past))]
    q, k, v = (rows(i + dim, int(c[-1]), n, dim, dtype) for i, (c, n) in enumerate(((cu_q, hq), (cu_k, hk), (cu_k, hk))))
    scale, outs = dim ** -0.5, []
    for _ in range(2):
        out, lse, err = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda"), i32([0])
        H.lora_prompt_attend(q, k, v, i32(cu_q), i32(cu_k), scale, out, lse=lse, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    check(q, k, v, [int(x) for x in cu_q], [int(x) for x in cu_k], scale, out, lse, dtype)


def test_as_many_requests_as_a_call_takes(H):
    n = np.random.default_rng(6).integers(0, 12, 4096)
    n[4000] = 700
    cu = [int(x) for x in np.r_[0, np.cumsum(n)]]
    q, k, v = (rows(i, cu[-1], m, 64, FP) for i, m in ((1, 2), (2, 1), (3, 1)))
    out, lse, err = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda"), i32([0])
    H.lora_prompt_attend(q, k, v, i32(cu), i32(cu), 0.125, out, lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(q, k, v, cu, cu, 0.125, out, lse, FP)
