"""GPU: attention over the 4-bit cache where every CTA has much to do: rings of
stages that go round, block tables fetched again, references of the scores and of
the values' steps that move, requests cut between CTAs.  Every row is compared
with a 64-bit reference by the norm of its error, which a lost, doubled or
wrongly scaled token shows in."""
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


class Contexts:
    """A cache on the device for requests of these lengths: random codes, steps near 0.3, lows near -7.5 steps; what lies past a
    request's end has NaN parameters.

    rise: what the lows of the keys grow by over a request, in proportion to the token's place (negative: fall);
    grow: the factor by which the values' steps and lows grow over a request."""

    def __init__(self, seed, lens, hk, dim, block, rise=0.0, grow=1.0):
        self.lens, self.hk, self.dim, self.block, self.ng = list(lens), hk, dim, block, dim // 64
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        held = [-(-n // block) for n in lens]
        n_pages, width = sum(held) + 3, max(max(held), 1)
        order = np.random.default_rng(seed).permutation(n_pages)
        self.table = np.full((len(lens), width), -1)
        half = 16 * dim // 2 + 16 * 4 * self.ng
        self.pages = torch.randint(0, 256, (n_pages, K.block_bytes(hk, dim, block)), generator=g, device="cuda", dtype=torch.uint8)
        view = self.pages.view(n_pages, hk, block // 16, 2, half)
        view[..., 16 * dim // 2:] = torch.full((16 * self.ng * 2,), math.nan, dtype=torch.float16, device="cuda").view(torch.uint8)
        at = 0
        for r, n in enumerate(lens):
            self.table[r, :held[r]] = order[at:at + held[r]]
            at += held[r]
            if n == 0:
                continue
            j = torch.arange(held[r] * block, device="cuda").view(held[r], 1, block // 16, 16, 1)       # token of the request
            shape = (held[r], hk, block // 16, 16, self.ng)
            par = []
            for which in (0, 1):
                step = torch.rand(shape, generator=g, device="cuda") * 0.2 + 0.2
                low = step * -7.5 + 0.1 * torch.randn(shape, generator=g, device="cuda")
                x = j / max(n, 1)
                if which == 0:
                    low = low + rise * x
                else:
                    step, low = step * grow ** (x - 1), low * grow ** (x - 1)
                p = torch.stack([step, low], -1)
                par.append(torch.where((j < n)[..., None], p, torch.full_like(p, math.nan)).half())
            p = torch.stack(par, 3).contiguous().view(torch.uint8).flatten(4)      # [blocks, heads, granules, 2, bytes]
            pages = torch.as_tensor(self.table[r, :held[r]], device="cuda")
            view[pages, ..., 16 * dim // 2:] = p

    def values(self, r, h):
        """float64 keys and values [n, D] of request r's kv head h, and the values' (and keys') steps [n]."""
        n, half = self.lens[r], 16 * self.dim // 2 + 16 * 4 * self.ng
        held = -(-n // self.block)
        pages = torch.as_tensor(self.table[r, :held].clip(0), device="cuda")
        x = self.pages[pages].view(held, self.hk, self.block // 16, 2, half)[:, h].transpose(1, 2).transpose(0, 1)  # [2, blocks, granules, half]
        x = x.reshape(2, -1, half)
        c = x[..., :16 * self.dim // 2].reshape(2, -1, self.dim // 2)[:, :n]
        p = x[..., 16 * self.dim // 2:].contiguous().view(torch.float16).reshape(2, -1, self.ng, 2)[:, :n].double()
        codes = torch.stack([c & 15, c >> 4], -1).flatten(-2).double()
        out = codes * p[..., 0].repeat_interleave(64, -1) + p[..., 1].repeat_interleave(64, -1)
        return out[0], out[1], p[0, :, :, 0].amax(-1)


def queries(seed, T, hq, dim, dtype, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((T, hq, dim), generator=g, device="cuda") + mean).to(dtype)


def run(H, c, q, q_lens, max_q, scale, ws=None, table=None):
    hq, err = q.shape[1], i32([0])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    if ws is None:
        ws = torch.randint(0, 256, (H.lora_kv_attend_workspace_size(hq, c.hk, c.dim, max_q),), dtype=torch.uint8, device="cuda")
    H.lora_kv_attend(q, c.pages, c.block, c.hk, i32(c.table if table is None else table), i32(np.r_[0, np.cumsum(q_lens)]), i32(c.lens),
                     max_q, scale, out, ws, lse=lse, err=err)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def check(c, q, q_lens, scale, out, lse, dtype, table=None):
    """The norm of a row's error against what the arithmetic allows:
      the rounding of the outputs, HALF of each element;
      that of a weight times its step to fp16, 2^-11 and independent from key to key: 2^-11 / sqrt(3) times the root of the sum of
      (weight * norm of the values)^2 on average, and twice 2^-11 times it at most;
      the score's, 8 products' accumulations of at most 2^-23 of 1032 times a step times the norm of the query, weighted alike.
    The last two are far below the first for bf16 and near it for fp16.  One token that is missing or counted twice in a request
    of n whose tokens weigh alike is an error of 1 / sqrt(n)."""
    G, at, worst = q.shape[1] // c.hk, 0, 0.0
    for r, (n, L) in enumerate(zip(q_lens, c.lens)):
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        for h in range(c.hk):
            k, v, step = c.values(r, h)
            a = q[rows, h * G:(h + 1) * G].double().transpose(0, 1)                  # [G, n, D]
            s = (a @ k.T) * scale
            hide = torch.arange(L, device="cuda") > (L - n) + torch.arange(n, device="cuda")[:, None]
            if table is not None:
                gone = torch.as_tensor(table[r] < 0, device="cuda").repeat_interleave(c.block)[:L]
                hide = hide | gone
            s = s.masked_fill(hide, -math.inf)
            l = torch.logsumexp(s, -1)
            p = (s - l[..., None]).exp()
            o = p @ v
            delta = 2.0 ** -20 * 1032 * abs(scale) * float(step.max()) * a.norm(dim=-1) + 2.0 ** -21 * s.masked_fill(hide, 0).abs().amax(-1)
            noise = (p.square() @ v.square().sum(-1)).sqrt()
            got = out[rows, h * G:(h + 1) * G].double().transpose(0, 1)
            allowed = K.HALF[dtype] * o.norm(dim=-1) + (2.0 ** -10 + 2 * delta) * noise
            e = (got - o).norm(dim=-1)
            assert (e <= allowed).all(), (r, h, float((e / o.norm(dim=-1)).max()), float((allowed / o.norm(dim=-1)).min()))
            worst = max(worst, float((e / o.norm(dim=-1)).max()))
            y = lse[rows, h * G:(h + 1) * G].double().transpose(0, 1)
            assert ((y - l).abs() <= delta + 2.0 ** -20 * l.abs().clamp(min=1)).all(), (r, h, float((y - l).abs().max()))
    return worst


def ragged(seed, R, top):
    n = np.random.default_rng(seed).integers(1, top + 1, R)
    n[0], n[R // 2] = top, 1
    return [int(x) for x in n]


SHAPES = [(128, 32, 8, 1, BF, 64), (64, 32, 8, 1, FP, 16), (128, 8, 8, 1, FP, 96), (128, 32, 8, 5, FP, 16), (64, 28, 4, 3, BF, 64)]


@pytest.mark.parametrize("dim,hq,hk,n,dtype,block", SHAPES)
@pytest.mark.parametrize("rise,grow", [(0.0, 1.0), (6.0, 64.0), (-6.0, 1.0 / 64)])
def test_much_to_do_for_every_cta(H, dim, hq, hk, n, dtype, block, rise, grow):
    """48 ragged requests: 20 to 70 rounds of 128 tokens for each of 296 or 444 CTAs.  rise: the scores climb by some 60 over the
    longest request, so that their reference moves every few hundred tokens and what was summed before still counts; grow: so do
    the values' steps, by 2^6."""
    lens = ragged(dim + hk, 48, 12000 if hk == 8 else 16384)
    c = Contexts(7 + dim, lens, hk, dim, block, rise, grow)
    q_lens = [min(1 + i % n, x) for i, x in enumerate(lens)]
    q = queries(dim + n, sum(q_lens), hq, dim, dtype, 1.0 if rise else 0.0)
    scale = dim ** -0.5
    out, lse, err = run(H, c, q, q_lens, n, scale)
    assert err == 0
    check(c, q, q_lens, scale, out, lse, dtype)
    again, lse2, _ = run(H, c, q, q_lens, n, scale)
    assert torch.equal(out, again) and torch.equal(lse, lse2)                        # and the same bits again


@pytest.mark.parametrize("lens", [[32749], [3001, 5, 1200], [16000, 16000], [1, 8191, 1, 1, 700], [128 * 40], [40000, 3, 129]])
@pytest.mark.parametrize("dim,hq,hk,n,dtype", [(128, 32, 8, 1, BF), (128, 4, 1, 1, FP), (64, 16, 1, 2, FP), (128, 12, 2, 3, BF)])
def test_few_requests_cut_between_ctas(H, lens, dim, hq, hk, n, dtype):
    c = Contexts(sum(lens), lens, hk, dim, 64, 2.0, 4.0)
    q_lens = [min(n, x) for x in lens]
    q = queries(len(lens), sum(q_lens), hq, dim, dtype, 0.3)
    out, lse, err = run(H, c, q, q_lens, n, 0.1)
    assert err == 0
    check(c, q, q_lens, 0.1, out, lse, dtype)


@pytest.mark.parametrize("n", [1, 4])
def test_blocks_that_are_not_there_in_long_contexts(H, n):
    """They are passed over and flagged; the requests attend to their other blocks."""
    lens = ragged(5, 24, 9000)
    c = Contexts(9, lens, 4, 128, 32)
    q_lens = [min(n, x) for x in lens]
    q = queries(3, sum(q_lens), 16, 128, FP)
    table = c.table.copy()
    r = np.random.default_rng(4)
    for i, x in enumerate(lens):
        held = -(-x // 32)
        table[i, r.random(table.shape[1]) < 0.2] = -1
        table[i, held - 1] = c.table[i, held - 1]                                    # the rows' own tokens stay
    out, lse, err = run(H, c, q, q_lens, n, 0.09, table=table)
    assert err == H.DEV_ERR_BAD_PAGE
    check(c, q, q_lens, 0.09, out, lse, FP, table)


def test_every_length_around_the_rounds(H):
    """Lengths beside the borders of granules, rounds and stages, many requests of each CTA."""
    lens = [x + d for x in (16, 32, 48, 64, 96, 112, 128, 160, 256, 384, 512, 640, 1024) for d in (-1, 0, 1)] * 12
    c = Contexts(3, lens, 8, 128, 16)
    q = queries(2, len(lens), 32, 128, FP)
    out, lse, err = run(H, c, q, [1] * len(lens), 1, 0.09)
    assert err == 0
    check(c, q, [1] * len(lens), 0.09, out, lse, FP)


def test_the_check_sees_single_tokens():
    """What check() is for: a reference with one token less, with values exchanged, or with a piece scaled, is refused.  At a scale
    of 0.01 the weights lie within a factor of some e^2, so that any token counts for about 1 / 3001 of the sum and its error,
    1 / sqrt(3001) of the norm, lies well above what is allowed."""
    c = Contexts(1, [3001], 1, 128, 64)
    q = queries(1, 1, 4, 128, FP)
    k, v, _ = c.values(0, 0)
    s = (q[0].double() @ k.T) * 0.01
    p = (s - s.amax(-1, keepdim=True)).exp()

    def refused(p, v):
        o, l = (p @ v / p.sum(-1, keepdim=True)).to(FP)[None], (s.amax(-1) + p.sum(-1).log()).float()[None]
        try:
            check(c, q, [1], 0.01, o, l, FP)
            return False
        except AssertionError:
            return True

    assert not refused(p, v)
    gone, twice, scaled, turned = p.clone(), p.clone(), p.clone(), v.clone()
    gone[:, 1700], scaled[:, :1500] = 0, scaled[:, :1500] * 1.01
    twice[:, 5] *= 2
    turned[1000:1016] = v[1000:1016].flip(0)
    assert refused(gone, v) and refused(twice, v) and refused(scaled, v) and refused(p, turned)


def test_the_longest_context_that_is_taken(H):
    """2^31 - 32 tokens in blocks of 16, every entry of the table the same page: as 16 tokens, each 134217726 times.

    A warp adds up 134217726 / 1776 = 75572 granules: accumulations of 2^-23 each come to 0.9 %, the two sums of weights a granule
    of 2^-24 each to 0.9 % more."""
    n = ((2 ** 31 - 1) // 16 - 1) * 16
    c = Contexts(2, [16], 1, 64, 16)
    table = torch.full((1, n // 16), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    q = queries(1, 1, 4, 64, FP)
    out, lse, err = torch.full_like(q, 7.0), torch.full((1, 4), 7.0, device="cuda"), i32([0])
    ws = torch.empty(H.lora_kv_attend_workspace_size(4, 1, 64, 1), dtype=torch.uint8, device="cuda")
    H.lora_kv_attend(q, c.pages, 16, 1, table, i32([0, 1]), i32([n]), 1, 0.125, out, ws, lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    k, v, _ = c.values(0, 0)
    s = (q[0].double() @ k.T) * 0.125
    o, l = torch.softmax(s, -1) @ v, torch.logsumexp(s, -1) + math.log(n // 16)
    assert ((out[0].double() - o).norm(dim=-1) <= 2.0 ** -5 * (torch.softmax(s, -1) @ v.abs()).norm(dim=-1)).all()
    assert ((lse[0].double() - l).abs() <= 2.0 ** -5).all()


def test_as_many_requests_as_a_call_takes(H):
    r = np.random.default_rng(8)
    lens = [int(x) for x in r.integers(0, 50, 4096)]
    c = Contexts(4, lens, 1, 64, 16)
    q_lens = [min(int(x), n) for x, n in zip(r.integers(0, 3, 4096), lens)]
    q = queries(5, sum(q_lens), 4, 64, FP)
    out, lse, err = run(H, c, q, q_lens, 2, 0.125)
    assert err == 0
    check(c, q, q_lens, 0.125, out, lse, FP)
