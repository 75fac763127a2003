"""GPU: the roundings of the 4-bit cache where floating-point steps in between
would move them, against rational arithmetic, and groups beyond fp16's range."""
import numpy as np
import pytest
import torch

from tests import _kv as K
from tests import _kv_exact as E

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def H():
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def cached(H, groups, dtype, src=None):
    """Groups [n, 64] of values of `dtype` as keys and values of one head of 64, one token each -> host cache and read-back."""
    n = groups.shape[0]
    x = groups.to(dtype)[:, None].to(src or dtype).cuda()
    pages = torch.zeros((n // 16 + 1, K.block_bytes(1, 64, 16)), dtype=torch.uint8, device="cuda")
    slots, err = i32(np.arange(n)), i32([0])
    H.lora_kv_append(None, x, x, i32(np.zeros(n)), None, slots, pages, 16, None, dtype=dtype, err=err)
    kb, vb = (torch.empty((n, 1, 64), device="cuda") for _ in range(2))
    H.lora_kv_gather(pages, 16, slots, kb, vb, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return K.Cache(pages.cpu().numpy(), 1, 64, 16), kb[:, 0].cpu(), vb[:, 0].cpu()


def spread(lo, hi, extra=()):
    """64 values of which lo is the least and hi the greatest."""
    x = torch.linspace(0, 1, 64, dtype=torch.float64) * (hi - lo) + lo
    x[0], x[63] = lo, hi
    for i, e in enumerate(extra):
        x[1 + i] = e
    return x


def check(H, groups, dtype, src=None):
    groups = torch.stack(list(groups)).to(dtype)
    cache, kb, vb = cached(H, groups, dtype, src)
    for t in range(groups.shape[0]):
        codes, step, low = E.quantise_group(groups[t].double().tolist())
        for which, back in ((0, kb), (1, vb)):
            c, s, lo = cache.read(t, 0, which)
            assert (float(s[0]), float(lo[0])) == (step, low), (t, which)
            assert c.tolist() == codes, (t, which)
            assert back[t].tolist() == [float(np.float32(n * step + low)) for n in codes]


# (greatest, least) of fp16 groups whose fifteenth of the span lies so near the middle of two fp16 numbers that a rounding to
# fp32 on the way takes it there
PAIRS = [(30.21875, -0.0009760856628417969)]


def pairs(limit=40):
    """More of them: greatest + j units = 15 middles exactly, and a least value of about j units, a last place off."""
    out = []
    for e in range(-13, 4):                                  # middles of fp16 numbers are odd multiples of 2^e, 2049 and up
        for m in range(2049, 4096, 2):
            for j in range(1, 4):
                hi, b = np.ldexp(15.0 * m - j, e), np.float16(np.ldexp(float(j), e))
                if hi > 65504 or np.float64(np.float16(hi)) != hi:
                    continue
                for lo in (-np.nextafter(b, np.float16(0)), -np.nextafter(b, np.float16(9))):
                    q = (hi - np.float64(lo)) / 15
                    if np.float16(np.float32(q)) != np.float16(q):
                        out.append((hi, float(lo)))
    return out[::max(1, len(out) // limit)][:limit]


def test_steps_are_rounded_once(H):
    found = PAIRS + pairs()
    assert len(found) > 8
    groups = [spread(lo, hi) for hi, lo in found] + [spread(-hi, -lo) for hi, lo in found]
    check(H, groups, FP)
    check(H, groups, FP, F32)


def test_steps_between_the_least_fp16_numbers(H):
    """Spans at 15 halves of fp16's least step, with a least value that 64 bits beside them cannot hold."""
    tiny = 2.0 ** -130
    groups = [spread(lo, n * 2.0 ** -24) for n in (7.5, 22.5, 37.5) for lo in (0.0, tiny, -tiny)]
    groups += [-g for g in groups]
    check(H, groups, BF)


def test_codes_beside_a_border(H):
    """Values that differ from a border between codes by less than 64 bits beside the least value hold."""
    tiny = [0.0, 2.0 ** -120, -2.0 ** -120, 2.0 ** -60, -2.0 ** -60, 2.0 ** -20, -2.0 ** -20]
    check(H, [spread(-1.0, 29.0, tiny), spread(-3.0, 27.0, tiny), spread(-5.0, 25.0, tiny), spread(-29.0, 1.0, tiny)], BF)
    tiny = [0.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -14, -2.0 ** -14]
    check(H, [spread(-1.0, 29.0, tiny), spread(-3.0, 27.0, tiny)], FP)


@pytest.mark.parametrize("lo,hi", [(-1e5, 0.0), (-1e5, -0.9e5), (-65536.0, 3.0), (-3e38, -3e38), (66048.0, 66048.0), (1e5, 1.2e5), (7e4, 3e38), (-1e6, 1e6)])
def test_groups_beyond_fp16_read_back_as_nan(H, lo, hi):
    """A least value or a step that fp16 does not hold makes its group NaN, and no other."""
    good = spread(-65280.0, 65280.0)                         # the widest least value that bf16 rows have within fp16's range
    cache, kb, vb = cached(H, torch.stack([good, spread(lo, hi).clamp(lo, hi), good]), BF)
    for back in (kb, vb):
        assert torch.isnan(back[1]).all() and torch.isfinite(back[0]).all() and torch.isfinite(back[2]).all()


def test_a_greatest_value_beyond_fp16_is_fine(H):
    """Codes reach above fp16's range as long as the least value and the step lie within it."""
    check(H, [spread(-6e4, 1e5), spread(0.0, 9e5)], BF)


def test_a_key_beyond_fp16_is_not_dropped(H):
    """Such a key shows as NaN in the attention that sees it; a score of minus infinity would leave it out without a word."""
    q = torch.ones((2, 2, 64), dtype=BF, device="cuda")
    k, v = (torch.randn((3, 1, 64), dtype=BF, device="cuda") for _ in range(2))
    k[2] = spread(-1e5, -0.9e5).to(BF).cuda()
    pages = torch.zeros((2, K.block_bytes(1, 64, 16)), dtype=torch.uint8, device="cuda")
    H.lora_kv_append(None, k, v, i32([0, 1, 2]), None, i32([0, 1, 2]), pages, 16, None)
    out = torch.empty_like(q)
    ws = torch.empty(H.lora_kv_attend_workspace_size(2, 1, 64, 2), dtype=torch.uint8, device="cuda")
    H.lora_kv_attend(q, pages, 16, 1, i32([[0]]), i32([0, 2]), i32([3]), 2, 0.125, out, ws)
    assert torch.isfinite(out[0].float()).all() and torch.isnan(out[1].float()).all()
