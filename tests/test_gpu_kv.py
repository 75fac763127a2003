"""GPU: block tables and slots, rotary positions, the 4-bit cache's write and
read-back, against 64-bit references."""
import numpy as np
import pytest
import torch

from tests import _kv as K

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def H():
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# --------------------------------------------------------------------------
# lora_kv_layout
# --------------------------------------------------------------------------

def run_layout(H, past, new, T, block, table, free, head=0, req_ids=None, stream=None):
    R = len(past)
    o = {"cu": i32(np.full(R + 1, -7)), "kv_len": i32(np.full(R, -7)), "positions": i32(np.full(T, -7)), "slots": i32(np.full(T, -7)),
         "ids": i32(np.full(T, -7)), "head": i32([-7]), "table": i32(table)}
    err = i32([0])
    H.lora_kv_layout(i32(past), i32(new), None if req_ids is None else i32(req_ids), block, o["table"], None if free is None else i32(free),
                     i32([head]), o["cu"], o["kv_len"], o["positions"], o["slots"], o["ids"], o["head"], err=err, stream=stream)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in o.items()}
    got["err"] = int(err.item())
    return got


def check_layout(H, past, new, T, block, table, free, head=0, req_ids=None):
    got = run_layout(H, past, new, T, block, table, free, head, req_ids)
    ref = K.layout(past, new, req_ids, T, block, np.asarray(table), free, head)
    for k in ("table", "cu", "kv_len", "positions", "slots", "ids"):
        assert np.array_equal(got[k], ref[k]), k
    assert int(got["head"][0]) == ref["head"] and got["err"] == ref["err"]
    return got


def batch(seed, R, block, width, max_new, pad):
    r = np.random.default_rng(seed)
    past = r.integers(0, width * block // 2, R)
    past[r.random(R) < 0.2] = 0
    past[r.random(R) < 0.2] = block * r.integers(0, width // 2 + 1)
    new = np.minimum(r.integers(0, max_new + 1, R), width * block - past)
    held = -(-past // block)
    need = -(-(past + new) // block) - held
    ids = r.permutation(int(held.sum() + need.sum()) + 8)
    table = np.full((R, width), -1)
    table[np.arange(width) < held[:, None]] = ids[:held.sum()]
    return past, new, int(new.sum()) + pad, table, ids[held.sum():], r.integers(-1, 40, R)


@pytest.mark.parametrize("R,block,width,max_new,pad", [
    (1, 16, 1, 1, 0), (1, 16, 3, 40, 5), (3, 32, 5, 1, 0), (64, 16, 20, 1, 64), (65, 64, 9, 200, 1), (255, 96, 4, 7, 0),
    (257, 16, 33, 300, 1000), (1024, 128, 3, 2, 0), (4096, 16, 5, 9, 77)])
def test_layout_matches_the_reference(H, R, block, width, max_new, pad):
    past, new, T, table, free, ids = batch(R + block, R, block, width, max_new, pad)
    got = check_layout(H, past, new, T, block, table, free, 0, ids)
    assert got["err"] == 0
    live = got["slots"][got["slots"] >= 0]
    assert len(np.unique(live)) == len(live) == new.sum()      # no two tokens share a slot


def test_layout_from_the_middle_of_the_list_and_without_ids(H):
    past, new, T, table, free, _ = batch(5, 40, 16, 12, 30, 3)
    check_layout(H, past, new, T, 16, table, np.concatenate([[99991, 99992, 99993], free]), head=3)


def test_layout_of_a_complete_table(H):
    """free_pages NULL: the slots of tokens that are cached already; past 0 lists a whole request."""
    past, new, T, table, free, ids = batch(6, 33, 32, 9, 80, 0)
    first = run_layout(H, past, new, T, 32, table, free, 0, ids)
    total = past + new
    got = check_layout(H, np.zeros_like(past), total, int(total.sum()), 32, first["table"], None, 0, ids)
    tail = np.concatenate([got["slots"][got["cu"][r] + past[r]:got["cu"][r + 1]] for r in range(33)])
    assert np.array_equal(tail, first["slots"][:new.sum()])


def test_layout_nothing_new(H):
    got = check_layout(H, np.array([5, 0, 16]), np.zeros(3, int), 4, 16, np.array([[3], [-1], [4]]), np.array([9]), 0, np.array([1, 2, 3]))
    assert got["err"] == 0 and (got["slots"] == -1).all() and got["head"][0] == 0
    got = check_layout(H, np.array([5]), np.zeros(1, int), 0, 16, np.array([[3]]), np.array([9]))
    assert got["kv_len"].tolist() == [5]


@pytest.mark.parametrize("case", ["dry", "dry, later ones need none", "too long", "negative", "rows", "bad page", "head beyond", "huge"])
def test_layout_failures_stay_with_their_request(H, case):
    block, width = 16, 4
    past, new = np.array([10, 16, 0, 30, 7]), np.array([3, 20, 33, 1, 1])
    table = np.full((5, width), -1)
    table[0, 0], table[1, 0], table[3, :2], table[4, 0] = 50, 51, (52, 53), 54
    free, head, T = np.arange(100, 105), 0, 60
    want = 0
    if case == "dry":
        free, want = free[:3], 16                            # two for request 1, one is not enough for request 2
    elif case == "dry, later ones need none":
        free, want = free[:1], 16
    elif case == "too long":
        past[1], want = 60, 32
        table[1] = [51, 55, 56, 57]
    elif case == "negative":
        past[0], new[2], want = -1, -5, 32
    elif case == "rows":
        T, want = 57, 32
    elif case == "bad page":
        table[0, 0], want = -3, 8
    elif case == "head beyond":
        head, want = 9, 16
    elif case == "huge":
        new[1], past[2], want = 2 ** 31 - 1, 2 ** 31 - 1, 32
    if case == "head beyond":                                # the reference has no such list: nothing can be handed out
        got = run_layout(H, past, new, T, block, table, free, head)
        assert got["err"] == 16 and got["kv_len"].tolist() == [13, 0, 0, 31, 8] and got["head"][0] == 9
        assert np.array_equal(got["table"], table)
        return
    got = check_layout(H, past, new, T, block, table, free, head, np.arange(5))
    assert got["err"] == want


def test_layout_on_a_side_stream_and_replayed(H):
    past, new, T, table, free, ids = batch(9, 50, 16, 9, 5, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = run_layout(H, past, new, T, 16, table, free, 0, ids, stream=side)
    ref = K.layout(past, new, ids, T, 16, table, free, 0)
    assert np.array_equal(a["slots"], ref["slots"])
    # captured once, replayed on lengths changed in place
    R = 50
    dp, dn, di, dt, df, dh = i32(past), i32(new), i32(ids), i32(table), i32(free), i32([0])
    cu, kl, po, sl, ii = i32(np.zeros(R + 1)), i32(np.zeros(R)), i32(np.zeros(T)), i32(np.zeros(T)), i32(np.zeros(T))
    H.lora_kv_layout(dp, dn, di, 16, dt, df, dh, cu, kl, po, sl, ii)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.lora_kv_layout(dp, dn, di, 16, dt, df, dh, cu, kl, po, sl, ii)
    dn.copy_(i32(np.maximum(new - 1, 0)))
    dt.copy_(i32(table))
    g.replay()
    torch.cuda.synchronize()
    ref = K.layout(past, np.maximum(new - 1, 0), ids, T, 16, table, free, 0)
    assert np.array_equal(sl.cpu().numpy(), ref["slots"]) and np.array_equal(dt.cpu().numpy(), ref["table"])


# --------------------------------------------------------------------------
# lora_rope
# --------------------------------------------------------------------------

def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None


def rope_bound(x, ref, dtype, rot, interleaved, mscale, src):
    """fp32 rotation: two products and a sum, sine and cosine rounded once each: within 4 * 2^-24 (|a| + |b|) mscale; then the rounding."""
    mag = x.double().abs()
    n = rot // 2
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    both = mag[..., a] + mag[..., b]
    slack = torch.zeros_like(mag)
    slack[..., a] = slack[..., b] = 4 * 2.0 ** -24 * both * abs(mscale)
    return K.HALF[dtype] * (ref.abs() + slack) + slack + K.TINY[dtype]


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32), (96, 96), (96, 48), (16, 16), (256, 256), (80, 32), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,dst", [(F32, BF), (BF, BF), (F32, FP), (FP, FP)])
def test_rope(H, dim, rot, interleaved, src, dst):
    T, hq, hk = 7, 5, 2
    x = torch.randn((T, hq + hk, dim), generator=gen(dim + rot)).to(src)
    pos = torch.tensor([0, 1, 17, 8191, 131071, 999983, 2 ** 31 - 1])
    f, m = freqs(rot), 1.25
    d = x.cuda()
    q, k = d[:, :hq], d[:, hq:]
    qo, ko = torch.empty((T, hq, dim), dtype=dst, device="cuda"), torch.empty((T, hk, dim), dtype=dst, device="cuda")
    H.lora_rope(q, k, i32(pos), None if f is None else f.cuda(), qo, ko, interleaved=interleaved, mscale=m)
    got = torch.cat([qo, ko], 1).double().cpu()
    ref = K.rotate(x, pos, f, m, interleaved)
    assert ((got - ref).abs() <= rope_bound(x, ref, dst, rot, interleaved, m, src)).all()


@pytest.mark.parametrize("T", [1, 2, 3, 5, 257, 2367, 2368, 2371])
def test_rope_batch_sizes_strides_and_rows_left_alone(H, T):
    """Views of a fused projection, rows with position -1 left as they were, no k."""
    x = torch.randn((T, 9, 64), generator=gen(T))
    pos = torch.arange(T) * 3
    pos[T // 2] = -1
    out = torch.full((T, 12, 64), 7.0, dtype=BF, device="cuda")
    H.lora_rope(x.cuda()[:, 2:8], None, i32(pos), freqs(64).cuda(), out[:, 3:9])
    ref = K.rotate(x[:, 2:8], pos, freqs(64), 1.0, False)
    got = out.double().cpu()
    live = pos >= 0
    assert ((got[:, 3:9] - ref).abs() <= rope_bound(x[:, 2:8], ref, BF, 64, False, 1.0, F32))[live].all()
    assert (got[:, :3] == 7).all() and (got[:, 9:] == 7).all() and (got[~live] == 7).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place(H, interleaved):
    x = torch.randn((33, 6, 128), generator=gen(4)).to(BF)
    pos = torch.randint(0, 5000, (33,), generator=gen(5))
    d, out = x.cuda(), torch.empty((33, 6, 128), dtype=BF, device="cuda")
    f = freqs(64).cuda()
    H.lora_rope(d, None, i32(pos), f, out, interleaved=interleaved)
    H.lora_rope(d, None, i32(pos), f, d, interleaved=interleaved)
    assert torch.equal(d, out)


# --------------------------------------------------------------------------
# lora_kv_append, lora_kv_gather
# --------------------------------------------------------------------------

def append_case(H, T, hq, hk, dim, rot, interleaved, src, dst, block, seed=0, edit=None, dense=True):
    """Append T rows to scattered slots of a cache with garbage in it; everything checked, the rest of the pages included."""
    g = gen(seed)
    x = torch.randn((T, hq + 2 * hk, dim), generator=g)
    x[:, hq:hq + hk, 5::16] *= 9
    if edit:
        edit(x, hq, hk)
    x = x.to(src)
    pos = torch.randint(0, 70000, (T,), generator=g)
    n_pages = T // block + 3
    slots = torch.randperm(n_pages * block, generator=g)[:T]
    if T > 4:
        slots[1], pos[3] = -1, -1
    pages = torch.randint(0, 256, (n_pages, K.block_bytes(hk, dim, block) + 32), generator=g, dtype=torch.uint8)
    f, d, dp, err = freqs(rot), x.cuda(), pages.cuda(), i32([0])
    q, k, v = d[:, :hq], d[:, hq:hq + hk], d[:, hq + hk:]
    qo = torch.full((T, hq, dim), 3.0, dtype=dst, device="cuda") if hq else None
    ko, vo = (torch.full((T, hk, dim), 3.0, dtype=dst, device="cuda") if dense else None for _ in range(2))
    H.lora_kv_append(q if hq else None, k, v, i32(pos), None if f is None else f.cuda(), i32(slots), dp, block, qo, ko, vo,
                     interleaved=interleaved, mscale=1.125, dtype=dst, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    kr = K.rotate(x[:, hq:hq + hk], pos, f, 1.125, interleaved).float().to(dst)
    vr = x[:, hq + hk:].float().to(dst)
    live = (pos >= 0).numpy()
    host = pages.numpy().copy()
    cache = K.Cache(host, hk, dim, block)
    kq, vq = K.quantise(kr), K.quantise(vr)
    for t in np.nonzero(live & (slots.numpy() >= 0))[0]:
        for h in range(hk):
            for which, (n, s, lo) in ((0, kq), (1, vq)):
                cache.write(int(slots[t]), h, which, n[t, h], s[t, h], lo[t, h])
    got = dp.cpu().numpy()
    finite = bool(torch.isfinite(kr.float()).all() and torch.isfinite(vr.float()).all())
    if finite:
        assert np.array_equal(got, host)                     # every byte: codes, parameters, and what was not written
    if dense:
        assert torch.equal(ko.cpu()[live].nan_to_num(), kr[live].nan_to_num()) and torch.equal(vo.cpu()[live].nan_to_num(), vr[live].nan_to_num())
        assert (ko.cpu()[~live] == 3).all() and (vo.cpu()[~live] == 3).all()
    if hq:
        ref = K.rotate(x[:, :hq], pos, f, 1.125, interleaved)
        ok = (qo.double().cpu() - ref).abs() <= rope_bound(x[:, :hq], ref, dst, rot, interleaved, 1.125, src)
        assert ok[live].all() and (qo.cpu()[~live] == 3).all()
    # read back
    for dt in (dst, F32):
        kb, vb = (torch.full((T, hk, dim), 5.0, dtype=dt, device="cuda") for _ in range(2))
        H.lora_kv_gather(dp, block, i32(slots), kb, vb, err=err)
        H.lora_kv_gather(dp, block, i32(slots), None, torch.empty_like(vb), err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        dev = K.Cache(got, hk, dim, block)
        for t in range(T):
            for h in range(hk):
                for which, b in ((0, kb), (1, vb)):
                    row = b[t, h].cpu()
                    if slots[t] < 0:
                        assert (row == 5).all()
                        continue
                    want = torch.from_numpy(K.value(*dev.read(int(slots[t]), h, which))).to(dt)
                    assert torch.equal(row.nan_to_num(nan=1e4), want.nan_to_num(nan=1e4))
    return kr, vr, kb.cpu(), vb.cpu(), live & (slots.numpy() >= 0)


@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 64, False), (128, 32, True), (128, 16, False),
                                                 (64, 64, False), (64, 32, False), (64, 64, True), (64, 16, True), (128, 0, False)])
@pytest.mark.parametrize("src,dst", [(F32, BF), (BF, BF), (F32, FP), (FP, FP)])
def test_append(H, dim, rot, interleaved, src, dst):
    append_case(H, 19, 3, 2, dim, rot, interleaved, src, dst, 32, seed=dim + rot)


@pytest.mark.parametrize("T,hq,hk,block", [(1, 4, 1, 16), (1, 1, 1, 1024), (2, 0, 3, 48), (3, 7, 1, 96), (37, 28, 4, 16), (70, 12, 2, 128), (2369, 1, 1, 64)])
def test_append_sizes(H, T, hq, hk, block):
    append_case(H, T, hq, hk, 128, 128, False, F32, BF, block, seed=T)
    append_case(H, T, hq, hk, 64, 64, False, FP, FP, block, seed=T + 1, dense=False)


def test_append_special_values(H):
    """Constant groups, groups of zeros, denormal ranges, the widest range fp16 parameters reach."""
    def edit(x, hq, hk):
        x[:, hq:] = x[:, hq:].clamp(-4, 4)
        x[0, hq + hk, :64] = 2.5
        x[0, hq + hk, 64:] = 0.0
        x[2, hq + hk, :64] = torch.linspace(-3e-7, 3e-7, 64)
        x[2, hq + hk, 64:] = torch.linspace(0, 6e4, 64)
        x[4, hq + hk, :64] = torch.arange(64) % 31 * 0.5     # codes on every border
        x[4, hq + hk, 64:] = -(torch.arange(64) % 31 * 0.5)
    for src, dst in ((F32, BF), (F32, FP), (FP, FP)):
        append_case(H, 6, 1, 2, 128, 64, False, src, dst, 16, seed=3, edit=edit)


def test_append_not_finite(H):
    """A NaN or an infinity makes its own group NaN and no other; so do values beyond fp16's range."""
    def edit(x, hq, hk):
        x[0, hq + hk, 3] = float("nan")
        x[0, hq + hk + 1, 70] = float("inf")
        x[2, hq + hk, 3] = -float("inf")
        x[2, hq + hk + 1, 64:] = torch.linspace(-3e6, 3e6, 64)
    _, vr, _, vb, live = append_case(H, 6, 1, 2, 128, 0, False, F32, BF, 16, seed=8, edit=edit)
    nan = torch.isnan(vb)
    want = torch.zeros((6, 2, 2), dtype=torch.bool)
    want[0, 0, 0] = want[0, 1, 1] = want[2, 0, 0] = want[2, 1, 1] = True
    got = nan.unflatten(-1, (2, 64)).all(-1)
    assert torch.equal(got[live], want[live]) and torch.equal(nan.unflatten(-1, (2, 64)).any(-1)[live], want[live])


def test_append_a_slot_beyond_the_cache(H):
    x = torch.randn((3, 4, 64), generator=gen(1)).cuda()
    pages = torch.zeros((2, K.block_bytes(2, 64, 16)), dtype=torch.uint8, device="cuda")
    err = i32([0])
    H.lora_kv_append(None, x[:, :2], x[:, 2:], i32([0, 1, 2]), freqs(64).cuda(), i32([5, 32, 2 ** 31 - 1]), pages, 16, None, dtype=BF, err=err)
    assert int(err.item()) == 8
    b = pages.cpu().numpy()
    assert b[1].max() == 0 and b[0].max() > 0
    out = torch.full((3, 2, 64), 5.0, device="cuda")
    err.zero_()
    H.lora_kv_gather(pages, 16, i32([5, 32, -1]), out, err=err)
    assert int(err.item()) == 8 and (out[1:] == 5).all() and not (out[0] == 5).any()


def test_pages_beyond_32_bits(H):
    """Byte offsets of pages and rows above 2^32."""
    big = torch.empty((3, 3 << 30), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([2 * 16 + 3, 1 * 16 + 15, 7])
    x = torch.randn((3, 2, 64), generator=gen(2)).to(BF)
    H.lora_kv_append(None, x.cuda()[:, :1], x.cuda()[:, 1:], i32([0, 0, 0]), None, i32(slots), big, 16, None)
    kb, vb = (torch.empty((3, 1, 64), device="cuda") for _ in range(2))
    H.lora_kv_gather(big, 16, i32(slots), kb, vb)
    for b, r in ((kb, x[:, :1]), (vb, x[:, 1:])):
        assert torch.equal(b.cpu(), torch.from_numpy(K.value(*K.quantise(r))))
    del big
    torch.cuda.empty_cache()
