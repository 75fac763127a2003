"""CPU checks of the KV-cache and attention calls: sizes, argument refusals before
any CUDA call, and the binding's own checks."""
import ctypes

import pytest
import torch

from tests import _kv as K

FAKE = 0x7F0000000000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def H():
    from heterogeneous_adapter_batching_b200 import build
    build.build()
    import heterogeneous_adapter_batching_b200 as H
    H.load_library()
    return H


def p(off=0):
    return ctypes.c_void_p(FAKE + off)


def rows(H, off=0, ts=1024, hs=128):
    return ctypes.byref(H.LoraRows(FAKE + off, ts, hs))


def cache(H, **kw):
    a = dict(pages=FAKE, page_bytes=1 << 20, num_pages=64, kv_heads=8, head_dim=128, block_tokens=64)
    a.update(kw)
    return ctypes.byref(H.LoraKvCache(**a))


def test_block_bytes(H):
    for heads in (1, 2, 8, 256):
        for dim in (64, 128):
            for block in (16, 96, 1024):
                n = H.lora_kv_block_bytes(heads, dim, block)
                assert n == K.block_bytes(heads, dim, block) and n % 128 == 0
    for bad in ((0, 128, 16), (257, 128, 16), (8, 96, 16), (8, 256, 16), (8, 128, 0), (8, 128, 17), (8, 128, 1040), (-1, 128, 16)):
        assert H.lora_kv_block_bytes(*bad) == 0


def test_layout_refusals(H):
    lib = H.load_library()

    def call(past=p(), new=p(), R=4, T=8, block=16, table=p(), width=4, free=p(), nfree=10, head=p(64), cu=p(), kv=p(), pos=p(),
             slots=p(), out=p(128)):
        return lib.lora_kv_layout(past, new, None, R, T, block, table, width, free, nfree, head, cu, kv, pos, slots, None, out, None, None)

    assert call(past=None) == -1 and call(new=None) == -1 and call(table=None) == -1 and call(cu=None) == -1 and call(kv=None) == -1
    assert call(pos=None) == -1 and call(slots=None) == -1
    assert call(R=0) == -1 and call(T=-1) == -1 and call(width=0) == -1 and call(nfree=-1) == -1
    assert call(block=0) == -1 and call(block=24) == -1 and call(block=1040) == -1
    assert call(head=p(64), out=p(64)) == -1                    # the list's head is not updated in place
    assert call(R=4097) == -8 and call(width=2 ** 31 // 16) == -8
    assert lib.lora_last_launch_count() == 0


def test_rope_refusals(H):
    lib = H.load_library()

    def call(q=None, hq=8, k=None, hk=2, src=0, T=4, dim=128, pos=p(), freq=p(), rot=128, qo=None, ko=None, dst=0):
        q, k, qo, ko = (rows(H) if x is None else x for x in (q, k, qo, ko))
        return lib.lora_rope(q, hq, k, hk, src, T, dim, pos, freq, rot, 0, 1.0, qo, ko, dst, None)

    assert call(T=0) == 0 and call(hq=0, hk=0) == 0             # nothing to do
    assert call(T=-1) == -1 and call(pos=None) == -1 and call(freq=None) == -1
    assert call(dim=120) == -1 and call(dim=272) == -1 and call(dim=0) == -1
    assert call(rot=8) == -1 and call(rot=144) == -1 and call(rot=-16) == -1
    assert call(src=3) == -1 and call(dst=2) == -1 and call(src=0, dst=1) == -1 and call(src=2, dst=2) == -1
    assert call(q=rows(H, 8)) == -1                             # 16-byte alignment
    assert call(k=rows(H, ts=1028)) == -1 and call(qo=rows(H, hs=132)) == -1 and call(ko=rows(H, ts=-1024)) == -1
    assert call(src=2, q=rows(H, ts=1020), k=rows(H, ts=1020), T=0) == 0   # four fp32 values are 16 bytes
    assert call(hq=-1) == -1 and call(hk=-1) == -1
    assert lib.lora_last_launch_count() == 0


def test_append_and_gather_refusals(H):
    lib = H.load_library()

    def app(kv=None, T=4, hq=8, q=None, k=None, v=None, slots=p(), ko=None, src=0, dst=0):
        kv = cache(H) if kv is None else kv
        q, k, v = (rows(H) if x is None else x for x in (q, k, v))
        return lib.lora_kv_append(q, hq, k, v, src, T, p(), p(), 128, 0, 1.0, slots, kv, rows(H), ko, None, dst, None, None)

    def gat(kv=None, slots=p(), T=4, ko=None, dst=0):
        return lib.lora_kv_gather(cache(H) if kv is None else kv, slots, T, rows(H) if ko is None else ko, None, dst, None, None)

    assert app(T=0) == 0 and gat(T=0) == 0
    assert lib.lora_kv_gather(cache(H), p(), 4, None, None, 0, None, None) == 0
    for bad in (dict(pages=None), dict(pages=FAKE + 8), dict(page_bytes=(1 << 20) + 8), dict(num_pages=0), dict(kv_heads=0),
                dict(head_dim=96), dict(block_tokens=40), dict(page_bytes=K.block_bytes(8, 128, 64) - 16)):
        assert app(kv=cache(H, **bad)) == -1, bad
        assert gat(kv=cache(H, **bad)) == -1, bad
    assert app(kv=cache(H, num_pages=2 ** 31 // 64)) == -8 and gat(kv=cache(H, num_pages=2 ** 31 // 64)) == -8
    assert app(slots=None) == -1 and gat(slots=None) == -1 and app(T=-1) == -1 and gat(T=-1) == -1
    assert app(v=rows(H, 4)) == -1 and app(ko=rows(H, ts=4)) == -1 and gat(ko=rows(H, hs=12)) == -1
    assert app(src=1, dst=0) == -1 and gat(dst=3) == -1
    assert lib.lora_last_launch_count() == 0


def test_attend_refusals(H):
    lib = H.load_library()
    n = H.lora_kv_attend_workspace_size(32, 8, 128, 1)
    assert n > 0 and n % 256 == 0
    assert H.lora_kv_attend_workspace_size(30, 8, 128, 1) == 0 and H.lora_kv_attend_workspace_size(32, 8, 96, 1) == 0
    assert H.lora_kv_attend_workspace_size(32, 8, 128, 0) == 0 and H.lora_kv_attend_workspace_size(0, 8, 128, 1) == 0

    def call(q=None, T=4, hq=32, dtype=0, kv=None, table=p(), width=4, cu=p(), lens=p(), R=4, mq=1, out=None, ws=p(), nb=n):
        q, out = (rows(H) if x is None else x for x in (q, out))
        return lib.lora_kv_attend(q, T, hq, dtype, cache(H) if kv is None else kv, table, width, cu, lens, R, mq, 1.0, out, None, ws, nb,
                                  None, None)

    assert call(T=0) == 0
    assert call(hq=30) == -1 and call(hq=0) == -1 and call(hq=8 * 65) == -1
    assert call(dtype=2) == -1 and call(T=-1) == -1 and call(R=0) == -1 and call(mq=0) == -1 and call(width=0) == -1
    assert call(table=None) == -1 and call(cu=None) == -1 and call(lens=None) == -1
    assert call(q=rows(H, 2)) == -1 and call(out=rows(H, ts=1025)) == -1
    assert call(ws=None) == -7 and call(ws=p(16)) == -7 and call(nb=n - 1) == -7
    assert call(R=4097) == -8 and call(width=2 ** 31 // 64) == -8
    assert call(kv=cache(H, head_dim=80)) == -1
    assert lib.lora_last_launch_count() == 0


def test_prompt_refusals(H):
    lib = H.load_library()

    def call(q=None, k=None, v=None, Tq=4, Tk=4, hq=32, hk=8, dim=128, dtype=0, cq=p(), ck=p(), R=1, out=None, scale=1.0):
        q, k, v, out = (rows(H) if x is None else x for x in (q, k, v, out))
        return lib.lora_prompt_attend(q, k, v, Tq, Tk, hq, hk, dim, dtype, cq, ck, R, scale, out, None, None, None)

    assert call(Tq=0) == 0
    assert call(Tq=-1) == -1 and call(Tk=-1) == -1 and call(R=0) == -1 and call(cq=None) == -1 and call(ck=None) == -1
    assert call(hq=31) == -1 and call(hk=0) == -1 and call(dim=96) == -1 and call(dim=256) == -1 and call(dtype=2) == -1
    assert call(k=rows(H, 8)) == -1 and call(v=rows(H, ts=1026)) == -1 and call(out=rows(H, hs=-128)) == -1
    assert call(R=4097) == -8
    assert call(scale=-1.0) == -1 and call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(q=rows(H, ts=0)) == -1 and call(k=rows(H, hs=0)) == -1 and call(v=rows(H, ts=1 << 39)) == -1   # what a descriptor takes
    assert lib.lora_last_launch_count() == 0


def test_layout_refuses_arrays_that_overlap(H):
    lib = H.load_library()
    R, T, width, nfree = 4, 8, 4, 10
    names = ("past", "new", "ids_in", "free", "head", "table", "cu", "kv", "pos", "slots", "ids", "out")
    size = dict(past=R, new=R, ids_in=R, free=nfree, head=1, table=R * width, cu=R + 1, kv=R, pos=T, slots=T, ids=T, out=1)

    def call(**at):
        a = {k: p(at.get(k, 4096 * (i + 1))) for i, k in enumerate(names)}
        return lib.lora_kv_layout(a["past"], a["new"], a["ids_in"], R, T, 16, a["table"], width, a["free"], nfree, a["head"], a["cu"],
                                  a["kv"], a["pos"], a["slots"], a["ids"], a["out"], None, None)

    where = {k: 4096 * (i + 1) for i, k in enumerate(names)}
    for o in names[5:]:
        for i in names:
            if i != o:   # the first and the last word of i
                assert call(**{o: where[i]}) == -1, (o, i)
                assert call(**{o: where[i] + 4 * (size[i] - 1)}) == -1, (o, i)
                assert call(**{o: where[i] - 4 * (size[o] - 1)}) == -1, (o, i)
    assert lib.lora_last_launch_count() == 0


def test_outputs_whose_rows_overlap_are_refused(H):
    lib = H.load_library()
    n = H.lora_kv_attend_workspace_size(32, 8, 128, 1)
    for bad in (dict(ts=0), dict(hs=0), dict(hs=64), dict(ts=64)):
        o = rows(H, **bad)
        assert lib.lora_rope(rows(H), 8, None, 0, 0, 4, 128, p(), p(), 128, 0, 1.0, o, None, 0, None) == -1, bad
        assert lib.lora_rope(rows(H), 8, rows(H), 2, 0, 4, 128, p(), p(), 128, 0, 1.0, rows(H), o, 0, None) == -1, bad
        for k in range(3):
            out = [o if i == k else rows(H) for i in range(3)]
            assert lib.lora_kv_append(rows(H), 8, rows(H), rows(H), 0, 4, p(), p(), 128, 0, 1.0, p(), cache(H), *out, 0, None, None) == -1, bad
        assert lib.lora_kv_gather(cache(H), p(), 4, o, None, 0, None, None) == -1, bad
        assert lib.lora_kv_gather(cache(H), p(), 4, None, o, 0, None, None) == -1, bad
        assert lib.lora_kv_attend(rows(H), 4, 32, 0, cache(H), p(), 4, p(), p(), 4, 1, 1.0, o, None, p(), n, None, None) == -1, bad
        assert lib.lora_prompt_attend(rows(H), rows(H), rows(H), 4, 4, 32, 8, 128, 0, p(), p(), 1, 1.0, o, None, None, None) == -1, bad
    # rows times heads of a group beyond 31 bits
    assert lib.lora_kv_attend(rows(H), 2 ** 30, 32, 0, cache(H), p(), 4, p(), p(), 4, 1, 1.0, rows(H), None, p(), n, None, None) == -8
    assert lib.lora_prompt_attend(rows(H), rows(H), rows(H), 2 ** 30, 4, 32, 8, 128, 0, p(), p(), 1, 1.0, rows(H), None, None, None) == -8
    assert lib.lora_last_launch_count() == 0


def test_binding_refuses_what_it_cannot_pass(H):
    t = torch.zeros
    q, i = t((4, 8, 128), dtype=torch.bfloat16), t(4, dtype=torch.int32)
    f = t(64)
    for call in (lambda: H.lora_rope(q, None, i, f, q), lambda: H.lora_prompt_attend(q, q, q, i, i, 1.0, q),
                 lambda: H.lora_kv_gather(q[0], 16, i, q), lambda: H.lora_kv_append(None, q, q, i, f, i, q[0], 16, None),
                 lambda: H.lora_kv_attend(q, q[0], 16, 8, t((4, 2), dtype=torch.int32), i, i, 1, 1.0, q, f),
                 lambda: H.lora_kv_layout(i, i, None, 16, t((4, 2), dtype=torch.int32), None, None, i, i, i, i)):
        with pytest.raises(H.LoraError):   # tensors of the host
            call()


def test_reference_quantiser_and_page_format():
    """The reference itself: closed forms, and a page written by hand."""
    import numpy as np
    x = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    x[0, 0, :64] = torch.arange(64) % 16                # low 0, step 1: codes are the values
    x[0, 0, 64:] = -2.5                                 # a constant group: step 0, low the value
    n, s, lo = K.quantise(x)
    assert n[0, 0, :64].tolist() == [i % 16 for i in range(64)] and n[0, 0, 64:].max() == 0
    assert s[0, 0].tolist() == [1.0, 0.0] and lo[0, 0].tolist() == [0.0, -2.5]
    assert K.value(n, s, lo)[0, 0].tolist() == x[0, 0].float().tolist()
    b = np.zeros((2, K.block_bytes(2, 128, 32)), dtype=np.uint8)
    c = K.Cache(b, 2, 128, 32)
    c.write(32 + 17, 1, 1, n[0, 0], s[0, 0], lo[0, 0])  # page 1, second granule, row 1, head 1, the V half
    base = (1 * 2 + 1) * 2304 + 1152
    assert b[1, base + 64:base + 128].tolist() == [(2 * j % 16) | ((2 * j + 1) % 16) << 4 for j in range(32)] + [0] * 32
    assert b[1, base + 1024 + 8:base + 1024 + 16].view(np.float16).tolist() == [1.0, 0.0, 0.0, -2.5]
    assert b[0].max() == 0
    got = c.read(49, 1, 1)
    assert all((a == w).all() for a, w in zip(got, (n[0, 0], s[0, 0], lo[0, 0])))


def test_rope_frequencies():
    """Closed forms of the scalings."""
    import math
    from heterogeneous_adapter_batching_b200 import rope_frequencies as rf
    f, m = rf(128)
    assert f.shape == (64,) and f[0] == 1 and m == 1.0 and abs(float(f[32]) - 10000.0 ** -0.5) < 1e-9
    lin, _ = rf(128, scaling={"kind": "linear", "factor": 4.0})
    assert torch.equal(lin, f / 4)
    ntk, _ = rf(128, scaling={"kind": "ntk", "factor": 4.0})
    assert ntk[0] == 1 and abs(float(ntk[-1] / f[-1]) - 0.25) < 1e-6
    y, m = rf(128, scaling={"kind": "yarn", "factor": 8.0, "original_max_position": 4096})
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-12 and y[0] == f[0] and abs(float(y[-1] / f[-1]) - 0.125) < 1e-6
    assert (y <= f).all() and (y >= f / 8 * (1 - 1e-6)).all()
    b, _ = rf(128, 500000.0, {"kind": "bands", "factor": 8.0, "original_max_position": 8192})
    g, _ = rf(128, 500000.0)
    wave = 2 * math.pi / g.double()
    assert torch.equal(b[wave < 8192 / 4], g[wave < 8192 / 4])
    slow = wave > 8192
    assert ((b[slow] * 8 / g[slow] - 1).abs() < 1e-6).all()
    with pytest.raises(ValueError):
        rf(63)
    with pytest.raises(ValueError):
        rf(64, scaling={"kind": "other", "factor": 2.0, "original_max_position": 1})


@pytest.mark.parametrize("rot_dim,scaling", [(0, None), (64, {"kind": "linear", "factor": 0.0}), (64, {"kind": "linear", "factor": -2.0}),
                                             (64, {"kind": "ntk", "factor": float("nan")}), (2, {"kind": "ntk", "factor": 2.0}),
                                             (64, {"kind": "bands", "factor": 2.0, "original_max_position": 64, "low_freq_factor": 4.0}),
                                             (64, {"kind": "yarn", "factor": float("inf"), "original_max_position": 64})])
def test_rope_frequencies_refusals(rot_dim, scaling):
    from heterogeneous_adapter_batching_b200 import rope_frequencies as rf
    with pytest.raises(ValueError):
        rf(rot_dim, scaling=scaling)


def test_layout_of_held_blocks_refusals(H):
    lib = H.load_library()

    def call(held=p(4096), held_out=p(8192), past=p(), kv=p(12288)):
        return lib.lora_kv_layout_held(past, p(256), None, 4, 0, 16, p(512), 4, p(1024), 10, p(2048), p(2304), kv, None, None, None,
                                       p(3328), held, held_out, None, None)

    assert call(held=None) == -1 and call(held_out=None) == -1 and call(past=None) == -1
    assert call(held_out=p(4096)) == -1 and call(held_out=p(4096 + 12)) == -1      # not in place
    assert call(held=p(12288)) == -1 and call(held_out=p(12288)) == -1             # nor over another array
    assert lib.lora_last_launch_count() == 0


def test_whole_prompt_refusals(H):
    lib = H.load_library()

    def call(q=None, T=4, hq=32, hk=8, dim=128, dtype=0, cu=p(), lens=p(), R=1, scale=1.0):
        return lib.lora_prompt_attend_whole(rows(H) if q is None else q, rows(H), rows(H), T, hq, hk, dim, dtype, cu, lens, R, scale,
                                            rows(H), None, None, None)

    assert call(T=0) == 0
    assert call(lens=None) == -1 and call(cu=None) == -1 and call(T=-1) == -1 and call(R=0) == -1 and call(hq=31) == -1
    assert call(q=rows(H, 8)) == -1 and call(dim=96) == -1 and call(dtype=2) == -1 and call(scale=-1.0) == -1 and call(R=4097) == -8
    assert lib.lora_last_launch_count() == 0


def test_no_rows_need_no_memory(H):
    """A step without tokens: the rows of an empty tensor have no address."""
    lib = H.load_library()
    none = ctypes.byref(H.LoraRows(None, 0, 0))
    assert lib.lora_rope(none, 8, none, 2, 2, 0, 128, None, p(), 128, 0, 1.0, none, none, 0, None) == 0
    assert lib.lora_kv_append(none, 8, none, none, 2, 0, None, p(), 128, 0, 1.0, None, cache(H), none, none, none, 0, None, None) == 0
    assert lib.lora_kv_gather(cache(H), None, 0, none, none, 0, None, None) == 0
    n = H.lora_kv_attend_workspace_size(32, 8, 128, 1)
    assert lib.lora_kv_attend(none, 0, 32, 0, cache(H), p(), 4, p(), p(), 4, 1, 1.0, none, None, p(), n, None, None) == 0
    assert lib.lora_prompt_attend(none, none, none, 0, 0, 32, 8, 128, 0, p(), p(), 1, 1.0, none, None, None, None) == 0
    # rows that are there need theirs as ever
    assert lib.lora_rope(none, 8, None, 0, 2, 1, 128, p(), p(), 128, 0, 1.0, rows(H), None, 0, None) == -1
    assert lib.lora_kv_gather(cache(H), p(), 1, none, None, 0, None, None) == -1
    assert lib.lora_last_launch_count() == 0


def test_a_build_with_other_register_counts_is_refused(H):
    """The prompt kernel's register split holds for the count it was written for; another compiler's fails in the build."""
    from heterogeneous_adapter_batching_b200 import build
    line = ("ptxas info    : Compiling entry function '_ZN4lora1{0}' for 'sm_100a'\nptxas info    : Function properties for _ZN4lora1{0}\n"
            "    8 bytes stack frame, 24 bytes spill stores, 12 bytes spill loads\nptxas info    : Used {1} registers, used 1 barriers\n")
    other = line.format("kv_join_kernelILi64E", 32)
    good = line.format("prompt_kernelILi128E", 168) + other + line.format("prompt_kernelILi64E", 168)
    assert build.check_registers(good, "prompt_kernel", 168) == 2
    for bad in (good + line.format("prompt_kernelILi64ELb1E", 160), good.replace("168", "255"), other, ""):
        with pytest.raises(RuntimeError, match="prompt_kernel"):
            build.check_registers(bad, "prompt_kernel", 168)
    assert set(build.EXACT_REGISTERS) <= {p.rsplit("/", 1)[-1] for p in build.sources()}


def test_attend_refuses_a_scale_that_is_not_finite(H):
    lib = H.load_library()
    n = H.lora_kv_attend_workspace_size(32, 8, 128, 1)
    for scale, rc in ((float("nan"), -1), (float("inf"), -1), (-float("inf"), -1), (-1.0, 0), (0.0, 0)):
        assert lib.lora_kv_attend(rows(H), 0, 32, 0, cache(H), p(), 4, p(), p(), 4, 1, scale, rows(H), None, p(), n, None, None) == rc
