"""Host tests of the chunk operators (include/mk_chunk.h): what they refuse before anything is
launched, and the rotary frequencies.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest

import persistent_moe_decode_megakernel_gb300 as mk


@pytest.fixture(scope="module", autouse=True)
def built():
    mk.build()


def i32(*v):
    return np.array(v, dtype=np.int32)


def shape(**over):
    s = mk.CacheShape(8, 2, 128, 16, 32, 8, 0)
    for k, v in over.items():
        setattr(s, k, v)
    return s


PTR = 1 << 20    # an aligned address that no refused call reads


def append(sh, cl=(3,), sl=(5,), n=None, rope=None, eps=1e-6, stride=None, qkv=PTR, kv=PTR, bt=PTR, q_out=PTR, qn=None,
           status=None):
    cl, sl = i32(*cl), i32(*sl)
    stride = (sh.num_q_heads + 2 * sh.num_kv_heads) * sh.head_dim if stride is None else stride
    return mk.lib().mk_append_chunk(ctypes.byref(sh), len(cl) if n is None else n, cl.ctypes.data, sl.ctypes.data, bt, qkv,
                                    stride, None if rope is None else ctypes.byref(rope.struct), qn, None, eps, q_out, kv,
                                    status, None)


def attend(sh, cl=(3,), sl=(5,), n=None, stride=None, q=PTR, kv=PTR, bt=PTR, out=PTR, ws=None, ws_bytes=0, status=None):
    cl, sl = i32(*cl), i32(*sl)
    stride = sh.num_q_heads * sh.head_dim if stride is None else stride
    return mk.lib().mk_chunk_attention(ctypes.byref(sh), len(cl) if n is None else n, cl.ctypes.data, sl.ctypes.data, bt, q,
                                       stride, kv, out, ws, ws_bytes, status, None)


def read(sh, cl=(3,), sl=(5,), n=None, kv=PTR, bt=PTR, k=PTR, v=PTR, status=None):
    cl, sl = i32(*cl), i32(*sl)
    return mk.lib().mk_read_cache(ctypes.byref(sh), len(cl) if n is None else n, cl.ctypes.data, sl.ctypes.data, bt, kv, k, v,
                                  status, None)


BAD, NO = mk.MK_ERR_INVALID_ARG, mk.MK_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [append, attend, read])
@pytest.mark.parametrize("over,code", [
    (dict(num_q_heads=0), BAD), (dict(num_kv_heads=-1), BAD), (dict(num_kv_heads=3), BAD), (dict(page_size=0), BAD),
    (dict(num_pages=0), BAD), (dict(max_pages_per_seq=0), BAD), (dict(flags=1), BAD), (dict(flags=4), BAD),
    (dict(head_dim=96), NO), (dict(num_q_heads=18), NO), (dict(page_size=12), NO), (dict(flags=2, head_dim=64), NO),
    (dict(num_q_heads=2048, num_kv_heads=2048), NO), (dict(page_size=1 << 28, max_pages_per_seq=8), NO),
    (dict(num_pages=1 << 30), NO)])
def test_refuses_shapes(call, over, code):
    assert call(shape(**over)) == code
    assert mk.lib().mk_last_error().decode() != ""


@pytest.mark.parametrize("call", [append, attend, read])
@pytest.mark.parametrize("cl,sl,n,code", [
    ((-1,), (5,), None, BAD), ((6,), (5,), None, BAD), ((1,), (129,), None, BAD), ((3,), (5,), 0, BAD),
    ((1,) * 65, (1,) * 65, None, BAD), ((1, 2, 9), (1, 2, 8), None, BAD)])
def test_refuses_lengths(call, cl, sl, n, code):
    assert call(shape(), cl, sl, n) == code


def test_refuses_too_many_rows():
    sh = shape(max_pages_per_seq=1 << 26)
    for call in (append, attend, read):
        assert call(sh, (1 << 24,), (1 << 24,)) == NO
    assert attend(shape(num_q_heads=1024, num_kv_heads=128, max_pages_per_seq=1 << 20), (1 << 21,), (1 << 21,)) == NO


def test_refuses_pointers_and_strides():
    sh = shape()
    for k in ("qkv", "kv", "q_out"):
        assert append(sh, **{k: None}) == BAD and append(sh, **{k: PTR + 8}) == BAD
    assert append(sh, bt=None) == BAD and append(sh, bt=PTR + 2) == BAD and append(sh, qn=PTR + 4) == BAD
    assert append(sh, stride=12 * 128 - 8) == BAD and append(sh, stride=12 * 128 + 4) == BAD
    for k in ("q", "kv", "out"):
        assert attend(sh, **{k: None}) == BAD and attend(sh, **{k: PTR + 8}) == BAD
    assert attend(sh, bt=None) == BAD and attend(sh, stride=8 * 128 - 8) == BAD and attend(sh, stride=8 * 128 + 2) == BAD
    assert attend(sh, ws=PTR + 4) == BAD
    for k in ("kv", "k", "v"):
        assert read(sh, **{k: None}) == BAD and read(sh, **{k: PTR + 8}) == BAD
    for call in (append, attend, read):
        assert call(sh, status=PTR + 1) == BAD
    assert mk.lib().mk_append_chunk(None, 1, None, None, None, None, 0, None, None, None, 0.0, None, None, None, None) == BAD


@pytest.mark.parametrize("eps", [-1.0, math.nan, math.inf])
def test_refuses_eps(eps):
    assert append(shape(), eps=eps) == BAD


def test_refuses_rotations():
    def rope(n, **over):
        r = mk.Rope(np.ones(n))
        for k, v in over.items():
            setattr(r.struct, k, v)
        return r
    for r in (rope(4), rope(72), rope(8, rotary_dim=-16), rope(8, interleaved=2), rope(8, mscale=math.nan),
              rope(8, inv_freq=None), mk.Rope([1.0] * 7 + [math.inf])):
        assert append(shape(), rope=r) == BAD


def test_no_rows_is_no_work():
    # nothing is launched, so no device is needed and pointers may be NULL
    for call in (append, attend, read):
        assert call(shape(), (0, 0), (5, 0)) == mk.MK_OK
    assert attend(shape(), (0,), (0,), q=None, kv=None, bt=None, out=None) == mk.MK_OK
    assert mk.chunk_attention_workspace(shape(), [0], [0]) == 0


def test_rope_frequencies():
    f = mk.rope_frequencies(128, 1e4)
    assert np.allclose(f, 1e4 ** (-2.0 * np.arange(64) / 128), rtol=1e-15)
    assert np.allclose(mk.rope_frequencies(128, 1e4, factor=4), f / 4, rtol=1e-15)
    # by parts: fast pairs kept, slow ones divided, a falling ramp of the kept share between
    g = mk.rope_frequencies(128, 1e4, factor=8, original_len=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(g[turns > 33], f[turns > 33]) or np.allclose(g[turns > 40], f[turns > 40], rtol=1e-15)
    assert np.allclose(g[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-12)
    share = (g / f - 1 / 8) / (1 - 1 / 8)
    assert np.all(np.diff(share) <= 1e-12) and share.min() >= -1e-12 and share.max() <= 1 + 1e-12
    lo = math.floor(128 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4)))
    hi = math.ceil(128 * math.log(4096 / (1 * 2 * math.pi)) / (2 * math.log(1e4)))
    assert np.allclose(share, 1 - np.clip((np.arange(64) - lo) / (hi - lo), 0, 1), atol=1e-12)
    for bad in ((127, 1e4), (0, 1e4), (128, 1.0), (128, math.inf)):
        with pytest.raises(mk.MkError):
            mk.rope_frequencies(*bad)
    for bad in (dict(factor=0.5), dict(factor=math.nan), dict(original_len=-1), dict(original_len=9, beta_fast=1.0),
                dict(original_len=9, beta_slow=0.0)):
        with pytest.raises(mk.MkError):
            mk.rope_frequencies(128, 1e4, **bad)


def check_plan(sh, cl, sl):
    """Every position tile of every (sequence, unit, KV head) in exactly one segment, a sequence in one
    launch, no segment empty, the cut items' partials distinct and in block order; returns the tiles of
    each launch's blocks."""
    seg = mk.plan_chunk_attention(sh, cl, sl)
    G = sh.num_q_heads // sh.num_kv_heads
    ut = 2 * (128 // G)
    want = {}
    for s, (c, n) in enumerate(zip(cl, sl)):
        for u in range(-(-c // ut)):
            for h in range(sh.num_kv_heads):
                want[s, u, h] = (n - c + min(c, (u + 1) * ut) - 1) // 128 + 1
    got, slots, load, where = {}, (set(), set()), ({}, {}), {}
    for launch, b, s, u, h, t0, n, total, slot in seg.tolist():
        assert where.setdefault(s, launch) == launch
        assert n > 0 and want[s, u, h] == total and t0 + n <= total
        assert got.get((s, u, h), 0) == t0       # segments of an item come in order, blocks ascending
        got[s, u, h] = t0 + n
        load[launch][b] = load[launch].get(b, 0) + n
        if n == total:
            assert slot == -1
        else:
            assert slot == 2 * b + (t0 == 0) and slot not in slots[launch]
            slots[launch].add(slot)
    assert got == want
    for launch in (0, 1):
        blocks = seg[seg[:, 0] == launch][:, 1]
        assert blocks.size == 0 or (blocks.max() < 152 and np.all(np.diff(blocks) >= 0))
    # staged sequences are q8_0 ones of many units, and the workspace holds their tiles and the partials
    staged = [s for s, launch in where.items() if launch == 1]
    assert all(sh.flags == mk.FLAG_KV_Q8 and -(-cl[s] // ut) >= 6 for s in staged)
    tiles = sum(-(-sl[s] // 128) for s in staged) * 2 * sh.num_kv_heads * 128 * sh.head_dim * 2
    assert tiles <= 1 << 30
    rows = max([min(c, ut) for c in cl], default=0) * G
    parts = (max(slots[0] | slots[1]) + 1) * (sh.head_dim + 4) * 4 if slots[0] | slots[1] else 0
    bytes_ = mk.chunk_attention_workspace(sh, cl, sl)
    assert bytes_ >= tiles and (bytes_ > tiles) == (parts > 0) and bytes_ <= tiles + 2 * 152 * rows * (sh.head_dim + 4) * 4
    return load


@pytest.mark.parametrize("seed", range(40))
def test_plan_covers_every_tile_once(seed):
    g = np.random.default_rng(seed)
    hkv, G = int(g.choice([1, 2, 4, 8])), int(g.integers(1, 9))
    sh = shape(num_q_heads=hkv * G, num_kv_heads=hkv, max_pages_per_seq=1 << 16, num_pages=1 << 10)
    n = int(g.integers(1, 65))
    sl = np.exp(g.uniform(0, np.log(g.choice([200, 5000, 200000])), n)).astype(int)
    top = int(g.choice([1, 64, 3000]))
    cl = [int(g.integers(0, min(x, top) + 1)) for x in sl]
    check_plan(sh, cl, sl.tolist())
    sh.flags = mk.FLAG_KV_Q8
    check_plan(sh, cl, sl.tolist())


@pytest.mark.parametrize("cl,sl", [([1], [131073]), ([1], [1]), ([8192], [8192]), ([2048], [32768]), ([1024], [16384]),
                                   ([1] * 64, [32768] * 64), ([200000], [200000]), ([1], [1 << 20])])
def test_plan_is_even(cl, sl):
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 16)
    load = check_plan(sh, cl, sl)[0]
    total = sum(load.values())
    if total > 152 * 8:      # enough to go round: the longest block within 15 % and a few tiles of even
        assert max(load.values()) <= 1.15 * total / 152 + 4


def test_plan_stages_at_most_a_gigabyte():
    # 8 KV heads: a tile of 128 positions is half a MiB staged
    sh = shape(num_q_heads=64, num_kv_heads=8, max_pages_per_seq=1 << 16, flags=mk.FLAG_KV_Q8)
    long, short = 2000 * 128, 100 * 128
    seg = mk.plan_chunk_attention(sh, [400, 400, 400], [long, short, short])
    launch = {s: k for k, s in zip(seg[:, 0].tolist(), seg[:, 2].tolist())}
    assert launch == {0: 1, 1: 0, 2: 0}        # the second and third no longer fit
    seg = mk.plan_chunk_attention(sh, [400, 400, 16], [2049 * 128, short, short])
    launch = {s: k for k, s in zip(seg[:, 0].tolist(), seg[:, 2].tolist())}
    assert launch == {0: 0, 1: 1, 2: 0}        # the first never fits, the last has too few rows


def test_binding_refuses_on_the_host():
    # what is no tensor, no length or not on a CUDA device ends as MkError before anything is launched
    torch = pytest.importorskip("torch")
    sh = mk.CacheShape(8, 2, 128, 16, 8, 4, 0)
    kv = torch.zeros(2 * 8 * 2 * 16 * 128, dtype=torch.bfloat16)
    ok = dict(q=torch.zeros(3, 8, 128, dtype=torch.bfloat16), chunk_lens=[3], seq_lens=[5],
              block_tables=torch.zeros(1, 4, dtype=torch.int32), kv_layer=kv)
    two = np.array([3, 0, 3, 0])
    for bad, word in ((dict(), "CUDA"), (dict(chunk_lens=np.array([3], np.int64)), "CUDA"), (dict(chunk_lens=two[:1]), "CUDA"),
                      (dict(chunk_lens=torch.tensor([3])), "CUDA"), (dict(chunk_lens=two[::2], seq_lens=[5, 5]), "CUDA"),
                      (dict(chunk_lens=[3.0]), "whole"), (dict(chunk_lens=np.array([3.0])), "whole"),
                      (dict(chunk_lens="3"), "whole"), (dict(chunk_lens=None), "whole"), (dict(seq_lens=[1 << 31]), "whole"),
                      (dict(seq_lens=np.array([1 << 40])), "32 bits"), (dict(seq_lens=[5, 5]), "one length"),
                      (dict(chunk_lens=[1 << 23] * 2, seq_lens=[1 << 23] * 2), "rows"), (dict(chunk_lens=[-1]), "rows"),
                      (dict(kv_layer=None), "kv_layer"), (dict(block_tables=[[0]]), "block_tables")):
        with pytest.raises(mk.MkError) as e:
            mk.chunk_attention(sh, **{**ok, **bad})
        assert e.value.code == mk.MK_ERR_INVALID_ARG and word in str(e.value), (bad, str(e.value))
    with pytest.raises(mk.MkError):
        mk.chunk_attention(None, **ok)
    with pytest.raises(mk.MkError):
        mk.append_chunk(sh, ok["q"], [3], [5], ok["block_tables"], kv)
    with pytest.raises(mk.MkError):
        mk.read_cache(sh, [3], [5], ok["block_tables"], kv)


@pytest.mark.parametrize("call", [mk.chunk_attention_workspace, mk.plan_chunk_attention])
def test_plan_and_workspace_refuse_lengths(call):
    sh = mk.CacheShape(8, 2, 128, 16, 8, 4, 0)
    for cl, sl in (([3, 1], [5]), ([3], [5, 5]), ([[3]], [[5]]), ([3.0], [5]), ([3], [5.5]), ([3], [1 << 40]), ([], []), ([6], [5])):
        with pytest.raises(mk.MkError) as e:
            call(sh, cl, sl)
        assert e.value.code == mk.MK_ERR_INVALID_ARG
    call(sh, np.array([3, 0, 3, 0])[::2], (5, 5))


def test_attention_refuses_an_output_over_its_query_rows():
    sh, row = shape(), 8 * 128 * 2                      # rows of 2048 bytes
    for n, stride, at in ((3, 1024, 0), (3, 1024, 16), (3, 1024, 3 * row - 16), (3, 1024, -3 * row + 16), (1, 1024, 0),
                          (3, 4096, 8192 - 3 * row + 16), (3, 4096, 2 * 8192 + row - 16), (2, 1 << 30, (1 << 31) + 16)):
        assert attend(sh, (n,), (n,), stride=stride, out=PTR + (1 << 20) + at, q=PTR + (1 << 20)) == BAD, (n, stride, at)
        assert "overlaps" in mk.lib().mk_last_error().decode()


def test_refused_lengths_are_let_go():
    # an array of lengths that is refused is not held afterwards
    import sys
    torch = pytest.importorskip("torch")
    sh = mk.CacheShape(8, 2, 128, 16, 8, 4, 0)
    args = (torch.zeros(2 * 8 * 2 * 16 * 128, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32))
    for bad in (np.array([1 << 40]), np.array([-(1 << 40), 3]), np.array([1.5]), np.array([3, 4])):
        before = sys.getrefcount(bad)
        for call in (lambda: mk.chunk_attention(sh, args[0], bad, [5], args[1], args[0]),
                     lambda: mk.append_chunk(sh, args[0], [3], bad, args[1], args[0]),
                     lambda: mk.read_cache(sh, bad, bad, args[1], args[0])):
            with pytest.raises(mk.MkError):
                call()
        assert sys.getrefcount(bad) == before


def test_binding_is_made_once(monkeypatch):
    # threads whose first call it is load and initialise the module once between them
    import importlib.util
    import threading
    import time
    pytest.importorskip("torch")
    mk.lib()
    monkeypatch.setattr(mk, "_bind", None)
    made, real = [], importlib.util.module_from_spec

    def slow(spec):
        made.append(spec.name)
        time.sleep(0.2)
        return real(spec)

    monkeypatch.setattr(importlib.util, "module_from_spec", slow)
    start, got = threading.Barrier(4), []

    def call():
        start.wait()
        got.append(mk._native())

    threads = [threading.Thread(target=call) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert made == ["_mk_torch"] and len(got) == 4 and all(m is mk._bind for m in got)


def test_rope_keeps_the_frequencies_that_its_calls_read():
    # the C structure points into the array: an assignment writes there, and none leaves it behind
    f = np.linspace(1.0, 0.1, 16)
    r = mk.Rope(f)
    f[:] = 7.0                                          # (a copy is kept)
    seen = lambda: np.ctypeslib.as_array(ctypes.cast(r.struct.inv_freq, ctypes.POINTER(ctypes.c_double)), (16,)).copy()  # noqa: E731
    want = np.linspace(1.0, 0.1, 16)
    r.inv_freq[3] = want[3] = 0.25
    assert np.array_equal(seen(), want) and r.struct.rotary_dim == 32
    r.inv_freq *= 2
    assert np.array_equal(seen(), 2 * want)
    r.inv_freq = np.ones(16)
    assert np.array_equal(seen(), np.ones(16)) and np.array_equal(r.inv_freq, np.ones(16))
    with pytest.raises(ValueError):
        r.inv_freq = np.ones(15)
