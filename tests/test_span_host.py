"""Host tests of attention over parts of the cache (mk_window_attention, mk_prefix_attention): what they refuse before
anything is launched, and their schedules.  No GPU needed."""
import ctypes

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
BAD, NO = mk.MK_ERR_INVALID_ARG, mk.MK_ERR_UNSUPPORTED


def window(sh, cl=(3,), sl=(5,), n=None, w=4, sinks=1, stride=None, q=PTR, kv=PTR, bt=PTR, out=PTR, ws=None, ws_bytes=0,
           status=None):
    cl, sl = i32(*cl), i32(*sl)
    stride = sh.num_q_heads * sh.head_dim if stride is None else stride
    return mk.lib().mk_window_attention(ctypes.byref(sh), len(cl) if n is None else n, cl.ctypes.data, sl.ctypes.data, w, sinks,
                                        bt, q, stride, kv, out, ws, ws_bytes, status, None)


def prefix(sh, cl=(3,), sl=(5,), n=None, groups=None, shared=None, ngroups=None, stride=None, q=PTR, kv=PTR, bt=PTR, out=PTR,
           ws=None, ws_bytes=0, status=None):
    groups, shared = i32(*((len(cl),) if groups is None else groups)), i32(*((0,) if shared is None else shared))
    cl, sl = i32(*cl), i32(*sl)
    stride = sh.num_q_heads * sh.head_dim if stride is None else stride
    return mk.lib().mk_prefix_attention(ctypes.byref(sh), len(cl) if n is None else n, cl.ctypes.data, sl.ctypes.data,
                                        len(groups) if ngroups is None else ngroups, groups.ctypes.data, shared.ctypes.data, bt,
                                        q, stride, kv, out, ws, ws_bytes, status, None)


@pytest.mark.parametrize("call", [window, prefix])
@pytest.mark.parametrize("over,code", [
    (dict(num_q_heads=0), BAD), (dict(page_size=-1), BAD), (dict(num_q_heads=9), BAD), (dict(flags=4), BAD),
    (dict(head_dim=96), NO), (dict(num_q_heads=18), NO), (dict(page_size=12), NO), (dict(flags=2, head_dim=64), NO),
    (dict(page_size=1 << 28, max_pages_per_seq=8), NO), (dict(num_pages=1 << 30), NO)])
def test_refuses_shapes(call, over, code):
    assert call(shape(**over)) == code
    assert mk.lib().mk_last_error().decode() != ""


@pytest.mark.parametrize("call", [window, prefix])
@pytest.mark.parametrize("cl,sl,n,code", [
    ((-1,), (5,), None, BAD), ((6,), (5,), None, BAD), ((1,), (129,), None, BAD), ((3,), (5,), 0, BAD),
    ((1,) * 65, (1,) * 65, None, BAD), ((1, 2, 9), (1, 2, 8), None, BAD)])
def test_refuses_lengths(call, cl, sl, n, code):
    assert call(shape(), cl, sl, n) == code


@pytest.mark.parametrize("call", [window, prefix])
def test_refuses_pointers_strides_and_workspaces(call):
    sh = shape()
    for k in ("q", "kv", "out"):
        assert call(sh, **{k: None}) == BAD and call(sh, **{k: PTR + 8}) == BAD
    far = 1 << 30
    assert call(sh, out=far, bt=None) == BAD and call(sh, out=far, bt=PTR + 2) == BAD
    assert call(sh, out=far, stride=8 * 128 - 8) == BAD and call(sh, out=far, stride=8 * 128 + 2) == BAD
    assert call(sh, out=far, stride=1 << 38) == NO
    assert call(sh, out=far, ws=PTR + 4) == BAD and call(sh, out=far, status=PTR + 1) == BAD
    assert call(sh, out=PTR + 16) == BAD and "overlaps" in mk.lib().mk_last_error().decode()
    big = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 16)
    kw = dict(w=1 << 20) if call is window else {}
    assert call(big, (1,), (100000,), out=far, **kw) == BAD and "workspace" in mk.lib().mk_last_error().decode()
    assert call(shape(max_pages_per_seq=1 << 26), (1 << 24,), (1 << 24,), out=far) == NO


def test_refuses_windows():
    for w, sinks in ((0, 0), (-1, 0), (1, -1), (-(1 << 31), 0), (1, -(1 << 31))):
        assert window(shape(), w=w, sinks=sinks) == BAD
        with pytest.raises(mk.MkError):
            mk.window_attention_workspace(shape(), [3], [5], w, sinks)
    for w, sinks in ((1 << 31, 0), (2.5, 0), ("3", 0), (None, 0), (3, 1 << 40), (3, 0.0)):
        with pytest.raises(mk.MkError) as e:
            mk.window_attention_workspace(shape(), [3], [5], w, sinks)
        assert e.value.code == BAD and "whole number" in str(e.value)


def test_refuses_groups():
    sh, cl, sl = shape(), (1, 2, 0, 1), (50, 40, 33, 60)
    for groups, shared, n in (((4,), (39,), None), ((4,), (34,), None), ((4,), (-1,), None), ((3,), (0,), None),
                              ((5,), (0,), None), ((2, 1), (0, 0), None), ((2, 3), (0, 0), None), ((4, 0), (0, 0), None),
                              ((0, 4), (0, 0), None), ((1,) * 5, (0,) * 5, None), ((4,), (0,), 0), ((4,), (0,), -1),
                              ((1 << 31) - 1, 5, None)):
        groups, shared = (groups, shared) if isinstance(groups, tuple) else ((groups, shared), (0, 0))
        assert prefix(sh, cl, sl, groups=groups, shared=shared, ngroups=n) == BAD, (groups, shared, n)
        if n is None:
            with pytest.raises(mk.MkError):
                mk.prefix_attention_workspace(sh, cl, sl, groups, shared)
    for groups, shared in (([4], [33]), ([2, 2], [38, 33]), ([1, 1, 1, 1], [49, 38, 33, 59]), ([3, 1], [0, 0])):
        mk.prefix_attention_workspace(sh, cl, sl, groups, shared)
    a = i32(1)
    for g, p in ((None, a.ctypes.data), (a.ctypes.data, None)):
        assert mk.lib().mk_prefix_attention(ctypes.byref(sh), 1, a.ctypes.data, i32(5).ctypes.data, 1, g, p, PTR, PTR, 1024, PTR,
                                            1 << 30, None, 0, None, None) == BAD
    for bad in (([4], [0, 0]), ([4.0], [0]), ([[4]], [[0]]), ([4], [1 << 40])):
        with pytest.raises(mk.MkError) as e:
            mk.prefix_attention_workspace(sh, cl, sl, *bad)
        assert e.value.code == BAD and "group_seqs" in str(e.value)


def test_no_rows_is_no_work():
    # nothing is launched, so no device is needed and pointers may be NULL
    for call in (window, prefix):
        assert call(shape(), (0, 0), (5, 0)) == mk.MK_OK
        assert call(shape(), (0,), (0,), q=None, kv=None, bt=None, out=None) == mk.MK_OK
    assert mk.window_attention_workspace(shape(), [0], [0], 1) == 0
    assert mk.prefix_attention_workspace(shape(), [0, 0], [0, 9], [2], [0]) == 0


def test_binding_refuses_on_the_host():
    torch = pytest.importorskip("torch")
    sh = mk.CacheShape(8, 2, 128, 16, 8, 4, 0)
    kv = torch.zeros(2 * 8 * 2 * 16 * 128, dtype=torch.bfloat16)
    args = (sh, torch.zeros(3, 8, 128, dtype=torch.bfloat16), [3], [5], torch.zeros(1, 4, dtype=torch.int32), kv)
    for call in (lambda *a: mk.window_attention(*a, 4), lambda *a: mk.prefix_attention(*a, [1], [0])):
        with pytest.raises(mk.MkError) as e:
            call(*args)
        assert e.value.code == BAD and "CUDA" in str(e.value)
        for i, bad, word in ((2, [3.0], "whole"), (3, [5, 5], "one length"), (3, [1 << 31], "whole"), (5, None, "kv_layer"),
                             (4, [[0]], "block_tables"), (0, None, "shape"), (2, [-1], "rows")):
            with pytest.raises(mk.MkError) as e:
                call(*args[:i], bad, *args[i + 1:])
            assert e.value.code == BAD and word in str(e.value), (i, bad, str(e.value))


# ---------------------------------------------------------------- schedules
COLS = ("launch", "block", "entry", "table", "row0", "ntok", "kvh", "head", "gap", "pos0", "len", "tile0", "n", "tiles", "slot",
        "stage0", "stage_tile0", "stage_head", "pair")
WHOLE = 304


def heads(segs):
    """Position tiles over all KV heads."""
    return sum(g["n"] * (1 + g["pair"]) for g in segs)


def segments(sh, cl, sl, **kw):
    return [dict(zip(COLS, row)) for row in mk.plan_span_attention(sh, cl, sl, **kw).tolist()]


def check_plan(sh, cl, sl, window=None, sinks=0, groups=(), shared=()):
    """Every position that a row sees is one place of one segment of each KV head, and no other place is seen; no copy
    reads a page that the call's rows do not see; copies stay within pages; partials are distinct."""
    G, Hkv, ps = sh.num_q_heads // sh.num_kv_heads, sh.num_kv_heads, sh.page_size
    box, TT = min(ps & -ps, 128), 128 // G
    kw = dict(group_seqs=groups, prefix_lens=shared) if len(groups) else dict(window=window, sinks=sinks)
    segs = segments(sh, cl, sl, **kw)
    w = window if window is not None else 1 << 30
    row0 = np.concatenate([[0], np.cumsum(cl)])
    seq_of = np.repeat(np.arange(len(cl)), cl)
    group_of = np.repeat(np.arange(len(groups)), groups) if len(groups) else np.arange(len(cl))
    count = [np.zeros((Hkv, c, n), dtype=np.int32) for c, n in zip(cl, sl)]
    visible = []
    for c, n in zip(cl, sl):
        row, pos = np.arange(n - c, n)[:, None], np.arange(n)[None, :]
        visible.append((pos <= row) & ((pos > row - w) | (pos < sinks)))
    slots, floats, staged = {0: set(), 1: set(), 2: set()}, {}, {}
    for g in segs:
        assert 0 < g["n"] and 0 <= g["tile0"] and g["tile0"] + g["n"] <= g["tiles"] and 0 < g["ntok"] <= 2 * TT
        assert g["head"] % box == 0 and g["gap"] % box == 0 and 0 <= g["block"] < 152
        v = np.arange(g["tile0"] * 128, min((g["tile0"] + g["n"]) * 128, g["len"]))
        pos = np.where(v < g["head"], v, v + g["gap"])
        for p in pos[v % box == 0]:                              # a copy's first position
            assert p % box == 0
            page = slice(p // ps * ps, p // ps * ps + ps)
            if window is not None:
                assert visible[g["table"]][:, page].any(), (p, g)
        if g["launch"] == 1:
            for t in np.unique(pos // 128):
                at = g["stage0"] + (t if t < g["stage_head"] else t - g["stage_tile0"] + g["stage_head"])
                assert (t < g["stage_head"] or t >= g["stage_tile0"]) and staged.setdefault(at, (g["entry"], t)) == (g["entry"], t)
        for i in range(g["ntok"]):
            r = g["row0"] + i
            s = seq_of[r]
            p0 = g["pos0"] + i
            seen = (v <= p0) & ((v < sinks) | (v > p0 - w))
            own = s == g["table"]
            if not own:                                          # another sequence's table: shared whole pages only
                assert group_of[s] == group_of[g["table"]]
                assert np.all(pos[seen] < shared[group_of[s]] // ps * ps)
            for h in range(g["kvh"], g["kvh"] + 1 + g["pair"]):
                count[s][h, r - row0[s], pos[seen]] += 1
        if 0 <= g["slot"] < WHOLE:
            assert g["slot"] == 2 * g["block"] + (g["tile0"] == 0) and g["slot"] not in slots[g["launch"]]
            slots[g["launch"]].add(g["slot"])
            assert g["n"] < g["tiles"]
        else:
            assert g["n"] == g["tiles"]
        if sh.flags == mk.FLAG_KV_Q8:
            assert (g["launch"] == 2) <= (g["ntok"] * G <= 32)
        else:
            assert g["launch"] == 0
    for s, c in enumerate(count):
        assert np.array_equal(c, np.broadcast_to(visible[s][None], c.shape)), s
    # who writes the output: a row that one entry has does so by itself, of two neither
    entries, hkv_even = {}, Hkv % 2 == 0
    units = {}
    for g in segs:
        units.setdefault((g["launch"], g["entry"]), set()).add(g["row0"])
    units = {k: len(v) for k, v in units.items()}
    for g in segs:
        for r in range(g["row0"], g["row0"] + g["ntok"]):
            assert not g["pair"] or (hkv_even and g["ntok"] <= TT and g["launch"] == 0 and units[g["launch"], g["entry"]] == 1)
            for h in range(g["kvh"], g["kvh"] + 1 + g["pair"]):
                entries.setdefault((r, h), set()).add((g["launch"], g["entry"]))
    for g in segs:
        many = {len(entries[r, g["kvh"]]) for r in range(g["row0"], g["row0"] + g["ntok"])}
        assert many in ({1}, {2})
        if g["n"] == g["tiles"]:
            assert g["slot"] == (-1 if many == {1} else WHOLE)
    return segs


@pytest.mark.parametrize("seed", range(60))
def test_window_plan_covers_what_rows_see(seed):
    g = np.random.default_rng(seed)
    hkv, G = int(g.choice([1, 2, 4])), int(g.integers(1, 9))
    sh = shape(num_q_heads=hkv * G, num_kv_heads=hkv, page_size=int(g.choice([8, 16, 24, 64, 128, 40, 256])), max_pages_per_seq=512,
               num_pages=64, flags=int(g.choice([0, 2])))
    n = int(g.integers(1, 9))
    sl = np.exp(g.uniform(0, np.log(g.choice([50, 1500])), n)).astype(int)
    top = int(g.choice([1, 40, 700]))
    cl = [int(g.integers(0, min(x, top) + 1)) for x in sl]
    w, sinks = int(np.exp(g.uniform(0, np.log(2000)))), int(g.choice([0, 1, 4, 17, 128, 300, 5000]))
    check_plan(sh, cl, sl.tolist(), w, sinks)


@pytest.mark.parametrize("seed", range(40))
def test_prefix_plan_covers_what_rows_see(seed):
    g = np.random.default_rng(1000 + seed)
    hkv, G = int(g.choice([1, 2, 4])), int(g.integers(1, 9))
    sh = shape(num_q_heads=hkv * G, num_kv_heads=hkv, page_size=int(g.choice([8, 16, 24, 64])), max_pages_per_seq=4096,
               num_pages=64, flags=int(g.choice([0, 2])))
    groups = [int(x) for x in g.integers(1, 20, int(g.integers(1, 4)))]
    shared = [int(np.exp(g.uniform(0, np.log(4000)))) for _ in groups]
    top = int(g.choice([1, 1, 5, 60]))
    cl = [int(g.integers(0, top + 1)) for _ in range(sum(groups))]
    sl = [c + int(g.integers(0, 200)) + p for c, p in zip(cl, np.repeat(shared, groups))]
    check_plan(sh, cl, sl, groups=groups, shared=shared)


def test_a_long_shared_prefix_is_read_once():
    # 64 sequences of one token behind 32768 shared positions: every shared tile is in the schedule for the group's
    # rows (two units of a KV head), not for each sequence
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 12)
    segs = segments(sh, [1] * 64, [32768 + 100] * 64, group_seqs=[64], prefix_lens=[32768])
    assert heads(segs) == 4 * 2 * 256 + 64 * 4
    # of two sequences over a few positions each takes its own way
    segs = segments(sh, [1] * 2, [200] * 2, group_seqs=[2], prefix_lens=[128])
    assert all(g["slot"] == -1 and g["len"] == 200 for g in segs)


def test_window_plan_skips_the_hidden_middle():
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 14)
    segs = segments(sh, [1], [131073], window=1000, sinks=4)
    # positions 130073..131072, from a multiple of 16 on: 1009 places, and 16 of the sinks' copy
    assert [(g["head"], g["len"], g["tiles"], g["pair"]) for g in segs if g["tile0"] == 0] == [(16, 1025, 9, 0)] * 4
    assert heads(segs) == 4 * 9
    segs = segments(sh, [8192], [8192], window=1024, sinks=4)
    assert max(g["tiles"] for g in segs) == 9


def test_window_plan_pairs_heads_of_many_tokens():
    # a block's two streams are two KV heads where there are more items than blocks without that, or four tiles a block
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 14)
    for n, ln, tiles, pair in ((64, 5000, 9, 1), (17, 5000, 9, 1), (16, 5000, 9, 0), (1, 5000, 9, 0), (39, 100, 1, 1),
                               (38, 100, 1, 0)):
        segs = segments(sh, [1] * n, [ln] * n, window=1024, sinks=4)
        assert {g["pair"] for g in segs} == {pair} and heads(segs) == n * 4 * tiles, (n, ln)
    sh.num_q_heads, sh.num_kv_heads = 24, 3
    assert {g["pair"] for g in segments(sh, [1] * 64, [5000] * 64, window=1024)} == {0}


def test_plans_of_the_largest_calls():
    # 2^20 rows, a sequence of 2^30 positions: planned in little time, and nothing overflows
    sh = shape(max_pages_per_seq=1 << 26)
    assert mk.window_attention_workspace(sh, [1 << 20], [1 << 30], 1 << 30, 1 << 30) >= 0
    segs = segments(sh, [1], [1 << 30], window=(1 << 31) - 1, sinks=(1 << 31) - 1)
    assert heads(segs) == 2 * (1 << 23)
    segs = segments(sh, [2], [1 << 30], window=5, sinks=16)
    assert [(g["head"], g["gap"], g["len"]) for g in segs] == [(16, (1 << 30) - 32, 32)] * 2
    segs = segments(sh, [1, 1], [1 << 30, 1 << 30], group_seqs=[2], prefix_lens=[(1 << 30) - 1])
    # 2^30 - 16 shared positions, and 16 of each sequence's own
    assert heads(segs) == 2 * (1 << 23) + 2 * 2


def blocks_of(segs):
    """Position tiles over all KV heads, and segments, of each launch's blocks."""
    load = {}
    for g in segs:
        at = load.setdefault((g["launch"], g["block"]), [0, 0])
        at[0] += g["n"] * (1 + g["pair"])
        at[1] += 1
    return load


@pytest.mark.parametrize("cl,sl,kw", [
    ([1] * 64, [9000] * 64, dict(window=4096, sinks=4)), ([1], [1 << 17], dict(window=1 << 16, sinks=4)),
    ([1] * 20, [5000 + 700 * i for i in range(20)], dict(window=1 << 20)),
    ([1] * 64, [40000] * 64, dict(group_seqs=[64], prefix_lens=[32768]))])
@pytest.mark.parametrize("flags", [0, mk.FLAG_KV_Q8])
def test_cuts_are_even(cl, sl, kw, flags):
    # a launch whose items are cut: no block has much more than its share (the costs differ by kind, by less than 2)
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 14, flags=flags)
    segs = segments(sh, cl, sl, **kw)
    assert any(0 <= g["slot"] < WHOLE for g in segs)
    load = blocks_of(segs)
    work = [t + 4 * n for t, n in load.values()]
    assert max(work) <= 2 * sum(work) / 152 + 4


def test_sequences_that_fill_units_read_for_themselves():
    # 30 tokens and two prompts behind 8192 shared positions: the tokens' runs go over these together, the prompts do not
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 12)
    cl = [1] * 10 + [500] + [1] * 15 + [400] + [1] * 5
    segs = segments(sh, cl, [8192 + 900] * 32, group_seqs=[32], prefix_lens=[8192])
    row0 = np.concatenate([[0], np.cumsum(cl)])
    runs = sorted({(g["row0"], g["ntok"]) for g in segs if g["len"] == 8192})
    assert runs == [(0, 10), (510, 15), (int(row0[27]), 5)]
    for s in (10, 26):
        mine = [g for g in segs if row0[s] <= g["row0"] < row0[s + 1]]
        assert mine and all(g["len"] == 9092 and g["slot"] != WHOLE and g["table"] == s for g in mine)


def test_runs_share_where_they_save_enough_together():
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 12)

    def shared(n, rows, prefix, groups=1):
        segs = segments(sh, [rows] * (n * groups), [prefix + 200] * (n * groups), group_seqs=[n] * groups,
                        prefix_lens=[prefix] * groups)
        return any(g["len"] == prefix for g in segs)
    assert shared(64, 1, 8192) and shared(16, 1, 8192) and not shared(64, 1, 512) and not shared(4, 1, 2048)
    assert not shared(8, 5, 8192) and shared(8, 5, 8192, groups=2)     # two groups for the price of one kernel


def test_q8_launches():
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 14, flags=mk.FLAG_KV_Q8)

    def launches(cl, sl, **kw):
        return sorted({g["launch"] for g in segments(sh, cl, sl, **kw)})
    assert launches([1] * 8, [5000] * 8, window=1000) == [2]                       # few rows of a unit
    assert launches([40], [5000], window=1000) == [0]
    assert launches([1] * 8 + [40], [5000] * 9, window=1000) == [0]                # with the launch that there is
    assert launches([1] * 60 + [40], [20000] * 61, window=16384) == [0, 2]         # but not so much of it
    assert launches([4096], [8192], window=512) == [1]                             # decoded once
    assert launches([512], [8192], window=256) == [0]
    assert launches([1] * 60 + [40, 4096], [20000] * 62, window=16384) == [0, 1, 2]


def test_staged_bytes_are_bounded():
    # 8 KV heads: a tile of 128 positions is half a MiB decoded; beyond a GiB sequences are read from their pages
    sh = shape(num_q_heads=64, num_kv_heads=8, max_pages_per_seq=1 << 16, flags=mk.FLAG_KV_Q8)
    segs = segments(sh, [2000] * 3, [1600 * 128, 600 * 128, 400 * 128], window=1 << 20)
    assert {g["table"]: g["launch"] for g in segs} == {0: 1, 1: 0, 2: 1}
    assert mk.window_attention_workspace(sh, [2000] * 3, [1600 * 128, 600 * 128, 400 * 128], 1 << 20) >= 2000 << 19


@pytest.mark.parametrize("kw", [dict(window=50, sinks=3), dict(group_seqs=[2, 1], prefix_lens=[64, 0])])
def test_workspace_is_what_the_plan_needs(kw):
    sh = shape(max_pages_per_seq=1 << 12)
    cl, sl = [3, 0, 5], [70, 64, 9]
    call = mk.window_attention_workspace if "window" in kw else mk.prefix_attention_workspace
    assert call(sh, cl, sl, *kw.values()) == 0                                     # whole items that write the output
    big = [1] * 64, [60000] * 64
    kw = dict(window=1 << 20, sinks=0) if "window" in kw else dict(group_seqs=[64], prefix_lens=[50000])
    segs = segments(sh, *big, **kw)
    cut = max(g["slot"] for g in segs if g["slot"] < WHOLE)
    assert call(sh, *big, *kw.values()) >= (cut + 1) * 4 * 132 * 4


def test_a_group_reads_the_table_of_a_sequence_with_rows():
    # sequences without new tokens stand first: nothing is read through their tables
    sh = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 12)
    cl = [0, 0] + [1] * 30
    segs = segments(sh, cl, [8192 + 100] * 32, group_seqs=[32], prefix_lens=[8192])
    joint = [g for g in segs if g["len"] == 8192]
    assert joint and all(g["table"] == 2 and (g["row0"], g["ntok"]) == (0, 30) for g in joint)
    assert all(cl[g["table"]] > 0 for g in segs)


def decoded(sh, cl, sl, window, sinks):
    """The positions that each sequence of launch 1 has looked up and decoded before it (none: not in that launch)."""
    out = {}
    for row in mk.plan_span_attention(sh, cl, sl, window=window, sinks=sinks).tolist():
        g = dict(zip(COLS + ("unseen", "unseen_n"), row))
        if g["launch"] == 1:
            pos = np.arange(sl[g["table"]])
            tile = (pos // 128 < g["stage_head"]) | (pos // 128 >= g["stage_tile0"])
            out[g["table"]] = tile & ~((pos >= g["unseen"]) & (pos < g["unseen"] + g["unseen_n"]))
    return out


def check_decoded(sh, cl, sl, window, sinks):
    got = decoded(sh, cl, sl, window, sinks)
    for s, looked in got.items():
        row, pos = np.arange(sl[s] - cl[s], sl[s])[:, None], np.arange(sl[s])[None, :]
        seen = ((pos <= row) & ((pos > row - window) | (pos < sinks))).any(0)
        pages = np.zeros(-(-sl[s] // sh.page_size), dtype=bool)
        pages[np.arange(sl[s])[seen] // sh.page_size] = True
        assert np.all(looked[seen])
        extra = np.unique(np.arange(sl[s])[looked] // sh.page_size)
        assert pages[extra].all(), (s, extra[~pages[extra]])
    return len(got)


@pytest.mark.parametrize("cl,sl,window,sinks,ps", [
    ([1024], [16384], 2048, 4, 16), ([4096], [12345], 512, 0, 16), ([4096], [9000], 512, 4, 16), ([4096, 3000], [9001, 8190], 700, 140, 8),
    ([4096], [9000], 512, 4, 64), ([4096], [9000], 500, 300, 40), ([3000], [20000], 900, 130, 256)])
def test_what_is_decoded_before_looks_up_no_page_that_no_row_sees(cl, sl, window, sinks, ps):
    # the window's beginning and the sinks' end lie inside tiles of 128 positions: the pages between are not looked up
    sh = shape(num_q_heads=32, num_kv_heads=4, page_size=ps, max_pages_per_seq=1 << 12, flags=mk.FLAG_KV_Q8)
    assert check_decoded(sh, cl, sl, window, sinks) == len(cl)


def test_what_is_decoded_before_over_random_windows():
    g, n = np.random.default_rng(5), 0
    for _ in range(400):
        hkv, G = int(g.choice([1, 2, 4])), int(g.integers(1, 9))
        sh = shape(num_q_heads=hkv * G, num_kv_heads=hkv, page_size=int(g.choice([8, 16, 24, 40, 64, 128, 256])),
                   max_pages_per_seq=2048, flags=mk.FLAG_KV_Q8)
        ln = int(g.integers(2000, 9000))
        n += check_decoded(sh, [int(g.integers(1, ln + 1))], [ln], int(np.exp(g.uniform(3, 8))), int(g.choice([0, 1, 4, 100, 128, 300])))
    assert n > 20


def test_rows_behind_the_most_shared_positions_see_the_first():
    # the second unit of 500 rows stands beyond 2^30 positions: its places begin at position 0 as the first one's do
    sh = shape(num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=64, max_pages_per_seq=1 << 24)
    segs = segments(sh, [100] * 5, [1 << 30] * 5, group_seqs=[5], prefix_lens=[(1 << 30) - 100])
    joint = [g for g in segs if g["len"] == (1 << 30) - 128]
    assert {(g["row0"], g["ntok"], g["pos0"]) for g in joint} == {(0, 256, (1 << 30) - 128), (256, 244, (1 << 30) + 128)}
    assert all(g["head"] == g["gap"] == 0 for g in joint) and sum(g["n"] for g in joint) == 2 * ((1 << 23) - 1)


def test_schedule_refuses_arguments_that_do_not_pair_up():
    sh = shape()
    for kw in (dict(group_seqs=[1, 1], prefix_lens=[0]), dict(group_seqs=[2], prefix_lens=[]), dict(group_seqs=[2.0], prefix_lens=[0]),
               dict(group_seqs=[[2]], prefix_lens=[[0]]), dict(group_seqs=[2], prefix_lens=[1 << 40])):
        with pytest.raises(mk.MkError) as e:
            mk.plan_span_attention(sh, [1, 1], [5, 6], **kw)
        assert e.value.code == BAD and "group_seqs" in str(e.value)
    for kw in (dict(window=1 << 32), dict(window=2.5), dict(window=None), dict(window=3, sinks=1 << 31), dict(window=3, sinks="1")):
        with pytest.raises(mk.MkError) as e:
            mk.plan_span_attention(sh, [1, 1], [5, 6], **kw)
        assert e.value.code == BAD and "whole number" in str(e.value)
    assert len(mk.plan_span_attention(sh, [1, 1], [5, 6], window=3)) == len(mk.plan_span_attention(sh, [1, 1], [5, 6], group_seqs=[2], prefix_lens=[0]))


def test_long_segments_have_room_for_their_sums():
    # more than 2048 position tiles of one row's in a segment: the workspace has [2][128][D + 4] floats for every block, and
    # without such segments nothing of the kind
    sh, long = shape(num_q_heads=32, num_kv_heads=4, max_pages_per_seq=1 << 20), 0
    for cl, sl, w in (([4000], [1 << 18], 1 << 20), ([4000], [(1 << 18) + 129], 1 << 20), ([5000], [1 << 20], 1 << 20), ([1], [1 << 23], 1 << 23),
                      ([1] * 64, [1 << 19] * 64, 1 << 20), ([4000], [1 << 20], 1 << 17), ([4000] * 2, [1 << 20] * 2, 300000),
                      ([1] * 64, [1 << 19] * 64, 200000)):
        segs = segments(sh, cl, sl, window=w)
        most = max(g["n"] if g["ntok"] > 16 or g["pair"] else (g["n"] + 1) // 2 for g in segs)
        cut = max((g["slot"] for g in segs if g["slot"] < WHOLE), default=-1)
        rows = max(min(g["ntok"], 32) << g["pair"] for g in segs) * 8
        blocks = len({g["block"] for g in segs})
        parts = 0 if cut < 0 else 2 * blocks * rows * 132 * 4
        folds = blocks * 2 * 128 * 132 * 4
        need = mk.window_attention_workspace(sh, cl, sl, w)
        long += most > 2048
        assert need == parts + (folds if most > 2048 else 0) or (most > 2045 and need == parts + folds), (cl, sl, w, need, parts, folds)
    assert long >= 3
