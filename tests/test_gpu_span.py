"""GPU tests of attention over parts of the paged cache (mk_window_attention, mk_prefix_attention), each against its
definition in 64 bits (tests/span_ref.py, with the error bounds of tests/chunk_ref.py), and runs of them with the
operators and the step that share the cache.  What no row may see holds NaNs throughout."""
import threading

import numpy as np
import pytest
import torch

import persistent_moe_decode_megakernel_gb300 as mk
from tests import chunk_ref as R
from tests import span_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mk.build()


def hide(st, window, sinks):
    """Marks the pages that no row of the call sees as given back: their entries name no page, and the pages' values
    are poison."""
    for s, (ln, n) in enumerate(zip(st.lens, st.news)):
        lo = max(0, ln - n - window + 1)
        first, last = -(-min(sinks, ln) // st.ps), lo // st.ps
        if n == 0:
            first, last = 0, -(-ln // st.ps)
        if last > first:
            S.poison(st, st.bt[s, first:last].long().clone())
            st.bt[s, first:last] = -1


def check_window(st, window, sinks, std=1.5, drop=None, status_want=mk.MK_OK, q=None, extra_rows=0):
    q = st.normal(st.rows + extra_rows, st.hq, st.d, std=std) if q is None else q
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    out = torch.full((st.rows + extra_rows, st.hq, st.d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, window, sinks, out=out, status=status)
    assert got is out and int(status) == status_want
    assert torch.all(out[st.rows:] == 7.0)           # rows behind the last sequence's
    ref, *scale = S.attention(st, q, st.kv, window, sinks, drop)
    far = (out[:st.rows].double() - ref).abs()
    bound = R.attention_bound(ref, *scale, st.q8)
    assert torch.all(far <= bound), float((far / bound).nan_to_num(9e9).max())
    return q, out


def check_prefix(st, groups, shared, std=1.5, drop=None, status_want=mk.MK_OK, q=None, extra_rows=0):
    q = st.normal(st.rows + extra_rows, st.hq, st.d, std=std) if q is None else q
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    out = torch.full((st.rows + extra_rows, st.hq, st.d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mk.prefix_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, groups, shared, out=out, status=status)
    assert got is out and int(status) == status_want
    assert torch.all(out[st.rows:] == 7.0)
    ref, *scale = S.attention(st, q, st.kv, drop=drop)
    far = (out[:st.rows].double() - ref).abs()
    bound = R.attention_bound(ref, *scale, st.q8)
    assert torch.all(far <= bound), float((far / bound).nan_to_num(9e9).max())
    return q, out


# ---------------------------------------------------------------- windows
WINDOW_SHAPES = [
    # hq, hkv, d, ps, lens, news, window, sinks: one token, one position, window edges inside pages and tiles, sinks that
    # meet the window, end inside a page or lie behind the row, odd groups
    (4, 2, 64, 16, [65], [65], 16, 2),
    (1, 1, 128, 8, [1], [1], 1, 0),
    (1, 1, 128, 8, [300], [300], 1, 0),
    (8, 1, 128, 16, [16, 17, 128, 129, 500], [1, 1, 1, 1, 1], 100, 4),
    (8, 1, 128, 16, [16, 17, 128, 129, 1], [16, 17, 128, 129, 1], 33, 5),
    (32, 4, 128, 16, [513, 40, 1000], [100, 0, 3], 129, 1),
    (3, 1, 64, 24, [200, 300], [200, 47], 50, 0),
    (10, 2, 128, 40, [333], [333], 64, 40),
    (12, 2, 128, 64, [400, 64], [31, 64], 128, 64),
    (7, 1, 64, 8, [700], [69], 13, 150),
    (16, 16, 64, 128, [130, 257], [130, 129], 127, 3),
    (14, 2, 128, 256, [700], [300], 200, 7),
    (32, 4, 128, 16, [5000], [1], 1024, 4),
    (16, 2, 128, 64, [9001, 3], [2, 1], 4000, 20),
    (16, 2, 128, 16, [2500], [2500], 300, 4),
    (8, 8, 128, 16, [900, 900], [700, 1], 128, 128),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,ps,lens,news,window,sinks", WINDOW_SHAPES)
def test_window(hq, hkv, d, ps, lens, news, window, sinks, q8):
    st = R.Setup(hq, hkv, 128 if q8 else d, ps, lens, news, q8=q8, seed=9)
    hide(st, window, sinks)
    check_window(st, window, sinks, extra_rows=1)


@pytest.mark.parametrize("q8", [False, True])
def test_window_of_everything_is_causal_attention(q8):
    for lens, news in (([700, 20, 5], [300, 1, 5]), ([5000], [1])):
        st = R.Setup(16, 2, 128, 16, lens, news, q8=q8, seed=21)
        q = st.normal(st.rows, 16, 128, std=1.5)
        want = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
        for window, sinks in ((5000, 0), ((1 << 31) - 1, 3), (1, 5000), (1, (1 << 31) - 1)):
            check_window(st, window, sinks, q=q)
            got = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, window, sinks)
            ref, *scale = S.attention(st, q, st.kv)
            assert torch.all((got.double() - want.double()).abs() <= 2 * R.attention_bound(ref, *scale, q8))


@pytest.mark.parametrize("q8", [False, True])
def test_window_64_sequences(q8):
    g = np.random.default_rng(1)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(3000), 64)).astype(int)]
    news = [min(ln, int(g.choice([0, 1, 1, 1, 5, 67]))) for ln in lens]
    st = R.Setup(16, 2, 128, 16, lens, news, q8=q8, seed=10)
    hide(st, 250, 4)
    check_window(st, 250, 4)
    st = R.Setup(16, 2, 128, 16, lens, [min(1, n) for n in news], q8=q8, seed=10)
    hide(st, 999, 0)
    check_window(st, 999, 0)


@pytest.mark.parametrize("std", [0.0, 30.0])
def test_window_flat_and_peaked_scores(std):
    check_window(R.Setup(8, 2, 128, 16, [1500], [70], seed=11), 400, 4, std=std)


@pytest.mark.parametrize("q8", [False, True])
def test_window_strided_query_rows_and_given_workspace(q8):
    st = R.Setup(6, 2, 128, 16, [3000, 30], [111, 30], q8=q8, seed=13)
    qkv = st.normal(141, (6 + 4) * 128 + 8)
    q = qkv[:, :6 * 128].unflatten(1, (6, 128))
    _, out = check_window(st, 1000, 9, q=q)
    need = mk.window_attention_workspace(st.shape(mk), st.news, st.lens, 1000, 9)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    again = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 1000, 9, workspace=ws)
    assert torch.equal(again, out) and torch.all(ws[need:] == 0xff)


@pytest.mark.parametrize("q8", [False, True])
def test_window_skips_pages_out_of_range(q8):
    st = R.Setup(8, 2, 128, 16, [100, 300, 20, 600], [100, 3, 20, 1], q8=q8, seed=14)
    drop = torch.zeros(4, 600, dtype=torch.bool, device="cuda")
    for s, p, bad in ((0, 0, st.P), (0, 3, -1), (1, 18, 1 << 30), (1, 12, -(1 << 31)), (2, 0, -5), (2, 1, 1 << 20), (3, 0, -1)):
        drop[s, p * 16:p * 16 + 16] = True
        st.bt[s, p] = bad
    check_window(st, 90, 8, drop=drop, status_want=mk.MK_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_window_rows_do_not_see_what_is_hidden(q8, what):
    # NaN or infinity in positions that some rows of a tile see and others do not: rows that see it take it in, rows
    # that do not are as if it were another number
    for hit, window, sinks in ((300, 64, 4), (2, 64, 4), (2, 64, 2), (431, 200, 0)):
        st = R.Setup(8, 2, 128, 16, [450], [180], q8=q8, seed=15)
        page, off = int(st.bt[0, hit // 16]), hit % 16
        if q8:
            _, scales = st.planes()
            scales[page, :, :, off] = what
        else:
            st.kv[page, :, :, off] = what
        q = st.normal(180, 8, 128, std=1.5)
        out = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, window, sinks)
        p = torch.arange(270, 450, device="cuda")
        sees = (hit <= p) & ((hit > p - window) | (hit < sinks))
        clean = st.kv.clone()
        if q8:
            n = st.P * 2 * st.hkv * st.ps * st.d
            clean[n:].view(torch.float16).view(st.P, 2, st.hkv, st.ps, st.d // 32)[page, :, :, off] = 0.01
        else:
            clean[page, :, :, off] = 0.5
        ref, *scale = S.attention(st, q, clean, window, sinks)
        bound = R.attention_bound(ref, *scale, q8)
        assert torch.all(((out.double() - ref).abs() <= bound)[~sees])
        # (an infinite key's score adds infinities of both signs)
        assert torch.all(out[sees].isnan())


def test_window_with_every_score_minus_infinity_is_nan():
    st = R.Setup(2, 1, 128, 16, [200], [1], seed=16)
    q = st.normal(1, 2, 128)
    q[...] = 1.0
    pos = torch.arange(200, device="cuda")
    st.kv[st.bt[0, pos // 16].long(), 0, 0, pos % 16] = -3e38
    out = mk.window_attention(st.shape(mk), q, [1], [200], st.bt, st.kv, 50, 4)
    assert torch.all(out.isnan())


# ---------------------------------------------------------------- shared prefixes
PREFIX_SHAPES = [
    # hq, hkv, d, ps, groups, shared, own lengths (repeated), news (repeated)
    (4, 2, 64, 16, [8], [200], [1, 40, 17], [1]),
    (32, 4, 128, 16, [16], [4000], [1, 100, 333], [1]),
    (32, 4, 128, 64, [5, 3], [2000, 777], [64, 5, 200], [5]),
    (8, 8, 128, 16, [20], [1500], [31, 2], [2]),
    (7, 1, 64, 24, [9, 1, 11], [3000, 50, 4001], [200, 1, 77], [1, 3]),
    (16, 2, 128, 8, [3, 12], [0, 5000], [3, 250], [3, 1]),
    (10, 2, 128, 40, [30], [2100], [39, 41], [1, 0]),
    (3, 1, 128, 128, [40], [6000], [1, 130], [1]),
    (6, 2, 64, 16, [10], [3000], [400, 50], [100, 1]),
    (1, 1, 128, 16, [64], [2500], [10, 2], [2]),
    (32, 4, 128, 16, [64], [1024], [1], [1]),
]


def prefix_setup(hq, hkv, d, ps, groups, shared, own, news, q8, seed, **kw):
    n = sum(groups)
    per = np.repeat(shared, groups)
    lens = [int(p) + own[i % len(own)] for i, p in enumerate(per)]
    st = R.Setup(hq, hkv, 128 if q8 else d, ps, lens, [min(news[i % len(news)], own[i % len(own)]) for i in range(n)], q8=q8,
                 seed=seed, **kw)
    S.share(st, groups, shared)
    return st


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,ps,groups,shared,own,news", PREFIX_SHAPES)
def test_prefix(hq, hkv, d, ps, groups, shared, own, news, q8):
    st = prefix_setup(hq, hkv, d, ps, groups, shared, own, news, q8, seed=31)
    check_prefix(st, groups, shared, extra_rows=1)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("std", [0.0, 1.5, 30.0])
def test_prefix_long(std, q8):
    # enough shared positions and rows that a group's part is cut over many blocks
    st = prefix_setup(32, 4, 128, 64, [40, 8], [20000, 9999], [1, 300, 1000], [1], q8, seed=32)
    check_prefix(st, [40, 8], [20000, 9999], std=std)


@pytest.mark.parametrize("q8", [False, True])
def test_prefix_with_prompts_among_single_tokens(q8):
    st = prefix_setup(16, 2, 128, 16, [12, 4], [5000, 3000], [300, 20, 700], [260, 1, 1, 513], q8, seed=33)
    check_prefix(st, [12, 4], [5000, 3000])


@pytest.mark.parametrize("q8", [False, True])
def test_prefix_skips_pages_out_of_range(q8):
    # in the shared part (every row of the group skips them), and in one sequence's own
    for shared in (3200, 160):
        st = prefix_setup(16, 2, 128, 16, [20], [shared], [50, 7], [1], q8, seed=34)
        drop = torch.zeros(20, max(st.lens), dtype=torch.bool, device="cuda")
        for p, bad in ((0, st.P), (5, -1), (9, 1 << 30)):
            drop[:, p * 16:p * 16 + 16] = True
            st.bt[:, p] = bad
        own = shared // 16
        st.bt[3, own], drop[3, shared:] = -9, True       # all of its own positions
        check_prefix(st, [20], [shared], drop=drop, status_want=mk.MK_ERR_DEVICE_BOUNDS)
        st.bt[:, :own], drop[:, :shared] = -1, True       # nothing is left of the shared part; of sequence 3 nothing at all
        check_prefix(st, [20], [shared], drop=drop, status_want=mk.MK_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("q8", [False, True])
def test_prefix_rows_with_a_poisoned_position(q8):
    # a NaN in a shared position is every row's, one in a sequence's own is that one's
    st = prefix_setup(32, 4, 128, 16, [24], [3000], [60, 9], [1], q8, seed=35)
    q = st.normal(st.rows, 32, 128, std=1.5)
    ref, *scale = S.attention(st, q, st.kv)
    bound = R.attention_bound(ref, *scale, q8)

    def poison(s, pos):
        page, off = int(st.bt[s, pos // 16]), pos % 16
        if q8:
            st.planes()[1][page, :, :, off] = float("nan")
        else:
            st.kv[page, :, :, off] = float("nan")
    poison(5, st.lens[5] - 1)
    out = mk.prefix_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, [24], [3000])
    other = torch.arange(24, device="cuda") != 5
    assert torch.all(out[5].isnan()) and torch.all(((out.double() - ref).abs() <= bound)[other])
    poison(0, 1000)
    out = mk.prefix_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, [24], [3000])
    assert torch.all(out.isnan())


# ---------------------------------------------------------------- both: streams, graphs, threads
def both(st, groups, shared, q, **kw):
    a = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 700, 4, **kw)
    return a, mk.prefix_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, groups, shared, **kw)


@pytest.mark.parametrize("q8", [False, True])
def test_calls_are_repeatable_captured_and_on_other_streams(q8):
    st = prefix_setup(16, 2, 128, 16, [20, 2], [3000, 500], [60, 9], [1, 2], q8, seed=41)
    q = st.normal(st.rows, 16, 128, std=1.5)
    want = both(st, [20, 2], [3000, 500], q)
    for _ in range(3):
        got = both(st, [20, 2], [3000, 500], q)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(st, [20, 2], [3000, 500], q, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured: a replay takes what its buffers hold then (values, tables), with the lengths of the capture
    graph = torch.cuda.CUDAGraph()
    q2, bt2 = st.normal(st.rows, 16, 128, std=1.5), st.bt.clone()
    qs, st.bt = q.clone(), st.bt.clone()
    with torch.cuda.graph(graph):
        got = both(st, [20, 2], [3000, 500], qs)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qs.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    captured = st.bt
    st.bt = bt2
    again = both(st, [20, 2], [3000, 500], q2)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    captured.fill_(-1)                                   # every page out of range: zeros
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.all(a == 0) for a in got)


def test_calls_of_several_threads():
    st = prefix_setup(16, 2, 128, 16, [20], [3000], [60, 9], [1], False, seed=42)
    q = st.normal(st.rows, 16, 128, std=1.5)
    want = both(st, [20], [3000], q)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            got = both(st, [20], [3000], q, stream=s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_binding_refuses_tensors():
    st = R.Setup(8, 2, 128, 16, [40], [40], seed=43)
    q = st.normal(40, 8, 128)
    args = (st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
    for call in (lambda *a, **k: mk.window_attention(*a, 4, 1, **k), lambda *a, **k: mk.prefix_attention(*a, [1], [0], **k)):
        for i, bad in ((1, q.float()), (1, q[:39]), (1, q.cpu()), (1, q.transpose(1, 2)), (4, st.bt.long()), (4, st.bt[:, :-1]),
                       (5, st.kv[1:]), (5, st.kv.view(torch.uint8)), (5, st.kv.float())):
            with pytest.raises(mk.MkError):
                call(*args[:i], bad, *args[i + 1:])
        for kw in (dict(out=q), dict(out=torch.empty(40, 8, 64, dtype=torch.bfloat16, device="cuda")), dict(status=q),
                   dict(workspace=torch.empty(4))):
            with pytest.raises(mk.MkError):
                call(*args, **kw)
    for bad in (("3", 0), (0, 0), (3, -1), (1 << 31, 0), (3, 0.5), (None, 0)):
        with pytest.raises(mk.MkError):
            mk.window_attention(*args, *bad)
    for bad in (([1], [41]), ([2], [0]), ([1, 1], [0, 0]), ([], []), ([1], [0.5]), (torch.ones(1, dtype=torch.int32, device="cuda"), [0]),
                ([1], [0, 0]), ([0], [0]), ([1], [-1])):
        with pytest.raises(mk.MkError):
            mk.prefix_attention(*args, *bad)


# ---------------------------------------------------------------- together, as a serving loop has them
@pytest.mark.parametrize("q8", [False, True])
def test_a_layer_of_a_batch_behind_a_common_prompt(q8):
    """The common prompt goes into the cache once; every sequence's own rows behind it; attention over both; then a
    token more each, in a full layer (shared pages) and in one of short sight (a window and sinks), whose pages
    between are given back."""
    hq, hkv, d, ps, n, shared = 16, 2, 128, 16, 6, 640
    own = [33, 5, 16, 70, 1, 48]
    lens = [shared + x for x in own]
    st = R.Setup(hq, hkv, d, ps, [x + 1 for x in lens], own, q8=q8, seed=51)
    S.share(st, [n], [shared])
    rope = mk.Rope(mk.rope_frequencies(d, 1e4))
    sh = st.shape(mk)
    first = st.normal(shared, (hq + 2 * hkv) * d, std=1.3)
    mk.append_chunk(sh, first, [shared], [shared], st.bt[:1], st.kv, rope)     # once, through the first one's table
    st.rows, st.lens, st.news = sum(own), lens, own
    q = mk.append_chunk(sh, st.normal(st.rows, (hq + 2 * hkv) * d, std=1.3), own, lens, st.bt, st.kv, rope)
    check_prefix(st, [n], [shared], q=q)
    check_window(st, 100, 4, q=q)
    st.lens, st.news, st.rows = [x + 1 for x in lens], [1] * n, n
    q = mk.append_chunk(sh, st.normal(n, (hq + 2 * hkv) * d, std=1.3), st.news, st.lens, st.bt, st.kv, rope)
    _, full = check_prefix(st, [n], [shared], q=q)
    ref, *scale = S.attention(st, q, st.kv)
    same = mk.chunk_attention(sh, q, st.news, st.lens, st.bt, st.kv)
    assert torch.all((full.double() - same.double()).abs() <= 2 * R.attention_bound(ref, *scale, q8))
    st.bt[:, 1:30] = -1                                   # (positions 16..479: nobody sees them through a window of 100)
    check_window(st, 100, 4, q=q)
