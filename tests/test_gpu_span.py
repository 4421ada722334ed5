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


@pytest.mark.parametrize("hq,hkv,d,q8", [(32, 4, 128, False), (32, 4, 128, True), (14, 2, 64, False), (6, 3, 128, False)])
def test_window_few_rows_of_many_partials(hq, hkv, d, q8):
    # long windows of one and two rows, cut over all blocks; and of more of them
    for lens, news, window in (([40000], [1], 30000), ([20000, 31000], [2, 1], 25000), ([9000] * 12, [1] * 12, 8000)):
        st = R.Setup(hq, hkv, d, 64, lens, news, q8=q8, seed=17)
        hide(st, window, 4)
        check_window(st, window, 4)


def test_window_three_launches():
    # q8_0: a prompt that is decoded once, forty rows, and tokens too many to go with these
    lens = [4500, 9000] + [9000 + 13 * i for i in range(40)]
    st = R.Setup(32, 4, 128, 64, lens, [4096, 40] + [1] * 40, q8=True, seed=18)
    hide(st, 8192, 4)
    seg = mk.plan_span_attention(st.shape(mk), st.news, st.lens, 8192, 4)
    assert sorted(set(seg[:, 0].tolist())) == [0, 1, 2]
    check_window(st, 8192, 4)


@pytest.mark.parametrize("lens,news,window,sinks,ps", [
    ([16384], [1024], 2048, 4, 16), ([9000], [4096], 512, 4, 16), ([12345], [4096], 512, 0, 8), ([9000, 40, 5000], [4096, 1, 2000], 500, 130, 40)])
def test_window_decoded_before_with_pages_given_back(lens, news, window, sinks, ps):
    # q8_0 prompts that are decoded once: what lies between the sinks and the first window is given back, inside the
    # tiles of 128 positions that these share too, and nothing is reported
    st = R.Setup(32, 4, 128, ps, lens, news, q8=True, seed=22)
    hide(st, window, sinks)
    seg = mk.plan_span_attention(st.shape(mk), st.news, st.lens, window, sinks)
    assert 1 in seg[:, 0]
    check_window(st, window, sinks)


@pytest.mark.parametrize("q8", [False, True])
def test_window_of_a_poisoned_position_in_cut_items(q8):
    # a NaN behind the sinks is nobody's, one in the window of a token whose item is cut is that token's alone
    st = R.Setup(32, 4, 128, 16, [20000] * 3, [1] * 3, q8=q8, seed=19)
    q = st.normal(3, 32, 128, std=1.5)
    ref, *scale = S.attention(st, q, st.kv, 9000, 4)
    bound = R.attention_bound(ref, *scale, q8)
    for s, pos in ((0, 5), (1, 15000)):
        page, off = int(st.bt[s, pos // 16]), pos % 16
        if q8:
            st.planes()[1][page, :, :, off] = float("nan")
        else:
            st.kv[page, :, :, off] = float("nan")
    out = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 9000, 4)
    good = torch.tensor([True, False, True], device="cuda")
    assert torch.all(((out.double() - ref).abs() <= bound)[good]) and torch.all(out[1].isnan())


@pytest.mark.parametrize("d,q8", [(128, False), (128, True), (64, False)])
def test_infinite_values_of_a_row_that_many_blocks_join(d, q8):
    # one token through a long window: 16 columns a block in the join.  Columns that are worked out again, those of a block
    # that has one which is not finite, are written by that block alone: the others keep what was joined, in every run
    st = R.Setup(32, 4, d, 64, [60000], [1], q8=q8, seed=23)
    q = st.normal(1, 32, d, std=1.5)
    args = (st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 50000, 4)
    clean = mk.window_attention(*args)
    page, off = int(st.bt[0, 59000 // 64]), 59000 % 64
    if q8:
        st.planes()[1][page, 1, 2, off, 1] = float("inf")          # dims 32..63 of KV head 2
        hit = slice(32, 64)
    else:
        st.kv[page, 1, 2, off, 37] = float("inf")
        hit = slice(32, 48)
    out = mk.window_attention(*args)
    other = torch.ones(1, 32, d, dtype=torch.bool, device="cuda")
    other[:, 16:24, hit] = False                                   # (KV head 2's query heads)
    assert torch.equal(out[other], clean[other]) and not torch.any(out[:, 16:24, 37].isfinite())
    if not q8:
        ref, *scale = S.attention(st, q, torch.where(st.kv.isinf(), 0.0, st.kv), 50000, 4)
        near = (out.double() - ref).abs() <= R.attention_bound(ref, *scale, q8)
        near[:, 16:24, 37] = True
        assert torch.all(near)
    for _ in range(20):
        assert torch.equal(mk.window_attention(*args).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("q8", [False, True])
def test_offsets_beyond_32_bits(q8):
    # a pool of more than 4 GiB, of which the sequences have the last pages and the first ones
    hq, hkv, d, ps = 16, 8, 128, 128
    P = (9 << 29) // (hkv * ps * d) if q8 else (9 << 28) // (hkv * ps * d)
    small = R.Setup(hq, hkv, d, ps, [1500, 1500, 900], [3, 1, 200], q8=q8, seed=20)
    S.share(small, [2, 1], [1280, 0])
    n = P * 2 * hkv * ps * d
    kv = torch.zeros(n + n // 16, dtype=torch.uint8, device="cuda") if q8 else torch.zeros(P, 2, hkv, ps, d, dtype=torch.bfloat16,
                                                                                       device="cuda")
    assert kv.nbytes > 1 << 32
    to = torch.tensor([P - 1 - i if i % 2 else i for i in range(small.P)], device="cuda")
    if q8:
        codes = kv[:n].view(torch.int8).view(P, 2, hkv, ps, d)
        scales = kv[n:].view(torch.float16).view(P, 2, hkv, ps, d // 32)
        a, b = small.planes()
        codes[to], scales.view(torch.int16)[to] = a, b.view(torch.int16)
    else:
        kv[to] = small.kv
    q = small.normal(small.rows, hq, d, std=1.5)
    bt = torch.where(small.bt >= 0, to[small.bt.clamp(min=0).long()].to(torch.int32), small.bt)
    sh = mk.CacheShape(hq, hkv, d, ps, P, small.maxpg, mk.FLAG_KV_Q8 if q8 else 0)
    for call in (lambda s, t, k: mk.window_attention(s, q, small.news, small.lens, t, k, 700, 4),
                 lambda s, t, k: mk.prefix_attention(s, q, small.news, small.lens, t, k, [2, 1], [1280, 0])):
        want = call(small.shape(mk), small.bt, small.kv)
        assert torch.equal(call(sh, bt, kv), want) and not want.isnan().any()


def test_output_aligned_to_16_bytes():
    st = R.Setup(16, 2, 128, 16, [900, 3000], [300, 1], seed=21)
    q = st.normal(301, 16, 128, std=1.5)
    for off in (8, 16, 24):
        buf = torch.full((301 * 2048 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[off:off + 301 * 2048].view(301, 16, 128)
        want = mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 500, 4)
        mk.window_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, 500, 4, out=out)
        assert torch.equal(out, want) and torch.all(buf[:off] == 7.0) and torch.all(buf[off + 301 * 2048:] == 7.0)


@pytest.mark.parametrize("window", [None, 1 << 30])
def test_segments_of_seconds(window):
    # 152 units over 3 * 2^27 positions: each block goes over 3 * 2^20 tiles in one segment, some 3 s, and the waits that last as
    # long (for the next query rows, for the last values) do not give up.  All scores are 0; values are 1 in every 64th
    # page and 0 in the others, so the sums of values are whole numbers up to 3 * 2^21, exact in fp32 in whatever groups they
    # are added, and those of weights multiples of 128 up to 3 * 2^27, exact too; two pages that repeat.
    rows, ps, ln = 152 * 256, 64, 3 << 27
    kv = torch.zeros(2, 2, 1, ps, 64, dtype=torch.bfloat16, device="cuda")
    kv[1, 1] = 1.0
    bt = (torch.arange(ln // ps, device="cuda", dtype=torch.int32) % 64 == 63).to(torch.int32)[None].contiguous()
    sh = mk.CacheShape(1, 1, 64, ps, 2, ln // ps, 0)
    q = torch.ones(rows, 1, 64, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    if window is None:
        seg = mk.plan_chunk_attention(sh, [rows], [ln])[:, 6]
        out = mk.chunk_attention(sh, q, [rows], [ln], bt, kv, status=status)
    else:
        seg = mk.plan_span_attention(sh, [rows], [ln], window=window)[:, 12]
        out = mk.window_attention(sh, q, [rows], [ln], bt, kv, window, status=status)
    assert seg.max() > 3_000_000 and int(status) == mk.MK_OK
    seen = torch.arange(ln - rows, ln, device="cuda") + 1
    want = (seen // 4096 * 64 + (seen % 4096 - 63 * 64).clamp(min=0)).double() / seen
    # (a row's last tile may hold any whole number of weights: the sum of all is off by at most 2^-24 there; the output
    # rounds to 2^-8)
    assert torch.all((out[:, 0].double() - want[:, None]).abs() <= want[:, None] * (2.0 ** -8 + 2.0 ** -20))


LONG = [
    # rows, sequences, hq, hkv, positions, q8: two tiles of rows a unit; streams of one token, cut over all blocks; many
    # tokens (two KV heads an item in a window); and over q8_0 few rows, more rows, and a prompt that is decoded before
    (152 * 256, 1, 1, 1, 1 << 21, False), (1, 1, 1, 1, 1 << 27, False), (1, 64, 4, 4, 1 << 20, False),
    (1, 1, 1, 1, 1 << 27, True), (5, 1, 8, 1, 1 << 27, True), (30000, 1, 1, 1, 1 << 20, True),
]


@pytest.mark.parametrize("window", [None, 1 << 30])
@pytest.mark.parametrize("rows,seqs,hq,hkv,ln,q8", LONG)
def test_sums_over_millions_of_positions(rows, seqs, hq, hkv, ln, q8, window):
    # Three kinds of pages of 64 positions: most have scores of 0 and values of 1, one in 5000 scores of 7.5 and values of
    # -3, one in 12000 scores of 11 and values of 2.  (All of the last lie further apart than what a block adds up before
    # it moves its sums to the workspace.)
    d, ps = (128 if q8 else 64), 64
    n = 3 * 2 * hkv * ps * d
    want_k, want_v = (0.0, 7.5 / d ** 0.5, 11 / d ** 0.5), (1.0, -3.0, 2.0)
    if q8:
        kv = torch.zeros(n + n // 16, dtype=torch.uint8, device="cuda")
        x = kv[:n].view(torch.int8).view(3, 2, hkv, ps, d)
        scale = kv[n:].view(torch.float16).view(3, 2, hkv, ps, d // 32)
        x[...] = 64
        for i in range(3):
            scale[i, 0], scale[i, 1] = want_k[i] / 64, want_v[i] / 64
        key = scale[:, 0, 0, 0, 0].double() * 64
    else:
        kv = torch.zeros(3, 2, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
        for i in range(3):
            kv[i, 0], kv[i, 1] = want_k[i], want_v[i]
        key = kv[:, 0, 0, 0, 0].double()
    at = torch.arange(ln // ps, device="cuda")
    kind = torch.where(at % 12000 == 7001, 2, torch.where(at % 5000 == 3001, 1, 0)).to(torch.int32)
    kind[-(rows // ps + 1):] = 0
    sh = mk.CacheShape(hq, hkv, d, ps, 3, ln // ps, mk.FLAG_KV_Q8 if q8 else 0)
    cl, sl, bt = [rows] * seqs, [ln] * seqs, kind[None].repeat(seqs, 1)
    q = torch.ones(rows * seqs, hq, d, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    if window is None:
        seg = mk.plan_chunk_attention(sh, cl, sl)[:, 6]
        out = mk.chunk_attention(sh, q, cl, sl, bt, kv, status=status)
    else:
        seg = mk.plan_span_attention(sh, cl, sl, window=window)[:, 12]
        out = mk.window_attention(sh, q, cl, sl, bt, kv, window, status=status)
    assert int(status) == mk.MK_OK and seg.max() > 4096
    w = (key * d ** 0.5).exp()
    value = torch.tensor(want_v, dtype=torch.float64, device="cuda")
    special = [ps * int((kind == i).sum()) for i in (1, 2)]
    common = (torch.arange(ln - rows, ln, device="cuda", dtype=torch.float64) + 1 - sum(special)).repeat(seqs)
    mass = torch.stack([common, *(torch.full_like(common, float(s)) * w[i + 1] for i, s in enumerate(special))])
    share = mass / mass.sum(0)
    want = (share * value[:, None]).sum(0)
    # A product adds 8 common weights and cuts off less than 2^-23 of the sum, which one page of the third kind makes up to
    # 128 w: 128 w / 2^23 of every 8 common ones at most, with what the page of the second kind has about as much again.
    # Weights round to 2^-8 (and to fp16, 2^-11, as do the q8_0 values), the output to 2^-8.
    cut = 2 * 128 * float(w[2]) / 2 ** 23 / 8
    assert cut < 0.25
    bound = share[0] * cut + (share * value[:, None].abs()).sum(0) * (2.0 ** -8 + 2.0 ** -10) + want.abs() * 2.0 ** -8
    assert torch.all((out.double() - want[:, None, None]).abs() <= bound[:, None, None])


@pytest.mark.parametrize("window", [None, 1 << 30])
@pytest.mark.parametrize("rows,seqs,hq,hkv,ln,q8", [(152 * 256, 1, 1, 1, 1 << 24, False), *LONG[1:]])
def test_sums_of_values_of_one_sign(rows, seqs, hq, hkv, ln, q8, window):
    # every score 0 and every value 1.3359375: a sum in one place loses 2 % of itself over four million positions
    d, ps = (128 if q8 else 64), 64
    n = 2 * hkv * ps * d
    if q8:
        kv = torch.zeros(n + n // 16, dtype=torch.uint8, device="cuda")
        kv[n // 2:n] = 1
        kv[n + n // 32:].view(torch.float16)[...] = 1.3359375
    else:
        kv = torch.zeros(1, 2, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
        kv[:, 1] = 1.3359375
    sh = mk.CacheShape(hq, hkv, d, ps, 1, ln // ps, mk.FLAG_KV_Q8 if q8 else 0)
    cl, sl = [rows] * seqs, [ln] * seqs
    bt = torch.zeros(seqs, ln // ps, dtype=torch.int32, device="cuda")
    q = torch.ones(rows * seqs, hq, d, dtype=torch.bfloat16, device="cuda")
    out = mk.chunk_attention(sh, q, cl, sl, bt, kv) if window is None else mk.window_attention(sh, q, cl, sl, bt, kv, window)
    # 2^18 positions are added up in one place, 8 at a time, each of which cuts off less than 2^-23 of a sum that is half of
    # its last on average: 2^-9; the output rounds to 2^-8
    assert torch.all((out.double() - 1.3359375).abs() <= 1.3359375 * (2.0 ** -8 + 2.0 ** -9))


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


def test_prefix_of_the_most_positions():
    # 2^30 - 128 shared positions: the rows of a second unit stand beyond 2^30, and still see the first page.  That holds
    # about half of the weight (64 e^16.625 against 2^30) and -1, every other position 1; its pages are one that repeats.
    n, rows, ps, ln = 5, 100, 64, 1 << 30
    kv = torch.zeros(2 + 2 * n, 2, 1, ps, 64, dtype=torch.bfloat16, device="cuda")
    kv[:, 1] = 1.0
    kv[0, 0], kv[0, 1] = 2.078125, -1.0                  # (q . k / 8 = 16.625, exactly)
    bt = torch.ones(n, ln // ps, dtype=torch.int32, device="cuda")
    bt[:, 0] = 0
    bt[:, -2:] = torch.arange(2, 2 + 2 * n, device="cuda", dtype=torch.int32).view(n, 2)
    sh = mk.CacheShape(1, 1, 64, ps, kv.shape[0], ln // ps, 0)
    args = (sh, [rows] * n, [ln] * n)
    q = torch.ones(n * rows, 1, 64, dtype=torch.bfloat16, device="cuda")
    seg = mk.plan_span_attention(*args, group_seqs=[n], prefix_lens=[ln - rows])
    assert {256} <= set(seg[:, 4].tolist())              # (the group's second unit of rows)
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    out = mk.prefix_attention(sh, q, *args[1:], bt, kv, [n], [ln - rows], status=status)
    assert int(status) == mk.MK_OK
    first = 64 * np.exp(16.625)
    rest = torch.arange(ln - rows, ln, device="cuda", dtype=torch.float64).repeat(n) + 1 - 64
    want = (rest - first) / (rest + first)
    # weights are powers of 2 times 1, so sums below 2^24 are exact; the segment that holds the first page may lose its
    # others' (2^-24 of that page's each), which moves numerator and denominator by as much; bf16 rounds to 2^-8
    lost = int(seg[:, 12].max()) * 128 / (ln + first)
    assert lost < 0.02
    assert torch.all((out[:, 0].double() - want[:, None]).abs() <= 2 * lost + 2.0 ** -8)


@pytest.mark.parametrize("q8", [False, True])
def test_prefix_with_prompts_among_single_tokens(q8):
    st = prefix_setup(16, 2, 128, 16, [12, 4], [5000, 3000], [300, 20, 700], [260, 1, 1, 513], q8, seed=33)
    check_prefix(st, [12, 4], [5000, 3000])


@pytest.mark.parametrize("hq,hkv,d,q8", [(32, 4, 128, False), (32, 4, 128, True), (4, 1, 64, False), (7, 1, 128, False)])
def test_prefix_with_many_rows_to_join(hq, hkv, d, q8):
    # rows of several 8s a unit, several blocks of them; and few rows of many partials
    for n, news, shared in ((64, 9, 6000), (48, 16, 9000), (3, 1, 60000)):
        st = prefix_setup(hq, hkv, d, 16, [n], [shared], [40, 21], [news], q8, seed=36)
        check_prefix(st, [n], [shared])


def test_prefix_groups_with_empty_sequences():
    # sequences without new tokens stand in groups (first, last and between), and a whole group of them
    lens = [5000] * 24 + [40, 900, 700]
    news = [0] + [1] * 10 + [0] * 2 + [1] * 10 + [0] + [0, 0, 5]
    st = R.Setup(32, 4, 128, 16, lens, news, seed=37)
    S.share(st, [24, 2, 1], [4800, 32, 0])
    check_prefix(st, [24, 2, 1], [4800, 32, 0])


@pytest.mark.parametrize("q8", [False, True])
def test_prefix_group_led_by_sequences_without_rows(q8):
    # their tables name no page: they are not read, and nothing is reported
    lens, news = [5000] * 30, [0, 0] + [1] * 27 + [0]
    st = R.Setup(32, 4, 128, 16, lens, news, q8=q8, seed=38)
    S.share(st, [30], [4800])
    st.bt[[0, 1, 29]] = -1
    check_prefix(st, [30], [4800])


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


@pytest.mark.parametrize("q8", [False, True])
def test_two_graphs_share_a_workspace(q8):
    # one after the other on a stream, each many times, with other calls between: a call owns the workspace while it runs
    st = prefix_setup(16, 2, 128, 16, [40], [6000], [60, 9], [1], q8, seed=44)
    q = st.normal(st.rows, 16, 128, std=1.5)
    args = (st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
    need = max(mk.prefix_attention_workspace(*[args[i] for i in (0, 2, 3)], [40], [6000]),
               mk.window_attention_workspace(*[args[i] for i in (0, 2, 3)], 5000, 4))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = mk.prefix_attention(*args, [40], [6000]), mk.window_attention(*args, 5000, 4)
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, call in zip(graphs, (lambda: mk.prefix_attention(*args, [40], [6000], workspace=ws),
                                lambda: mk.window_attention(*args, 5000, 4, workspace=ws))):
        call()
        with torch.cuda.graph(g):
            got.append(call())
    for i in (0, 1, 0, 0, 1, 1, 0, 1):
        got[i].zero_()
        graphs[i].replay()
        mk.chunk_attention(*args)
        graphs[1 - i].replay()
        ws.fill_(0xff)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_follow_each_other_without_a_pause():
    # each call's first kernel may set itself up while the one before ends: what it reads is what that one wrote
    st = prefix_setup(16, 2, 128, 16, [20], [3000], [60, 9], [1], False, seed=45)
    args = (st.shape(mk), st.news, st.lens, st.bt, st.kv)
    first = st.normal(st.rows, 16, 128, std=1.5)

    def chain(wait):
        q = first.clone()
        for _ in range(12):
            q = mk.window_attention(args[0], q * 3, *args[1:], 700, 4)
            if wait:
                torch.cuda.synchronize()
            q = mk.prefix_attention(args[0], q, *args[1:], [20], [3000])
            if wait:
                torch.cuda.synchronize()
        return q
    want = chain(True)
    for _ in range(3):
        assert torch.equal(chain(False), want)


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
