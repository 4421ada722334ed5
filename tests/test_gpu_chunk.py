"""GPU tests of the operators on chunks of new tokens over the paged cache (include/mk_chunk.h):
append (norms, rotary positions, the bf16 and q8_0 write), causal attention, read-back, each
against its definition in 64 bits (tests/chunk_ref.py), and a run of them together with the
decode step.  Pages that no sequence owns and positions behind a last one hold NaNs throughout."""
import numpy as np
import pytest
import torch

import workloads as W
import persistent_moe_decode_megakernel_gb300 as mk
from tests import chunk_ref as R

pytestmark = pytest.mark.gpu

H = 2.0 ** -8    # a bf16 rounding is off by at most this much of the value


@pytest.fixture(scope="module", autouse=True)
def built():
    mk.build()


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.uint8 else t.view(torch.int16)


# ---------------------------------------------------------------- append
def append_case(st, rot, inter, norm, theta=1e4, mscale=1.0, seed=1, extra_rows=0, stride_pad=0, freq=None):
    width = (st.hq + 2 * st.hkv) * st.d
    buf = st.normal(st.rows + extra_rows, width + stride_pad, std=1.3)
    qkv = buf[:, :width]
    freq = (mk.rope_frequencies(rot, theta) if rot else ()) if freq is None else freq
    gains = [(1 + 0.2 * torch.randn(st.d, generator=st.g, device="cuda")).to(torch.bfloat16) if norm else None
             for _ in range(2)]
    return qkv, mk.Rope(freq, inter, mscale) if rot else None, torch.from_numpy(np.asarray(freq)), gains


def check_append(st, rot, inter, norm, eps=1e-6, mscale=1.0, **kw):
    qkv, rope, freq, gains = append_case(st, rot, inter, norm, mscale=mscale, **kw)
    before = st.kv.clone()
    extra = qkv.shape[0] - st.rows
    q_out = torch.full((st.rows + extra, st.hq, st.d), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    got = mk.append_chunk(st.shape(mk), qkv, st.news, st.lens, st.bt, st.kv, rope=rope, q_norm=gains[0], k_norm=gains[1],
                          eps=eps, q_out=q_out, status=status)
    assert got is q_out and int(status) == mk.MK_OK
    assert torch.all(q_out[st.rows:] == 7.0)        # rows behind the last sequence's
    x = qkv[:st.rows].double().reshape(st.rows, st.hq + 2 * st.hkv, st.d)
    seq, pos = st.positions()
    q, k, v = x[:, :st.hq], x[:, st.hq:st.hq + st.hkv], x[:, st.hq + st.hkv:]
    if norm:
        q, k = R.head_norm(q, gains[0], eps), R.head_norm(k, gains[1], eps)
    # fp32 noise: the norm's sum of D squares and its square root (D/8 + 16 roundings of 2^-24), the
    # angle's cos and sin (4 of 2^-24, scaled by mscale) and two products, all of the pair's magnitude
    scale = max(1.0, abs(mscale))
    pair = lambda t: scale * t.abs().amax(-1, keepdim=True)  # noqa: E731
    nq, nk = pair(q) * 64 * 2.0 ** -24, pair(k) * 64 * 2.0 ** -24
    if rot:
        q, k = R.rotate(q, pos, freq, inter, mscale), R.rotate(k, pos, freq, inter, mscale)
    assert torch.all((q_out[:st.rows].double() - q).abs() <= q.abs() * H + nq * (1 + H))
    page, off = st.bt[seq, pos // st.ps].long(), pos % st.ps
    if st.q8:
        codes, scales = st.planes()
        c, s = codes[page, :, :, off].double(), scales[page, :, :, off]
        want = torch.stack([k, v], 1)                # [rows][2][Hkv][D]
        step = want.unflatten(-1, (-1, 32)).abs().amax(-1) / 127
        noise = torch.stack([nk.expand_as(k), torch.zeros_like(v)], 1)
        # the scale: fp32 noise, then half a step of f16 (2^-11 of it)
        sn = noise.unflatten(-1, (-1, 32)).amax(-1) / 127 + step * 2.0 ** -23
        assert torch.all((s.double() - step).abs() <= (step + sn) * 2.0 ** -11 + sn + 2.0 ** -25)
        full = step.repeat_interleave(32, -1)
        # the code: half a step, and the noise of the value and of the scale over 127 steps
        assert torch.all((c * full - want).abs() <= full * (0.5 + 127 * 2.0 ** -22) + 2 * noise + 1e-30)
        assert c.abs().max() <= 127
    else:
        assert torch.all((st.kv[page, 0, :, off].double() - k).abs() <= k.abs() * H + nk * (1 + H))
        assert torch.equal(st.kv[page, 1, :, off], v.to(torch.bfloat16))
    # nothing but the new positions was written
    touched = torch.zeros(st.P, st.ps, dtype=torch.bool, device="cuda")
    touched[page, off] = True
    if st.q8:
        for a, b in zip(st.planes(), st.planes(before)):
            same = (a.contiguous().view(torch.uint8) == b.contiguous().view(torch.uint8)).all(-1)
            assert torch.all(same | touched[:, None, None, :])
    else:
        same = (bits(st.kv) == bits(before)).all(-1)
        assert torch.all(same | touched[:, None, None, :])


APPEND_SHAPES = [
    # hq, hkv, d, ps, lens, news
    (4, 2, 64, 16, [65], [65]),
    (32, 4, 128, 16, [1, 512, 33], [1, 1, 1]),
    (7, 1, 128, 24, [100, 40], [37, 40]),
    (8, 8, 64, 8, [9, 300], [2, 299]),
    (6, 2, 128, 40, [2000, 77, 5], [1400, 0, 5]),
    (5, 5, 128, 128, [129], [129]),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rot,inter,norm", [(1.0, False, False), (1.0, True, True), (0.5, False, True), (0.25, True, False),
                                            (0, False, True), (0.75, False, False)])
@pytest.mark.parametrize("hq,hkv,d,ps,lens,news", APPEND_SHAPES)
def test_append(hq, hkv, d, ps, lens, news, rot, inter, norm, q8):
    if q8 and d != 128:
        d = 128
    st = R.Setup(hq, hkv, d, ps, lens, news, q8=q8, seed=3)
    check_append(st, int(rot * d), inter, norm, extra_rows=2)


@pytest.mark.parametrize("q8", [False, True])
def test_append_strided_rows_eps_and_mscale(q8):
    st = R.Setup(8, 2, 128, 16, [70, 3], [50, 3], q8=q8, seed=4)
    check_append(st, 128, False, True, eps=0.5, mscale=1.37, stride_pad=72, extra_rows=1)


@pytest.mark.parametrize("pos", [0, 1, 131071, 1048575, (1 << 29) + 12345])
def test_rotary_angles_of_far_positions(pos):
    # one token at a far position: its page alone exists (earlier block-table entries are not read)
    ps = 128
    maxpg = pos // ps + 1
    sh = mk.CacheShape(2, 1, 128, ps, 2, maxpg)
    kv = torch.zeros(2, 2, 1, ps, 128, dtype=torch.bfloat16, device="cuda")
    bt = torch.full((1, maxpg), -1, dtype=torch.int32, device="cuda")
    bt[0, pos // ps] = 1
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    qkv = torch.randn(1, 4 * 128, generator=g, device="cuda").to(torch.bfloat16)
    freq = mk.rope_frequencies(128, 1e4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = mk.append_chunk(sh, qkv, [1], [pos + 1], bt, kv, rope=mk.Rope(freq), status=status)
    x = qkv.double().view(1, 4, 128)
    want = R.rotate(x, torch.tensor([pos], device="cuda"), torch.from_numpy(freq), False)
    # the angle itself: a 64-bit frequency is off by 2^-53 of itself and its turns by as much
    far = pos * 2.0 ** -52 * x.abs().max()
    assert int(status) == 0
    assert torch.all((q.double() - want[:, :2]).abs() <= want[:, :2].abs() * H + 2.0 ** -18 * x.abs().max() + far)
    assert torch.all((kv[1, 0, :, pos % ps].double() - want[:, 2]).abs()
                     <= want[:, 2].abs() * H + 2.0 ** -18 * x.abs().max() + far)


def test_append_reports_pages_out_of_range():
    st = R.Setup(4, 2, 128, 16, [40, 20], [40, 20], seed=6)
    good = st.bt.clone()
    st.bt[0, 1], st.bt[1, 0] = st.P, -7
    qkv, rope, freq, _ = append_case(st, 128, False, False)
    before = st.kv.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = mk.append_chunk(st.shape(mk), qkv, st.news, st.lens, st.bt, st.kv, rope=rope, status=status)
    assert int(status) == mk.MK_ERR_DEVICE_BOUNDS
    kv_bad, st.kv = st.kv, before
    q2 = mk.append_chunk(st.shape(mk), qkv, st.news, st.lens, good, st.kv, rope=rope, status=status)
    assert int(status) == mk.MK_OK and torch.equal(q, q2)
    for s, p in ((0, 0), (0, 2), (1, 1)):            # the pages that were in range hold the same
        n = min(st.lens[s] - p * 16, 16)
        assert torch.equal(bits(kv_bad[good[s, p].long(), :, :, :n]), bits(st.kv[good[s, p].long(), :, :, :n]))


# ---------------------------------------------------------------- read-back
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hkv,d,ps,lens,counts", [(2, 64, 16, [65], [65]), (4, 128, 24, [100, 7, 1], [33, 0, 1]),
                                                  (1, 128, 8, [1000], [999]), (8, 128, 64, [64, 129], [64, 2])])
def test_read_cache(hkv, d, ps, lens, counts, q8):
    st = R.Setup(hkv, hkv, 128 if q8 else d, ps, lens, counts, q8=q8, seed=7)
    k, v = mk.read_cache(st.shape(mk), counts, lens, st.bt, st.kv)
    want = torch.cat([st.cached(st.kv, s, ln)[:, :, ln - n:] for s, (ln, n) in enumerate(zip(lens, counts))], 2)
    want = want.transpose(1, 2)
    assert torch.equal(k, want[0].float().to(torch.bfloat16))     # code * scale is exact in fp32
    assert torch.equal(v, want[1].float().to(torch.bfloat16))


def test_read_cache_zeros_for_pages_out_of_range():
    st = R.Setup(2, 2, 64, 16, [40], [40], seed=8)
    st.bt[0, 1] = 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = mk.read_cache(st.shape(mk), [40], [40], st.bt, st.kv, status=status)
    assert int(status) == mk.MK_ERR_DEVICE_BOUNDS
    assert torch.all(k[16:32] == 0) and torch.all(v[16:32] == 0) and torch.all(k[:16] != 0) and torch.all(v[32:] != 0)


# ---------------------------------------------------------------- attention
def check_attention(st, std=1.5, drop=None, status_want=mk.MK_OK, q=None, extra_rows=0):
    q = st.normal(st.rows + extra_rows, st.hq, st.d, std=std) if q is None else q
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    out = torch.full((st.rows + extra_rows, st.hq, st.d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, out=out, status=status)
    assert got is out and int(status) == status_want
    assert torch.all(out[st.rows:] == 7.0)
    ref, *scale = R.attention(st, q, st.kv, drop)
    far = (out[:st.rows].double() - ref).abs()
    bound = R.attention_bound(ref, *scale, st.q8)
    assert torch.all(far <= bound), float((far / bound).max())
    return q, out


ATTN_SHAPES = [
    # hq, hkv, d, ps, lens, news: one token, one position, page edges, tiles' edges, ragged, odd groups
    (4, 2, 64, 16, [65], [65]),
    (1, 1, 128, 8, [1], [1]),
    (8, 1, 128, 16, [16, 17, 128, 129], [1, 1, 1, 1]),
    (8, 1, 128, 16, [16, 17, 128, 129, 1], [16, 17, 128, 129, 1]),
    (32, 4, 128, 16, [513, 40, 1000], [100, 0, 3]),
    (3, 1, 64, 24, [200, 300], [200, 47]),
    (10, 2, 128, 40, [333], [333]),
    (12, 2, 128, 64, [400, 64], [31, 64]),
    (7, 1, 64, 8, [700], [69]),
    (16, 16, 64, 128, [130, 257], [130, 129]),
    (14, 2, 128, 256, [700], [300]),
    (32, 4, 128, 16, [5000], [1]),
    (16, 2, 128, 64, [9001, 3], [2, 1]),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,ps,lens,news", ATTN_SHAPES)
def test_attention(hq, hkv, d, ps, lens, news, q8):
    st = R.Setup(hq, hkv, 128 if q8 else d, ps, lens, news, q8=q8, seed=9)
    check_attention(st, extra_rows=1)


@pytest.mark.parametrize("q8", [False, True])
def test_attention_64_sequences(q8):
    g = np.random.default_rng(1)
    lens = [int(x) for x in np.exp(g.uniform(0, np.log(3000), 64)).astype(int)]
    news = [min(ln, int(g.choice([0, 1, 1, 1, 5, 67]))) for ln in lens]
    check_attention(R.Setup(16, 2, 128, 16, lens, news, q8=q8, seed=10))


@pytest.mark.parametrize("std", [0.0, 30.0])
def test_attention_flat_and_peaked_scores(std):
    # all scores equal; and scores so far apart that the running maximum moves often and by much
    check_attention(R.Setup(8, 2, 128, 16, [1500], [70], seed=11), std=std)


def test_attention_rising_scores():
    # every later key scores higher than all before: the running maximum moves with every tile
    st = R.Setup(8, 1, 128, 16, [2000], [50], seed=12)
    pos = torch.arange(2000, device="cuda")
    page, off = st.bt[0, pos // 16].long(), pos % 16
    k = torch.zeros(2000, 128, device="cuda")
    k[:, 0] = pos * 0.25
    st.kv[page, 0, 0, off] = k.to(torch.bfloat16)
    q = st.normal(50, 8, 128)
    q[..., 0] = 4.0
    check_attention(st, q=q)


def test_attention_strided_query_rows():
    st = R.Setup(6, 2, 128, 16, [300, 30], [111, 30], seed=13)
    qkv = st.normal(141, (6 + 4) * 128 + 8)
    check_attention(st, q=qkv[:, :6 * 128].unflatten(1, (6, 128)))


@pytest.mark.parametrize("q8", [False, True])
def test_attention_skips_pages_out_of_range(q8):
    st = R.Setup(8, 2, 128, 16, [100, 300, 20], [100, 3, 20], q8=q8, seed=14)
    drop = torch.zeros(3, 300, dtype=torch.bool, device="cuda")
    for s, p, bad in ((0, 0, st.P), (0, 3, -1), (1, 18, 1 << 30), (1, 2, -(1 << 31)), (2, 0, -5), (2, 1, 1 << 20)):
        drop[s, p * 16:p * 16 + 16] = True          # rows 0..15 of sequence 0 and all of sequence 2 see nothing
    ref_bt = st.bt.clone()
    bad_bt = st.bt.clone()
    for s, p, bad in ((0, 0, st.P), (0, 3, -1), (1, 18, 1 << 30), (1, 2, -(1 << 31)), (2, 0, -5), (2, 1, 1 << 20)):
        bad_bt[s, p] = bad
    q = st.normal(st.rows, 8, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, bad_bt, st.kv, status=status)
    assert int(status) == mk.MK_ERR_DEVICE_BOUNDS
    st.bt = ref_bt
    ref, *scale = R.attention(st, q, st.kv, drop)
    assert torch.all((out.double() - ref).abs() <= R.attention_bound(ref, *scale, q8))
    assert torch.all(out[:16] == 0) and torch.all(out[103:] == 0)


@pytest.mark.parametrize("hq,hkv,d,len_,new", [(4, 1, 64, 90, 90), (8, 1, 128, 5000, 90)])
@pytest.mark.parametrize("which,value", [(0, "nan"), (1, "nan"), (1, "inf")])
def test_attention_nan_in_a_later_position_stays_there(hq, hkv, d, len_, new, which, value):
    # a NaN or infinity of the sequence reaches the rows that see it, and no other row of its tile
    st = R.Setup(hq, hkv, d, 16, [len_], [new], seed=15)
    q = st.normal(new, hq, d)
    ref, *scale = R.attention(st, q, st.kv)
    pos, row = len_ - 10, new - 10
    st.kv[st.bt[0, pos // 16].long(), which, 0, pos % 16, 5] = float(value)
    out = mk.chunk_attention(st.shape(mk), q, [new], [len_], st.bt, st.kv)
    bound = R.attention_bound(ref, *scale, False)
    assert torch.all((out[:row].double() - ref[:row]).abs() <= bound[:row])
    hit = out[row:] if which == 0 else out[row:, :, 5]
    assert torch.isnan(hit).all() if value == "nan" else torch.isinf(hit).all()


@pytest.mark.parametrize("q8", [False, True])
def test_attention_all_rows_poisoned(q8):
    # a NaN at position 0 is every row's: each is worked out again, and none but NaN comes of it
    st = R.Setup(16, 2, 128, 16, [3000, 40], [300, 7], q8=q8, seed=21)
    q = st.normal(st.rows, 16, 128)
    page = st.bt[0, 0].long()
    if q8:
        st.planes()[1][page, 0, :, 0] = float("nan")
    else:
        st.kv[page, 0, :, 0] = float("nan")
    out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
    assert torch.isnan(out[:300]).all() and torch.isfinite(out[300:]).all()


@pytest.mark.parametrize("len_,new", [(90, 90), (5000, 2)])
def test_attention_q8_values_beyond_fp16(len_, new):
    # decoded values above 65504 (scales up to f16's largest) in a few positions, K and V
    st = R.Setup(8, 2, 128, 16, [len_], [new], q8=True, seed=19)
    codes, scales = st.planes()
    for pos, which, sc in ((3, 1, 60000.0), (len_ - 5, 1, 3000.0), (len_ // 2, 0, 600.0), (len_ - 1, 0, 40000.0)):
        page = st.bt[0, pos // 16].long()
        scales[page, which, :, pos % 16, 1] = sc
    check_attention(st, std=0.02)


def test_attention_q8_sequences_of_many_rows_and_of_few():
    # those of many rows are decoded into the workspace first; pages out of range, values beyond fp16 and a
    # tail inside a page on both sides
    lens, news = [700, 300, 40, 513], [650, 2, 40, 300]
    st = R.Setup(16, 2, 128, 24, lens, news, q8=True, seed=25)
    assert set(mk.plan_chunk_attention(st.shape(mk), news, lens)[:, 0].tolist()) == {0, 1}
    codes, scales = st.planes()
    for s, pos, which, sc in ((0, 3, 1, 50000.0), (0, 600, 0, 700.0), (3, 511, 1, 65504.0), (1, 100, 1, 2000.0)):
        scales[st.bt[s, pos // 24].long(), which, :, pos % 24, 2] = sc
    drop = torch.zeros(4, 700, dtype=torch.bool, device="cuda")
    good, bad = st.bt.clone(), st.bt.clone()
    for s, p, v in ((0, 0, -1), (0, 7, st.P), (3, 20, 1 << 30), (1, 3, -9)):
        drop[s, p * 24:p * 24 + 24] = True
        bad[s, p] = v
    q = st.normal(st.rows, 16, 128, std=0.02)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mk.chunk_attention(st.shape(mk), q, news, lens, bad, st.kv, status=status)
    assert int(status) == mk.MK_ERR_DEVICE_BOUNDS
    st.bt = good
    ref, *scale = R.attention(st, q, st.kv, drop)
    far, bound = (out.double() - ref).abs(), R.attention_bound(ref, *scale, True)
    assert torch.all(far <= bound), float((far / bound).max())


# q8_0 units of at most 32 rows stand in each warp's lanes once: group sizes and tokens on both sides of that,
# contexts on both sides of a tile's quarters, split over blocks and whole
@pytest.mark.parametrize("hq,hkv,new", [(8, 1, 1), (8, 1, 4), (8, 1, 5), (3, 1, 10), (3, 1, 11), (10, 2, 6), (14, 2, 4), (2, 2, 32),
                                        (2, 2, 33), (2, 1, 16), (24, 4, 5)])
def test_attention_q8_few_rows(hq, hkv, new):
    lens = [new, max(new, 31), max(new, 33), max(new, 97), 128, 129, 160 + new, 2000, 9000]
    check_attention(R.Setup(hq, hkv, 128, 24, lens, [new] * len(lens), q8=True, seed=26), extra_rows=1)


def test_attention_q8_few_rows_large_scales_and_lost_pages():
    # scales on both sides of 2 and of what fp16 holds, in other quarters of other tiles; pages out of range, a whole
    # quarter's (32 positions) and a whole tile's among them
    lens, news = [1500, 130, 700], [2, 1, 3]
    st = R.Setup(8, 2, 128, 16, lens, news, q8=True, seed=27)
    codes, scales = st.planes()
    for s, pos, which, sc in ((0, 40, 0, 1.9990), (0, 300, 0, 2.0), (0, 301, 1, 511.0), (0, 900, 1, 520.0), (0, 1499, 0, 65504.0),
                              (1, 129, 1, 3.0), (2, 5, 0, 2.0)):
        scales[st.bt[s, pos // 16].long(), which, :, pos % 16, 3] = sc
    drop = torch.zeros(3, 1500, dtype=torch.bool, device="cuda")
    good, bad = st.bt.clone(), st.bt.clone()
    for s, p in [(0, 2), (0, 3), (0, 50), (1, 0), (1, 7)] + [(2, p) for p in range(8, 16)]:
        drop[s, p * 16:p * 16 + 16] = True
        bad[s, p] = st.P + p
    q = st.normal(st.rows, 8, 128, std=0.02)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mk.chunk_attention(st.shape(mk), q, news, lens, bad, st.kv, status=status)
    assert int(status) == mk.MK_ERR_DEVICE_BOUNDS
    st.bt = good
    ref, *scale = R.attention(st, q, st.kv, drop)
    far, bound = (out.double() - ref).abs(), R.attention_bound(ref, *scale, True)
    assert torch.all(far <= bound), float((far / bound).max())


def test_attention_q8_few_rows_rising_scores():
    # every later key scores higher than all before: each quarter's maximum moves with every tile
    st = R.Setup(8, 1, 128, 16, [2000], [3], q8=True, seed=28)
    codes, scales = st.planes()
    pos = torch.arange(2000, device="cuda")
    page, off = st.bt[0, pos // 16].long(), pos % 16
    codes[page, 0, 0, off] = 0
    codes[page, 0, 0, off, 0] = 100
    scales[page, 0, 0, off, 0] = (pos * 0.0008).to(torch.float16)
    q = st.normal(3, 8, 128)
    q[..., 0] = 4.0
    check_attention(st, q=q)


@pytest.mark.parametrize("q8", [False, True])
def test_attention_queries_of_any_magnitude(q8):
    # rows scaled by powers of two from 2^-100 to 2^100 against keys scaled the other way
    st = R.Setup(8, 2, 128, 16, [200], [60], q8=q8, seed=20)
    if q8:
        q = st.normal(60, 8, 128)
        e = torch.arange(60, device="cuda") * 3.0 - 100
        q = (q.float() * torch.exp2(e.clamp(max=4.0))[:, None, None]).to(torch.bfloat16)
    else:
        st.kv[:, 0] = (st.kv[:, 0].float() * 2.0 ** -60).to(torch.bfloat16)
        q = (st.normal(60, 8, 128).float() * 2.0 ** 60).to(torch.bfloat16)
    check_attention(st, q=q)


def test_attention_pool_beyond_32_bit_offsets():
    # a 5 GB layer whose used pages lie at its end
    ps, hkv, d = 128, 8, 128
    P = 5 * (1 << 30) // (2 * hkv * ps * d * 2)
    st = R.Setup(16, hkv, d, ps, [300], [40], seed=16)
    big = torch.empty(P, 2, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    n = st.kv.shape[0]
    big[P - n:] = st.kv
    bt = torch.where(st.bt >= 0, st.bt + (P - n), st.bt)
    sh = mk.CacheShape(16, hkv, d, ps, P, st.maxpg)
    q = st.normal(40, 16, d)
    assert torch.equal(mk.chunk_attention(sh, q, [40], [300], bt, big),
                       mk.chunk_attention(st.shape(mk), q, [40], [300], st.bt, st.kv))
    k, v = mk.read_cache(sh, [300], [300], bt, big)
    k2, v2 = mk.read_cache(st.shape(mk), [300], [300], st.bt, st.kv)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    qkv = st.normal(40, (16 + 2 * hkv) * d)
    mk.append_chunk(sh, qkv, [40], [300], bt, big)
    mk.append_chunk(st.shape(mk), qkv, [40], [300], st.bt, st.kv)
    assert torch.equal(bits(big[P - n:]), bits(st.kv))


# ---------------------------------------------------------------- streams, graphs, repeats
@pytest.mark.parametrize("q8", [False, True])
def test_repeats_are_bit_identical_on_any_stream_and_in_graphs(q8):
    st = R.Setup(16, 2, 128, 16, [4000, 70, 333], [1, 70, 40], q8=q8, seed=17)
    width = (16 + 4) * 128
    qkv = st.normal(st.rows, width)
    rope = mk.Rope(mk.rope_frequencies(128, 1e4))
    sh = st.shape(mk)

    def layer(kv, stream=None):
        q = mk.append_chunk(sh, qkv, st.news, st.lens, st.bt, kv, rope=rope, stream=stream)
        o = mk.chunk_attention(sh, q, st.news, st.lens, st.bt, kv, stream=stream)
        return q, o, *mk.read_cache(sh, st.news, st.lens, st.bt, kv, stream=stream)

    kv0 = st.kv.clone()
    first = layer(st.kv)
    again = layer(st.kv)                     # appending the same rows again changes nothing
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv2 = kv0.clone()
    side.wait_stream(torch.cuda.current_stream())
    other = layer(kv2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    kv3 = kv0.clone()
    graphs, outs = [], []
    for _ in range(2):                       # two graphs over the same inputs, replayed at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(kv3))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for r in (again, other, *outs):
        for a, b in zip(first, r):
            assert torch.equal(bits(a), bits(b))
    assert torch.equal(bits(st.kv), bits(kv2)) and torch.equal(bits(st.kv), bits(kv3))


def test_calls_of_several_threads():
    # each thread on a stream of its own, over its own cache type and rows, again and again: the first answers
    import threading
    cases = [R.Setup(8, 2, 128, 16, [3000, 129], [1, 1], q8=True, seed=30), R.Setup(8, 2, 128, 16, [3000, 129], [1, 1], seed=31),
             R.Setup(8, 2, 128, 16, [700, 5], [300, 5], q8=True, seed=32), R.Setup(4, 2, 64, 16, [700, 5], [300, 5], seed=33)]
    args = [(st.shape(mk), st.normal(st.rows, st.hq, st.d), st.news, st.lens, st.bt, st.kv) for st in cases]
    want = [mk.chunk_attention(*a) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        outs = [mk.chunk_attention(*args[i], stream=stream) for _ in range(20)]
        stream.synchronize()
        wrong.extend(i for o in outs if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_no_rows_and_reused_outputs():
    st = R.Setup(8, 2, 128, 16, [40, 5], [0, 0], seed=22)
    status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert mk.chunk_attention(st.shape(mk), q, [0, 0], st.lens, st.bt, st.kv, out=out, status=status) is out
    assert int(status) == mk.MK_OK and torch.all(out == 7.0)
    assert mk.append_chunk(st.shape(mk), q.new_empty(0, 12 * 128), [0, 0], st.lens, st.bt, st.kv).shape == (0, 8, 128)
    k, v = mk.read_cache(st.shape(mk), [0, 0], st.lens, st.bt, st.kv)
    assert k.shape == v.shape == (0, 2, 128)


def test_binding_refuses_wrong_tensors():
    st = R.Setup(8, 2, 128, 16, [40, 5], [4, 5], seed=23)
    sh, q = st.shape(mk), st.normal(9, 8, 128)
    ok = dict(q=q, chunk_lens=st.news, seq_lens=st.lens, block_tables=st.bt, kv_layer=st.kv)
    mk.chunk_attention(sh, **ok)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(q=q[:8]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q.transpose(1, 2)), dict(q=q[:, :7]),
                dict(block_tables=st.bt.long()), dict(block_tables=st.bt[:, :-1]), dict(block_tables=st.bt[:1]),
                dict(block_tables=st.bt.cpu()), dict(kv_layer=st.kv[1:]), dict(kv_layer=st.kv.half()),
                dict(chunk_lens=[4]), dict(chunk_lens=[4, 6]), dict(seq_lens=[3, 5]), dict(chunk_lens=[-1, 5]),
                dict(out=torch.empty(8, 8, 128, dtype=torch.bfloat16, device="cuda")),
                dict(out=torch.empty(9, 8, 128, device="cuda")), dict(status=torch.zeros(1, device="cuda")),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(workspace=ws.cpu())):
        with pytest.raises(mk.MkError) as e:
            mk.chunk_attention(sh, **{**ok, **bad})
        assert e.value.code == mk.MK_ERR_INVALID_ARG, bad
    big = R.Setup(8, 2, 128, 16, [20000], [1], seed=24)
    need = mk.chunk_attention_workspace(big.shape(mk), [1], [20000])
    assert need > 16
    with pytest.raises(mk.MkError) as e:    # too small a workspace
        mk.chunk_attention(big.shape(mk), big.normal(1, 8, 128), [1], [20000], big.bt, big.kv, workspace=ws)
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    with pytest.raises(mk.MkError):
        mk.append_chunk(sh, st.normal(9, 12 * 128), st.news, st.lens, st.bt, st.kv, q_norm=st.normal(64))


def test_splitting_a_prompt_gives_the_same_cache_and_close_rows():
    # a prompt in one call, and in slices with another sequence's tokens between
    st = R.Setup(8, 2, 128, 16, [300, 9], [300, 9], seed=18)
    sh = st.shape(mk)
    qkv = st.normal(309, 12 * 128)
    rope = mk.Rope(mk.rope_frequencies(128, 1e4))
    kv1, kv2 = st.kv.clone(), st.kv.clone()
    q1 = mk.append_chunk(sh, qkv, [300, 9], [300, 9], st.bt, kv1, rope=rope)
    o1 = mk.chunk_attention(sh, q1, [300, 9], [300, 9], st.bt, kv1)
    got = []
    for a, b, n2, l2 in ((0, 129, 0, 0), (129, 130, 9, 9), (130, 300, 0, 9)):
        rows = torch.cat([qkv[a:b], qkv[300:300 + n2]])
        q2 = mk.append_chunk(sh, rows, [b - a, n2], [b, l2], st.bt, kv2, rope=rope)
        got.append((mk.chunk_attention(sh, q2, [b - a, n2], [b, l2], st.bt, kv2), b - a))
    assert torch.equal(bits(kv1), bits(kv2))
    o2 = torch.cat([o[:n] for o, n in got] + [got[1][0][1:]])
    st.kv = kv1
    ref, *scale = R.attention(st, q1, kv1)
    bound = R.attention_bound(ref, *scale, False)
    assert torch.all((o1.double() - ref).abs() <= bound) and torch.all((o2.double() - ref).abs() <= bound)


# ---------------------------------------------------------------- together with the decode step
@pytest.mark.parametrize("q8", [False, True])
def test_prefill_then_decode_step(q8):
    """A prompt goes through every layer with the chunk operators (the products in between are plain
    torch in fp32), then mk_decode_step decodes the next token from the cache they left: its logits
    against the oracle's, which prefilled token by token."""
    from oracle import Oracle
    from tests.gpu_common import MEDIUM, check_rows, engine_for, gpu_step, to_device
    from tests.helpers import tiny_setup
    lens = [90, 33]
    s = tiny_setup(MEDIUM, lens, kv_q8=q8)
    m = s["model"]
    w = to_device(s["wt"])
    ps, P = s["page_size"], s["num_pages"]
    flags = mk.FLAG_KV_Q8 if q8 else 0
    sh = mk.cache_shape(m, ps, P, s["max_pages"], flags)
    kv = (torch.zeros(m["layers"], W.kv_q8_layer_bytes(m, P, ps), dtype=torch.uint8, device="cuda") if q8 else
          torch.zeros(W.kv_shape(m, P, ps), dtype=torch.bfloat16, device="cuda"))
    bt = torch.from_numpy(s["bt"]).cuda()
    news = [ln - 1 for ln in lens]
    tokens = torch.from_numpy(np.concatenate([s["seqs"][b][:news[b]] for b in range(2)])).cuda().long()
    rope = mk.Rope(mk.rope_frequencies(m["head_dim"], m["rope_theta"]))

    def norm(x, g):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + m["rms_eps"]) * g.float()

    x = w["embed"][tokens].float()
    for l, lw in enumerate(w["layers"]):
        qkv = (norm(x, lw["attn_norm"]) @ lw["w_qkv"].float().T).to(torch.bfloat16)
        q = mk.append_chunk(sh, qkv, news, news, bt, kv[l], rope=rope)
        o = mk.chunk_attention(sh, q, news, news, bt, kv[l])
        x = x + o.flatten(1).float() @ lw["w_o"].float().T
        y = norm(x, lw["ffn_norm"])
        top, ids = torch.softmax(y @ lw["w_router"].float().T, -1).topk(m["top_k"])
        top = top / top.sum(-1, keepdim=True)
        for k in range(m["top_k"]):
            gu = torch.einsum("th,tfh->tf", y, lw["w_gate_up"][ids[:, k]].float())
            act = torch.nn.functional.silu(gu[:, :m["ffn"]]) * gu[:, m["ffn"]:]
            x = x + top[:, k:k + 1] * torch.einsum("tf,thf->th", act, lw["w_down"][ids[:, k]].float())
    eng = engine_for(s, w, flags=flags)
    got = gpu_step(eng, s["tokens"], s["seq_lens"], s["bt"], kv)
    ref = Oracle("f32").decode_step(s["dims"], s["wn"], s["tokens"], s["seq_lens"], s["bt"], s["kv"].copy())
    # bf16 q, k, v rows and attention outputs where the oracle keeps fp32: 2^-9 each on average, over
    # three layers; the bound of the step's own parity tests holds
    errs = check_rows(got, ref)
    print("prefill + step: rel L2", errs)
    eng.close()


# ---------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("rot,norm", [(0, False), (128, False), (128, True)])
def test_append_keeps_what_is_not_finite(rot, norm, value, q8):
    # one value of one row's k, of another's v and of a third's q: no cached block of 32 (bf16: no value) that it
    # is part of reads back as finite, and every other is what it is without it
    st = R.Setup(4, 2, 128, 16, [70], [70], q8=q8, seed=34)
    qkv, rope, _, gains = append_case(st, rot, False, norm)
    sh = st.shape(mk)
    args = dict(rope=rope, q_norm=gains[0], k_norm=gains[1])
    q1 = mk.append_chunk(sh, qkv, [70], [70], st.bt, st.kv, **args)
    k1, v1 = mk.read_cache(sh, [70], [70], st.bt, st.kv)
    bad = qkv.clone()
    bad[3, (4 + 1) * 128 + 37] = float(value)        # k head 1 of row 3
    bad[20, (4 + 2) * 128 + 100] = float(value)      # v head 0 of row 20
    bad[41, 2 * 128 + 64] = float(value)             # q head 2 of row 41
    q2 = mk.append_chunk(sh, bad, [70], [70], st.bt, st.kv, **args)
    k2, v2 = mk.read_cache(sh, [70], [70], st.bt, st.kv)
    # dims that the value reaches: itself, with a rotation its pair, with a norm the head (an infinity: its own
    # dim, inf * 0, and for the others x * 0)
    reach = {37, 101} if rot else {37}
    if norm:
        reach = set(range(128)) if value == "nan" else reach
    kblocks = sorted({d // 32 for d in reach})
    hit = torch.zeros_like(k1, dtype=torch.bool)
    for d in reach:
        hit[3, 1, d] = True
    if q8:
        for b in kblocks:
            hit[3, 1, 32 * b:32 * b + 32] = True
    assert not torch.isfinite(k2[hit]).any()
    if value == "nan" or q8:
        assert torch.isnan(k2[hit]).any()
    same = ~hit
    if norm:
        same[3, 1] = False                            # (the norm's sum is the head's)
    assert torch.equal(bits(k2)[same], bits(k1)[same])
    hit = torch.zeros_like(v1, dtype=torch.bool)
    hit[20, 0, 96:128 if q8 else 101] = True
    if not q8:
        hit[20, 0, 96:100] = False
    assert not torch.isfinite(v2[hit]).any() and torch.equal(bits(v2)[~hit], bits(v1)[~hit])
    assert not torch.isfinite(q2[41, 2, 64])
    rows = torch.arange(70, device="cuda") != 41
    assert torch.equal(bits(q2)[rows], bits(q1)[rows])


SCORE_SHAPES = [(8, 1, 90, 90), (8, 1, 300, 3), (16, 2, 5000, 2), (8, 1, 9000, 40), (4, 1, 700, 700)]


@pytest.mark.parametrize("hq,hkv,len_,new", SCORE_SHAPES)
def test_attention_rows_whose_scores_are_all_minus_infinity(hq, hkv, len_, new):
    # exp(-inf) / 0: a NaN, as softmax has it; zeros are what a row without a position gets.  Query heads of the
    # other sign see scores of +inf, a NaN too; a second sequence is as it was
    st = R.Setup(hq, hkv, 128, 16, [len_, 50], [new, 9], seed=35)
    pos = torch.arange(len_, device="cuda")
    page, off = st.bt[0, pos // 16].long(), pos % 16
    q = st.normal(st.rows, hq, 128)
    q[..., 0] = torch.where(torch.arange(hq, device="cuda") % 2 == 0, 1.0, -1.0).to(torch.bfloat16)
    ref, *scale = R.attention(st, q, st.kv)
    st.kv[page, 0, :, off, 0] = float("-inf")
    out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
    assert torch.isnan(out[:new]).all()
    assert torch.all((out[new:].double() - ref[new:]).abs() <= R.attention_bound(ref, *scale, False)[new:])


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hq,hkv,len_,new", SCORE_SHAPES)
def test_attention_q8_scores_beyond_fp32(hq, hkv, len_, new, sign):
    # every score of a row is beyond what fp32 holds although its key and its query row are well within fp16 and
    # bf16: NaN, not zeros
    st = R.Setup(hq, hkv, 128, 16, [len_, 50], [new, 9], q8=True, seed=36)
    pos = torch.arange(len_, device="cuda")
    page, off = st.bt[0, pos // 16].long(), pos % 16
    codes, scales = st.planes()
    q = st.normal(st.rows, hq, 128)
    ref, *scale = R.attention(st, q, st.kv)
    codes[page, 0, :, off] = 0
    codes[page, 0, :, off, 0] = 127 * sign
    scales[page, 0, :, off, 0] = 500.0
    q[:new, :, 0] = 2.0 ** 120
    out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv)
    assert torch.isnan(out[:new]).all()
    assert torch.all((out[new:].double() - ref[new:]).abs() <= R.attention_bound(ref, *scale, True)[new:])


@pytest.mark.parametrize("len_,new", [(40, 1), (40, 9), (300, 200), (6000, 2)])
def test_attention_q8_code_minus_128(len_, new):
    # the one code that the quantizer does not make, under scales whose 127-fold fp16 still holds and whose 128-fold
    # it does not: keys that a query row meets with a small value, so that the score is an ordinary one
    st = R.Setup(8, 1, 128, 16, [len_], [new], q8=True, seed=37)
    codes, scales = st.planes()
    for p, sc in ((3, 514.0), (len_ // 2, 515.0), (len_ - new, 512.0), (len_ // 3, 511.5)):
        page = st.bt[0, p // 16].long()
        codes[page, :, :, p % 16, :32] = 0
        codes[page, 0, :, p % 16, 7] = -128
        scales[page, 0, :, p % 16, 0] = sc
    q = st.normal(new, 8, 128, std=0.1)
    q[..., :32] = 0
    q[..., 7] = 2.0 ** -14
    check_attention(st, q=q)


def test_attention_a_poisoned_prompt_ends_soon():
    # a NaN in an early key is every row's: each is worked out again only as far as that key.  (To the end it would be
    # about a thousand times the prompt's time; a hundred times leave room for any clock.)
    st = R.Setup(16, 2, 128, 16, [4096], [4096], seed=38)
    q = st.normal(st.rows, 16, 128)
    out = torch.empty_like(q)

    def took():
        best = None
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, out=out)
            b.record()
            b.synchronize()
            best = a.elapsed_time(b) if best is None else min(best, a.elapsed_time(b))
        return best

    clean = took()
    st.kv[st.bt[0, 0].long(), 0, :, 1, 9] = float("nan")
    poisoned = took()
    print("prompt of 4096:", clean, "ms, poisoned", poisoned, "ms")
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()
    assert poisoned < 100 * clean


def test_attention_output_beside_strided_query_rows():
    # an output that lies between the rows of q is no overlap; one that shares a value with a row is refused
    st = R.Setup(2, 1, 128, 16, [20], [3], seed=39)
    buf = st.normal(3, 8 * 256)
    q = buf[:, :256].unflatten(1, (2, 128))
    ref, *scale = R.attention(st, q, st.kv)
    flat = buf.flatten()
    out = flat[256:256 + 3 * 256].view(3, 2, 128)       # in the gap behind row 0
    assert mk.chunk_attention(st.shape(mk), q, [3], [20], st.bt, st.kv, out=out) is out
    assert torch.all((out.double() - ref).abs() <= R.attention_bound(ref, *scale, False))
    before = flat.clone()
    for at in (0, 8, 256 - 8, 8 * 256 - 2 * 256, 7 * 256 + 8, 16 * 256 + 248):
        with pytest.raises(mk.MkError) as e:
            mk.chunk_attention(st.shape(mk), q, [3], [20], st.bt, st.kv, out=flat[at:at + 768].view(3, 2, 128))
        assert e.value.code == mk.MK_ERR_INVALID_ARG and "overlap" in str(e.value)
    assert torch.equal(bits(flat), bits(before))


# ---------------------------------------------------------------- blocks that run several segments
def ragged(n, top, choices, seed=2):
    g = np.random.default_rng(seed)
    lens = [int(x) for x in np.exp(g.uniform(np.log(20), np.log(top), n))]
    return lens, [min(ln, int(g.choice(choices))) for ln in lens]


MIXED, FEW = ragged(64, 900, [1, 1, 3, 40, 140, 300]), ragged(64, 900, [1, 2, 3])
STAGED = [300, 700, 513, 260, 900, 170, 400, 333, 220, 640], [200, 300, 170, 260, 180, 170, 210, 190, 220, 300]
SEGMENTS = {
    # name: hq, hkv, d, ps, q8, lens, news, launch, ranged, segments a block, pairs of (one or two tiles) in a row
    "whole d128": (16, 8, 128, 16, False, *MIXED, 0, False, 5, {"11", "12", "21", "22"}),
    "whole d64": (16, 8, 64, 24, False, *MIXED, 0, False, 5, {"11", "12", "21", "22"}),
    "whole q8": (16, 8, 128, 16, True, *MIXED, 0, False, 5, {"11", "12", "21", "22"}),
    "ranged d128": (8, 4, 128, 24, False, [9000] + MIXED[0][:40], [200] + MIXED[1][:40], 0, True, 4, {"11", "12", "21", "22"}),
    "ranged d64": (8, 4, 64, 16, False, [9000] + MIXED[0][:40], [200] + MIXED[1][:40], 0, True, 4, {"11", "12", "21", "22"}),
    "ranged q8": (8, 4, 128, 24, True, [9000] + MIXED[0][:40], [200] + MIXED[1][:40], 0, True, 4, {"11", "12", "21", "22"}),
    "whole few rows": (64, 8, 128, 16, True, *FEW, 0, False, 4, {"11"}),
    "ranged few rows": (64, 8, 128, 24, True, [6000] + FEW[0][:63], [3] + FEW[1][:63], 0, True, 5, {"11"}),
    "whole staged": (64, 8, 128, 16, True, *STAGED, 1, False, 4, {"11", "12", "21", "22"}),
    "ranged staged": (32, 4, 128, 16, True, [12000] + STAGED[0][:8], [170] + STAGED[1][:8], 1, True, 4, {"11", "12", "21", "22"}),
}


@pytest.mark.parametrize("name", SEGMENTS)
def test_attention_blocks_of_several_segments(name):
    # a persistent block's later segments: query tiles used again, phases and rings carried on, rows converted under
    # the segment before, tails of V that are not the block's first, units of one tile behind units of two
    hq, hkv, d, ps, q8, lens, news, launch, ranged, most, pairs = SEGMENTS[name]
    st = R.Setup(hq, hkv, d, ps, lens, news, q8=q8, seed=40)
    seg = mk.plan_chunk_attention(st.shape(mk), news, lens)
    assert set(seg[:, 0].tolist()) == {launch} and bool((seg[:, 8] >= 0).any()) == ranged
    TT = 128 // (hq // hkv)
    assert (max(min(n, 2 * TT) for n in news) * (hq // hkv) <= 32) == ("few" in name)
    count, seen, tails = {}, set(), 0
    for a, b in zip(seg[:-1].tolist(), seg[1:].tolist()):
        count[b[1]] = count.get(b[1], 1) + 1 if a[1] == b[1] else 1
        if a[1] == b[1]:
            seen.add("".join("12"[news[x[2]] - x[3] * 2 * TT > TT] for x in (a, b)))
            tails += (b[5] + b[6]) * 128 > lens[b[2]]
    assert max(count.values()) >= most and seen == pairs and tails >= 20
    q, out = check_attention(st, extra_rows=1)
    # the same with one sequence poisoned: its rows are worked out again between the block's segments
    s = int(np.argmax(news))
    page = st.bt[s, 0].long()
    (st.planes()[1] if q8 else st.kv)[page, 0, :, 0] = float("nan")
    got = mk.chunk_attention(st.shape(mk), q, news, lens, st.bt, st.kv)
    at = sum(news[:s])
    assert torch.isnan(got[at:at + news[s]]).all()
    keep = torch.ones(st.rows, dtype=torch.bool, device="cuda")
    keep[at:at + news[s]] = False
    assert torch.equal(bits(got[:st.rows])[keep], bits(out[:st.rows])[keep])


def test_calls_of_several_threads_are_right():
    # every thread's calls end, report no error and give the first answers, which are the reference's
    from concurrent.futures import ThreadPoolExecutor
    cases = [R.Setup(8, 2, 128, 16, [3000, 129], [1, 1], q8=True, seed=30), R.Setup(8, 2, 128, 16, [3000, 129], [1, 1], seed=31),
             R.Setup(8, 2, 128, 16, [700, 5], [300, 5], q8=True, seed=32), R.Setup(4, 2, 64, 16, [700, 5], [300, 5], seed=33)]
    checked = [check_attention(st) for st in cases]
    torch.cuda.synchronize()

    def work(i):
        st, (q, want) = cases[i], checked[i]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            status = torch.full((1,), -99, dtype=torch.int32, device="cuda")
        done = 0
        for _ in range(20):
            out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, st.bt, st.kv, status=status, stream=stream)
            stream.synchronize()
            assert int(status) == mk.MK_OK and torch.equal(out, want)
            done += 1
        return done

    with ThreadPoolExecutor(4) as pool:
        assert [f.result() for f in [pool.submit(work, i) for i in range(4)]] == [20] * 4


def test_attention_q8_single_tokens_beside_a_few_rows_more():
    # one sequence of 40 rows among single tokens: the launch takes the general form for all of them
    lens, news = [700, 129, 33, 1, 260, 400, 2000, 6], [1, 1, 1, 1, 5, 1, 1, 1]
    check_attention(R.Setup(16, 2, 128, 16, lens, news, q8=True, seed=41))


# ---------------------------------------------------------------- at the limits
@pytest.mark.parametrize("hq,hkv,d,q8", [(1024, 1024, 64, False), (1024, 128, 128, False), (1024, 128, 128, True),
                                         (1024, 1024, 128, True)])
def test_most_heads(hq, hkv, d, q8):
    st = R.Setup(hq, hkv, d, 8, [130, 3], [2, 3], q8=q8, seed=42)
    check_append(st, d, False, True)
    check_attention(st)
    k, v = mk.read_cache(st.shape(mk), st.lens, st.lens, st.bt, st.kv)
    want = torch.cat([st.cached(st.kv, s, ln) for s, ln in enumerate(st.lens)], 2).transpose(1, 2).float().to(torch.bfloat16)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("ps", [4096, 1000, 136])
def test_large_and_odd_pages(ps, q8):
    st = R.Setup(8, 2, 128, ps, [4500, 70, 1001], [3, 70, 170], q8=q8, seed=43)
    check_append(st, 128, True, False)
    check_attention(st)


@pytest.mark.parametrize("q8", [False, True])
def test_sequences_that_share_pages(q8):
    # a common prefix lies in the pool once; one sequence is listed twice
    st = R.Setup(8, 2, 128, 16, [500, 400, 500], [40, 7, 40], q8=q8, seed=44)
    st.bt[1, :20] = st.bt[0, :20]
    st.bt[2] = st.bt[0]
    q = st.normal(st.rows, 8, 128)
    q[47:] = q[:40]
    _, out = check_attention(st, q=q)
    assert torch.equal(out[:40], out[47:])
    k, v = mk.read_cache(st.shape(mk), st.lens, st.lens, st.bt, st.kv)
    assert torch.equal(k[:320], k[500:820]) and torch.equal(v[:500], v[900:])


@pytest.mark.parametrize("q8", [False, True])
def test_graph_follows_its_block_tables(q8):
    # a replay reads the tables and the cache as they are then; lengths are the capture's
    st = R.Setup(8, 2, 128, 16, [900, 40], [1, 40], q8=q8, seed=45)
    q = st.normal(st.rows, 8, 128)
    bt, kv = st.bt.clone(), st.kv.clone()
    mk.chunk_attention(st.shape(mk), q, st.news, st.lens, bt, kv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mk.chunk_attention(st.shape(mk), q, st.news, st.lens, bt, kv)
    other = R.Setup(8, 2, 128, 16, [900, 40], [1, 40], q8=q8, seed=46)
    bt.copy_(other.bt)
    kv.copy_(other.kv)
    g.replay()
    ref, *scale = R.attention(other, q, other.kv)
    assert torch.all((out.double() - ref).abs() <= R.attention_bound(ref, *scale, q8))
