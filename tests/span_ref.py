"""Attention over parts of the cache in 64 bits: a window with first positions that stay visible, and caches whose
sequences share their first pages.  Beside tests/chunk_ref.py, whose setups and error bounds it takes."""
from __future__ import annotations

import math

import torch

from tests import chunk_ref as R


def attention(st: R.Setup, q, kv, window=None, sinks=0, drop=None):
    """As ``chunk_ref.attention``, of rows that see the ``window`` positions which end with their own (None: all up to
    it) and the first ``sinks``; only pages that hold a visible position are looked at."""
    out = torch.zeros(st.rows, st.hq, st.d, dtype=torch.float64, device=q.device)
    weight, total = torch.zeros_like(out), torch.zeros_like(out)
    shift = torch.zeros(st.rows, st.hq, 1, dtype=torch.float64, device=q.device)
    G, at = st.hq // st.hkv, 0
    for s, (ln, n) in enumerate(zip(st.lens, st.news)):
        if n == 0:
            continue
        row, pos = torch.arange(ln - n, ln, device=q.device)[:, None], torch.arange(ln, device=q.device)[None, :]
        seen = pos <= row
        if window is not None:
            seen &= (pos > row - window) | (pos < sinks)
        if drop is not None:
            seen &= ~drop[s, :ln][None, :]
        used = seen.any(0)
        k, v = cached(st, kv, s, used)
        seen = seen[:, used]
        for h in range(st.hq):
            x, kk, vv = q[at:at + n, h].double(), k[h // G], v[h // G]
            w = (x @ kk.T / math.sqrt(st.d)).masked_fill(~seen, -math.inf)
            p = torch.softmax(w, -1).nan_to_num(0.0)   # a row without a position: zeros
            out[at:at + n, h] = p @ vv
            weight[at:at + n, h] = p @ vv.abs()
            total[at:at + n, h] = seen.double() @ vv.abs()
            if kk.shape[0]:
                shift[at:at + n, h, 0] = (x.abs() @ kk.abs().T / math.sqrt(st.d)).masked_fill(~seen, 0).amax(-1)
        at += n
    return out, weight, shift, total


def cached(st, kv, s, used):
    """K and V of the positions that ``used`` marks, each [Hkv][n][D] in 64 bits."""
    pos = used.nonzero()[:, 0]
    page, off = st.bt[s, pos // st.ps].long(), pos % st.ps
    if st.q8:
        codes, scales = st.planes(kv)
        x = codes[page, :, :, off].double() * scales[page, :, :, off].double().repeat_interleave(32, -1)
    else:
        x = kv[page, :, :, off].double()
    return x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1)


def share(st: R.Setup, group_seqs, prefix_lens):
    """Makes the sequences of each group share the pages that lie within their first ``prefix_len`` positions: all take
    the first one's, and the others' own ones hold what no sequence owns."""
    s = 0
    for size, shared in zip(group_seqs, prefix_lens):
        n = shared // st.ps
        for i in range(s + 1, s + size):
            given = st.bt[i, :n].clone().long()
            st.bt[i, :n] = st.bt[s, :n]
            poison(st, given)
        s += size


def poison(st, pages):
    if st.q8:
        codes, scales = st.planes()
        codes[pages] = -1
        scales.view(torch.int16)[pages] = -1
    else:
        st.kv[pages] = math.nan
