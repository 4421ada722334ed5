"""The chunk operators' definitions in 64 bits, on torch tensors of any device, and the setups
that their tests share.  Nothing here uses the library's kernels."""
from __future__ import annotations

import math

import torch

import workloads as W


class Setup:
    """A paged cache of one layer with shuffled pages.  Everything that no sequence owns -- spare
    pages and what lies behind a last position -- holds NaN (bf16) or all-ones bits (q8_0, whose
    f16 scale is then a NaN), and a row per spare block-table entry holds -1."""

    def __init__(self, hq, hkv, d, ps, lens, news, q8=False, seed=0, dev="cuda", extra_pages=2, wide_tables=1, std=1.0):
        self.hq, self.hkv, self.d, self.ps, self.q8, self.dev = hq, hkv, d, ps, q8, dev
        self.lens, self.news = list(lens), list(news)
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        self.g = g
        need = [-(-ln // ps) for ln in self.lens]
        self.P = sum(need) + extra_pages
        self.maxpg = max(max(need), 1) + wide_tables
        perm = torch.randperm(self.P, generator=g, device=dev)
        self.bt = torch.full((len(lens), self.maxpg), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, n in enumerate(need):
            self.bt[s, :n] = perm[at:at + n].to(torch.int32)
            at += n
        used = torch.zeros(self.P, ps, dtype=torch.bool, device=dev)
        for s, ln in enumerate(self.lens):
            pos = torch.arange(ln, device=dev)
            used[self.bt[s, pos // ps].long(), pos % ps] = True
        self.used = used
        mask = used[:, None, None, :, None]
        if q8:
            n = self.P * 2 * hkv * ps * d
            self.kv = torch.empty(n + n // 16, dtype=torch.uint8, device=dev)
            codes, scales = self.planes()
            c = (torch.randn(codes.shape, generator=g, device=dev) * 42).round().clamp(-127, 127).to(torch.int8)
            sc = (torch.rand(scales.shape, generator=g, device=dev) * 0.012 + 0.012).to(torch.float16)
            codes.copy_(torch.where(mask, c, torch.full_like(c, -1)))
            scales.view(torch.int16).copy_(torch.where(mask, sc.view(torch.int16), torch.full_like(sc.view(torch.int16), -1)))
        else:
            x = (torch.randn(self.P, 2, hkv, ps, d, generator=g, device=dev) * std).to(torch.bfloat16)
            self.kv = torch.where(mask, x, torch.full_like(x, math.nan))
        self.rows = sum(self.news)

    def shape(self, mk):
        return mk.CacheShape(self.hq, self.hkv, self.d, self.ps, self.P, self.maxpg, mk.FLAG_KV_Q8 if self.q8 else 0)

    def planes(self, kv=None):
        return W.kv_q8_planes(self.kv if kv is None else kv, dict(n_kv=self.hkv, head_dim=self.d), self.P, self.ps)

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.g, device=self.dev) * std).to(torch.bfloat16)

    def positions(self):
        """(sequence, position) of each packed row."""
        seq = torch.repeat_interleave(torch.arange(len(self.news)), torch.tensor(self.news)).to(self.dev)
        pos = torch.cat([torch.arange(ln - n, ln) for ln, n in zip(self.lens, self.news)]).to(self.dev)
        return seq, pos

    def cached(self, kv, s, ln):
        """K and V of positions 0..ln-1 of sequence s, [2][Hkv][ln][D] in 64 bits."""
        page = self.bt[s, :-(-ln // self.ps)].long()
        if self.q8:
            codes, scales = self.planes(kv)
            x = (codes[page].double().unflatten(-1, (-1, 32)) * scales[page].double()[..., None]).flatten(-2)
        else:
            x = kv[page].double()
        return x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :ln]


def rotate(x, pos, inv_freq, interleaved, mscale=1.0):
    """x [rows][heads][D] in 64 bits, rotated."""
    r = 2 * inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.to(pos.device)
    z = torch.polar(torch.full_like(ang, mscale), ang)[:, None]
    first = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    second = first + (1 if interleaved else r // 2)
    y = x.clone()
    w = torch.complex(x[..., first], x[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def head_norm(x, gain, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()


def attention(st: Setup, q, kv, drop=None):
    """(out, weight, shift, total) in 64 bits for query rows q [rows][Hq][D]: the attention output;
    sum_t p_t |v_t|, what a relative error of the weights scales with; the largest
    sum_d |q_d k_td| / sqrt(D) of a row, what a relative error of the keys shifts scores by; and
    sum_t |v_t|, what an absolute error of the weights scales with.
    ``drop``: bool [num_seqs][max length], positions whose page is out of range."""
    out = torch.zeros(st.rows, st.hq, st.d, dtype=torch.float64, device=q.device)
    weight, total, shift = torch.zeros_like(out), torch.zeros_like(out), torch.zeros(st.rows, st.hq, 1, dtype=torch.float64, device=q.device)
    at = 0
    G = st.hq // st.hkv
    for s, (ln, n) in enumerate(zip(st.lens, st.news)):
        if n == 0:
            continue
        k, v = st.cached(kv, s, ln)
        gone = torch.zeros(ln, dtype=torch.bool, device=q.device) if drop is None else drop[s, :ln]
        k, v = torch.where(gone[:, None], 0.0, k), torch.where(gone[:, None], 0.0, v)
        late = torch.arange(ln, device=q.device)[None, :] > torch.arange(ln - n, ln, device=q.device)[:, None]
        hide = late | gone[None, :]
        for h in range(st.hq):
            x = q[at:at + n, h].double()
            kk = k[h // G]
            w = (x @ kk.T / math.sqrt(st.d)).masked_fill(hide, -math.inf)
            p = torch.softmax(w, -1).nan_to_num(0.0)   # a row without a position: zeros
            out[at:at + n, h] = p @ v[h // G]
            weight[at:at + n, h] = p @ v[h // G].abs()
            total[at:at + n, h] = (~hide).double() @ v[h // G].abs()
            shift[at:at + n, h, 0] = (x.abs() @ kk.abs().T / math.sqrt(st.d)).masked_fill(hide, 0).amax(-1)
        at += n
    return out, weight, shift, total


def attention_bound(ref, weight, shift, total, q8):
    """How far a correct kernel may be from the 64-bit attention, value by value.  The output is
    rounded to bf16 (off by at most 2^-8 of it), and so is each softmax weight over a bf16 cache
    (the sum uses the unrounded ones); fp32 scores and sums add less than 2^-12 of the weighted
    values for the lengths tested (D terms of 2^-24 each times a shift below 100).  Over a q8_0
    cache the weights, V and K round to fp16, 2^-11 of each: K moves every score by at most
    ``shift * 2^-11`` and so every normalised weight by a factor within exp(+-2 of that).  (A
    query row's power of two is exact, and what fp16 loses of its values 2^-14 below the row's
    largest is less than 2^-25 of that: 1 % more of the shift covers it.)  Small weights become
    fp16 subnormals, spaced 2^-24 and so off by at most 2^-25 where the largest weight is 2^6 or
    more (weights carry a factor 2^6 and are relative to a reference no larger than the row's
    maximum): 2^-31 of each |v|."""
    h = 2.0 ** -8
    rel = h + 2.0 ** -12
    tiny = total * 2.0 ** -31 if q8 else 0.0
    if q8:
        e = 2.0 ** -11
        rel = 2 * e + 2.0 ** -12 + (2 * 1.01 * shift * e).expm1()
    # an out value is rounded after it is off by the rest
    return (weight * rel + tiny) * (1 + h) + ref.abs() * h + 1e-30
