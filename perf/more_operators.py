"""Measured cases of attention over parts of the paged KV cache.

Two operators beside ``chunk_attention`` of ``persistent_moe_decode_megakernel_gb300``, over the same
pages, block tables and packed rows (a ragged batch of prompts, slices of prompts and single tokens):

* ``window``: a row at position p sees the ``window`` positions that end with its own, and the first
  ``sinks`` positions of its sequence, which stay visible;
* ``prefix``: causal attention of sequences that share their first positions in groups, whose block
  tables name the same pages there: a shared position is read for all rows of its group together.

``own`` selects the framework's kernels; otherwise ``run`` computes the plain form in torch.
A case: ``op``; ``hq``, ``hkv``, ``d`` heads; ``ps`` page size; ``q8`` cache type; ``seqs`` sequences;
``len_lo``/``len_hi`` the range of their lengths (prefix: of what lies behind the shared positions;
log-uniform); ``chunk`` new tokens per sequence (at most that length); ``wide`` of the sequences bring
``chunk`` new tokens, the others one; window also ``window`` and ``sinks``; prefix also ``groups`` of
about as many sequences each and ``pre_lo``/``pre_hi``, the range of their shared lengths.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False


def _case(name, op, hq=32, hkv=4, d=128, ps=16, q8=False, seqs=1, len_lo=1, len_hi=1, chunk=1, wide=1, **more):
    c = dict(op=op, hq=hq, hkv=hkv, d=d, ps=ps, q8=q8, seqs=seqs, len_lo=len_lo, len_hi=len_hi, chunk=chunk, wide=wide, **more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest call: a short prompt of the tiny model (4 query heads of 64 over 2 KV heads)
        _case("window_tiny_prompt", "window", 4, 2, 64, len_lo=65, len_hi=65, chunk=65, window=16, sinks=2),
        # a whole prompt into an empty cache, the 30B shape's heads, in a layer of short sight
        _case("window_prompt_8k", "window", len_lo=8192, len_hi=8192, chunk=8192, window=1024, sinks=4),
        # a slice of a long prompt in a layer of longer sight (chunked prefill)
        _case("window_chunk_2k_of_32k", "window", ps=64, len_lo=32768, len_hi=32768, chunk=2048, window=4096, sinks=4),
        # a continuous batch: most rows decode one token, four bring an odd slice of a prompt; no sinks
        _case("window_mixed_64", "window", seqs=64, len_lo=512, len_hi=32768, chunk=509, wide=4, window=1023, sinks=0),
        # a batch that decodes: only the visible positions' bytes count; heads of 64
        _case("window_tokens_64_d64", "window", 16, 4, 64, seqs=64, len_lo=2048, len_hi=65536, window=4096, sinks=4),
        # the two ends over the quantised cache
        _case("window_q8_chunk_1k_of_16k", "window", q8=True, len_lo=16384, len_hi=16384, chunk=1024, window=2048, sinks=4),
        _case("window_q8_tokens_16", "window", ps=64, q8=True, seqs=16, len_lo=16384, len_hi=131072, window=8192, sinks=16),
        # a few requests behind a short common instruction
        _case("prefix_tiny_8", "prefix", 4, 2, 64, seqs=8, len_lo=1, len_hi=40, groups=1, pre_lo=200, pre_hi=200),
        # a batch that decodes behind one long document
        _case("prefix_tokens_64_of_32k", "prefix", ps=64, seqs=64, len_lo=64, len_hi=1024, groups=1, pre_lo=32768, pre_hi=32768),
        # several documents, and five speculative tokens a sequence
        _case("prefix_groups_4", "prefix", seqs=32, len_lo=33, len_hi=700, chunk=5, wide=32, groups=4, pre_lo=1000, pre_hi=12001),
        # a batch that decodes behind a common instruction while two of its sequences still bring their prompts
        _case("prefix_mixed_32", "prefix", seqs=32, len_lo=100, len_hi=2000, chunk=509, wide=2, groups=1, pre_lo=8191, pre_hi=8191),
        # the same over the quantised cache
        _case("prefix_q8_tokens_64_of_32k", "prefix", ps=64, q8=True, seqs=64, len_lo=64, len_hi=1024, groups=1, pre_lo=32768,
              pre_hi=32768),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "prefix"])
    q8 = rng.random() < 0.4
    d = 128 if q8 else rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8])
    ps = rng.choice([8, 16, 16, 24, 32, 40, 64, 64, 128])
    seqs = _log_int(rng, 1, 64)
    chunk_most, wide, more = 8192, _log_int(rng, 1, seqs), {}
    if op == "window":
        len_hi = _log_int(rng, 40, 65536)
        while seqs * len_hi * hkv * d > 1 << 30:         # a pool of 4 GB at most
            len_hi //= 2
        more = dict(window=_log_int(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 4, rng.randint(2, 200)]))
    else:
        len_hi, chunk_most = _log_int(rng, 1, 2048), 600
        pre_hi = _log_int(rng, 8, 32768)
        more = dict(groups=rng.randint(1, 4), pre_lo=rng.choice([pre_hi, _log_int(rng, 1, pre_hi)]), pre_hi=pre_hi)
    len_lo = rng.choice([len_hi, _log_int(rng, 1, len_hi)])
    chunk = _log_int(rng, 1, min(len_hi, chunk_most))
    while True:
        if op == "prefix":
            more["groups"] = min(more["groups"], seqs)
        c = _case(None, op, hkv * g, hkv, d, ps, q8, seqs, len_lo, len_hi, chunk, wide, **more)
        w = work(c)
        if w["flops"] <= 1.37e11 and w["bytes"] <= 2.5e8:   # no more than the largest listed ones
            return c
        if chunk > 1 and wide * 4 <= seqs or wide == 1 and chunk > 1:
            chunk = chunk * 3 // 4
        elif wide > 1 and chunk > 1:
            wide -= 1
        else:
            seqs -= 1
            wide = min(wide, seqs)


# ---------------------------------------------------------------- shapes and inputs
def _spread(lo, hi, n):
    return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i + 0.5) / n))) for i in range(n)]


def _groups(case):
    """(sequences, shared positions) of each group; a window case has none."""
    if case["op"] == "window":
        return [(1, 0)] * case["seqs"]
    n, k = case["seqs"], case["groups"]
    return list(zip([(i + 1) * n // k - i * n // k for i in range(k)], _spread(case["pre_lo"], case["pre_hi"], k)))


def _lengths(case, seed):
    """(lengths with the new tokens, new tokens) of the sequences: the case fixes how much work
    they are together, the seed only which sequence (of a group) has which length."""
    n = case["seqs"]
    lens = _spread(case["len_lo"], case["len_hi"], n)
    news = [min(ln, case["chunk"] if i * case["wide"] // n != (i - 1) * case["wide"] // n or i == 0 else 1)
            for i, ln in enumerate(lens)]
    groups = _groups(case)
    # (lengths rise with i: dealt out so that each group has short and long ones)
    order = sorted(range(n), key=lambda i: i % len(groups)) if case["op"] == "prefix" else list(range(n))
    rng, at, out = random.Random(seed), 0, []
    if case["op"] == "window":
        rng.shuffle(order)
        return [lens[i] for i in order], [news[i] for i in order]
    for size, shared in groups:
        part = order[at:at + size]
        at += size
        rng.shuffle(part)
        out += [(lens[i] + shared, news[i]) for i in part]
    return [ln for ln, _ in out], [n for _, n in out]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    lens, news = _lengths(case, seed)
    groups = _groups(case)
    maxpg = max(-(-ln // ps) for ln in lens)
    first = np.concatenate([[0], np.cumsum([size for size, _ in groups])])
    total = sum(-(-ln // ps) for ln in lens)
    num_pages = total - sum((size - 1) * (shared // ps) for size, shared in groups) + 3
    perm = torch.randperm(num_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    bt = torch.full((len(lens), maxpg), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, (size, shared) in enumerate(groups):
        common = perm[at:at + shared // ps]              # whole pages that the group shares
        at += shared // ps
        for s in range(int(first[i]), int(first[i + 1])):
            n = -(-lens[s] // ps) - shared // ps
            bt[s, :shared // ps] = common
            bt[s, shared // ps:shared // ps + n] = perm[at:at + n]
            at += n
    st = dict(case=case, lens=np.array(lens, dtype=np.int32), news=np.array(news, dtype=np.int32), bt=bt, num_pages=num_pages)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)

    if case["q8"]:
        # decoded values about N(0, 0.76^2): codes round(N(0, 42^2)), scales U(0.012, 0.024)
        n = num_pages * 2 * hkv * ps * d
        codes = normal(n, dtype=torch.float32, scale=42.0).round_().clamp_(-127, 127).to(torch.int8)
        scales = (torch.rand(n // 32, generator=g, device=dev) * 0.012 + 0.012).to(torch.float16)
        st["kv"] = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8)])
    else:
        st["kv"] = normal(num_pages, 2, hkv, ps, d)
    st["q"] = normal(sum(news), hq, d, scale=1.5)
    st["sizes"] = np.array([size for size, _ in groups], dtype=np.int32)
    st["shared"] = np.array([shared for _, shared in groups], dtype=np.int32)
    if own:
        import persistent_moe_decode_megakernel_gb300 as mk
        st["mk"] = mk
        st["shape"] = mk.CacheShape(hq, hkv, d, ps, num_pages, maxpg, mk.FLAG_KV_Q8 if case["q8"] else 0)
    return st


# ---------------------------------------------------------------- the plain form
def _planes(st):
    """(codes [P][2][Hkv][ps][D], scales [P][2][Hkv][ps][D/32]) of a q8_0 cache."""
    c = st["case"]
    shape = (st["num_pages"], 2, c["hkv"], c["ps"])
    n = math.prod(shape) * c["d"]
    return st["kv"][:n].view(torch.int8).view(*shape, c["d"]), st["kv"][n:].view(torch.float16).view(*shape, c["d"] // 32)


def _gather(st, page, off, which):
    """fp32 rows [n][Hkv][D] of K (0) or V (1) at (page, offset) pairs."""
    if st["case"]["q8"]:
        codes, scales = _planes(st)
        return codes[page, which, :, off].float() * scales[page, which, :, off].float().repeat_interleave(32, dim=-1)
    return st["kv"][page, which, :, off].float()


def _plain(st):
    c = st["case"]
    hq, hkv, d, ps = c["hq"], c["hkv"], c["d"], c["ps"]
    g = hq // hkv
    window, sinks = c.get("window", 1 << 30), c.get("sinks", 0)
    out = torch.empty_like(st["q"])
    at = 0
    for s, (ln, n) in enumerate(zip(st["lens"].tolist(), st["news"].tolist())):   # ragged: one sequence at a time
        lo = max(0, ln - n - window + 1)                 # the first position in some row's window
        pos = torch.arange(lo, ln, device=out.device)
        if min(sinks, lo) > 0:
            pos = torch.cat([torch.arange(min(sinks, lo), device=out.device), pos])
        page, off = st["bt"][s, torch.div(pos, ps, rounding_mode="floor")].long(), pos % ps
        k, v = _gather(st, page, off, 0).permute(1, 2, 0), _gather(st, page, off, 1).permute(1, 0, 2)
        q = st["q"][at:at + n].float().view(n, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * n, d)
        w = torch.matmul(q * (1.0 / math.sqrt(d)), k).view(hkv, g, n, pos.numel())
        if n > 1:   # (a single new token sees every position that is gathered)
            mine = torch.arange(ln - n, ln, device=out.device)[:, None]
            w.masked_fill_((pos[None, :] > mine) | ((pos[None, :] <= mine - window) & (pos[None, :] >= sinks)), -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True)).exp_()
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.view(hkv, g * n, pos.numel()), v).view(hkv, g, n, d) / total
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, d).to(torch.bfloat16)
        at += n
    return out


def run(state):
    st, c = state, state["case"]
    if not own:
        return _plain(st)
    args = (st["shape"], st["q"], st["news"], st["lens"], st["bt"], st["kv"])
    if c["op"] == "window":
        return st["mk"].window_attention(*args, c["window"], c["sinks"])
    return st["mk"].prefix_attention(*args, st["sizes"], st["shared"])


# ---------------------------------------------------------------- the work
def work(case):
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    lens, news = _lengths(case, 0)
    per = 2 * hkv * d * (17.0 / 16 if case["q8"] else 2.0)   # cached bytes of one position
    rows = sum(news)
    if case["op"] == "window":
        window, sinks = case["window"], case["sinks"]
        read = seen = 0
        for ln, n in zip(lens, news):
            lo = max(0, ln - n - window + 1)
            read += ln - lo + min(sinks, lo)
            p = np.arange(ln - n, ln, dtype=np.int64)
            below = np.maximum(p - window + 1, 0)            # positions before the window
            seen += int((p + 1 - below + np.minimum(below, sinks)).sum())
    else:
        read, s, seen = 0, 0, 0
        for size, shared in _groups(case):
            common = shared // ps * ps
            read += common + sum(lens[s:s + size]) - size * common
            s += size
        seen = sum(n * (ln - n) + n * (n + 1) // 2 for ln, n in zip(lens, news))
    return {"bytes": 2 * rows * hq * d * 2 + per * read, "flops": 4.0 * d * hq * seen}


# ---------------------------------------------------------------- the definition in 64 bits
def _cached64(st, s, lo, hi):
    """K and V of positions lo..hi-1 of sequence s, [2][Hkv][hi - lo][D] in 64 bits, page by page in order."""
    c = st["case"]
    a = lo // c["ps"]
    page = st["bt"][s, a:-(-hi // c["ps"])].long()
    if c["q8"]:
        codes, scales = _planes(st)
        x = codes[page].double().unflatten(-1, (-1, 32)) * scales[page].double()[..., None]
        x = x.flatten(-2)
    else:
        x = st["kv"][page].double()
    return x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, lo - a * c["ps"]:hi - a * c["ps"]]


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    window, sinks = case.get("window"), case.get("sinks", 0)
    out = torch.empty(sum(st["news"].tolist()), hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for s, (ln, n) in enumerate(zip(st["lens"].tolist(), st["news"].tolist())):
        whole = _cached64(st, s, 0, ln) if window is None else None
        for lo in range(0, n, 512):
            hi = min(n, lo + 512)
            row = torch.arange(ln - n + lo, ln - n + hi, device="cuda")
            end = ln - n + hi                            # no row of this block sees a later position
            if window is None:
                at_pos, kv = torch.arange(end, device="cuda"), whole[:, :, :end]
            else:
                begin = max(0, ln - n + lo - window + 1)
                few = min(sinks, begin)
                at_pos = torch.cat([torch.arange(few, device="cuda"), torch.arange(begin, end, device="cuda")])
                kv = _cached64(st, s, begin, end)
                if few:
                    kv = torch.cat([_cached64(st, s, 0, few), kv], dim=2)
            back = row[:, None] - at_pos[None, :]
            seen = back >= 0
            if window is not None:
                seen &= (back < window) | (at_pos[None, :] < sinks)
            for h in range(hkv):
                q = st["q"][at + lo:at + hi, h * G:(h + 1) * G].double()
                w = torch.einsum("rgd,td->rgt", q, kv[0, h]) / math.sqrt(d)
                w = torch.where(seen[:, None, :], w, -math.inf)
                p = (w - torch.logsumexp(w, -1, keepdim=True)).exp()
                out[at + lo:at + hi, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", p, kv[1, h])
        at += n
    return out
