"""Measured cases of the chunk operators over the paged KV cache.

Three operators, all over the pages, block tables and packed rows that a serving loop keeps
(``persistent_moe_decode_megakernel_gb300``: ``append_chunk``, ``chunk_attention``,
``read_cache``):

* ``append``: the fused QKV rows of a chunk of new tokens -> optional per-head RMSNorm of q and
  k, rotary positions, q rows out, k and v into the cache (bf16, or q8_0 codes and scales);
* ``attend``: causal attention of packed chunks of different lengths over the cached positions,
  grouped heads, bf16 or q8_0 cache;
* ``read``: positions of the cache back as contiguous bf16 rows.

``own`` selects the framework's kernels; otherwise ``run`` computes the plain form in torch.
A case: ``op``; ``hq``, ``hkv``, ``d`` heads; ``ps`` page size; ``q8`` cache type; ``seqs``
sequences; ``len_lo``/``len_hi`` the range of their lengths (log-uniform by seed, ``len_lo`` ==
``len_hi`` fixes them); ``chunk`` new tokens per sequence (at most its length); ``wide`` of the
sequences bring ``chunk`` new tokens, the others one; append also ``rot`` rotary dims,
``inter`` interleaved pairs, ``norm`` per-head norms.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1e4


def _case(name, op, hq=32, hkv=4, d=128, ps=16, q8=False, seqs=1, len_lo=1, len_hi=1, chunk=1, wide=1, rot=128,
          inter=False, norm=False):
    c = dict(op=op, hq=hq, hkv=hkv, d=d, ps=ps, q8=q8, seqs=seqs, len_lo=len_lo, len_hi=len_hi, chunk=chunk, wide=wide)
    if op == "append":
        c.update(rot=rot, inter=inter, norm=norm)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest call: a short prompt of the tiny model (4 query heads of 64 over 2 KV heads)
        _case("attend_tiny_prompt", "attend", 4, 2, 64, len_lo=65, len_hi=65, chunk=65),
        # a whole prompt into an empty cache, the 30B shape's heads
        _case("attend_prompt_8k", "attend", len_lo=8192, len_hi=8192, chunk=8192),
        # a slice of a long prompt over what its earlier slices left (chunked prefill)
        _case("attend_chunk_2k_of_32k", "attend", ps=64, len_lo=32768, len_hi=32768, chunk=2048),
        # a continuous batch: most rows decode one token, four bring an odd slice of a prompt
        _case("attend_mixed_64", "attend", seqs=64, len_lo=512, len_hi=32768, chunk=509, wide=4),
        # one new token over a long context: only the cache's bytes count
        _case("attend_token_of_128k", "attend", ps=64, len_lo=131073, len_hi=131073),
        # the same two ends over the quantised cache
        _case("attend_q8_chunk_1k_of_16k", "attend", q8=True, len_lo=16384, len_hi=16384, chunk=1024),
        _case("attend_q8_token_of_256k", "attend", ps=64, q8=True, len_lo=262145, len_hi=262145),
        # what goes into the cache before each of these
        _case("append_8_tokens", "append", seqs=8, len_lo=1, len_hi=512),
        _case("append_prompt_8k", "append", len_lo=8192, len_hi=8192, chunk=8192),
        _case("append_q8_ragged_norm", "append", q8=True, seqs=16, len_lo=257, len_hi=2048, chunk=257, wide=16, norm=True),
        # a sequence taken out of the pool (moved, or kept for later)
        _case("read_bf16_1k", "read", len_lo=1021, len_hi=1021),
        _case("read_q8_ragged", "read", q8=True, seqs=32, len_lo=512, len_hi=8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "read"])
    q8 = rng.random() < 0.4
    d = 128 if q8 else rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8])
    ps = rng.choice([8, 16, 16, 24, 32, 40, 64, 64, 128])
    seqs = _log_int(rng, 1, 64)
    if op == "attend":
        len_hi = _log_int(rng, 40, 32768)
        len_lo = rng.choice([len_hi, _log_int(rng, 1, len_hi)])
        chunk = _log_int(rng, 1, min(len_hi, 4096))
        wide = _log_int(rng, 1, seqs)
        # no more scores than the largest listed case, nor more cached bytes
        while wide * chunk * len_hi * hkv * g > 32 * 2048 * 32768:
            if wide > 1:
                wide -= 1
            else:
                chunk = max(1, chunk * 3 // 4)
        while seqs * len_hi * hkv * d > 64 * 8192 * 4 * 128 and seqs > wide:
            seqs -= 1
        return _case(None, op, hkv * g, hkv, d, ps, q8, seqs, len_lo, len_hi, chunk, wide)
    budget = 8192 * 32 * 128   # values of q in the largest append
    if op == "append":
        chunk = _log_int(rng, 1, max(1, min(8192, budget // (hkv * g * d))))
        seqs = max(1, min(seqs, budget // (chunk * hkv * g * d)))
        len_hi = chunk + rng.choice([0, _log_int(rng, 1, 16384)])
        rot = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
        return _case(None, op, hkv * g, hkv, d, ps, q8, seqs, rng.randint(1, len_hi), len_hi, chunk, rng.randint(1, seqs),
                     rot, rng.random() < 0.4, rng.random() < 0.5)
    len_hi = _log_int(rng, 3, 16384)
    seqs = max(1, min(seqs, 32 * 4096 * 4 * 128 // (len_hi * hkv * d)))
    return _case(None, op, hkv * g, hkv, d, ps, q8, seqs, rng.randint(1, len_hi), len_hi, 1, seqs)


# ---------------------------------------------------------------- shapes and inputs
def _lengths(case, seed):
    """(lengths with the new tokens, new tokens) of the sequences: the case fixes how much work
    they are together, the seed only which sequence has which length."""
    n, lo, hi = case["seqs"], case["len_lo"], case["len_hi"]
    lens = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i + 0.5) / n))) for i in range(n)]
    news = [min(ln, case["chunk"] if i * case["wide"] // n != (i - 1) * case["wide"] // n or i == 0 else 1)
            for i, ln in enumerate(lens)]
    order = list(range(n))
    random.Random(seed).shuffle(order)
    return [lens[i] for i in order], [news[i] for i in order]


def _pages(case, lens):
    return sum(-(-ln // case["ps"]) for ln in lens)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["ps"]
    lens, news = _lengths(case, seed)
    num_pages = _pages(case, lens) + 3
    maxpg = max(-(-ln // ps) for ln in lens)
    perm = torch.randperm(num_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    bt = torch.full((len(lens), maxpg), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, ln in enumerate(lens):
        n = -(-ln // ps)
        bt[s, :n] = perm[at:at + n]
        at += n
    st = dict(case=case, lens=np.array(lens, dtype=np.int32), bt=bt, num_pages=num_pages)

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
    rows = sum(news)
    if case["op"] != "read":
        st["news"] = np.array(news, dtype=np.int32)
        # sequence and position of each packed row, as a serving loop keeps them
        st["seq"] = torch.from_numpy(np.repeat(np.arange(len(news)), news)).to(dev)
        st["pos"] = torch.from_numpy(np.concatenate([np.arange(ln - n, ln) for ln, n in zip(lens, news)])).to(dev)
    if case["op"] == "attend":
        st["q"] = normal(rows, hq, d, scale=1.5)
    elif case["op"] == "append":
        st["qkv"] = normal(rows, (hq + 2 * hkv) * d, scale=1.3)
        st["freq"] = THETA ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])
        st["freq_dev"] = torch.from_numpy(st["freq"]).to(dev)
        st["q_norm"] = (1 + normal(d, scale=0.1).float()).to(torch.bfloat16) if case["norm"] else None
        st["k_norm"] = (1 + normal(d, scale=0.1).float()).to(torch.bfloat16) if case["norm"] else None
    if own:
        import persistent_moe_decode_megakernel_gb300 as mk
        st["mk"] = mk
        st["shape"] = mk.CacheShape(hq, hkv, d, ps, num_pages, maxpg, mk.FLAG_KV_Q8 if case["q8"] else 0)
        if case["op"] == "append":
            st["rope"] = mk.Rope(st["freq"], interleaved=case["inter"])
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


def _slots(st, seq, pos):
    ps = st["case"]["ps"]
    return st["bt"][seq, torch.div(pos, ps, rounding_mode="floor")].long(), pos % ps


def _read_plain(st, seq, pos):
    page, off = _slots(st, seq, pos)
    return _gather(st, page, off, 0).to(torch.bfloat16), _gather(st, page, off, 1).to(torch.bfloat16)


def _head_norm(x, gain):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()


def _rotate(x, cos, sin, rot, inter):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], dim=-1).flatten(-2) if inter else torch.cat([u, w], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _append_plain(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = st["qkv"].float().view(-1, hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if c["norm"]:
        q, k = _head_norm(q, st["q_norm"]), _head_norm(k, st["k_norm"])
    ang = st["pos"].double()[:, None] * st["freq_dev"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q, k = _rotate(q, cos, sin, c["rot"], c["inter"]), _rotate(k, cos, sin, c["rot"], c["inter"])
    page, off = _slots(st, st["seq"], st["pos"])
    out = {"q": q.to(torch.bfloat16)}
    if not c["q8"]:
        st["kv"][page, 0, :, off] = k.to(torch.bfloat16)
        st["kv"][page, 1, :, off] = v.to(torch.bfloat16)
        out["kv"] = st["kv"]
        return out
    codes, scales = _planes(st)
    x = torch.stack([k, v], dim=1).reshape(-1, 2, hkv, d // 32, 32)
    step = x.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(step != 0, 1.0 / step, torch.zeros_like(step))
    y = (x * inv).double()
    code = (y.sign() * (y.abs() + 0.5).floor()).to(torch.int8).reshape(-1, 2, hkv, d)
    codes[page, :, :, off] = code
    scales[page, :, :, off] = step[..., 0].to(torch.float16)
    out["k"], out["v"] = _read_plain(st, st["seq"], st["pos"])
    return out


def _attend_plain(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    out = torch.empty_like(st["q"])
    at = 0
    for s, (ln, n) in enumerate(zip(st["lens"].tolist(), st["news"].tolist())):   # ragged: one sequence at a time
        pos = torch.arange(ln, device=out.device)
        page, off = _slots(st, s, pos)
        k, v = _gather(st, page, off, 0).permute(1, 2, 0), _gather(st, page, off, 1).permute(1, 0, 2)
        q = st["q"][at:at + n].float().view(n, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * n, d)
        w = torch.matmul(q * (1.0 / math.sqrt(d)), k).view(hkv, g, n, ln)
        if n > 1:   # (the last row, a single new token's only one, sees every position)
            w.masked_fill_(pos[None, :] > pos[ln - n:, None], -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True)).exp_()
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.view(hkv, g * n, ln), v).view(hkv, g, n, d) / total
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, d).to(torch.bfloat16)
        at += n
    return out


def _every_position(st):
    lens = torch.from_numpy(st["lens"]).to(st["bt"].device, torch.int64)
    ends = lens.cumsum(0)
    total = int(st["lens"].sum())
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens, output_size=total)
    return seq, torch.arange(total, device=lens.device) - (ends - lens)[seq]


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        if op == "append":
            return _append_plain(st)
        if op == "attend":
            return _attend_plain(st)
        return _read_plain(st, *_every_position(st))
    mk, shape = st["mk"], st["shape"]
    if op == "attend":
        return mk.chunk_attention(shape, st["q"], st["news"], st["lens"], st["bt"], st["kv"])
    if op == "read":
        return mk.read_cache(shape, st["lens"], st["lens"], st["bt"], st["kv"])
    q = mk.append_chunk(shape, st["qkv"], st["news"], st["lens"], st["bt"], st["kv"], rope=st["rope"],
                        q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS)
    if not st["case"]["q8"]:
        return {"q": q, "kv": st["kv"]}
    k, v = mk.read_cache(shape, st["news"], st["lens"], st["bt"], st["kv"])   # the new rows as they will be read
    return {"q": q, "k": k, "v": v}


# ---------------------------------------------------------------- the work
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens, news = _lengths(case, 0)
    per = 2 * hkv * d * (17.0 / 16 if case["q8"] else 2.0)   # cached bytes of one position
    rows = sum(news)
    if case["op"] == "attend":
        seen = sum(n * (ln - n) + n * (n + 1) // 2 for ln, n in zip(lens, news))
        return {"bytes": 2 * rows * hq * d * 2 + per * sum(lens), "flops": 4.0 * d * hq * seen}
    if case["op"] == "append":
        back = rows * 2 * hkv * d * 2 + per * rows if case["q8"] else 0   # the new rows read back
        return {"bytes": rows * (hq + 2 * hkv) * d * 2 + rows * hq * d * 2 + per * rows + back,
                "flops": 6.0 * rows * (hq + hkv) * d}
    return {"bytes": sum(lens) * (per + 2 * hkv * d * 2), "flops": 2.0 * sum(lens) * hkv * d if case["q8"] else 0.0}


# ---------------------------------------------------------------- the definition in 64 bits
def _cached64(st, s, ln):
    """K and V of positions 0..ln-1 of sequence s, [2][Hkv][ln][D] in 64 bits, page by page in order."""
    c = st["case"]
    page = st["bt"][s, :-(-ln // c["ps"])].long()
    if c["q8"]:
        codes, scales = _planes(st)
        x = codes[page].double().unflatten(-1, (-1, 32)) * scales[page].double()[..., None]
        x = x.flatten(-2)
    else:
        x = st["kv"][page].double()
    return x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :ln]


def exact(case, seed):
    st = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = st["lens"].tolist()
    if case["op"] == "read":
        kv = torch.cat([_cached64(st, s, ln) for s, ln in enumerate(lens)], dim=2)
        return kv[0].transpose(0, 1).contiguous(), kv[1].transpose(0, 1).contiguous()
    news = st["news"].tolist()
    if case["op"] == "attend":
        out = torch.empty(sum(news), hq, d, dtype=torch.float64, device="cuda")
        at = 0
        for s, (ln, n) in enumerate(zip(lens, news)):
            kv = _cached64(st, s, ln)
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                end = ln - n + hi    # no row of this block sees a later position
                late = torch.ones(hi - lo, end, dtype=torch.bool, device="cuda").triu(ln - n + lo + 1)
                for h in range(hq):
                    k, v = kv[0, h // (hq // hkv), :end], kv[1, h // (hq // hkv), :end]
                    w = st["q"][at + lo:at + hi, h].double() @ k.T / math.sqrt(d)
                    w = torch.where(late, -math.inf, w)
                    out[at + lo:at + hi, h] = (w - torch.logsumexp(w, 1, keepdim=True)).exp() @ v
            at += n
        return out
    x = st["qkv"].double().view(-1, hq + 2 * hkv, d)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(st["pos"].double(), torch.from_numpy(st["freq"]).cuda()))
    r = case["rot"]
    done = []
    for h in range(hq + hkv):
        y = x[:, h].clone()
        if case["norm"]:
            y = y / (y.square().sum(1, keepdim=True) / d + EPS).sqrt() * st["q_norm" if h < hq else "k_norm"].double()
        first = torch.arange(0, r, 2, device="cuda") if case["inter"] else torch.arange(r // 2, device="cuda")
        second = first + (1 if case["inter"] else r // 2)
        z = torch.complex(y[:, first], y[:, second]) * turn
        y[:, first], y[:, second] = z.real, z.imag
        done.append(y)
    q, k, v = torch.stack(done[:hq], 1), torch.stack(done[hq:], 1), x[:, hq + hkv:]
    if case["q8"]:
        def kept(t):
            b = t.unflatten(-1, (-1, 32))
            s = b.abs().amax(-1, keepdim=True) / 127
            code = torch.where(s > 0, b / s, torch.zeros_like(b))
            code = torch.where(code < 0, (code - 0.5).ceil(), (code + 0.5).floor())
            return (code * s.to(torch.float16).double()).flatten(-2)
        return {"q": q, "k": kept(k), "v": kept(v)}
    kv = st["kv"].double()
    table = st["bt"].tolist()
    for row, (s, p) in enumerate(zip(st["seq"].tolist(), st["pos"].tolist())):
        slot, off = table[s][p // case["ps"]], p % case["ps"]
        kv[slot, 0, :, off], kv[slot, 1, :, off] = k[row], v[row]
    return {"q": q, "kv": kv}
