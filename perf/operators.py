"""Timed cases of the paged-cache operators: rotary positions, the page write, attention of new
tokens over the pages, accumulated attention weights, and eviction by them.

``run`` computes an operator in plain torch operations (fp32, angles in fp64), or, with ``own``
set, through the library. A case is a dict of plain values; ragged lengths follow from it alone.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128
BF = torch.bfloat16


def listed():
    """Shapes of the repository's workloads (32 / 8, 32 / 32 and 4 / 1 heads of 128 dims)."""
    return [
        # queries of one decode step of a batch, rotated in place of use
        dict(name="rope_decode_queries", op="rope", B=1, T=33, H=32, rot=128, inter=False,
             scaling="bands", dtype="bf16", transpose=False, far=131072),
        # a whole head-major prompt cache rotated back (gradient / un-rotation), part of the head
        dict(name="rope_transpose_prompt", op="rope", B=2, T=16001, H=8, rot=64, inter=True,
             scaling="yarn", dtype="f32", transpose=True, far=1000000),
        # one decode step of 64 sequences: rotate q and k, write k and v into the pages
        dict(name="append_decode_b64", op="append", B=64, Hq=32, Hkv=8, max_q=1, max_kv=4096,
             page=16, ragged=7, scaling="plain"),
        # a ragged prompt batch: up to 4001 new tokens a sequence
        dict(name="append_prompts", op="append", B=5, Hq=32, Hkv=8, max_q=4001, max_kv=8192,
             page=64, ragged=11, scaling="linear"),
        # the smallest call: one token of one short sequence, 4 query heads on 1 KV head
        dict(name="attend_one_token", op="attend", B=1, Hq=4, Hkv=1, max_q=1, max_kv=2048, page=16,
             ragged=0, window=0),
        # a full decode batch over long ragged caches: the KV read
        dict(name="attend_decode_b64", op="attend", B=64, Hq=32, Hkv=8, max_q=1, max_kv=16384,
             page=64, ragged=3, window=0),
        # mixed batch without head sharing: chunks and single tokens, sliding window, odd lengths
        dict(name="attend_mixed_window", op="attend", B=6, Hq=32, Hkv=32, max_q=701, max_kv=5003,
             page=32, ragged=5, window=1024),
        # a prompt chunk late in a long prompt: the matrix products
        dict(name="attend_chunk_4k_16k", op="attend", B=1, Hq=32, Hkv=8, max_q=4096, max_kv=16384,
             page=128, ragged=0, window=0),
        # key weights of one decode step
        dict(name="weights_decode_b32", op="weights", B=32, Hq=32, Hkv=8, max_q=1, max_kv=8192,
             page=64, ragged=9, window=0),
        # key weights of the last chunk of a prompt
        dict(name="weights_chunk_1k_32k", op="weights", B=1, Hq=32, Hkv=8, max_q=1024,
             max_kv=32768, page=128, ragged=0, window=0),
        # one long cache cut to an eighth
        dict(name="evict_b1_128k", op="evict", B=1, Hq=32, Hkv=8, max_kv=131072, keep=16384,
             sink=32, recent=1024, page=64, dst_page=64, ragged=0),
        # a ragged batch cut to an odd budget, pages of another size
        dict(name="evict_b24_8k", op="evict", B=24, Hq=32, Hkv=8, max_kv=8191, keep=2001,
             sink=4, recent=333, page=16, dst_page=48, ragged=13),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weights", "evict"])
    page = 16 * rng.choice([1, 2, 3, 4, 8, 16])
    Hq, Hkv = rng.choice([(32, 8), (32, 32), (4, 1), (32, 4), (7, 1), (30, 6), (16, 16)])
    if op == "rope":
        T = _spread(rng, 1, 8000)
        return dict(op=op, B=rng.randint(1, 4), T=T, H=rng.randint(1, 40), rot=2 * rng.randint(2, 64),
                    inter=rng.random() < 0.5, scaling=rng.choice(list(SCALINGS)),
                    dtype=rng.choice(["bf16", "f32"]), transpose=rng.random() < 0.5,
                    far=_spread(rng, 16, 2000000))
    if op == "append":
        max_q = _spread(rng, 1, 4000)
        return dict(op=op, B=rng.randint(1, max(1, min(64, 16000 // max_q))), Hq=Hq, Hkv=Hkv,
                    max_q=max_q, max_kv=max_q + _spread(rng, 1, 4000), page=page,
                    ragged=rng.randint(1, 999), scaling=rng.choice(list(SCALINGS)))
    if op in ("attend", "weights"):
        if rng.random() < 0.5:
            max_q = rng.randint(1, 4)
            max_kv = max_q + _spread(rng, 1, 30000)
            B = rng.randint(1, max(1, min(64, 600000 // max_kv)))
        else:
            max_q = _spread(rng, 5, 4000)
            max_kv = max_q + rng.choice([0, _spread(rng, 1, 12000)])
            B = rng.randint(1, max(1, min(8, 40000000 // (max_q * max_kv))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, max_q=max_q, max_kv=max_kv, page=page,
                    ragged=rng.randint(0, 999),
                    window=rng.choice([0, 0, _spread(rng, 1, 5000)]))
    max_kv = _spread(rng, 40, 130000)
    keep = max(1, int(max_kv * rng.uniform(0.05, 0.9)))
    sink = rng.randint(0, min(64, keep))
    return dict(op=op, B=rng.randint(1, max(1, min(48, 200000 // max_kv))), Hq=Hq, Hkv=Hkv,
                max_kv=max_kv, keep=keep, sink=sink, recent=rng.randint(0, min(2048, keep - sink)),
                page=page, dst_page=16 * rng.choice([1, 2, 3, 4, 8]), ragged=rng.randint(0, 999))


# --------------------------------------------------------------------------- lengths and frequencies

def _lengths(c):
    """(new tokens, cached tokens) of each sequence; ragged = 0 gives every sequence the largest."""
    max_q, max_kv = c.get("max_q", 1), c["max_kv"]
    if not c["ragged"]:
        return [max_q] * c["B"], [max_kv] * c["B"]
    rng = random.Random(c["ragged"])
    qs, kvs = [], []
    for b in range(c["B"]):
        n = max_q if b == 0 else rng.randint(1, max_q) if rng.random() < 0.7 else 1
        qs.append(n)
        kvs.append(max_kv if b == 0 else rng.randint(n, max_kv))
    return qs, kvs


SCALINGS = {  # base, factor, low / high band, length before scaling
    "plain": (10000.0, 1.0, 1.0, 4.0, 0),
    "linear": (10000.0, 4.0, 1.0, 4.0, 0),
    "ntk": (10000.0, 8.0, 1.0, 4.0, 0),
    "bands": (500000.0, 8.0, 1.0, 4.0, 8192),
    "yarn": (10000.0, 16.0, 1.0, 32.0, 4096),
}


def _frequencies(scaling, rot):
    """(angle per position of each pair, magnitude) in fp64."""
    base, factor, low, high, orig = SCALINGS[scaling]
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling in ("bands", "yarn"):
        out = []
        if scaling == "yarn":  # pairs that turn more than `high` / fewer than `low` times
            a = max(0.0, math.floor(rot * math.log(orig / (high * 2 * math.pi)) / (2 * math.log(base))))
            z = min(rot - 1.0, math.ceil(rot * math.log(orig / (low * 2 * math.pi)) / (2 * math.log(base))))
            z = max(z, a + 0.001)
        for i, x in enumerate(f):
            if scaling == "bands":
                keep = (orig * x / (2 * math.pi) - low) / (high - low)
            else:
                keep = 1.0 - (i - a) / (z - a)
            keep = min(1.0, max(0.0, keep))
            out.append(x / factor * (1.0 - keep) + x * keep)
        f = out
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def _library_rope(scaling, rot, inter):
    import fourier_basis_attention_b200 as fa
    base, factor, low, high, orig = SCALINGS[scaling]
    return fa.fa_rope_init(rot_dim=rot, base=base, interleaved=inter, scaling=scaling,
                           factor=factor, low=low, high=high, original_len=orig)


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = case
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    rand = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    s = dict(c=c)
    if c["op"] == "rope":
        dt = BF if c["dtype"] == "bf16" else torch.float32
        # head-major storage, seen as [B, T, H, 128]
        s["x"] = rand(c["B"], c["H"], c["T"], D).to(dt).transpose(1, 2)
        s["out"] = torch.empty(c["B"], c["T"], c["H"], D, dtype=dt, device=dev)
        s["pos"] = torch.randint(0, c["far"], (c["B"], c["T"]), generator=gen, device=dev,
                                 dtype=torch.int32)
        f, s["mag"] = _frequencies(c["scaling"], c["rot"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        if own:
            s["rope"] = _library_rope(c["scaling"], c["rot"], c["inter"])
        return s
    qs, kvs = _lengths(c)
    B, Hq, Hkv, page = c["B"], c["Hq"], c["Hkv"], c["page"]
    max_pages = -(-c["max_kv"] // page)
    used = sum(-(-n // page) for n in kvs)
    order = torch.randperm(used, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(kvs):
        m = -(-n // page)
        table[b, :m] = order[at:at + m]
        at += m
    s["table"] = table
    s["kv_len"] = torch.tensor(kvs, dtype=torch.int32, device=dev)
    s["q_start"] = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    s["K"] = rand(used, Hkv, page, D).to(BF)
    s["V"] = (rand(used, Hkv, page, D) + 0.5 * rand(1, Hkv, 1, D)).to(BF)
    total = sum(qs)
    if c["op"] == "append":
        # q, k, v as slices of one fused projection's rows
        qkv = rand(total, Hq + 2 * Hkv, D).to(BF)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.empty(total, Hq, D, dtype=BF, device=dev)
        f, s["mag"] = _frequencies(c["scaling"], D)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
    elif c["op"] in ("attend", "weights"):
        s["q"] = (1.5 * rand(total, Hq, D)).to(BF)
        s["out"] = torch.empty(total, Hq, D, dtype=BF, device=dev)
        s["lse"] = torch.empty(total, Hq, dtype=torch.float32, device=dev)
    if c["op"] == "weights":
        # the attention pass of the same step has left each row's log-sum-exp
        s["lse"] = _plain_scores(s)[1]
        s["acc"] = torch.zeros(B, Hkv, c["max_kv"], dtype=torch.float32, device=dev)
    if c["op"] == "evict":
        # few heavy keys, many light ones
        s["w"] = torch.exp(2.0 * rand(B, Hkv, c["max_kv"]))
        dst_pages = -(-c["keep"] // c["dst_page"])
        s["dst_table"] = torch.randperm(B * dst_pages, generator=gen, device=dev).to(
            torch.int32).view(B, dst_pages)
        s["dst_K"] = torch.zeros(B * dst_pages, Hkv, c["dst_page"], D, dtype=BF, device=dev)
        s["dst_V"] = torch.zeros_like(s["dst_K"])
        s["dst_w"] = torch.zeros(B, Hkv, c["keep"], dtype=torch.float32, device=dev)
        s["index"] = torch.empty(B, Hkv, c["keep"], dtype=torch.int32, device=dev)
        s["dst_len"] = torch.empty(B, dtype=torch.int32, device=dev)
    if own:
        import fourier_basis_attention_b200 as fa
        cache = fa.PagedCache(s["K"], s["V"], s["table"])
        s["batch"] = fa.PagedBatch(cache, Hq, s["q_start"], s["kv_len"], total_q=total,
                                   max_q=c.get("max_q", 1), max_kv=c["max_kv"])
        if c["op"] == "append":
            s["rope"] = _library_rope(c["scaling"], D, False)
        if c["op"] == "attend":
            s["ws"] = torch.empty(fa.fa_paged_attend_workspace_size(s["batch"], c["window"]),
                                  dtype=torch.uint8, device=dev)
        if c["op"] == "evict":
            s["dst"] = fa.PagedCache(s["dst_K"], s["dst_V"], s["dst_table"])
            s["ws"] = torch.empty(fa.fa_evict_workspace_size(s["batch"], c["keep"]),
                                  dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, mag, inter, transpose):
    """x [..., H, 128] fp32, pos [...]: the first 2 * len(freq) dims rotated, the rest as they are."""
    ang = pos.double()[..., None, None] * freq
    co, si = (mag * torch.cos(ang)).float(), (mag * torch.sin(ang)).float()
    if transpose:
        si = -si
    n = freq.numel()
    if inter:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack([a * co - b * si, b * co + a * si], dim=-1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat([a * co - b * si, b * co + a * si], dim=-1)
    return torch.cat([r, x[..., 2 * n:]], dim=-1)


def _rows(s):
    """Sequence and position of every new token (the last token of b is at kv_len[b] - 1)."""
    i = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["q_start"], i, right=True) - 1
    n = s["q_start"][1:] - s["q_start"][:-1]
    return b, s["kv_len"][b] - n[b] + (i - s["q_start"][b])


def _dense(pool, table):
    """[B, Hkv, tokens, 128] fp32 of a pool of pages."""
    x = pool[table.long()].permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, D).float()


def _plain_scores(s):
    """Softmax weights [B, Hkv, rows, keys] of the padded batch, lse and row numbers of it."""
    c, q = s["c"], s["q"]
    B, Hq, Hkv, Q = c["B"], c["Hq"], c["Hkv"], c["max_q"]
    G = Hq // Hkv
    n = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    i = torch.arange(Q, device="cuda", dtype=torch.int32)[None]
    row = (s["q_start"][:-1, None] + torch.minimum(i, n - 1)).long()      # padded rows repeat the last
    pos = s["kv_len"][:, None] - n + torch.minimum(i, n - 1)
    x = q[row].float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    K = _dense(s["K"], s["table"])[:, :, :c["max_kv"]]
    a = torch.matmul(x, K.transpose(-1, -2)).view(B, Hkv, Q, G, -1)
    a *= D ** -0.5
    j = torch.arange(c["max_kv"], device="cuda", dtype=torch.int32)
    hidden = j > pos[..., None]
    if c["window"]:
        hidden |= j <= pos[..., None] - c["window"]
    a.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    a -= top
    a.exp_()
    total = a.sum(-1, keepdim=True)
    a /= total
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(B, Q, Hq)
    live = (i < n)
    out = torch.empty(q.shape[0], Hq, dtype=torch.float32, device="cuda")
    out[row] = lse
    return a, out, row, live


def _plain(s):
    c = s["c"]
    if c["op"] == "rope":
        y = _rotate(s["x"].float(), s["pos"], s["freq"], s["mag"], c["inter"], c["transpose"])
        s["out"].copy_(y)
        return s["out"]
    if c["op"] == "append":
        b, pos = _rows(s)
        s["q_out"].copy_(_rotate(s["q"].float(), pos, s["freq"], s["mag"], False, False))
        k = _rotate(s["k"].float(), pos, s["freq"], s["mag"], False, False).to(BF)
        pg = s["table"][b, pos // c["page"]].long()
        s["K"][pg, :, (pos % c["page"]).long()] = k
        s["V"][pg, :, (pos % c["page"]).long()] = s["v"]
        return s["q_out"], s["K"], s["V"]
    if c["op"] == "attend":
        p, lse, row, live = _plain_scores(s)
        V = _dense(s["V"], s["table"])[:, :, :c["max_kv"]]
        B, Hkv, Q, G, _ = p.shape
        o = torch.matmul(p.view(B, Hkv, Q * G, -1), V).view(B, Hkv, Q, G, D)
        s["out"][row] = o.permute(0, 2, 1, 3, 4).reshape(B, Q, Hkv * G, D).to(BF)
        return s["out"], lse
    if c["op"] == "weights":
        p, _, _, live = _plain_scores(s)
        p *= live[:, None, :, None, None]
        s["acc"] += p.sum((2, 3))
        return s["acc"]
    return _plain_evict(s)


def _plain_evict(s):
    c = s["c"]
    keep, n = c["keep"], s["kv_len"][:, None, None]
    j = torch.arange(c["max_kv"], device="cuda", dtype=torch.int32)
    w = s["w"]
    held = (j < c["sink"]) | (j >= n - c["recent"])
    w = torch.where(j < n, torch.where(held, math.inf, w), -math.inf)
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = torch.minimum(s["kv_len"], torch.full_like(s["kv_len"], keep))
    here = torch.arange(keep, device="cuda", dtype=torch.int32) < count[:, None, None]
    first = torch.where(here, first, c["max_kv"]).sort(dim=-1).values
    if first.shape[-1] < keep:
        first = torch.cat([first, first.new_full((*first.shape[:2], keep - first.shape[-1]),
                                                 c["max_kv"])], dim=-1)
    idx = first.clamp(max=c["max_kv"] - 1)
    s["index"].copy_(torch.where(here, first, -1))
    s["dst_len"].copy_(count)
    s["dst_w"].copy_(torch.where(here, torch.gather(s["w"], 2, idx), s["dst_w"]))
    g = torch.arange(c["Hkv"], device="cuda")[None, :, None]
    pg = torch.gather(s["table"].long()[:, None].expand(-1, c["Hkv"], -1), 2, idx // c["page"])
    at = torch.arange(keep, device="cuda")
    dpg = s["dst_table"].long()[:, at // c["dst_page"]][:, None].expand(-1, c["Hkv"], -1)
    for pool, dst in ((s["K"], s["dst_K"]), (s["V"], s["dst_V"])):
        old = dst[dpg, g, at % c["dst_page"]]
        dst[dpg, g, at % c["dst_page"]] = torch.where(here[..., None], pool[pg, g, idx % c["page"]], old)
    return s["index"], s["dst_len"], s["dst_w"], s["dst_K"], s["dst_V"]


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fourier_basis_attention_b200 as fa
    c = s["c"]
    if c["op"] == "rope":
        fa.fa_rope(s["rope"], s["x"], s["pos"], s["out"], transpose=c["transpose"])
        return s["out"]
    if c["op"] == "append":
        fa.fa_paged_append(s["batch"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], rope=s["rope"])
        return s["q_out"], s["K"], s["V"]
    if c["op"] == "attend":
        fa.fa_paged_attend(s["batch"], s["q"], s["out"], s["ws"], lse=s["lse"], window=c["window"])
        return s["out"], s["lse"]
    if c["op"] == "weights":
        fa.fa_paged_weights(s["batch"], s["q"], s["lse"], s["acc"], window=c["window"])
        return s["acc"]
    fa.fa_evict(s["batch"], s["w"], c["keep"], s["dst"], s["index"], s["dst_len"], s["ws"],
                sink=c["sink"], recent=c["recent"], dst_weights=s["dst_w"])
    return s["index"], s["dst_len"], s["dst_w"], s["dst_K"], s["dst_V"]


# --------------------------------------------------------------------------- work

def _visible(n, kv, window):
    """(query, key) pairs of n new tokens at the end of kv cached ones, and keys that some query sees."""
    pairs = 0
    lo = kv - n
    if not window:
        return n * lo + n * (n + 1) // 2, kv
    # position p sees min(p + 1, window) keys
    short = max(0, min(kv, window) - lo)                 # positions p < window
    pairs = short * lo + short * (short + 1) // 2 + (n - short) * window
    return pairs, min(kv, n - 1 + window)


def work(case):
    c = case
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"]
        return dict(bytes=2 * n * c["H"] * D * e + 4 * n, flops=6 * n * c["H"] * c["rot"] // 2)
    qs, kvs = _lengths(c)
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["op"] == "append":
        n = sum(qs)
        return dict(bytes=2 * n * (Hq + 2 * Hkv) * D * 2, flops=6 * n * (Hq + Hkv) * D // 2)
    if c["op"] == "evict":
        kept = sum(min(k, c["keep"]) for k in kvs)
        return dict(bytes=Hkv * (4 * sum(kvs) + kept * (2 * 2 * D * 2 + 8 + 4)), flops=Hkv * sum(kvs))
    pairs = keys = 0
    for n, kv in zip(qs, kvs):
        a, k = _visible(n, kv, c["window"])
        pairs, keys = pairs + a, keys + k
    rows = sum(qs) * Hq
    if c["op"] == "attend":
        return dict(bytes=keys * Hkv * 2 * D * 2 + rows * (2 * D * 2 + 4), flops=4 * D * pairs * Hq)
    return dict(bytes=keys * Hkv * (D * 2 + 8) + rows * (D * 2 + 4), flops=2 * D * pairs * Hq)


# --------------------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(s["x"], s["pos"], c["scaling"], c["rot"], c["inter"], c["transpose"])
    qs, kvs = _lengths(c)
    start = [sum(qs[:b]) for b in range(c["B"])]
    if c["op"] == "append":
        K, V = s["K"].double(), s["V"].double()
        pos = torch.cat([torch.arange(kv - n, kv, device="cuda") for n, kv in zip(qs, kvs)])
        q = _exact_rope(s["q"], pos, c["scaling"], D, False, False)
        k = _exact_rope(s["k"], pos, c["scaling"], D, False, False)
        for b, (n, kv) in enumerate(zip(qs, kvs)):
            t = torch.arange(kv - n, kv, device="cuda")
            pg = s["table"][b].long()[t // c["page"]]
            K[pg, :, t % c["page"]] = k[start[b]:start[b] + n]
            V[pg, :, t % c["page"]] = s["v"][start[b]:start[b] + n].double()
        return q, K, V
    if c["op"] in ("attend", "weights"):
        return _exact_attend(s, qs, kvs, start)
    index = torch.full((c["B"], c["Hkv"], c["keep"]), -1, dtype=torch.int32)
    w, dst_w = s["w"].cpu().double(), s["dst_w"].cpu().double()
    dK, dV = s["dst_K"].double(), s["dst_V"].double()
    for b, kv in enumerate(kvs):
        m = min(kv, c["keep"])
        for g in range(c["Hkv"]):
            held = [j for j in range(kv) if j < c["sink"] or j >= kv - c["recent"]] if kv > m else list(range(kv))
            rest = set(range(kv)) - set(held)
            row = w[b, g].tolist()
            best = sorted(rest, key=lambda j: (-row[j], j))[:m - len(held)]
            kept = torch.tensor(sorted(held + best))
            index[b, g, :m] = kept.int()
            dst_w[b, g, :m] = w[b, g, kept]
            kept, at = kept.cuda(), torch.arange(m, device="cuda")
            src = s["table"][b].long()[kept // c["page"]]
            to = s["dst_table"][b].long()[at // c["dst_page"]]
            dK[to, g, at % c["dst_page"]] = s["K"][src, g, kept % c["page"]].double()
            dV[to, g, at % c["dst_page"]] = s["V"][src, g, kept % c["page"]].double()
    return index.cuda(), s["kv_len"].clamp(max=c["keep"]), dst_w.cuda(), dK, dV


def _exact_rope(x, pos, scaling, rot, inter, transpose):
    """Each pair as a complex number times magnitude * exp(i * position * frequency)."""
    f, mag = _frequencies(scaling, rot)
    turn = torch.polar(torch.tensor(mag, dtype=torch.float64, device="cuda"),
                       pos.double()[..., None] * torch.tensor(f, dtype=torch.float64, device="cuda"))
    turn = (turn.conj() if transpose else turn).unsqueeze(-2)
    y = x.double().clone()
    pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if inter else (2, rot // 2))
    if not inter:
        pairs = pairs.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y[..., :rot] = (z if inter else z.transpose(-1, -2)).flatten(-2)
    return y


def _exact_attend(s, qs, kvs, start):
    c = s["c"]
    G, total = c["Hq"] // c["Hkv"], sum(qs)
    out = torch.empty(total, c["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(total, c["Hq"], dtype=torch.float64, device="cuda")
    acc = torch.zeros(c["B"], c["Hkv"], c["max_kv"], dtype=torch.float64, device="cuda")
    for b, (n, kv) in enumerate(zip(qs, kvs)):
        pages = s["table"][b, :-(-kv // c["page"])].long()
        rows = slice(start[b], start[b] + n)
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None]
        seen = (j <= p) & (j > p - c["window"]) if c["window"] else j <= p
        for g in range(c["Hkv"]):
            k = s["K"][pages, g].reshape(-1, D)[:kv].double()
            v = s["V"][pages, g].reshape(-1, D)[:kv].double()
            for h in range(g * G, g * G + G):
                a = (s["q"][rows, h].double() @ k.T) / math.sqrt(D)
                a[~seen] = -math.inf
                lse[rows, h] = torch.logsumexp(a, dim=1)
                a = torch.exp(a - lse[rows, h][:, None])
                if c["op"] == "attend":
                    out[rows, h] = a @ v
                else:
                    acc[b, g, :kv] += a.sum(0)
    return (out, lse) if c["op"] == "attend" else acc
