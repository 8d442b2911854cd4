"""What is measured of the cached-decode operators, and their plain forms.

Four operators that sit between the quantized projections of a decoder layer and its next
token:

* ``append``     per-head RMSNorm and position rotation of new queries and keys, and the write of
                 the rotated keys and of the values into a paged cache;
* ``attention``  causal attention over that cache for a batch whose sequences may share a long
                 prefix, stored once and read once for all of them;
* ``select``     one beam-search selection over beams and vocabulary;
* ``reorder``    the matching reorder of the beams' cached states.

A case is a dict of plain values.  ``prepare`` makes the inputs on the GPU, ``run`` makes one
pass: the plain form in elementary torch operations, or (``own``) the library's calls.
``exact`` computes the same outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ----------------------------------------------------------------------------------
# Head layouts: 32 query heads over 8 key/value heads of 128 (the repository's Qwen3-4B
# shape) and 32 over 4 (its Qwen3-30B-A3B shape); vocabulary 151936, 36 layers.

def _append(name, **kw):
    c = dict(op="append", name=name, B=1, n_lo=1, n_hi=1, own_lo=1, own_hi=64, groups=0, prefix=0, Hq=32, Hkv=8,
             D=128, rot=128, style="half", norm=True, page=16, dtype="f16", layout="nhd", shapes=1)
    c.update(kw)
    return c


def _attention(name, **kw):
    c = dict(op="attention", name=name, B=1, n_lo=1, n_hi=1, own_lo=1, own_hi=64, groups=0, prefix=0, Hq=32, Hkv=8,
             D=128, page=16, dtype="f16", out="f32", layout="nhd", shapes=1)
    c.update(kw)
    return c


def _select(name, **kw):
    c = dict(op="select", name=name, N=1, W=4, K=4, V=151936, done=0, masked=0)
    c.update(kw)
    return c


def _reorder(name, **kw):
    c = dict(op="reorder", name=name, N=1, W=4, layers=36, own_lo=20, own_hi=60, Hkv=8, D=128, page=16, dtype="f16",
             layout="nhd", shapes=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user's decode step: the smallest call, all latency
        _append("append one token", own_lo=4097, own_hi=4097),
        # a served batch's decode step, positions far into a shared prompt
        _append("append 96 sequences", B=96, own_lo=1, own_hi=700, groups=1, prefix=120000, dtype="bf16"),
        # prompts entering the cache, ragged, partial rotation of interleaved pairs, head-major pages
        _append("append prompts", B=6, n_lo=900, n_hi=3001, own_lo=0, own_hi=333, rot=64, style="pair", page=64,
                dtype="bf16", layout="hnd"),
        # one user's decode step over a few thousand cached tokens
        _attention("attend one token", own_lo=4097, own_hi=4097),
        # a served batch without anything shared: ragged contexts, some just begun
        _attention("attend 64 ragged", B=64, own_lo=1, own_hi=8191, dtype="bf16", out="same"),
        # a served batch under one long system prompt
        _attention("attend 64 under a prefix", B=64, own_lo=1, own_hi=500, groups=1, prefix=32768, Hkv=4, dtype="bf16",
                   out="same", page=64),
        # beam search: 8 requests of 6 beams, each request's beams under its own prompt
        _attention("attend beams", B=48, own_lo=9, own_hi=75, groups=8, prefix=2999),
        # prompts of a shared system prompt: ragged, many query tokens each
        _attention("attend prompts", B=7, n_lo=257, n_hi=2048, own_lo=0, own_hi=0, groups=1, prefix=4001,
                   dtype="bf16", out="same", page=32, layout="hnd"),
        # one request's selection
        _select("select 4 beams"),
        # a served batch of beam searches, some beams ended, some tokens banned
        _select("select 16 x 8 beams", N=16, W=8, K=8, done=9, masked=1),
        # one request's states, a page just begun
        _reorder("reorder 4 beams"),
        # a batch of beam searches
        _reorder("reorder 6 x 8 beams", N=6, W=8, own_lo=33, own_hi=62),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the same ranges, never costlier than the largest listed one."""
    op = rng.choice(["append", "append", "attention", "attention", "attention", "select", "reorder"])
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in t:
            t[k] = max(t[k], w[k])
    while True:
        c = _draw(op, rng)
        w = work(c)
        if all(w[k] <= top[op][k] for k in w):
            return c


def _draw(op, rng):
    if op == "select":
        W = rng.randint(1, 16)
        V = rng.choice([151936, _logint(rng, 50, 262144)])
        c = _select("", N=_logint(rng, 1, 32), W=W, K=min(W * V, W * rng.choice([1, 1, 2])), V=V,
                    masked=rng.randint(0, 1))
        c["done"] = rng.choice([0, rng.randint(0, c["N"] * W)])
    elif op == "reorder":
        lo = rng.randint(1, 60)
        c = _reorder("", N=_logint(rng, 1, 8), W=rng.randint(2, 16), layers=_logint(rng, 1, 48), own_lo=lo,
                     own_hi=lo + rng.randint(0, 30), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]),
                     page=rng.choice([8, 16, 32]), dtype=rng.choice(["f16", "bf16"]),
                     layout=rng.choice(["nhd", "hnd"]), shapes=rng.randint(1, 10 ** 6))
    else:
        Hkv = rng.choice([1, 2, 4, 4, 8, 8])
        D = rng.choice([64, 128, 128, 128, 256])
        common = dict(Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8]), D=D, page=rng.choice([1, 8, 16, 32, 64, 128]),
                      dtype=rng.choice(["f16", "bf16"]), layout=rng.choice(["nhd", "hnd"]),
                      shapes=rng.randint(1, 10 ** 6))
        kind = rng.choice(["one", "ragged", "prefix", "beams", "few", "prompts"])
        groups, prefix, n_lo, n_hi = 0, 0, 1, 1
        if kind == "one":
            B = 1
            own_lo = own_hi = _logint(rng, 1, 100000)
        elif kind == "ragged":
            B = _logint(rng, 2, 128)
            own_lo, own_hi = rng.randint(0, 3), _logint(rng, 8, 12000)
        elif kind == "prefix":
            B = _logint(rng, 2, 128)
            groups, prefix = 1, _logint(rng, 100, 60000)
            own_lo, own_hi = 1, _logint(rng, 1, 1000)
        elif kind == "beams":
            groups = _logint(rng, 1, 12)
            B = groups * rng.randint(2, 16)
            prefix = _logint(rng, 10, 6000)
            own_lo, own_hi = 1, _logint(rng, 1, 100)
        elif kind == "few":  # several new tokens a sequence: a draft to verify, a prompt's last piece
            B = _logint(rng, 1, 64)
            n_lo, n_hi = 1, rng.randint(2, 17)
            groups = rng.choice([0, 1])
            prefix = groups * _logint(rng, 10, 20000)
            own_lo, own_hi = 0, _logint(rng, 20, 4000)
        else:
            common["D"] = D = min(D, 128)
            B = _logint(rng, 1, 12)
            n_lo, n_hi = 1, _logint(rng, 30, 5000)
            groups = rng.choice([0, 1])
            prefix = groups * _logint(rng, 10, 8000)
            own_lo, own_hi = 0, rng.choice([0, _logint(rng, 10, 2000)])
        common.update(B=B, groups=groups, prefix=prefix, n_lo=n_lo, n_hi=n_hi, own_lo=own_lo, own_hi=own_hi)
        if op == "append":
            if kind in ("one", "ragged"):
                common["own_lo"] = max(1, common["own_lo"])
                common["own_hi"] = max(1, common["own_hi"])
            c = _append("", rot=rng.choice([D, D, D // 2, D // 4]), style=rng.choice(["half", "pair"]),
                        norm=rng.random() < 0.6, **common)
        else:
            c = _attention("", out=rng.choice(["f32", "same"]), **common)
    del c["name"]
    return c


# ---- the batch a case describes ---------------------------------------------------------------
# Sequence b has n[b] new query tokens and len[b] tokens of its own in the cache, the new ones
# among them; its group's prefix precedes them.

def _shape(c):
    r = random.Random(c["shapes"])
    B = c["B"]
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(B)]
    if c["n_hi"] == 1:
        length = [r.randint(c["own_lo"], c["own_hi"]) for _ in range(B)]
    else:
        length = [x + r.randint(c["own_lo"], c["own_hi"]) for x in n]
    G = c["groups"]
    gstart = [B * g // G for g in range(G + 1)] if G else []
    plen = [c["prefix"] if G == 1 else r.randint(3 * c["prefix"] // 4, c["prefix"]) for _ in range(G)]
    if G > 1:  # the beams of a request advance together
        for g in range(G):
            for b in range(gstart[g], gstart[g + 1]):
                length[b] = length[gstart[g]] if n[b] == 1 else length[b]
    return n, length, gstart, plen


def _group_of(b, gstart):
    for g in range(len(gstart) - 1):
        if gstart[g] <= b < gstart[g + 1]:
            return g
    return -1


def _visible(n, length, pre, i):
    """Keys that query token i of n sees: the prefix and its own tokens up to itself."""
    return max(0, pre + length - n + i + 1)


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"] == "select":
        rows = c["N"] * c["W"]
        return {"bytes": (rows - c["done"]) * c["V"] * 4 + rows * 5 + c["N"] * c["K"] * 13,
                "flops": (rows - c["done"]) * c["V"] * 4}
    if c["op"] == "reorder":
        length, parents = _beam_shape(c)
        tok = c["Hkv"] * c["D"] * 2 * 2 * c["layers"]
        nbytes = 0
        for ln, par in zip(length, parents):
            moved = [(i, p) for i, p in enumerate(par) if i != p]
            nbytes += (ln % c["page"]) * tok * (len(moved) + len({p for _, p in moved}))
            nbytes += (ln // c["page"]) * 4 * 2 * len(moved)
        return {"bytes": nbytes + 8 * c["N"] * c["W"], "flops": 0}
    n, length, gstart, plen = _shape(c)
    T = sum(n)
    if c["op"] == "append":
        per = (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": T * per * (4 + 2) + 8 * c["B"] + 4 * T,
                "flops": T * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + (4 * c["D"] if c["norm"] else 0))}
    keys = 0
    pairs = 0
    for b in range(c["B"]):
        g = _group_of(b, gstart)
        pre = plen[g] if g >= 0 else 0
        keys += length[b]
        first, last = pre + length[b] - n[b] + 1, pre + length[b]
        lo = max(0, first)
        if last >= lo:
            pairs += (lo + last) * (last - lo + 1) // 2
    keys += sum(plen)
    return {"bytes": keys * c["Hkv"] * c["D"] * 2 * 2 + T * c["Hq"] * c["D"] * (2 + (4 if c["out"] == "f32" else 2)),
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(n_pages, c, gen, layers=1):
    """One allocation of page pools, [2 * layers][pages][tokens][heads][D]: a layer's keys, then
    its values (head-major pools are permuted views)."""
    nhd = c["layout"] == "nhd"
    dims = (c["page"], c["Hkv"]) if nhd else (c["Hkv"], c["page"])
    pool = torch.empty((2 * layers, n_pages, *dims, c["D"]), dtype=DTYPES[c["dtype"]], device="cuda")
    for x in pool:
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    return pool if nhd else pool.permute(0, 1, 3, 2, 4)


def _batch(c, gen, with_prefix_pages):
    n, length, gstart, plen = _shape(c)
    page = c["page"]
    B, G = c["B"], c["groups"]
    npp = [(x + page - 1) // page for x in length]
    gpp = [(x + page - 1) // page if with_prefix_pages else 0 for x in plen]
    total = max(1, sum(npp) + sum(gpp))
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    st = {"n": n, "len": length, "gstart": gstart, "plen": plen, "n_pages": total}
    at = 0

    def table(counts):
        nonlocal at
        t = torch.zeros((len(counts), max(1, max(counts, default=1))), dtype=torch.int32, device="cuda")
        for i, k in enumerate(counts):
            t[i, :k] = order[at:at + k]
            at += k
        return t

    st["pages"] = table(npp)
    st["kv_len"] = _i32(length)
    qs = [0]
    for x in n:
        qs.append(qs[-1] + x)
    st["qs"] = qs
    st["T"] = qs[-1]
    st["q_start"] = None if c["n_hi"] == 1 else _i32(qs)
    if G:
        st["group_start"] = _i32(gstart)
        st["prefix_len"] = _i32(plen)
        st["prefix_pages"] = table(gpp)
    else:
        st["group_start"] = st["prefix_len"] = st["prefix_pages"] = None
    return st


def _beam_shape(c):
    """Per request: tokens held by each beam, and the picks' parents.  Children are laid out so
    that a parent's first child keeps the parent's place, as an engine does that copies little."""
    r = random.Random(c["shapes"])
    length, parents = [], []
    for _ in range(c["N"]):
        length.append(r.randint(c["own_lo"], c["own_hi"]))
        live = sorted(r.sample(range(c["W"]), max(1, (c["W"] + 1) // 2)))
        parents.append([i if i in live else r.choice(live) for i in range(c["W"])])
    return length, parents


def _package():
    import gguf_block_dequant_gb300 as qg

    return qg


def prepare(c, seed):
    gen = _gen(seed)
    st = {"case": c}
    if c["op"] == "select":
        rows = c["N"] * c["W"]
        logits = torch.randn((rows, c["V"]), generator=gen, device="cuda") * 2.5
        if c["masked"]:  # banned tokens: the type's lowest value, or minus infinity
            ban = torch.rand((rows, c["V"]), generator=gen, device="cuda") < 0.1
            low = torch.where(torch.arange(rows, device="cuda") % 2 == 0, torch.finfo(torch.float32).min, -math.inf)
            logits = torch.where(ban, low[:, None], logits)
        st["logits"] = logits
        st["scores"] = -20.0 * torch.rand((rows,), generator=gen, device="cuda") / 4 - 10.0
        done = torch.zeros((rows,), dtype=torch.uint8, device="cuda")
        if c["done"]:
            done[torch.randperm(rows, generator=gen, device="cuda")[:c["done"]]] = 1
        st["done"] = done
        st["eos"] = c["V"] - 3
        st["out"] = (torch.empty((c["N"], c["K"]), device="cuda"),
                     torch.empty((c["N"], c["K"]), dtype=torch.int32, device="cuda"),
                     torch.empty((c["N"], c["K"]), dtype=torch.int32, device="cuda"),
                     torch.empty((c["N"], c["K"]), dtype=torch.uint8, device="cuda"))
        if own:
            qg = _package()
            st["ws"] = torch.zeros(qg.beam_workspace_size(c["N"], c["W"], c["K"], c["V"]), dtype=torch.uint8,
                                   device="cuda")
        return st
    if c["op"] == "reorder":
        length, parents = _beam_shape(c)
        W, page = c["W"], c["page"]
        cols = max(length) // page + 1
        total = c["N"] * W * cols
        st["pages"] = torch.randperm(total, generator=gen, device="cuda").to(torch.int32).view(c["N"] * W, cols)
        st["kv_len"] = _i32([x for x in length for _ in range(W)])
        st["len"] = length
        st["parents"] = _i32(parents)
        st["pool"] = _cache(total, c, gen, c["layers"])
        if own:
            qg = _package()
            st["caches"] = qg.kv_caches(list(st["pool"][0::2]), list(st["pool"][1::2]))
            st["batch"] = qg.kv_batch(st["kv_len"], st["pages"])
        return st
    st.update(_batch(c, gen, c["op"] == "attention"))
    T, Hq, Hkv, D = st["T"], c["Hq"], c["Hkv"], c["D"]
    st["k"], st["v"] = _cache(st["n_pages"], c, gen)
    if c["op"] == "append":
        # one projection's output row holds the queries, keys and values side by side
        st["qkv"] = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda") * 1.7
        st["wq"] = st["wk"] = None
        if c["norm"]:
            st["wq"] = 1.0 + 0.3 * torch.randn((D,), generator=gen, device="cuda")
            st["wk"] = 1.0 + 0.3 * torch.randn((D,), generator=gen, device="cuda")
        st["q_out"] = torch.zeros((T, Hq, D), dtype=DTYPES[c["dtype"]], device="cuda")
    else:
        st["q"] = (torch.randn((T, Hq, D), generator=gen, device="cuda") * 2.0).to(DTYPES[c["dtype"]])
        st["out"] = torch.empty((T, Hq, D), dtype=torch.float32 if c["out"] == "f32" else DTYPES[c["dtype"]],
                                device="cuda")
    if own:
        qg = _package()
        st["cache"] = qg.kv_cache(st["k"], st["v"])
        st["batch"] = qg.kv_batch(st["kv_len"], st["pages"], st["q_start"], T, st["group_start"], st["prefix_len"],
                                  st["prefix_pages"])
        if c["op"] == "append":
            st["freqs"] = qg.rope_freqs(c["rot"], THETA).cuda()
        else:
            st["ws"] = torch.zeros(qg.attn_workspace_size(st["cache"], st["batch"], Hq), dtype=torch.uint8,
                                   device="cuda")
    return st


THETA = 1000000.0
EPS = 1e-6


# ---- one pass ---------------------------------------------------------------------------------

def run(st):
    c = st["case"]
    return (_own if own else _plain)[c["op"]](c, st)


def _own_append(c, st):
    qg = _package()
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = st["qkv"]
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    qg.kv_append(st["cache"], st["batch"], q, k, v, st["q_out"], st["freqs"], pairs=c["style"] == "pair",
                 q_norm=st["wq"], k_norm=st["wk"], eps=EPS)
    return st["q_out"], st["k"], st["v"]


def _own_attention(c, st):
    return _package().attn_paged(st["cache"], st["batch"], st["q"], st["out"], _scale(c), st["ws"])


def _own_select(c, st):
    score, parent, token, done = st["out"]
    _package().beam_select(st["logits"], st["scores"], c["N"], c["W"], score, parent, token, st["ws"],
                           done=st["done"], eos=st["eos"], done_out=done)
    return score, parent, token, done


def _own_reorder(c, st):
    _package().beam_reorder(st["caches"], st["batch"], st["parents"], c["W"])
    return st["pages"], st["pool"]


def _scale(c):
    return 1.0 / math.sqrt(c["D"])


def _slots(c, st):
    """Page, row and position of every new token."""
    page_of, row_of, pos = [], [], []
    for b in range(c["B"]):
        g = _group_of(b, st["gstart"])
        pre = st["plen"][g] if g >= 0 else 0
        s = torch.arange(st["len"][b] - st["n"][b], st["len"][b], device="cuda")
        page_of.append(st["pages"][b][s // c["page"]].long())
        row_of.append(s % c["page"])
        pos.append(s + pre)
    return torch.cat(page_of), torch.cat(row_of), torch.cat(pos)


def _plain_append(c, st):
    T, Hq, Hkv, D, rot = st["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    page_of, row_of, pos = _slots(c, st)
    x = st["qkv"].view(T, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * st["wq"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * st["wk"]
    # far positions: the angle in 64 bits
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    ang = pos.double()[:, None] * THETA ** (-2.0 * i / rot)
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def turn(t):
        t = t.clone()
        if c["style"] == "pair":
            a, b = t[..., 0:rot:2].clone(), t[..., 1:rot:2].clone()
            t[..., 0:rot:2], t[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = t[..., :rot // 2].clone(), t[..., rot // 2:rot].clone()
            t[..., :rot // 2], t[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
        return t

    st["q_out"].copy_(turn(q))
    st["k"][page_of, row_of] = turn(k).to(st["k"].dtype)
    st["v"][page_of, row_of] = v.to(st["v"].dtype)
    return st["q_out"], st["k"], st["v"]


def _keys(pool, table, length, page):
    """The first `length` cached rows [length][heads][D] of a page list."""
    s = torch.arange(length, device="cuda")
    return pool[table[s // page].long(), s % page]


def _plain_attention(c, st):
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    scale = _scale(c)
    pre = {}
    for g, ln in enumerate(st["plen"]):
        pre[g] = [_keys(st[x], st["prefix_pages"][g], ln, page).float() for x in ("k", "v")]
    out = st["out"]
    for b in range(c["B"]):
        n, ln = st["n"][b], st["len"][b]
        t0 = st["qs"][b]
        g = _group_of(b, st["gstart"])
        k, v = [_keys(st[x], st["pages"][b], ln, page).float() for x in ("k", "v")]
        if g >= 0:
            k, v = torch.cat([pre[g][0], k]), torch.cat([pre[g][1], v])
        S = k.shape[0]
        if S == 0:
            out[t0:t0 + n] = 0
            continue
        k, v = k.permute(1, 2, 0), v.permute(1, 0, 2)  # [Hkv][D][S], [Hkv][S][D]
        step = max(1, (1 << 28) // (Hq * S))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            q = st["q"][t0 + i0:t0 + i1].float().view(i1 - i0, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
            s = torch.matmul(q.reshape(Hkv, -1, D), k).view(Hkv, i1 - i0, Hq // Hkv, S) * scale
            last = torch.arange(i0, i1, device="cuda") + (S - n)  # the last key each token sees
            seen = torch.arange(S, device="cuda")[None] <= last[:, None]
            s = s.masked_fill(~seen[None, :, None], -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            p = torch.where(seen[None, :, None], p, 0.0)
            l = p.sum(-1)
            o = torch.matmul(p.view(Hkv, -1, S), v).view(Hkv, i1 - i0, Hq // Hkv, D)
            o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
            out[t0 + i0:t0 + i1] = o.permute(1, 0, 2, 3).reshape(i1 - i0, Hq, D).to(out.dtype)
    return out


def _plain_select(c, st):
    N, W, K, V = c["N"], c["W"], c["K"], c["V"]
    # candidates next to each other in score are told apart in 64 bits
    x = st["logits"].double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - torch.where(torch.isinf(m), 0.0, m)).sum(-1, keepdim=True)) - torch.where(
        torch.isinf(m), m, 0.0)
    lp = x - lse
    lp = torch.where(torch.isnan(lp), -math.inf, lp)
    ended = st["done"].bool()[:, None]
    only = torch.where(torch.arange(V, device="cuda")[None] == st["eos"], 0.0, -math.inf).double()
    cand = st["scores"].double()[:, None] + torch.where(ended, only, lp)
    val, idx = torch.sort(cand.view(N, W * V), dim=-1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    parent, token = idx // V, idx % V
    fin = st["done"].view(N, W).gather(1, parent).bool() | (token == st["eos"])
    return val.float(), parent.int(), token.int(), fin.to(torch.uint8)


def _plain_reorder(c, st):
    W, page = c["W"], c["page"]
    par = st["parents"].long()
    for r in range(c["N"]):
        full, rem = st["len"][r] // page, st["len"][r] % page
        rows = st["pages"][r * W:(r + 1) * W]
        if rem:
            dst, src = rows[:, full].long(), rows[par[r], full].long()
            for pool in st["pool"]:
                pool[dst, :rem] = pool[src, :rem]
        rows[:, :full] = rows[par[r], :full]
    return st["pages"], st["pool"]


_plain = {"append": _plain_append, "attention": _plain_attention, "select": _plain_select, "reorder": _plain_reorder}
_own = {"append": _own_append, "attention": _own_attention, "select": _own_select, "reorder": _own_reorder}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(c, seed):
    """The outputs of ``run`` for these inputs, each from its definition."""
    global own
    keep, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = keep
    if c["op"] == "append":
        return _exact_append(c, st)
    if c["op"] == "attention":
        return _exact_attention(c, st)
    if c["op"] == "select":
        return _exact_select(c, st)
    return _exact_reorder(c, st)


def _exact_append(c, st):
    Hq, Hkv, D, rot, page = c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    heads = st["qkv"].double().view(st["T"], Hq + 2 * Hkv, D)
    q_out = torch.empty((st["T"], Hq, D), dtype=torch.float64, device="cuda")
    kc, vc = st["k"].double(), st["v"].double()
    half = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * half, 2 * half + 1) if c["style"] == "pair" else (half, half + rot // 2)
    freq = torch.exp(half.double() * (-2.0 / rot) * math.log(THETA))
    for b in range(c["B"]):
        t0, n, ln = st["qs"][b], st["n"][b], st["len"][b]
        g = _group_of(b, st["gstart"])
        slot = torch.arange(ln - n, ln, device="cuda")
        ang = (slot + (st["plen"][g] if g >= 0 else 0)).double()[:, None, None] * freq
        z = torch.complex(torch.cos(ang), torch.sin(ang))
        done = []
        for x, w in ((heads[t0:t0 + n, :Hq], st["wq"]), (heads[t0:t0 + n, Hq:Hq + Hkv], st["wk"])):
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            y = x.clone()
            r = torch.complex(x[..., ia].contiguous(), x[..., ib].contiguous()) * z
            y[..., ia], y[..., ib] = r.real, r.imag
            done.append(y)
        q_out[t0:t0 + n] = done[0]
        pg, row = st["pages"][b][slot // page].long(), slot % page
        kc[pg, row] = done[1]
        vc[pg, row] = heads[t0:t0 + n, Hq + Hkv:]
    return q_out, kc, vc


def _exact_attention(c, st):
    if work(c)["flops"] > 6e12:
        return None
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros((st["T"], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n, ln, t0 = st["n"][b], st["len"][b], st["qs"][b]
        g = _group_of(b, st["gstart"])
        rows = [(st["prefix_pages"][g], st["plen"][g])] if g >= 0 else []
        rows.append((st["pages"][b], ln))
        where = [(t[torch.arange(x, device="cuda") // page].long(), torch.arange(x, device="cuda") % page)
                 for t, x in rows]
        pg, rw = torch.cat([w[0] for w in where]), torch.cat([w[1] for w in where])
        S = pg.numel()
        for h in range(Hkv):
            K, V = st["k"][pg, rw, h].double(), st["v"][pg, rw, h].double()
            step = max(1, (1 << 27) // max(1, S * (Hq // Hkv)))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                q = st["q"][t0 + i0:t0 + i1, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
                s = torch.einsum("tgd,sd->tgs", q, K) / math.sqrt(D)
                for_token = torch.tensor([_visible(n, ln, S - ln, i) for i in range(i0, i1)], device="cuda")
                hid = torch.arange(S, device="cuda") >= for_token[:, None]
                s[hid[:, None, :].expand_as(s)] = -math.inf
                some = for_token > 0
                if S and bool(some.any()):
                    w = torch.softmax(s[some], -1)
                    blk = out[t0 + i0:t0 + i1, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)]
                    blk[some] = torch.einsum("tgs,sd->tgd", w, V)
    return out


def _exact_select(c, st):
    N, W, K, V = c["N"], c["W"], c["K"], c["V"]
    score = torch.empty((N, K), dtype=torch.float64, device="cuda")
    parent = torch.empty((N, K), dtype=torch.int32, device="cuda")
    token, fin = torch.empty_like(parent), torch.empty((N, K), dtype=torch.uint8, device="cuda")
    for r in range(N):
        best = []
        for w in range(W):
            base, row = float(st["scores"][r * W + w]), st["logits"][r * W + w].double()
            if int(st["done"][r * W + w]):
                lp = torch.full((V,), -math.inf, dtype=torch.float64, device="cuda")
                lp[st["eos"]] = 0.0
            else:
                row = torch.nan_to_num(row, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
                lp = torch.nan_to_num(row - torch.logsumexp(row, 0), nan=-math.inf, neginf=-math.inf)
            # a row's K best, ties to the lowest token
            o = torch.argsort(lp, descending=True, stable=True)[:K]
            best += [(base + x, w, t) for x, t in zip(lp[o].tolist(), o.tolist())]
        best.sort(key=lambda e: (-e[0], e[1], e[2]))
        for i, (x, w, t) in enumerate(best[:K]):
            score[r, i], parent[r, i], token[r, i] = x, w, t
            fin[r, i] = 1 if int(st["done"][r * W + w]) or t == st["eos"] else 0
    return score, parent, token, fin


def _exact_reorder(c, st):
    W, page = c["W"], c["page"]
    pages, pool, par = st["pages"].clone(), st["pool"].clone(), st["parents"].tolist()
    for r in range(c["N"]):
        full, rem = divmod(st["len"][r], page)
        for i in range(W):
            p = par[r][i]
            if p == i:
                continue
            pages[r * W + i, :full] = st["pages"][r * W + p, :full]
            if rem:
                d, s = int(st["pages"][r * W + i, full]), int(st["pages"][r * W + p, full])
                pool[:, d, :rem] = st["pool"][:, s, :rem]
    return pages, pool
