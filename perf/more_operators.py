"""What is measured of the drafted-decode operators, and their plain forms.

Five operators of a server that drafts tokens, verifies them and branches its contexts, on decoders whose
layers are partly recurrent:

* ``delta``    the gated delta rule of a linear-attention layer: one state matrix per value head, for single
               tokens, for drafted ones (the state after each of them is kept) and for whole prompts;
* ``probs``    the next token's probabilities from logits, a temperature for each row;
* ``verify``   drafted tokens against the target's probabilities from given random numbers;
* ``branch``   several continuations of cached prompts: their pages are shared, the page begun is copied
               when a continuation gets its next tokens;
* ``compact``  chosen tokens of cached contexts moved into pages of their own.

A case is a dict of plain values.  ``prepare`` makes the inputs on the GPU, ``run`` makes one pass: the
plain form in elementary torch operations, or (``own``) the library's calls.  ``exact`` computes the same
outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
L2_EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------
# Recurrent layers of 16 key and 32 value heads of 128; caches of 8 key/value heads of 128 over 36 layers
# and a vocabulary of 151936 (the repository's Qwen3-4B shape).

def _delta(name, **kw):
    c = dict(op="delta", name=name, B=1, n_lo=1, n_hi=1, Hk=16, Hv=32, Dk=128, Dv=128, gates="raw", l2=True,
             keep=False, fresh=False, tiled=False, shapes=1)
    c.update(kw)
    return c


def _probs(name, **kw):
    c = dict(op="probs", name=name, T=1, V=151936, temp="mixed", masked=False)
    c.update(kw)
    return c


def _verify(name, **kw):
    c = dict(op="verify", name=name, B=1, n_lo=4, n_hi=4, V=151936, draft="probs", shapes=1)
    c.update(kw)
    return c


def _branch(name, **kw):
    c = dict(op="branch", name=name, R=1, ways=4, lo=1001, hi=1001, add=1, layers=36, Hkv=8, D=128, page=16,
             dtype="f16", layout="nhd", shapes=1)
    c.update(kw)
    return c


def _compact(name, **kw):
    c = dict(op="compact", name=name, R=1, lo=40, hi=40, part=0.33, layers=36, Hkv=8, D=128, page=16, dtype="f16",
             layout="nhd", shapes=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user's decode step in one recurrent layer: the smallest call, all latency
        _delta("delta one token"),
        # a served batch's decode step
        _delta("delta 64 sequences", B=64),
        # a served batch with drafts of several lengths: every token's state is kept for the verification to choose from
        _delta("delta drafts", B=16, n_lo=2, n_hi=7, keep=True),
        # ragged prompts
        _delta("delta prompts", B=5, n_lo=900, n_hi=8000, fresh=True),
        # one user's drafts and the token behind them
        _probs("probs 5 rows", T=5),
        # a served batch's drafts, some rows greedy, some tokens banned
        _probs("probs 200 rows", T=200, masked=True),
        # one user's four drafts
        _verify("verify 4 drafts"),
        # a served batch, ragged drafts
        _verify("verify 64 sequences", B=64, n_lo=1, n_hi=8),
        # four continuations of one prompt, each about to get one token
        _branch("branch 4 of a prompt"),
        # a batch of prompts, four continuations each, each about to get a few drafted tokens
        _branch("branch 4 of 12 prompts", R=12, lo=20, hi=90, add=5, dtype="bf16"),
        # a short context's chosen tokens
        _compact("compact 40 tokens"),
        # long contexts, half of their tokens kept
        _compact("compact 2 contexts", R=2, lo=1200, hi=1900, part=0.5, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the same ranges, never costlier than the largest listed one."""
    op = rng.choice(["delta", "delta", "delta", "probs", "verify", "branch", "compact"])
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in t:
            t[k] = max(t[k], w[k])
    longest = max(c["n_hi"] for c in listed() if c["op"] == "delta")
    while True:
        c = _draw(op, rng, longest)
        w = work(c)
        if all(w[k] <= top[op][k] for k in w) and _pool_bytes(c) <= 1 << 30 and w["bytes"] > 0:
            del c["name"]
            return c


def _draw(op, rng, longest):
    shapes = rng.randint(1, 10 ** 6)
    if op == "probs":
        return _probs("", T=_logint(rng, 1, 256), V=rng.choice([151936, _logint(rng, 50, 262144)]),
                      temp=rng.choice(["none", "mixed"]), masked=rng.random() < 0.5)
    if op == "verify":
        lo = rng.randint(0, 3)
        return _verify("", B=_logint(rng, 1, 128), n_lo=lo, n_hi=lo + rng.randint(0, 9),
                       V=rng.choice([151936, _logint(rng, 400, 262144)]), draft=rng.choice(["probs", "probs", "none"]),
                       shapes=shapes)
    pool = dict(layers=_logint(rng, 1, 48), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]),
                page=rng.choice([1, 8, 16, 32, 64]), dtype=rng.choice(["f16", "bf16"]),
                layout=rng.choice(["nhd", "hnd"]), shapes=shapes)
    if op == "branch":
        lo = _logint(rng, 1, 1500)
        return _branch("", R=_logint(rng, 1, 24), ways=rng.randint(1, 8), lo=lo, hi=lo + _logint(rng, 1, 300),
                       add=rng.choice([1, 1, rng.randint(1, 20)]), **pool)
    if op == "compact":
        lo = _logint(rng, 1, 2000)
        return _compact("", R=_logint(rng, 1, 16), lo=lo, hi=lo + _logint(rng, 1, 500),
                        part=rng.choice([0.1, 0.33, 0.5, 0.8]), **pool)
    kind = rng.choice(["one", "tokens", "drafts", "prompts", "prompts"])
    Hk = rng.choice([1, 2, 4, 8, 16, 16])
    c = _delta("", Hk=Hk, Hv=Hk * rng.choice([1, 2, 2, 4]), Dk=rng.choice([64, 128, 128]),
               Dv=rng.choice([32, 64, 96, 128, 128, 256]), gates=rng.choice(["raw", "direct"]), l2=rng.random() < 0.7,
               tiled=rng.random() < 0.3, fresh=rng.random() < 0.5, shapes=shapes)
    if kind == "tokens":
        c.update(B=_logint(rng, 2, 256))
    elif kind == "drafts":
        c.update(B=_logint(rng, 1, 64), n_lo=rng.randint(0, 3), n_hi=rng.randint(3, 12), keep=rng.random() < 0.7)
    elif kind == "prompts":
        hi = _logint(rng, 13, longest)
        c.update(B=_logint(rng, 1, 12), n_lo=rng.randint(0, hi), n_hi=hi)
    return c


# ---- the shapes a case describes --------------------------------------------------------------

def _counts(c):
    r = random.Random(c["shapes"])
    return [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]


def _starts(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def _branch_shape(c):
    """Tokens of each prompt, and the new tokens of each continuation."""
    r = random.Random(c["shapes"])
    length = [r.randint(c["lo"], c["hi"]) for _ in range(c["R"])]
    return length, [r.randint(1, c["add"]) for _ in range(c["R"] * c["ways"])]


def _compact_shape(c):
    """Tokens of each context, and the slots that are kept: the first ones, the latest ones, some of the rest."""
    r = random.Random(c["shapes"])
    length = [r.randint(c["lo"], c["hi"]) for _ in range(c["R"])]
    kept = []
    for n in length:
        want = max(1, int(n * c["part"]))
        always = sorted(set(range(min(4, n))) | set(range(max(0, n - 8), n)))
        rest = [i for i in range(n) if i not in set(always)]
        kept.append(sorted((always + r.sample(rest, max(0, min(len(rest), want - len(always)))))[:max(want, 1)]))
    return length, kept


def _pool_bytes(c):
    """What a case's caches hold."""
    if c["op"] == "branch":
        length, add = _branch_shape(c)
        tokens = sum(-(-x // c["page"]) for x in length) * c["page"] + len(add) * (c["add"] + 2 * c["page"])
    elif c["op"] == "compact":
        tokens = sum(len(k) + x + 2 * c["page"] for x, k in zip(*_compact_shape(c)))
    else:
        return 0
    return tokens * c["Hkv"] * c["D"] * 2 * 2 * c["layers"]


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"] == "delta":
        n = _counts(c)
        T, state = sum(n), c["Hv"] * c["Dk"] * c["Dv"] * 4
        live = sum(1 for x in n if x)
        moved = (0 if c["fresh"] else live) + (T if c["keep"] else live)
        return {"bytes": T * 4 * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"] + 2 * c["Hv"]) + moved * state,
                "flops": 6 * T * c["Hv"] * c["Dk"] * c["Dv"]}
    if c["op"] == "probs":
        return {"bytes": 8 * c["T"] * c["V"], "flops": 4 * c["T"] * c["V"]}
    if c["op"] == "verify":  # one row of the target's and, where there are drafts, one of the drafter's
        n = _counts(c)
        rows = sum(2 if x and c["draft"] == "probs" else 1 for x in n)
        return {"bytes": rows * c["V"] * 4 + sum(n) * 16 + 24 * c["B"], "flops": 2 * rows * c["V"]}
    token = c["Hkv"] * c["D"] * 2 * 2 * c["layers"]
    if c["op"] == "branch":
        length, _ = _branch_shape(c)
        moved = sum(x % c["page"] for x in length) * c["ways"]
        pages = sum(-(-x // c["page"]) for x in length) * c["ways"]
        return {"bytes": 2 * moved * token + 12 * pages, "flops": 0}
    _, kept = _compact_shape(c)
    return {"bytes": sum(len(k) for k in kept) * (2 * token + 4), "flops": 0}


# ---- inputs -------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pools(n_pages, c, gen):
    """One allocation of page pools, [2 * layers][pages][tokens][heads][D]: a layer's keys, then its values
    (head-major pools are permuted views)."""
    nhd = c["layout"] == "nhd"
    dims = (c["page"], c["Hkv"]) if nhd else (c["Hkv"], c["page"])
    pool = torch.empty((2 * c["layers"], n_pages, *dims, c["D"]), dtype=DTYPES[c["dtype"]], device="cuda")
    for x in pool:
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    return pool if nhd else pool.permute(0, 1, 3, 2, 4)


def _package():
    import gguf_block_dequant_gb300 as qg

    return qg


def prepare(c, seed):
    gen = _gen(seed)
    st = {"case": c}
    {"delta": _prepare_delta, "probs": _prepare_probs, "verify": _prepare_verify, "branch": _prepare_branch,
     "compact": _prepare_compact}[c["op"]](c, st, gen)
    return st


def _prepare_delta(c, st, gen):
    n = _counts(c)
    T, B, Hk, Hv, Dk, Dv = sum(n), c["B"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    st["n"], st["starts"] = n, _starts(n)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    def rand(*s):
        return torch.rand(s, generator=gen, device="cuda")

    # one projection's output row holds the queries, keys and values side by side, another one both gates
    x = randn(T, 2 * Hk * Dk + Hv * Dv)
    if not c["l2"]:  # normalised by the caller
        x[:, :2 * Hk * Dk] /= x[:, :2 * Hk * Dk].view(T, 2 * Hk, Dk).norm(dim=-1).repeat_interleave(Dk, 1)
    st["q"], st["k"] = x[:, :Hk * Dk].unflatten(1, (Hk, Dk)), x[:, Hk * Dk:2 * Hk * Dk].unflatten(1, (Hk, Dk))
    st["v"] = x[:, 2 * Hk * Dk:].unflatten(1, (Hv, Dv))
    ba = randn(T, 2 * Hv)
    st["a_scale"] = st["a_bias"] = None
    if c["gates"] == "raw":
        st["a_scale"] = -torch.exp(rand(Hv) * math.log(16.0))
        dt = torch.exp(math.log(1e-3) + rand(Hv) * math.log(100.0))
        st["a_bias"] = dt + torch.log(-torch.expm1(-dt))  # softplus of it is dt
    else:
        ba[:, Hv:] = -torch.exp(ba[:, Hv:] - 3.0)
        ba[:, :Hv] = torch.sigmoid(ba[:, :Hv])
    st["b"], st["a"] = ba[:, :Hv], ba[:, Hv:]
    # states are read from some slots of a pool and left in others
    slots = B + (T if c["keep"] else B)
    order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
    st["states"] = 0.3 * randn(slots, Hv, Dk, Dv)
    st["state_in"] = torch.full_like(order[:B], -1) if c["fresh"] else order[:B].clone()
    st["state_out"] = None if c["keep"] else order[B:].clone()
    st["state_each"] = order[B:].clone() if c["keep"] else None
    st["q_start"] = None if c["n_lo"] == c["n_hi"] == 1 else _i32(st["starts"])
    st["out"] = torch.zeros((T, Hv, Dv), device="cuda")
    st["scale"] = 1.0 / math.sqrt(Dk)
    if own:
        qg = _package()
        st["ws"] = torch.empty(qg.delta_workspace_size(T, B, Hk, Hv, Dk, Dv, c["n_hi"]), dtype=torch.uint8, device="cuda")


def _prepare_probs(c, st, gen):
    T, V = c["T"], c["V"]
    x = torch.randn((T, V), generator=gen, device="cuda") * 2.5
    if c["masked"]:  # banned tokens: the type's lowest value, or minus infinity
        ban = torch.rand((T, V), generator=gen, device="cuda") < 0.1
        low = torch.where(torch.arange(T, device="cuda") % 2 == 0, torch.finfo(torch.float32).min, -math.inf)
        x = torch.where(ban, low[:, None], x)
    st["logits"] = x
    st["temperature"] = None
    if c["temp"] == "mixed":  # from sharp to flat, and rows that take the largest logit
        t = 0.3 + 1.2 * torch.rand((T,), generator=gen, device="cuda")
        st["temperature"] = torch.where(torch.rand((T,), generator=gen, device="cuda") < 0.15, 0.0, t)
    st["out"] = torch.empty((T, V), device="cuda")


def _prepare_verify(c, st, gen):
    n, V, B = _counts(c), c["V"], c["B"]
    rows = [x + 1 for x in n]  # the last sampled token, then the drafts
    starts = _starts(rows)
    T = starts[-1]
    x = torch.randn((T, V), generator=gen, device="cuda") * 2.5
    st["p"] = torch.softmax(x + 0.7 * torch.randn((T, V), generator=gen, device="cuda"), -1)
    q = torch.softmax(x, -1)
    # row t holds what follows token t: draft t + 1 was drawn from the drafter's row t
    drawn = torch.multinomial(q, 1, generator=gen)[:, 0] if c["draft"] == "probs" else q.argmax(-1)
    st["q"] = q if c["draft"] == "probs" else None
    first = torch.randint(0, V, (1,), generator=gen, device="cuda")
    st["tokens"] = torch.cat([first, drawn[:-1]]).to(torch.int32)
    st["u"] = torch.rand((T,), generator=gen, device="cuda")
    st["u_next"] = torch.rand((B,), generator=gen, device="cuda")
    st["n"], st["starts"] = n, starts
    st["q_start"] = _i32(starts)
    st["kv_len"] = _i32([100 + x for x in rows])
    st["out"] = [torch.zeros((B,), dtype=torch.int32, device="cuda") for _ in range(3)]


def _prepare_branch(c, st, gen):
    length, add = _branch_shape(c)
    R, ways, page = c["R"], c["ways"], c["page"]
    have = [-(-x // page) for x in length]
    # a prompt's row is followed by those of its continuations, which are empty
    B = R * (ways + 1)
    cols = max(-(-(x + c["add"]) // page) for x in length)
    most = sum(have) + sum(-(-(length[i // ways] + a) // page) - length[i // ways] // page for i, a in enumerate(add))
    total = most + 5
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((B, cols), dtype=torch.int32, device="cuda")
    refs = torch.zeros((total,), dtype=torch.int32, device="cuda")
    at = 0
    kv_len, src, more = [0] * B, list(range(B)), [0] * B
    for r in range(R):
        p = r * (ways + 1)
        table[p, :have[r]] = order[at:at + have[r]]
        at += have[r]
        kv_len[p] = length[r]
        for i in range(ways):
            src[p + 1 + i], more[p + 1 + i] = p, add[r * ways + i]
    refs[order[:at].long()] = 1
    st.update(pages=table, refs=refs, kv_len=_i32(kv_len), src=_i32(src), add=_i32(more), pool=_pools(total, c, gen))
    st["short"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    if own:
        qg = _package()
        st["caches"] = qg.kv_caches(list(st["pool"][0::2]), list(st["pool"][1::2]))
        st["batch"] = qg.kv_batch(st["kv_len"], st["pages"])
        st["ws"] = torch.empty(qg.reserve_workspace_size(st["caches"], st["batch"]), dtype=torch.uint8, device="cuda")


def _prepare_compact(c, st, gen):
    length, kept = _compact_shape(c)
    R, page = c["R"], c["page"]
    # the contexts' rows, then those that receive what is kept, with pages of their own
    size = length + [len(k) for k in kept]
    have = [-(-x // page) for x in size]
    total = sum(have) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((2 * R, max(have)), dtype=torch.int32, device="cuda")
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    st.update(pages=table, kv_len=_i32(size), src=_i32([-1] * R + list(range(R))), size=size,
              keep_start=_i32([0] * R + _starts([len(k) for k in kept])), keep=_i32([i for k in kept for i in k]),
              pool=_pools(total, c, gen))
    st["dst_of"] = torch.repeat_interleave(torch.arange(R, 2 * R, device="cuda"), _i32([len(k) for k in kept]))
    st["slot_of"] = torch.cat([torch.arange(len(k), device="cuda") for k in kept])
    if own:
        qg = _package()
        st["caches"] = qg.kv_caches(list(st["pool"][0::2]), list(st["pool"][1::2]))
        st["batch"] = qg.kv_batch(st["kv_len"], st["pages"])


# ---- one pass ---------------------------------------------------------------------------------

def run(st):
    c = st["case"]
    return (_own if own else _plain)[c["op"]](c, st)


def _own_delta(c, st):
    _package().delta_rule(st["q"], st["k"], st["v"], st["a"], st["b"], st["states"], st["state_in"], st["state_out"],
                          st["out"], st["ws"], q_start=st["q_start"], max_new=c["n_hi"], state_each=st["state_each"],
                          a_scale=st["a_scale"], a_bias=st["a_bias"], l2norm_eps=L2_EPS if c["l2"] else None,
                          scale=st["scale"], tiled=c["tiled"])
    return st["out"], st["states"]


def _own_probs(c, st):
    return _package().token_probs(st["logits"], st["out"], temperature=st["temperature"])


def _own_verify(c, st):
    accepted, token, length = st["out"]
    _package().draft_verify(st["p"], st["tokens"], st["u"], st["u_next"], accepted, token, draft_probs=st["q"],
                            q_start=st["q_start"], kv_len=st["kv_len"], kept_len=length)
    return accepted, token, length


def _own_branch(c, st):
    qg = _package()
    qg.kv_fork(st["caches"], st["batch"], st["refs"], src=st["src"])
    qg.kv_reserve(st["caches"], st["batch"], st["refs"], st["add"], st["short"], st["ws"])
    return st["pages"], st["kv_len"], st["refs"], st["short"], st["pool"]


def _own_compact(c, st):
    _package().kv_compact(st["caches"], st["batch"], st["src"], st["keep_start"], st["keep"])
    return st["pool"]


def _heads(c, x):
    """The key heads' rows, one for each value head."""
    r = c["Hv"] // c["Hk"]
    return x.repeat(1, r, 1) if c["tiled"] else x.repeat_interleave(r, 1)


def _gates(c, st):
    if c["gates"] != "raw":
        return st["a"], st["b"]
    x = st["a"] + st["a_bias"]
    softplus = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    return st["a_scale"] * softplus, 1.0 / (1.0 + torch.exp(-st["b"]))


def _plain_delta(c, st):
    """One token or a few: token after token, all sequences and heads at once.  Longer: chunk after chunk, each
    chunk's updates from a triangular system.  A sequence that has ended keeps its state."""
    n = st["n"]
    q, k = st["q"], st["k"]
    if c["l2"]:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    q, k, v = _heads(c, q * st["scale"]), _heads(c, k), st["v"]
    g, beta = _gates(c, st)
    N, T = max(n), q.shape[0]
    first, live = torch.tensor(st["starts"][:-1], device="cuda"), torch.tensor(n, device="cuda")
    C = 1 if c["keep"] or N <= 16 else 64
    # tokens [B][N'], those past a sequence's end without decay and without update
    i = torch.arange(-(-N // C) * C, device="cuda")
    on = i[None] < live[:, None]
    at = torch.where(on, first[:, None] + i, T - 1)
    g, beta = torch.where(on[..., None], g[at], 0.0), torch.where(on[..., None], beta[at], 0.0)
    slot = st["state_in"].long()
    S = torch.where((slot >= 0)[:, None, None, None], st["states"][slot.clamp(min=0)], 0.0)
    some = on.nonzero(as_tuple=True)
    if C == 1:
        o = []
        for j in range(N):
            t = at[:, j]
            S = S * torch.exp(g[:, j])[..., None, None]
            u = beta[:, j][..., None] * (v[t] - torch.matmul(k[t].unsqueeze(-2), S).squeeze(-2))
            S = S + k[t][..., None] * u[..., None, :]
            o.append(torch.matmul(q[t].unsqueeze(-2), S).squeeze(-2))
            if c["keep"]:
                b = on[:, j].nonzero()[:, 0]
                st["states"][st["state_each"][t[b]].long()] = S[b]
        o = torch.stack(o, 1)
    else:
        def split(x):  # [B][N'][H][..] -> [B][H][chunks][C][..]
            return x.unflatten(1, (-1, C)).movedim(3, 1)

        q, k, v, beta = split(q[at]), split(k[at]), split(v[at]), split(beta)
        G = torch.cumsum(split(g.double()), -1)
        decay = torch.exp(G[..., :, None] - G[..., None, :]).float().tril()  # of token j's update at token i
        G, last = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
        A = (beta[..., None] * decay * torch.matmul(k, k.transpose(-1, -2))).tril(-1)
        X = torch.diag_embed(beta)  # the solution X of (1 + A) X = diag(beta), row after row
        for j in range(1, C):
            X[..., j, :] -= torch.matmul(A[..., j, None, :j], X[..., :j, :]).squeeze(-2)
        w, y = torch.matmul(X, G * k), torch.matmul(X, v)
        within = decay * torch.matmul(q, k.transpose(-1, -2))
        q, k, whole = G * q, last * k, G[..., -1:, :]
        o = []
        for j in range(at.shape[1] // C):
            u = y[:, :, j] - torch.matmul(w[:, :, j], S)
            o.append(torch.matmul(q[:, :, j], S) + torch.matmul(within[:, :, j], u))
            S = whole[:, :, j] * S + torch.matmul(k[:, :, j].transpose(-1, -2), u)
        o = torch.cat(o, 2).transpose(1, 2)
    st["out"][at[some]] = o[some]
    if not c["keep"]:  # a sequence without tokens leaves no state
        b = (live > 0).nonzero()[:, 0]
        st["states"][st["state_out"][b].long()] = S[b]
    return st["out"], st["states"]


def _plain_probs(c, st):
    x = st["logits"]
    m = x.amax(-1, keepdim=True)
    t = st["temperature"]
    if t is None:
        e = torch.exp(x - m)
        st["out"].copy_(e / e.sum(-1, keepdim=True))
        return st["out"]
    e = torch.exp((x - m) / torch.where(t > 0, t, 1.0)[:, None])
    best = torch.arange(c["V"], device="cuda")[None] == x.argmax(-1, keepdim=True)
    st["out"].copy_(torch.where(t[:, None] > 0, e / e.sum(-1, keepdim=True), best.float()))
    return st["out"]


def _plain_verify(c, st):
    B, V = c["B"], c["V"]
    p, q = st["p"], st["q"]
    T = p.shape[0]
    t = torch.arange(T - 1, device="cuda")
    drafted = st["tokens"][1:].long()
    # next to a border: in 64 bits
    want = p[t, drafted].double()
    have = q[t, drafted].double() if q is not None else torch.ones_like(want)
    ok = torch.cat([st["u"][:-1].double() * have < want, torch.zeros((1,), dtype=torch.bool, device="cuda")])
    start = st["q_start"].long()
    last = start[1:] - 1
    ok[last] = False  # the last row has no draft behind it
    # the first row of each sequence that is not ok
    row = torch.arange(T, device="cuda")
    stop = torch.where(ok, T, row).flip(0).cummin(0).values.flip(0)[start[:-1]]
    accepted, token, length = st["out"]
    accepted.copy_(stop - start[:-1])
    r = p[stop]
    refused = (stop < last)[:, None]
    if q is not None:
        r = torch.where(refused, torch.clamp(r - q[stop], min=0), r)
    else:
        at = st["tokens"][torch.clamp(stop + 1, max=T - 1)].long()
        hit = torch.arange(V, device="cuda")[None] == at[:, None]
        r = torch.where(refused & hit, torch.clamp(r - 1, min=0), r)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, p[stop])
    run_sum = torch.cumsum(r.double(), -1)
    over = run_sum > st["u_next"].double()[:, None] * run_sum[:, -1:]
    token.copy_(over.to(torch.uint8).argmax(-1))
    length.copy_(st["kv_len"] - (last - stop).int())
    return accepted, token, length


def _plain_branch(c, st):
    page = c["page"]
    table, refs, kv = st["pages"], st["refs"], st["kv_len"]
    B, cols = table.shape
    src, add = st["src"].long(), st["add"]
    col = torch.arange(cols, device="cuda")[None]
    me = torch.arange(B, device="cuda")
    other = src != me
    # fork: what a row held is released, what its source holds is shared
    held = (col < ((kv + page - 1) // page)[:, None]) & other[:, None]
    refs.index_add_(0, table[held].long(), torch.full_like(table[held], -1))
    new_len = kv[src]
    shared = (col < ((new_len + page - 1) // page)[:, None]) & other[:, None]
    table.copy_(torch.where(shared, table[src], table))
    refs.index_add_(0, table[shared].long(), torch.ones_like(table[shared]))
    kv.copy_(new_len)
    # reserve: the lowest free pages in the order of the rows; a shared page that was begun is copied
    old_pages, new_pages = (kv + page - 1) // page, (kv + add + page - 1) // page
    begun = torch.clamp(kv // page, max=cols - 1)
    own_page = table.gather(1, begun.long()[:, None])[:, 0]
    copy = (add > 0) & (kv % page > 0) & (refs[own_page.long()] > 1)
    need = torch.where(add > 0, new_pages - old_pages, 0) + copy.int()
    upto = torch.cumsum(need, 0)
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True)
    lowest = torch.where(copy, kv // page, old_pages)  # the first column that gets a page
    gets = (col >= lowest[:, None]) & (col < (lowest + need)[:, None])
    rank = (upto - need)[:, None] + col - lowest[:, None]
    st["short"].copy_(torch.clamp(upto[-1:] - (refs == 0).sum(), min=0))
    table.copy_(torch.where(gets, free[torch.where(gets, rank, 0).long()].int(), table))
    refs.index_add_(0, own_page[copy].long(), torch.full_like(own_page[copy], -1))
    refs[table[gets].long()] = 1
    rows = torch.arange(page, device="cuda")
    b = copy.nonzero()[:, 0]
    begun_rows = rows[None] < (kv[b] % page)[:, None]
    which, r = begun_rows.nonzero(as_tuple=True)
    dst, frm = table[b, begun[b].long()].long()[which], own_page[b].long()[which]
    for pool in st["pool"]:
        pool[dst, r] = pool[frm, r]
    kv.add_(add)
    return table, kv, refs, st["short"], st["pool"]


def _plain_compact(c, st):
    page = c["page"]
    src = st["src"].long()[st["dst_of"]]
    keep = st["keep"].long()
    dst_page, dst_row = st["pages"][st["dst_of"], st["slot_of"] // page].long(), st["slot_of"] % page
    src_page, src_row = st["pages"][src, keep // page].long(), keep % page
    for pool in st["pool"]:
        pool[dst_page, dst_row] = pool[src_page, src_row]
    return st["pool"]


_plain = {"delta": _plain_delta, "probs": _plain_probs, "verify": _plain_verify, "branch": _plain_branch,
          "compact": _plain_compact}
_own = {"delta": _own_delta, "probs": _own_probs, "verify": _own_verify, "branch": _own_branch,
        "compact": _own_compact}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(c, seed):
    """The outputs of ``run`` for these inputs, each from its definition."""
    global own
    keep, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = keep
    return {"delta": _exact_delta, "probs": _exact_probs, "verify": _exact_verify, "branch": _exact_branch,
            "compact": _exact_compact}[c["op"]](c, st)


def _exact_delta(c, st):
    """S <- e^g S;  S <- S + beta k (v - S^T k)^T;  o = S^T q: one sequence, one token after another."""
    n, Hk, Hv = st["n"], c["Hk"], c["Hv"]
    if sum(n) > 40000:
        return None
    key = [h % Hk for h in range(Hv)] if c["tiled"] else [h // (Hv // Hk) for h in range(Hv)]
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    if c["l2"]:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + L2_EPS)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + L2_EPS)
    q, k = q[:, key] / math.sqrt(c["Dk"]), k[:, key]
    g, beta = st["a"].double(), st["b"].double()
    if c["gates"] == "raw":
        g = st["a_scale"].double() * torch.logaddexp(g + st["a_bias"].double(), torch.zeros_like(g))
        beta = torch.sigmoid(beta)
    alpha = torch.exp(g)[..., None, None]
    out, states = st["out"].double(), st["states"].double()
    for b, N in enumerate(n):
        slot = int(st["state_in"][b])
        S = states[slot].clone() if slot >= 0 else torch.zeros_like(states[0])
        for t in range(st["starts"][b], st["starts"][b] + N):
            S *= alpha[t]
            miss = v[t] - torch.bmm(k[t, :, None], S)[:, 0]
            S.baddbmm_(k[t, :, :, None], (beta[t, :, None] * miss)[:, None])
            out[t] = torch.bmm(q[t, :, None], S)[:, 0]
            if c["keep"]:
                states[int(st["state_each"][t])] = S
        if N and not c["keep"]:
            states[int(st["state_out"][b])] = S
    return out, states


def _exact_probs(c, st):
    x, t = st["logits"].double(), st["temperature"]
    out = torch.empty_like(x)
    for r in range(c["T"]):
        tau = 1.0 if t is None else float(t[r])
        if tau > 0:
            out[r] = torch.softmax(x[r] / tau, -1)
        else:
            out[r] = 0
            out[r, int((x[r] == x[r].max()).nonzero()[0])] = 1
    return out


def _exact_verify(c, st):
    got = [[], [], []]
    for b in range(c["B"]):
        s, e = st["starts"][b], st["starts"][b + 1]
        t = s
        while t + 1 < e:
            x = int(st["tokens"][t + 1])
            q = float(st["q"][t, x]) if st["q"] is not None else 1.0
            if not float(st["u"][t]) * q < float(st["p"][t, x]):
                break
            t += 1
        r = st["p"][t].clone()
        if t + 1 < e:
            if st["q"] is not None:
                r = (r - st["q"][t]).clamp(min=0)
            else:
                x = int(st["tokens"][t + 1])
                r[x] = max(float(r[x]) - 1.0, 0.0)
        if float(r.double().sum()) == 0.0:
            r = st["p"][t].clone()
        run_sum = torch.cumsum(r.double(), 0)
        over = (run_sum > float(st["u_next"][b]) * float(run_sum[-1])).nonzero()
        got[0].append(t - s)
        got[1].append(int(over[0]))
        got[2].append(int(st["kv_len"][b]) - (e - 1 - t))
    return tuple(_i32(x) for x in got)


def _exact_branch(c, st):
    page, pool = c["page"], st["pool"]
    table, refs = st["pages"].tolist(), st["refs"].tolist()
    kv, src, add = st["kv_len"].tolist(), st["src"].tolist(), st["add"].tolist()
    for b, s in enumerate(src):
        if s != b:
            for i in range(-(-kv[b] // page)):
                refs[table[b][i]] -= 1
            kv[b] = kv[s]
            for i in range(-(-kv[b] // page)):
                table[b][i] = table[s][i]
                refs[table[s][i]] += 1
    free = [i for i, x in enumerate(refs) if x == 0]
    many = [x > 1 for x in refs]
    need = 0
    for b in range(len(kv)):
        if not add[b]:
            continue
        full, rem = divmod(kv[b], page)
        if rem and many[table[b][full]]:
            old, table[b][full] = table[b][full], free[need]
            refs[old] -= 1
            refs[free[need]] = 1
            pool[:, free[need], :rem] = pool[:, old, :rem]
            need += 1
        for i in range(-(-kv[b] // page), -(-(kv[b] + add[b]) // page)):
            table[b][i] = free[need]
            refs[free[need]] = 1
            need += 1
        kv[b] += add[b]
    return _i32(table), _i32(kv), _i32(refs), _i32([max(0, need - len(free))]), pool


def _exact_compact(c, st):
    page, pool = c["page"], st["pool"]
    table, start, keep = st["pages"].tolist(), st["keep_start"].tolist(), st["keep"].tolist()
    for b, s in enumerate(st["src"].tolist()):
        if s < 0:
            continue
        for i, at in enumerate(keep[start[b]:start[b + 1]]):
            pool[:, table[b][i // page], i % page] = pool[:, table[s][at // page], at % page]
    return pool
