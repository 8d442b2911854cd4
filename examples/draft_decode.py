"""Drafted decoding of several continuations of each prompt, on a small synthetic hybrid decoder.

One layer is recurrent (delta_rule), one attends over the paged cache (kv_append, attn_paged); projections are
quantized GEMVs.  The prompts are read once (kv_reserve, the delta rule in chunks), then forked: a continuation
shares its prompt's pages until it writes (kv_fork, kv_reserve), and starts from its prompt's recurrent state.
The last continuation of a prompt gets a copy of its own instead (kv_compact).  Every step drafts a few tokens with a
bigram model (the embedding and the head alone), runs the decoder over all of them at once, keeping the recurrent
state after each, and lets draft_verify say how many stay: kv_fork drops the others from the cache, and the next step
starts from the state after the last one kept.  Nothing but the finished tokens comes back to the host.

Run from the repository root on a GPU:  python examples/draft_decode.py
"""
import math
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import gguf_block_dequant_gb300 as qg  # noqa: E402
import gguf_synth as gs  # noqa: E402


class Config:
    H, V, eps = 256, 512, 1e-6
    mix = 1e-3                                # of a layer's output: the bigram drafts are then worth something
    Hk, Hv, Dk, Dv = 2, 4, 64, 64             # recurrent layer
    Hq, Hkv, D, theta, page = 4, 2, 64, 1e4, 8  # attention layer


class Weights:
    """Synthetic Q8_0 blocks (host, numpy) and vectors."""

    def __init__(self, c=Config, seed=0):
        q = lambda rows, n, s: gs.quant_blocks(gs.Q8_0, rows, n, seed=seed, stream=s)  # noqa: E731
        rng = np.random.default_rng(seed)
        self.embed = q(c.V, c.H, 1)
        self.delta = [q(m, c.H, 10 + i) for i, m in enumerate((c.Hk * c.Dk, c.Hk * c.Dk, c.Hv * c.Dv))]
        self.gates = [q(c.Hv, c.H, 20 + i) for i in range(2)]
        self.delta_out = q(c.H, c.Hv * c.Dv, 30)
        self.attn = [q(m, c.H, 40 + i) for i, m in enumerate((c.Hq * c.D, c.Hkv * c.D, c.Hkv * c.D))]
        self.attn_out = q(c.H, c.Hq * c.D, 50)
        self.a_scale = -rng.uniform(0.02, 0.5, c.Hv).astype(np.float32)
        self.a_bias = rng.uniform(-2, 0, c.Hv).astype(np.float32)
        self.final = np.full(c.H, 0.01, np.float32)  # keeps the synthetic head's logits within a few units
        self.ones = np.ones(c.H, np.float32)
        self.head_norm = np.ones(c.D, np.float32)


class Decoder:
    def __init__(self, w, n_pages, n_slots, c=Config):
        self.c, dev = c, torch.device("cuda")
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.w = {k: [up(x) for x in v] if isinstance(v, list) else up(v) for k, v in vars(w).items()}
        pool = torch.zeros((2, n_pages, c.page, c.Hkv, c.D), dtype=torch.float16, device=dev)
        self.caches = qg.kv_caches([pool[0]], [pool[1]])
        self.states = torch.zeros((n_slots, c.Hv, c.Dk, c.Dv), device=dev)
        self.freqs = qg.rope_freqs(c.D, c.theta).to(dev)

    def _project(self, weights, x, sizes):
        c, T = self.c, x.shape[0]
        out = torch.empty((T, sum(sizes)), device="cuda")
        for i in range(0, T, 16):  # the GEMVs take 16 tokens at a time
            j = min(T, i + 16)
            ys = [torch.empty((j - i, m), device="cuda") for m in sizes]
            qg.qgemv_multi(gs.Q8_0, weights, ys, x[i:j], c.H, j - i)
            out[i:j] = torch.cat(ys, 1)
        return out

    def _back(self, weight, x, n):
        c, T = self.c, x.shape[0]
        y = torch.empty((T, c.H), device="cuda")
        for i in range(0, T, 16):
            j = min(T, i + 16)
            qg.qgemv_t(gs.Q8_0, weight, x[i:j].reshape(j - i, n), y[i:j], c.H, n, j - i)
        return y

    def forward(self, tokens, batch, q_start, most, state_in, state_out=None, state_each=None):
        """Hidden rows of the batch's new tokens (at most `most` of a sequence); both layers' states move on."""
        c, w, T = self.c, self.w, tokens.numel()
        x, xn = (torch.empty((T, c.H), device="cuda") for _ in range(2))
        qg.embed_rows(gs.Q8_0, w["embed"], c.V, c.H, tokens, x)
        # the recurrent layer
        qg.rmsnorm(x, w["ones"], c.eps, xn)
        a, b = c.Hk * c.Dk, 2 * c.Hk * c.Dk
        qkv = self._project(w["delta"], xn, (a, a, c.Hv * c.Dv))
        ab = self._project(w["gates"], xn, (c.Hv, c.Hv))
        o = torch.empty((T, c.Hv, c.Dv), device="cuda")
        ws = torch.empty(qg.delta_workspace_size(T, batch.n_seqs, c.Hk, c.Hv, c.Dk, c.Dv, most), dtype=torch.uint8, device="cuda")
        qg.delta_rule(qkv[:, :a].unflatten(1, (c.Hk, c.Dk)), qkv[:, a:b].unflatten(1, (c.Hk, c.Dk)),
                      qkv[:, b:].unflatten(1, (c.Hv, c.Dv)), ab[:, :c.Hv], ab[:, c.Hv:], self.states, state_in, state_out, o, ws,
                      q_start=q_start, max_new=most, state_each=state_each, a_scale=w["a_scale"], a_bias=w["a_bias"],
                      l2norm_eps=c.eps, scale=c.Dk ** -0.5)
        x.add_(self._back(w["delta_out"], o, c.Hv * c.Dv), alpha=c.mix)
        # the attention layer
        qg.rmsnorm(x, w["ones"], c.eps, xn)
        a, b = c.Hq * c.D, (c.Hq + c.Hkv) * c.D
        qkv = self._project(w["attn"], xn, (a, b - a, b - a))
        q16, att = torch.empty((T, c.Hq, c.D), dtype=torch.float16, device="cuda"), torch.empty((T, c.Hq, c.D), device="cuda")
        ws = torch.empty(qg.attn_workspace_size(self.caches[0], batch, c.Hq), dtype=torch.uint8, device="cuda")
        qg.kv_append(self.caches[0], batch, qkv[:, :a], qkv[:, a:b], qkv[:, b:], q16, self.freqs, q_norm=w["head_norm"],
                     k_norm=w["head_norm"], eps=c.eps)
        qg.attn_paged(self.caches[0], batch, q16, att, c.D ** -0.5, ws)
        x.add_(self._back(w["attn_out"], att, c.Hq * c.D), alpha=c.mix)
        return x

    def logits(self, x):
        c, T = self.c, x.shape[0]
        y, out = torch.empty_like(x), torch.empty((T, c.V), device="cuda")
        qg.rmsnorm(x, self.w["final"], c.eps, y)
        for i in range(0, T, 16):
            j = min(T, i + 16)
            qg.qgemv_t(gs.Q8_0, self.w["embed"], y[i:j], out[i:j], c.V, c.H, j - i)  # tied head
        return out

    def bigram(self, tokens):
        x = torch.empty((tokens.numel(), self.c.H), device="cuda")
        qg.embed_rows(gs.Q8_0, self.w["embed"], self.c.V, self.c.H, tokens, x)
        return self.logits(x)


def generate(weights, prompts, ways, drafts, steps, temperature=1.0, seed=0, c=Config, trace=None):
    """Per prompt, `ways` continuations of `steps` steps: lists of tokens.  trace: a list that receives each step's tokens,
    random numbers, probabilities, accepted counts and next tokens."""
    N, page = len(prompts), c.page
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, n = N * (ways + 1), drafts + 1  # a prompt's row is followed by its continuations'
    longest = max(len(p) for p in prompts) + steps * n
    cols = -(-longest // page) + 1
    n_pages = B * cols
    model = Decoder(weights, n_pages, N + 2 * N * ways * n, c)
    pages = torch.zeros((B, cols), dtype=torch.int32, device="cuda")
    kv_len, refs = i32([0] * B), i32([0] * n_pages)
    table = qg.kv_batch(kv_len, pages)
    room = torch.empty(qg.reserve_workspace_size(model.caches, table), dtype=torch.uint8, device="cuda")
    missing = i32([0])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda k: torch.rand((k,), generator=gen, device="cuda")  # noqa: E731

    # the prompts
    counts = [len(prompts[b // (ways + 1)]) if b % (ways + 1) == 0 else 0 for b in range(B)]
    start = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
    T = sum(counts)
    qg.kv_reserve(model.caches, table, refs, i32(counts), missing, room)
    slots = [b // (ways + 1) if b % (ways + 1) == 0 else -1 for b in range(B)]
    x = model.forward(i32(np.concatenate(prompts).tolist()), qg.kv_batch(kv_len, pages, start, T), start, max(counts),
                      i32([-1] * B), i32(slots))
    ends = start[1:].long()[:: ways + 1] - 1
    p = model.logits(x[ends])
    # continuations share their prompt's pages; the last one gets a copy of its own
    src = [b - b % (ways + 1) for b in range(B)]
    own = [b for b in range(B) if b % (ways + 1) == ways]
    qg.kv_fork(model.caches, table, refs, src=i32([b if b in own else s for b, s in enumerate(src)]))
    lens = [len(prompts[b // (ways + 1)]) if b in own else 0 for b in range(B)]
    qg.kv_reserve(model.caches, table, refs, i32(lens), missing, room)
    qg.kv_compact(model.caches, table, i32([src[b] if b in own else -1 for b in range(B)]),
                  i32(np.concatenate([[0], np.cumsum(lens)]).tolist()), i32([s for k in lens for s in range(k)]))
    # each continuation's first token
    live = [b for b in range(B) if b % (ways + 1)]
    L = len(live)
    temp = torch.full((L,), float(temperature), device="cuda")
    probs = torch.empty((L, c.V), device="cuda")
    qg.token_probs(p[[b // (ways + 1) for b in live]].contiguous(), probs, temperature=temp)
    pending, none = (torch.empty((L,), dtype=torch.int32, device="cuda") for _ in range(2))
    un = rand(L)
    qg.draft_verify(probs, None, None, un, none, pending)
    if trace is not None:
        trace.append(dict(first=True, u_next=un.cpu(), next=pending.cpu()))

    counts = [n if b % (ways + 1) else 0 for b in range(B)]
    start = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
    T, rows = L * n, torch.arange(L, device="cuda")
    batch = qg.kv_batch(kv_len, pages, start, T)
    adds, live_t = i32(counts), torch.tensor(live, device="cuda")
    state_in = i32([b // (ways + 1) if b % (ways + 1) else -1 for b in range(B)])
    accepted, token, kept = (i32([0] * B) for _ in range(3))
    tokens = torch.empty((L, n), dtype=torch.int32, device="cuda")
    q = torch.empty((L, n, c.V), device="cuda")
    p = torch.empty((T, c.V), device="cuda")
    temps = temp.repeat_interleave(n)
    history = [[pending.clone()[:, None], None]]
    for step in range(steps):
        tokens[:, 0] = pending
        for i in range(drafts):  # row i: what follows token i, and a draw from it
            qi = torch.empty((L, c.V), device="cuda")
            qg.token_probs(model.bigram(tokens[:, i].contiguous()), qi, temperature=temp)
            nxt = torch.empty((L,), dtype=torch.int32, device="cuda")
            qg.draft_verify(qi, None, None, rand(L), none, nxt)
            q[:, i], tokens[:, i + 1] = qi, nxt
        qg.kv_reserve(model.caches, table, refs, adds, missing, room)
        each = i32(list(range(N + (step % 2) * T, N + (step % 2 + 1) * T)))
        x = model.forward(tokens.view(-1), batch, start, n, state_in, None, each)
        qg.token_probs(model.logits(x), p, temperature=temps)
        u, un = rand(T), rand(B)
        qg.draft_verify(p, tokens.view(-1), u, un, accepted, token, draft_probs=q.view(T, c.V), q_start=start, kv_len=kv_len,
                        kept_len=kept)
        qg.kv_fork(model.caches, table, refs, keep=kept)
        got = accepted[live_t].long()
        state_in[live_t] = each[rows * n + got]
        pending = token[live_t]
        history.append([torch.cat([tokens[:, 1:], pending[:, None]], 1), got])
        if trace is not None:
            trace.append(dict(tokens=tokens.cpu().clone(), u=u.cpu().view(L, n), u_next=un[live_t].cpu(), q=q.cpu().clone(),
                              accepted=got.cpu(), next=pending.cpu().clone()))
    out = [[[] for _ in range(ways)] for _ in range(N)]
    for i in range(L):
        line = out[i // ways][i % ways]
        line.append(int(history[0][0][i]))
        for rows_, got in history[1:]:
            k = int(got[i])
            line += rows_[i, :k].tolist() + [int(rows_[i, -1])]
    if int(missing) or int(refs.min()) < 0:
        raise RuntimeError("the pages ran out")
    return out


def main():
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, Config.V, n).astype(np.int32) for n in (45, 9)]
    qg.load()
    for i, lines in enumerate(generate(Weights(), prompts, ways=3, drafts=3, steps=6, temperature=0.8)):
        print(f"prompt {i} ({len(prompts[i])} tokens)")
        for t in lines:
            print("  ", t)
    if qg.device_status():
        raise SystemExit("device status set")


if __name__ == "__main__":
    main()
