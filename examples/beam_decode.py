"""Beam search on a small synthetic MoE decoder, every step through the library.

Per layer: RMSNorm, q/k/v projections (quantized GEMVs), kv_append (per-head norm, rotation,
write into the paged cache), attn_paged, output projection, RMSNorm, moe_layer; then the head,
beam_select and beam_reorder.  The W beams of a request share their prompt's pages as a prefix:
the prompt is cached once and read once for all of them.

Run from the repository root on a GPU:  python examples/beam_decode.py
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
    layers, H, Hq, Hkv, D, V = 2, 256, 8, 2, 64, 1024
    E, k, F = 8, 2, 256
    theta, eps, page = 10000.0, 1e-6, 8


class Weights:
    """Synthetic Q8_0 blocks (host, numpy) and norm vectors of the decoder."""

    def __init__(self, c=Config, seed=0):
        q = lambda rows, n, s: gs.quant_blocks(gs.Q8_0, rows, n, seed=seed, stream=s)  # noqa: E731
        self.embed = q(c.V, c.H, 1)
        self.layers = []
        for i in range(c.layers):
            s = 100 * (i + 1)
            self.layers.append(dict(q=q(c.Hq * c.D, c.H, s), k=q(c.Hkv * c.D, c.H, s + 1), v=q(c.Hkv * c.D, c.H, s + 2),
                                    o=q(c.H, c.Hq * c.D, s + 3), experts=gs.moe_experts(c.E, c.H, c.F, seed=seed, stream=s + 10),
                                    router=gs.router_weights(c.E, c.H, seed=seed, stream=s + 20)))
        self.final = np.full(c.H, 0.1, np.float32)  # keeps the synthetic head's logits within a few units
        self.ones = np.ones(c.H, np.float32)
        self.head_norm = np.ones(c.D, np.float32)


class Decoder:
    def __init__(self, w, n_pages, c=Config):
        self.c, dev = c, torch.device("cuda")
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.embed, self.final, self.ones, self.qk_norm = up(w.embed), up(w.final), up(w.ones), up(w.head_norm)
        self.layers = [{k: up(v.reshape(-1)) if k != "router" else up(v) for k, v in x.items()} for x in w.layers]
        self.gate, self.up, self.down, self.stride = gs.moe_expert_record_layout(c.H, c.F, gs.Q8_0)
        pool = torch.zeros((2 * c.layers, n_pages, c.page, c.Hkv, c.D), dtype=torch.float16, device=dev)
        self.caches = qg.kv_caches(list(pool[0::2]), list(pool[1::2]))
        self.freqs = qg.rope_freqs(c.D, c.theta).to(dev)
        self.moe_ws = torch.zeros(qg.moe_workspace_size(16, c.k, c.E, c.H, c.F), dtype=torch.uint8, device=dev)

    def forward(self, tokens, batch):
        """Hidden rows [T][H] of the batch's new tokens, whose keys and values join the cache."""
        c, T = self.c, tokens.numel()
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
        x, xn, qkv = f32(T, c.H), f32(T, c.H), f32(T, (c.Hq + 2 * c.Hkv) * c.D)
        q16 = torch.empty((T, c.Hq, c.D), dtype=torch.float16, device="cuda")
        att, proj = f32(T, c.Hq, c.D), f32(T, c.H)
        a, b = c.Hq * c.D, (c.Hq + c.Hkv) * c.D
        ws = torch.empty(qg.attn_workspace_size(self.caches[0], batch, c.Hq), dtype=torch.uint8, device="cuda")
        parts = [(i, min(T, i + 16)) for i in range(0, T, 16)]  # the GEMVs and the MoE layer take 16 tokens at a time
        qg.embed_rows(gs.Q8_0, self.embed, c.V, c.H, tokens, x)
        for cache, w in zip(self.caches, self.layers):
            qg.rmsnorm(x, self.ones, c.eps, xn)
            for i, j in parts:
                ys = [f32(j - i, n) for n in (a, b - a, b - a)]
                qg.qgemv_multi(gs.Q8_0, [w["q"], w["k"], w["v"]], ys, xn[i:j], c.H, j - i)
                qkv[i:j] = torch.cat(ys, 1)
            qg.kv_append(cache, batch, qkv[:, :a], qkv[:, a:b], qkv[:, b:], q16, self.freqs, q_norm=self.qk_norm,
                         k_norm=self.qk_norm, eps=c.eps)
            qg.attn_paged(cache, batch, q16, att, 1.0 / math.sqrt(c.D), ws)
            for i, j in parts:
                qg.qgemv_t(gs.Q8_0, w["o"], att[i:j], proj[i:j], c.H, c.Hq * c.D, j - i)
            x += proj
            qg.rmsnorm(x, self.ones, c.eps, xn)
            for i, j in parts:
                n = j - i
                ids = torch.empty((n, c.k), dtype=torch.int32, device="cuda")
                wts, act = f32(n, c.k), f32(n * c.k, c.F)
                e = w["experts"]
                qg.moe_layer(gs.Q8_0, xn[i:j], w["router"], e[self.gate:], e[self.up:], e[self.down:], self.stride, None,
                             c.E, n, c.H, c.F, c.E, c.k, ids, wts, act, x[i:j], self.moe_ws)
        return x

    def logits(self, x):
        c, n = self.c, x.shape[0]
        y = torch.empty_like(x)
        qg.rmsnorm(x, self.final, c.eps, y)
        out = torch.empty((n, c.V), dtype=torch.float32, device="cuda")
        for i in range(0, n, 16):
            j = min(n, i + 16)
            qg.qgemv_t(gs.Q8_0, self.embed, y[i:j], out[i:j], c.V, c.H, j - i)  # tied head
        return out


def beam_search(weights, prompts, W, steps, eos=-1, c=Config):
    """Per prompt: (scores [W], tokens [W][steps]) of the W best continuations, best first."""
    N, page = len(prompts), c.page
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pre_pages = [-(-len(p) // page) for p in prompts]
    own_cols = -(-steps // page)
    n_pages = sum(pre_pages) + N * W * own_cols
    model = Decoder(weights, n_pages, c)

    # pages: the prompts' first, then every beam's own
    table = np.zeros((N, max(pre_pages)), np.int32)
    at = 0
    for i, n in enumerate(pre_pages):
        table[i, :n] = np.arange(at, at + n)
        at += n
    prefix_pages = torch.from_numpy(table).cuda()
    own_pages = torch.arange(at, n_pages, dtype=torch.int32, device="cuda").view(N * W, own_cols)

    # the prompts, as the only tokens of N sequences
    lens = [len(p) for p in prompts]
    starts = np.concatenate([[0], np.cumsum(lens)])
    batch = qg.kv_batch(i32(lens), prefix_pages, i32(starts.tolist()), int(starts[-1]))
    x = model.forward(i32(np.concatenate(prompts).tolist()), batch)
    logits = model.logits(x[i32([s - 1 for s in starts[1:]]).long()]).repeat_interleave(W, 0)

    # the W beams of a request start equal: only the first may be continued
    scores = torch.full((N, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    done = torch.zeros((N, W), dtype=torch.uint8, device="cuda")
    kv_len = torch.zeros((N * W,), dtype=torch.int32, device="cuda")
    batch = qg.kv_batch(kv_len, own_pages, None, None, i32([W * i for i in range(N + 1)]), i32(lens), prefix_pages)
    sel_ws = torch.empty(qg.beam_workspace_size(N, W, W, c.V), dtype=torch.uint8, device="cuda")
    history = torch.zeros((N, W, steps), dtype=torch.int32, device="cuda")
    for step in range(steps):
        new_scores, new_done = torch.empty_like(scores), torch.empty_like(done)
        parents, tokens = (torch.empty((N, W), dtype=torch.int32, device="cuda") for _ in range(2))
        qg.beam_select(logits, scores, N, W, new_scores, parents, tokens, sel_ws, done=done, eos=eos, done_out=new_done)
        qg.beam_reorder(model.caches, batch, parents, W)
        scores, done = new_scores, new_done
        history = history.gather(1, parents.long()[..., None].expand_as(history))
        history[..., step] = tokens
        if step + 1 < steps:
            kv_len += 1
            logits = model.logits(model.forward(tokens.view(-1), batch))
    return [(scores[i].cpu(), history[i].cpu()) for i in range(N)]


def main():
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, Config.V, n).astype(np.int32) for n in (37, 5, 20)]
    qg.load()
    for i, (scores, tokens) in enumerate(beam_search(Weights(), prompts, W=4, steps=12)):
        print(f"request {i} ({len(prompts[i])} prompt tokens)")
        for s, t in zip(scores.tolist(), tokens.tolist()):
            print(f"  {s:9.4f}  {t}")
    if qg.device_status():
        raise SystemExit("device status set")


if __name__ == "__main__":
    main()
