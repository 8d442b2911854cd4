"""The beam-search example against a plain 64-bit forward pass without a cache: every returned
sequence's score is the sum of its tokens' log-probabilities under the model (the example's
pages, shared prefixes, appends, reorders and picks all have to be right for that), and the
beams come best first."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_dequant_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("beam_decode", os.path.join(ROOT, "examples", "beam_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.qg.load()
    m.qg.device_status()
    return m


class Plain:
    """The same model in 64 bits from dequantized weights; q, k and v round to f16 as the cache does."""

    def __init__(self, w, c, oracle, gs):
        d = lambda b, r, n: torch.from_numpy(oracle.dequant(gs.Q8_0, b.reshape(-1), r, n)).double()  # noqa: E731
        self.c, self.embed, self.final = c, d(w.embed, c.V, c.H), torch.from_numpy(w.final).double()
        go, uo, do, st = gs.moe_expert_record_layout(c.H, c.F, gs.Q8_0)
        self.layers = []
        for x in w.layers:
            ex = x["experts"].reshape(c.E, st)
            self.layers.append(dict(
                q=d(x["q"], c.Hq * c.D, c.H), k=d(x["k"], c.Hkv * c.D, c.H), v=d(x["v"], c.Hkv * c.D, c.H),
                o=d(x["o"], c.H, c.Hq * c.D), r=torch.from_numpy(x["router"]).double(),
                e=[(d(e[go:uo].copy(), c.F, c.H), d(e[uo:do].copy(), c.F, c.H), d(e[do:].copy(), c.H, c.F)) for e in ex]))

    def norm(self, x, w=1.0):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + self.c.eps) * w

    def rope(self, x):
        h = self.c.D // 2
        f = self.c.theta ** (-2.0 * torch.arange(h, dtype=torch.float64) / self.c.D)
        a = torch.arange(x.shape[0], dtype=torch.float64)[:, None, None] * f
        u, v = x[..., :h], x[..., h:]
        return torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1)

    def log_probs(self, tokens):
        c, n = self.c, len(tokens)
        x = self.embed[torch.as_tensor(tokens, dtype=torch.long)]
        r16 = lambda t: t.float().half().double()  # noqa: E731
        for w in self.layers:
            xn = self.norm(x)
            q, k, v = [(xn @ w[m].T).view(n, -1, c.D) for m in "qkv"]
            q, k, v = r16(self.rope(self.norm(q))), r16(self.rope(self.norm(k))), r16(v)
            g = c.Hq // c.Hkv
            s = torch.einsum("thd,shd->hts", q, k.repeat_interleave(g, 1)) / math.sqrt(c.D)
            s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool), 1), -math.inf)
            x = x + torch.einsum("hts,shd->thd", torch.softmax(s, -1), v.repeat_interleave(g, 1)).reshape(n, -1) @ w["o"].T
            xn = self.norm(x)
            top, ids = (xn @ w["r"].T).topk(c.k, -1)
            p = torch.softmax(top, -1)
            out = torch.zeros_like(x)
            for t in range(n):
                for j in range(c.k):
                    ga, up, dn = w["e"][ids[t, j]]
                    a = ga @ xn[t]
                    out[t] += p[t, j] * (dn @ (a / (1 + torch.exp(-a)) * (up @ xn[t])))
            x = x + out
        return torch.log_softmax(self.norm(x, self.final) @ self.embed.T, -1)


@pytest.mark.parametrize("W,lens,steps", [(4, (37, 5), 11), (3, (8, 1, 24), 18), (1, (9,), 4)])
def test_scores_are_the_sequences_log_probabilities(ex, oracle_lib, W, lens, steps):
    rng = np.random.default_rng(W)
    prompts = [rng.integers(0, ex.Config.V, n).astype(np.int32) for n in lens]
    w = ex.Weights(seed=W)
    res = ex.beam_search(w, prompts, W, steps)
    assert ex.qg.device_status() == 0
    plain = Plain(w, ex.Config, oracle_lib, ex.gs)
    for prompt, (scores, tokens) in zip(prompts, res):
        assert (scores[:-1] >= scores[1:]).all()
        assert len({tuple(t) for t in tokens.tolist()}) == W
        for s, t in zip(scores.tolist(), tokens.tolist()):
            lp = plain.log_probs([*prompt.tolist(), *t])
            want = sum(lp[len(prompt) - 1 + i, x].item() for i, x in enumerate(t))
            # f32 arithmetic (2^-24 steps, sums of up to 512 terms: about 2^-18 of a hidden row), and
            # f16 roundings that fall the other way for it (2^-11 of an element, one in 2^7): about
            # 2^-15 of a row; logits of up to 10 over at most 18 steps
            assert abs(s - want) <= 18 * 10 * 2.0 ** -15, (s, want)
